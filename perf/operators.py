"""Operators of the 8-bit latent cache and of eviction: cases, inputs and plain forms.

Four operators of one serving loop over the latent cache (512 latent columns
and 64 rotary columns a position, one latent head shared by 128 query heads):

  append      new tokens' latents rounded to E4M3 and written with their
              rotary keys; one power-of-two scale for each block of tokens
  decode      the sparse decode step (or prefill rows, or a head shard) that
              reads that cache
  accumulate  the attention weight that every selected position got, summed
              over the heads and added to its running total
  evict       the positions of least total weight leave the cache, the others
              move up in their order

The 8-bit cache holds codes e4m3 [slots, S, 512], rotary keys bf16
[slots, S, 64] and scale f32 [slots, ceil(S / block)]; position t of a slot
stands for the latent code * s and the rotary key pe * s, s = scale[t // block].
"""
import math

import torch

own = False

D_LAT, D_ROPE, D_NOPE, D_V, HEADS = 512, 64, 128, 128, 128
SCALE = 192.0 ** -0.5
MIN_SCALE = 2.0 ** -40


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new token of each of 64 sequences, a scale a token
        {"name": "append_b64_token", "op": "append", "B": 64, "S": 4096, "new": 1, "ragged": False, "block": 1},
        # the same where 64 tokens share a scale: the block's earlier rows may have to be rounded again
        {"name": "append_b64_token_block64", "op": "append", "B": 64, "S": 4096, "new": 1, "ragged": False, "block": 64},
        # prompts of 8 sequences written at once, ragged, up to 4096 tokens each
        {"name": "append_b8_prompt", "op": "append", "B": 8, "S": 8192, "new": 4096, "ragged": True, "block": 16},
        # a single request: 1001 cached positions, 256 selected
        {"name": "decode_b1_ctx1001_top256", "op": "decode", "B": 1, "S": 1001, "lo": 1001, "K": 256, "heads": 128,
         "block": 1, "prefill": False},
        # a tensor-parallel rank's 16 heads, 32 requests of up to 8K
        {"name": "decode_b32_heads16", "op": "decode", "B": 32, "S": 8192, "lo": 2048, "K": 2048, "heads": 16,
         "block": 16, "prefill": False},
        # the large batch: contexts of 1K to 32K, top 2048
        {"name": "decode_b64_ctx32k_top2048", "op": "decode", "B": 64, "S": 32768, "lo": 1024, "K": 2048,
         "heads": 128, "block": 1, "prefill": False},
        # a prefill chunk: 500 query positions of one sequence, each with its own selection
        {"name": "prefill_r500_top2048", "op": "decode", "B": 500, "S": 4096, "lo": 3597, "K": 2048, "heads": 128,
         "block": 64, "prefill": True},
        # the weights of a small batch over the 8-bit cache, padded selections
        {"name": "weights_b8_ctx4096_fp8", "op": "accumulate", "B": 8, "S": 4096, "lo": 700, "K": 1000, "block": 16},
        # the weights of the large batch over the bf16 cache (block 0)
        {"name": "weights_b64_ctx8k_bf16", "op": "accumulate", "B": 64, "S": 8192, "lo": 1024, "K": 2048, "block": 0},
        # one request's cache halved
        {"name": "evict_b1_4096_fp8", "op": "evict", "B": 1, "S": 4096, "lo": 4096, "keep": 2048, "recent": 256,
         "block": 1},
        # a batch of ragged 8-bit caches brought to 2500 positions, 64 tokens a scale
        {"name": "evict_b64_8k_fp8_block64", "op": "evict", "B": 64, "S": 8192, "lo": 2048, "keep": 2500,
         "recent": 512, "block": 64},
        # long bf16 caches (block 0) halved
        {"name": "evict_b8_32k_bf16", "op": "evict", "B": 8, "S": 32768, "lo": 32768, "keep": 16384, "recent": 512,
         "block": 0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "decode", "decode", "accumulate", "evict"])
    if op == "append":
        B = spread(1, 64)
        new = spread(1, 4096 if B <= 8 else 64)
        return {"op": op, "B": B, "S": new + spread(16, 4096), "new": new, "ragged": rng.random() < 0.5,
                "block": rng.choice([1, 2, 4, 8, 16, 32, 64, 128])}
    if op == "decode":
        S = spread(64, 16384)
        return {"op": op, "B": spread(1, 64), "S": S, "lo": rng.randint(1, S), "K": spread(16, 2048),
                "heads": rng.choice([1, 16, 40, 64, 127, 128]), "block": rng.choice([1, 1, 8, 64, 128]),
                "prefill": rng.random() < 0.25}
    if op == "accumulate":
        S = spread(64, 8192)
        return {"op": op, "B": spread(1, 64), "S": S, "lo": rng.randint(1, S), "K": spread(16, 2048),
                "block": rng.choice([0, 0, 1, 16, 128])}
    S = spread(64, 16384)
    keep = rng.randint(1, S)
    return {"op": op, "B": spread(1, 32), "S": S, "lo": rng.randint(1, S), "keep": keep,
            "recent": rng.randint(0, keep), "block": rng.choice([0, 1, 4, 32, 128])}


# ------------------------------------------------------------------- inputs
def _ints(g, lo, hi, n):
    """n whole numbers of [lo, hi] (int32)."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _selection(g, end, K, S):
    """Distinct positions of [0, end) in a random order, -1 where a row has fewer than K."""
    rows = []
    for e in end.tolist():
        take = torch.randperm(e, generator=g, device="cuda")[:K].to(torch.int32)
        rows.append(torch.cat([take, torch.full((K - take.numel(),), -1, dtype=torch.int32, device="cuda")]))
    return torch.stack(rows)


def _latent_cache(g, slots, S, block):
    """A filled cache of normalised latents: (codes, pe, scale), or (kv, pe) in bf16 where block is 0."""
    bf = torch.bfloat16
    pe = torch.randn(slots, S, D_ROPE, generator=g, device="cuda", dtype=bf)
    if block == 0:
        return torch.randn(slots, S, D_LAT, generator=g, device="cuda", dtype=bf), pe, None
    n_blocks = -(-S // block)
    codes = torch.empty(slots, S, D_LAT, dtype=torch.uint8, device="cuda")
    scale = torch.empty(slots, n_blocks, dtype=torch.float32, device="cuda")
    at = torch.arange(S, device="cuda") // block
    for i in range(slots):
        x = torch.randn(S, D_LAT, generator=g, device="cuda") * torch.exp2(torch.randint(-1, 2, (S, 1), generator=g,
                                                                                         device="cuda").float())
        top = torch.zeros(n_blocks, device="cuda").scatter_reduce(0, at, x.abs().amax(1), "amax")
        scale[i] = _power_scale(top)
        s = scale[i][at][:, None]
        codes[i] = (x / s).to(torch.float8_e4m3fn).view(torch.uint8)
        pe[i] = (pe[i].float() / s).to(bf)
    return codes, pe, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf, B, S, op = torch.bfloat16, case["B"], case["S"], case["op"]
    st = dict(case)
    if op == "append":
        n = _ints(g, 1, case["new"], B) if case["ragged"] else torch.full((B,), case["new"], dtype=torch.int32,
                                                                          device="cuda")
        start = torch.floor(torch.rand(B, generator=g, device="cuda") * (S - n + 1)).to(torch.int32)
        cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        cu[1:] = torch.cumsum(n, 0)
        N = int(cu[-1])
        st["codes"], st["pe"], st["sc"] = _latent_cache(g, B, S, case["block"])
        # one token in eight is four times as large: its block's scale grows
        loud = 1 + 3 * (torch.rand(N, 1, generator=g, device="cuda") < 0.125).to(bf)
        st |= {"kv_new": torch.randn(N, D_LAT, generator=g, device="cuda", dtype=bf) * loud,
               "pe_new": torch.randn(N, D_ROPE, generator=g, device="cuda", dtype=bf), "cu": cu, "start": start}
        return st
    if op == "evict":
        end = _ints(g, case["lo"], S, B)
        kv, pe, sc = _latent_cache(g, B, S, case["block"])
        # totals fall off like attention's do: most positions small, a few large, some never selected
        acc = torch.exp(2 * torch.randn(B, S, generator=g, device="cuda"))
        acc *= torch.rand(B, S, generator=g, device="cuda") < 0.7
        st |= {"kv": kv, "pe": pe, "sc": sc, "acc": acc, "end": end, "kv_to": torch.zeros_like(kv),
               "pe_to": torch.zeros_like(pe), "sc_to": None if sc is None else torch.zeros_like(sc),
               "acc_to": torch.zeros_like(acc)}
        return st
    slots = 1 if case.get("prefill") else B
    st["kv"], st["pe"], st["sc"] = _latent_cache(g, slots, S, case["block"])
    st["end"] = _ints(g, case["lo"], S, B)
    if case.get("prefill"):
        st["end"] = torch.linspace(case["lo"], S, B, device="cuda").to(torch.int32)
        st["slot"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    st["idx"] = _selection(g, st["end"], case["K"], S)
    heads = case.get("heads", HEADS)
    st["q_pe"] = torch.randn(B, heads, D_ROPE, generator=g, device="cuda", dtype=bf)
    if op == "decode":
        st["q_nope"] = torch.randn(B, heads, D_NOPE, generator=g, device="cuda", dtype=bf)
        st["wkv_b"] = (torch.randn(heads * (D_NOPE + D_V), D_LAT, generator=g, device="cuda") * D_LAT ** -0.5).to(bf)
        return st
    st["q_lat"] = (torch.randn(B, heads, D_LAT, generator=g, device="cuda") * 0.5).to(bf)
    # the log-sum-exps that the decode step left behind
    st["lse"] = torch.logsumexp(_scores(st, st["q_lat"].float(), _rows(st)), -1)
    st["lse"] = torch.where(torch.isfinite(st["lse"]), st["lse"], torch.full_like(st["lse"], -math.inf))
    st["acc"] = torch.rand(B, S, generator=g, device="cuda")
    return st


# ------------------------------------------------------------------- plain forms
def _power_scale(top):
    """The smallest power of two that brings `top` to at most 448, E4M3's largest value."""
    m, e = torch.frexp(top / 448)  # top / 448 = m 2^e, m in [1/2, 1)
    return torch.ldexp(torch.ones_like(top), torch.where(m == 0.5, e - 1, e)).clamp_min(MIN_SCALE)


def _rows(st):
    """The selected positions' latents and rotary keys in f32, and which of them count."""
    idx, end = st["idx"].long(), st["end"].long().clamp(0, st["S"])
    ok = (idx >= 0) & (idx < end[:, None])
    t = torch.where(ok, idx, torch.zeros_like(idx))
    slot = st["slot"].long()[:, None] if "slot" in st else torch.arange(idx.shape[0], device="cuda")[:, None]
    c, r = st["kv"][slot, t], st["pe"][slot, t].float()
    if st["sc"] is None:
        return c.float(), r, ok, t
    s = st["sc"][slot, t // st["block"]][..., None]
    return c.view(torch.float8_e4m3fn).float() * s, r * s, ok, t


def _scores(st, q_lat, rows):
    c, r, ok, _ = rows
    s = torch.matmul(q_lat, c.transpose(1, 2)) + torch.matmul(st["q_pe"].float(), r.transpose(1, 2))
    return (s * SCALE).masked_fill(~ok[:, None], -math.inf)


def _append(st):
    T, S, B = st["block"], st["S"], st["B"]
    codes, pe, sc, cu, start = st["codes"], st["pe"], st["sc"], st["cu"].long(), st["start"].long()
    x, r = st["kv_new"].float(), st["pe_new"].float()
    i = torch.arange(x.shape[0], device="cuda")
    slot = torch.searchsorted(cu, i, right=True) - 1
    t = start[slot] + i - cu[slot]
    n_blocks = sc.shape[1]
    flat = slot * n_blocks + t // T
    need = torch.zeros(B * n_blocks, device="cuda").scatter_reduce(0, flat, x.abs().amax(1), "amax")
    need = _power_scale(need).view(B, n_blocks)
    touched = torch.zeros(B * n_blocks, dtype=torch.bool, device="cuda").index_fill(0, flat, True).view(B, n_blocks)
    # only the block that the first new token falls into can hold earlier rows
    earlier = torch.zeros_like(touched)
    seq = torch.arange(B, device="cuda")
    earlier[seq, start.clamp_max(S - 1) // T] = start % T != 0
    new = torch.where(touched, torch.where(earlier, torch.maximum(need, sc), need), sc)
    # earlier rows of that block, rounded again where the scale grew
    first = start.clamp_max(S - 1) // T
    old_t = first[:, None] * T + torch.arange(T, device="cuda")
    keep = old_t < start[:, None]
    old_t = torch.where(keep, old_t, torch.zeros_like(old_t))
    ratio = (sc[seq, first] / new[seq, first])[:, None, None]
    was, was_r = codes[seq[:, None], old_t], pe[seq[:, None], old_t]
    again = (was.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
    again_r = (was_r.float() * ratio).to(torch.bfloat16)
    at = (seq[:, None].expand_as(old_t)[keep], old_t[keep])
    codes[at], pe[at] = again[keep], again_r[keep]
    s = new[slot, t // T][:, None]
    codes[slot, t] = (x / s).to(torch.float8_e4m3fn).view(torch.uint8)
    pe[slot, t] = (r / s).to(torch.bfloat16)
    sc.copy_(new)
    return {"codes": codes.view(torch.float8_e4m3fn), "pe": pe, "scale": sc}


def _decode(st):
    w = st["wkv_b"].float().view(-1, D_NOPE + D_V, D_LAT)
    q_lat = torch.einsum("bhd,hdc->bhc", st["q_nope"].float(), w[:, :D_NOPE])
    rows = c, _, ok, _ = _rows(st)
    p = torch.softmax(_scores(st, q_lat, rows), -1)
    p = torch.where(ok.any(1)[:, None, None], p, torch.zeros_like(p))
    return torch.einsum("bhc,hdc->bhd", torch.matmul(p, c), w[:, D_NOPE:]).to(torch.bfloat16)


def _accumulate(st):
    rows = _, _, ok, t = _rows(st)
    p = torch.exp(_scores(st, st["q_lat"].float(), rows) - st["lse"][..., None])
    got = torch.where(ok, p.sum(1), torch.zeros_like(ok, dtype=torch.float32))
    return st["acc"].scatter_add_(1, t, got)


def _kept(acc, end, keep, recent):
    """Each row's kept positions in rising order, -1 behind the last, and their number."""
    B, S = acc.shape
    t = torch.arange(S, device="cuda")
    end = end.long().clamp(0, S)
    inside = t < end[:, None]
    late = inside & (t >= (end - recent)[:, None])
    key = torch.where(late, torch.full_like(acc, math.inf), acc).masked_fill(~inside, -math.inf)
    order = torch.argsort(key, dim=1, descending=True, stable=True)  # ties: the lower position first
    n = torch.minimum(end, torch.full_like(end, keep))
    chosen = torch.where(torch.arange(S, device="cuda") < n[:, None], order, torch.full_like(order, S))
    kept = torch.sort(chosen, 1).values[:, :keep]
    return torch.where(kept < S, kept, torch.full_like(kept, -1)), n


def _evict(st):
    acc, keep, T = st["acc"], st["keep"], st["block"]
    B, S = acc.shape
    kept, n = _kept(acc, st["end"], keep, st["recent"])
    ok = kept >= 0
    frm = kept.clamp_min(0)
    b, i = ok.nonzero(as_tuple=True)
    kv, pe = st["kv"][b, kept[b, i]], st["pe"][b, kept[b, i]]
    if T:
        s = st["sc"].gather(1, frm // T)
        at = (torch.arange(keep, device="cuda") // T).expand(B, keep)
        top = torch.zeros_like(st["sc"]).scatter_reduce(1, at, torch.where(ok, s, torch.zeros_like(s)), "amax")
        st["sc_to"].copy_(torch.where(top > 0, top, st["sc_to"]))
        ratio = (s / top.gather(1, at))[b, i][:, None]
        kv = (kv.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
        pe = (pe.float() * ratio).to(torch.bfloat16)
    st["kv_to"][b, i], st["pe_to"][b, i] = kv, pe
    st["acc_to"].zero_()
    st["acc_to"][b, i] = acc[b, kept[b, i]]
    return _evicted(st, kept.to(torch.int32), n.to(torch.int32))


def _evicted(st, kept, n):
    got = {"kv": st["kv_to"].view(torch.float8_e4m3fn) if st["block"] else st["kv_to"], "pe": st["pe_to"],
           "acc": st["acc_to"], "kept": kept, "end": n}
    return got | {"scale": st["sc_to"]} if st["block"] else got


# ------------------------------------------------------------------- one pass
def run(st):
    op = st["op"]
    if own:
        return _run_own(st)
    if op == "append":
        return _append(st)
    if op == "decode":
        return _decode(st)
    return _accumulate(st) if op == "accumulate" else _evict(st)


def _run_own(st):
    import sparse_latent_attention_absorb_b200 as mla
    op = st["op"]
    if op == "append":
        cache = mla.Fp8Cache(st["codes"], st["pe"], st["sc"], st["block"])
        mla.mla_append_fp8(cache, st["kv_new"], st["pe_new"], st["cu"], st["start"])
        return {"codes": st["codes"].view(torch.float8_e4m3fn), "pe": st["pe"], "scale": st["sc"]}
    cache = mla.Fp8Cache(st["kv"], st["pe"], st["sc"], st["block"]) if st["block"] else None
    if op == "decode":
        return mla.mla_sparse_decode_fp8(st["q_nope"], st["q_pe"], cache, st["end"], st["idx"], st["wkv_b"], SCALE,
                                         cache_slot=st.get("slot"))
    if op == "accumulate":
        if cache is None:
            return mla.mla_accumulate_weights(st["q_lat"], st["q_pe"], st["kv"], st["pe"], st["end"], st["idx"], SCALE,
                                              st["lse"], st["acc"])
        return mla.mla_accumulate_weights_fp8(st["q_lat"], st["q_pe"], cache, st["end"], st["idx"], SCALE, st["lse"],
                                              st["acc"])
    if cache is None:
        kept, n = mla.mla_evict(st["kv"], st["pe"], st["acc"], st["end"], st["keep"], st["recent"],
                                kv_out=st["kv_to"], pe_out=st["pe_to"], acc_out=st["acc_to"])
    else:
        to = mla.Fp8Cache(st["kv_to"], st["pe_to"], st["sc_to"], st["block"])
        kept, n = mla.mla_evict_fp8(cache, st["acc"], st["end"], st["keep"], st["recent"], cache_out=to,
                                    acc_out=st["acc_to"])
    return _evicted(st, kept, n)


# ------------------------------------------------------------------- least work
def work(case):
    """Bytes read and written once and operations of one pass; a ragged case counts the middle of its range."""
    B, S, op = case["B"], case["S"], case["op"]
    row = D_LAT * (1 if case["block"] else 2) + D_ROPE * 2
    if op == "append":
        n = B * ((1 + case["new"]) / 2 if case["ragged"] else case["new"])
        return {"bytes": n * ((D_LAT + D_ROPE) * 2 + row) + 8 * n / case["block"] + 8 * B, "flops": 4 * n * D_LAT}
    end = (case["lo"] + S) / 2
    if op == "evict":
        kept = min(case["keep"], end)
        scales = 8 * kept / case["block"] if case["block"] else 0
        return {"bytes": B * (4 * end + kept * (2 * row + 8) + 4 * (S - kept) + scales + 8), "flops": B * end}
    heads = case.get("heads", HEADS)
    keys = B * min(case["K"], end)
    # prefill rows share one slot: each of its rows is read once
    rows = min(keys, S) if case.get("prefill") else keys
    cache = rows * row + (4 * rows / case["block"] if case["block"] else 0)
    score = 2 * heads * (D_LAT + D_ROPE)
    if op == "accumulate":
        return {"bytes": cache + B * heads * ((D_LAT + D_ROPE) * 2 + 4) + 4 * B * case["K"] + 8 * keys,
                "flops": keys * (score + 2 * heads)}
    return {"bytes": cache + heads * (D_NOPE + D_V) * D_LAT * 2 + B * heads * (D_NOPE + D_ROPE + D_V) * 2
            + 4 * B * case["K"] + 4 * B,
            "flops": B * heads * 2 * D_LAT * (D_NOPE + D_V) + keys * (score + 2 * heads * D_LAT)}


# ------------------------------------------------------------------- 64 bits
def _e4m3(x):
    """The nearest E4M3 value of each number of at most 448 (ties to even), in float64."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -40)))
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e)  # log2 may fall short next to a power of two
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    step = torch.exp2(e.clamp_min(-6) - 3)
    return torch.round(x / step) * step


def _codes64(u8):
    """What E4M3 codes stand for: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    k = u8.long()
    e, m = (k >> 3) & 15, (k & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    return torch.where(k >= 128, -v, v)


def _scale64(top):
    v = MIN_SCALE
    while v * 448 < top:
        v *= 2
    return v


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "append":
        T, codes, pe, sc = st["block"], _codes64(st["codes"]), st["pe"].double(), st["sc"].double()
        cu, start = st["cu"].tolist(), st["start"].tolist()
        if cu[-1] / T > 20000:
            return None
        for b in range(case["B"]):
            n, p = cu[b + 1] - cu[b], start[b]
            x, r = st["kv_new"][cu[b]:cu[b + 1]].double(), st["pe_new"][cu[b]:cu[b + 1]].double()
            tops = x.abs().amax(1).tolist()
            while n > 0:
                k, lo = p // T, p - p % T
                m = min(n, lo + T - p)
                s = _scale64(max(tops[:m]))
                if p > lo and s > sc[b, k]:
                    f = float(sc[b, k]) / s
                    codes[b, lo:p], pe[b, lo:p] = _e4m3(codes[b, lo:p] * f), pe[b, lo:p] * f
                elif p > lo:
                    s = float(sc[b, k])
                sc[b, k] = s
                codes[b, p:p + m], pe[b, p:p + m] = _e4m3(x[:m] / s), r[:m] / s
                x, r, tops, p, n = x[m:], r[m:], tops[m:], p + m, n - m
        return {"codes": codes, "pe": pe, "scale": sc}
    if op == "evict":
        return None  # every output is copied, counted or a rounding of an 8-bit value
    out, slots = [], st["slot"].tolist() if "slot" in st else range(case["B"])
    w = st["wkv_b"].double().view(-1, D_NOPE + D_V, D_LAT) if op == "decode" else None
    for b, slot in enumerate(slots):
        t = st["idx"][b].long()
        t = t[(t >= 0) & (t < int(st["end"][b]))]
        c, r = st["kv"][slot, t], st["pe"][slot, t].double()
        if case["block"]:
            s = st["sc"][slot, t // case["block"]].double()[:, None]
            c, r = _codes64(c) * s, r * s
        c = c.double()
        q = st["q_lat"][b].double() if op == "accumulate" else torch.einsum("hd,hdc->hc", st["q_nope"][b].double(),
                                                                            w[:, :D_NOPE])
        x = (q @ c.T + st["q_pe"][b].double() @ r.T) * SCALE
        if op == "accumulate":
            row = st["acc"][b].double()
            row[t] += torch.exp(x - st["lse"][b].double()[:, None]).sum(0)
            out.append(row)
        else:
            x = torch.exp(x - x.amax(1, keepdim=True))
            mix = (x / x.sum(1, keepdim=True)) @ c
            out.append(torch.einsum("hc,hdc->hd", mix, w[:, D_NOPE:]))
    return torch.stack(out)
