"""Plain 64-bit forms of the 8-bit cache's operators and of eviction, for the
tests: written from the definitions in the public header, with no code of the
package."""
import math

import torch

D_LAT, D_ROPE, D_V = 512, 64, 128


def e4m3_values(codes):
    """What E4M3 codes stand for (sign, 4 exponent bits of bias 7, 3 mantissa bits, 0x7f / 0xff NaN)."""
    k = codes.long()
    e, m = (k >> 3) & 15, (k & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    v = torch.where((k & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(k >= 128, -v, v)


def e4m3_codes(x):
    """The nearest E4M3 code of each number of magnitude <= 448 (ties to even); what is not finite gives NaN."""
    a = x.abs()
    fin = torch.isfinite(x)
    a = torch.where(fin, a, torch.zeros_like(a))
    _, e = torch.frexp(a)  # a = m 2^e, m in [1/2, 1)
    q = torch.clamp(e - 1, min=-6) - 3
    n = torch.round(a / torch.exp2(q.double()))  # a whole number of steps, 16 at the most
    up = n >= 16
    n, q = torch.where(up, n / 2, n), torch.where(up, q + 1, q)
    code = torch.where(n >= 8, ((q + 10) << 3) + n.long() - 8, n.long())
    code = torch.where(fin, code, torch.full_like(code, 127))
    neg = torch.signbit(x) & ~torch.isnan(x) & torch.isfinite(x)
    return (code + 128 * neg.long()).to(torch.uint8)


def block_scale(top):
    s = 2.0 ** -40
    while 448 * s < top:
        s *= 2
    return s


def append(codes, pe, scale, block, kv_new, pe_new, cu, start, slots=None):
    """In place on copies in memory (codes uint8, pe bf16, scale f32)."""
    S = codes.shape[1]
    for q in range(len(start)):
        slot = q if slots is None else slots[q]
        rows = [(start[q] + i, cu[q] + i) for i in range(cu[q + 1] - cu[q])]
        rows = [(t, r) for t, r in rows if 0 <= t < S]
        if not 0 <= slot < codes.shape[0] or not rows:
            continue
        for k in sorted({t // block for t, _ in rows}):
            mine = [(t, r) for t, r in rows if t // block == k]
            x = kv_new[[r for _, r in mine]].double()
            fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
            s, lo = block_scale(float(fin.max())), k * block
            earlier = mine[0][0] - lo
            if earlier:
                old = float(scale[slot, k])
                s = max(s, old)
                if s != old:
                    was = e4m3_values(codes[slot, lo:lo + earlier]) * (old / s)
                    codes[slot, lo:lo + earlier] = e4m3_codes(was)
                    pe[slot, lo:lo + earlier] = (pe[slot, lo:lo + earlier].double() * (old / s)).to(torch.bfloat16)
            scale[slot, k] = s
            for (t, r), row in zip(mine, x):
                codes[slot, t] = e4m3_codes(row / s)
                pe[slot, t] = (pe_new[r].double() / s).to(torch.bfloat16)


def selected(idx, end, S):
    e = max(0, min(int(end), S))
    return idx[(idx >= 0) & (idx < e)].long()


def rows_of(cache, slot, t):
    """Latents and rotary keys of positions t, float64."""
    kv, pe, scale, block = cache
    if scale is None:
        return kv[slot, t].double(), pe[slot, t].double()
    s = scale[slot, t // block].double()[:, None]
    return e4m3_values(kv[slot, t]) * s, pe[slot, t].double() * s


def attend(q_lat, q_pe, cache, slot, t, scale):
    """One row: (scores [h, t], mix [h, 512], lse [h]) in float64; an empty selection mixes to 0, lse -inf."""
    c, r = rows_of(cache, slot, t)
    x = (q_lat.double() @ c.T + q_pe.double() @ r.T) * scale
    if x.shape[1] == 0:
        return x, torch.zeros(q_lat.shape[0], D_LAT, dtype=torch.float64, device=c.device), torch.full(
            (q_lat.shape[0],), -math.inf, dtype=torch.float64, device=c.device)
    return x, torch.softmax(x, 1) @ c, torch.logsumexp(x, 1)


def decode(q_nope, q_pe, cache, slots, end, idx, wkv_b, scale):
    R, h = q_nope.shape[:2]
    w = wkv_b.double().view(h, 256, D_LAT)
    S = cache[0].shape[1]
    out = torch.zeros(R, h, D_V, dtype=torch.float64, device=q_nope.device)
    lse = torch.full((R, h), -math.inf, dtype=torch.float64, device=q_nope.device)
    for b in range(R):
        slot = int(slots[b])
        t = selected(idx[b], end[b], S) if 0 <= slot < cache[0].shape[0] else idx[b][:0].long()
        if not len(t):
            continue
        q_lat = torch.einsum("hd,hdc->hc", q_nope[b].double(), w[:, :128])
        _, mix, lse[b] = attend(q_lat, q_pe[b], cache, slot, t, scale)
        out[b] = torch.einsum("hc,hdc->hd", mix, w[:, 128:])
    return out, lse


def keep_positions(acc, n, keep, recent):
    """The kept positions of one row of totals (a list of floats), rising."""
    if n <= keep:
        return list(range(n))
    late = n - recent
    order = sorted(range(late), key=lambda i: (0 if math.isnan(acc[i]) else 1, 0.0 if math.isnan(acc[i]) else -acc[i], i))
    return sorted(order[:keep - recent]) + list(range(late, n))
