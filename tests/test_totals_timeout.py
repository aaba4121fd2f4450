"""After a wait that timed out, a totals call adds nothing.  No wait of that
kernel can be made to run out on a sound GPU, so this reads the source: the one
place that adds to the totals looks at the abort flag, behind the barrier that
gathers the warps' sums."""
import os
import re

import sparse_latent_attention_absorb_b200 as mla


def test_the_totals_addition_looks_at_the_abort_flag():
    path = os.path.join(os.path.dirname(mla.__file__), "csrc", "weights.cuh")
    src = open(path).read()
    assert src.count("atomicAdd(") == 1
    at = src.index("atomicAdd(")
    guard = src[src.rindex("if (", 0, at):at]
    assert re.match(r"if \(!\*ab\.flag && ", guard), guard
    # every warp's waits for the scores lie before that barrier
    barrier = src.rindex("named_bar_sync(1, 256)", 0, at)
    assert src.rindex("bars->s_full[j & 1]), (j >> 1) & 1, ab)", 0, at) < barrier < at
