"""The tiles of qkv_prefix_attn at their limits (GPU): long ranges of key blocks per tile, scales and values near the
ends of their ranges, and padding and flagged rows where no merge follows.

Compared with the fp64 oracle ("[Perf][SM70][FP8] Hoist QSA E4M3 KV scales" §Changes: hoisted scales; "[Model][SM70]
[FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope: paged storage, split-K workspace)."""

import numpy as np
import pytest
import torch

from dense_harness import Batch, Pool, bits16, dev16
from test_gpu_prefix import FMTS, call, check

pytestmark = pytest.mark.gpu


def prefix_slots(b):
    p = np.arange(b.prefix)
    return b.prefix_blocks[p // b.block].astype(np.int64) * b.block + p % b.block


# One SM and a pair of SMs, one tile and two: each with several blocks per team, so that its score buffers are used
# again and again. A block's values differ from all others' and its keys weigh about the same: weights that a later
# block's scores had overwritten before they were multiplied would show.
@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,rows,prefix", [(128, 16, 70001), (128, 32, 70001), (256, 8, 70001), (256, 16, 70001), (128, 32, 9001)])
def test_score_buffers_used_again_and_again(fmt, act, D, rows, prefix):
    rng = np.random.default_rng(40)
    b = Batch(rng, prefix, [1] * rows, 1, 64)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, 1, D)
    order = prefix_slots(b)
    src = order[np.arange(prefix) // 64 % 61]  # one of 61 tokens per 64 keys
    for name in ("K", "V"):
        getattr(pool, name)[order] = getattr(pool, name)[src]
    to, frm = torch.from_numpy(order).cuda(), torch.from_numpy(src).cuda()
    for t in (*pool.cache, *(x for x in pool.kw.values() if torch.is_tensor(x))):
        t[to] = t[frm].clone()
    q = bits16(rng.standard_normal((rows, 16, D)), act)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, act), 1, 0.25 * D ** -0.5, status=status)
    check(pool, b, q, act, 1, 0.25 * D ** -0.5, out, lse, what=f"{fmt} {D} {rows}")
    assert int(status.item()) == 0
    for _ in range(10):
        o2, l2 = call(pool, b, dev16(q, act), 1, 0.25 * D ** -0.5)
        assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)
