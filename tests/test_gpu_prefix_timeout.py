"""qkv_prefix_attn's tcgen05 tiles when a wait runs out, made to happen on purpose (GPU).

The tiles' warps hand blocks to each other through mbarriers, and every wait is bounded: one that runs out sets
QKV_DEV_TIMEOUT, and the CTA drains its MMAs, frees its tensor memory and returns.
QKV_TEST_PREFIX_DROP_HANDOFF=<block> makes the warp that looks up the keys' records leave out one block's hand-off in
each CTA, a barrier that nothing will complete: the waits of the producers and of the scales' warp for that block run
out (after two seconds), and those of the MMA warp for its slots and of the softmax warps for its
scores. Nothing faults and nothing hangs. The call must come back with the bit set, and the
same context must then run it normally and match the oracle. On one SM per team and on a pair of SMs."""

import os
import time

import pytest
import torch

from dense_harness import dev16
from test_gpu_prefix import call, case, check

pytestmark = pytest.mark.gpu

ENV = "QKV_TEST_PREFIX_DROP_HANDOFF"


@pytest.mark.parametrize("fmt,act,D,rows,block", [("e4m3", "bf16", 128, 8, 1), ("e4m3", "bf16", 128, 32, 0), ("e4m3", "bf16", 128, 32, 2),
                                                  ("int8_side", "bf16", 256, 8, 2), ("int8_side", "bf16", 256, 16, 1),
                                                  ("bf16", "bf16", 128, 32, 1), ("f16", "f16", 256, 16, 0),
                                                  ("int8_inline", "f16", 256, 8, 3)])
def test_a_lost_handoff_times_out_and_the_context_stays_usable(fmt, act, D, rows, block):
    import quantized_kv_cache_write_gb300 as qkv
    assert ENV not in os.environ
    b, pool, q, scale = case(50, fmt, act, D, 1, 16, 70001, [1] * rows, 1, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = dev16(q, act)
    started = time.monotonic()
    os.environ[ENV] = str(block)
    try:
        call(pool, b, qd, 1, scale, status=status)
    finally:
        del os.environ[ENV]
    assert status.item() & qkv.QKV_DEV_TIMEOUT, status.item()
    assert time.monotonic() - started < 30
    status.zero_()
    out, lse = call(pool, b, qd, 1, scale, status=status)
    assert status.item() == 0
    check(pool, b, q, act, 1, scale, out, lse, what="after the timeout")
