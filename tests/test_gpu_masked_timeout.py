"""qkv_masked_attn's tcgen05 tiles when a wait runs out, made to happen on purpose (GPU), as test_gpu_prefix_timeout.py does
for the shared prefix: one block's hand-off is left out, every wait for it is bounded, the call comes back with
QKV_DEV_TIMEOUT set, and the same context then runs it normally and matches the oracle."""

import os
import time

import numpy as np
import pytest
import torch

from masked_harness import Pool, Seqs, call, check, chunk_rows, dev16, query
from test_gpu_prefix_timeout import ENV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,act,D,G,new,block", [("e4m3", "bf16", 128, 8, 200, 0), ("int8_side", "bf16", 256, 16, 90, 2),
                                                   ("bf16", "bf16", 256, 2, 40, 1), ("int8_inline", "f16", 128, 4, 300, 3)])
def test_a_lost_handoff_times_out_and_the_context_stays_usable(fmt, act, D, G, new, block, monkeypatch):
    import quantized_kv_cache_write_gb300 as qkv
    assert ENV not in os.environ
    rng = np.random.default_rng(block)
    lengths = (9000, 8000)
    seqs = Seqs(rng, lengths, 64)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, 2, D)
    rows = chunk_rows(lengths, (new, new))
    q = query(rng, len(rows), 2 * G, D, act)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", "tcgen05")
    started = time.monotonic()
    os.environ[ENV] = str(block)
    try:
        call(pool, fmt, dev16(q, act), seqs, rows, 2, D ** -0.5, status=status, window=5000, softcap=30.0)
    finally:
        del os.environ[ENV]
    assert status.item() & qkv.QKV_DEV_TIMEOUT, status.item()
    assert time.monotonic() - started < 30
    sub = np.concatenate([rows[:30], rows[-30:]])
    qs = np.concatenate([q[:30], q[-30:]])
    out, lse = call(pool, fmt, dev16(q, act), seqs, rows, 2, D ** -0.5, window=5000, softcap=30.0)
    torch.cuda.synchronize()
    pick = torch.cat([torch.arange(30), torch.arange(len(rows) - 30, len(rows))]).cuda()
    check(pool, fmt, act, qs, seqs, sub, 2, D ** -0.5, window=5000, softcap=30.0, got=(out[pick], lse[pick]), want_status=0)
