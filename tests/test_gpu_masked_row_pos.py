"""qkv_masked_attn's row_pos is looked at for the window and the bias only (GPU): without either it may hold anything.

Pools and block tables are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

from masked_harness import Pool, Seqs, call, check, chunk_rows, dev16, query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tiles", ["mma", "tcgen05"])
@pytest.mark.parametrize("fmt,act,H,G,D", [("int8_side", "bf16", 1, 16, 256), ("bf16", "bf16", 2, 4, 128)])
@pytest.mark.parametrize("n", [1, 70])
def test_positions_that_nothing_asks_for_may_be_anything(monkeypatch, tiles, fmt, act, H, G, D, n):
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", tiles)
    rng = np.random.default_rng(n + D)
    lengths = (200, 90)
    seqs = Seqs(rng, lengths, 16)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, H, D)
    rows = chunk_rows(lengths, (n, n))
    q = query(rng, len(rows), H * G, D, act)
    for cap in (0.0, 30.0):
        want = check(pool, fmt, act, q, seqs, rows, H, D ** -0.5, softcap=cap, use_pos=False)
        anything = rows.copy()
        anything[:, 3] = rng.choice(np.array([-1, -(1 << 31), (1 << 31) - 1, 7], dtype=np.int64), len(rows))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(pool, fmt, dev16(q, act), seqs, anything, H, D ** -0.5, softcap=cap, status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    anything[:, 3] = -1  # asked for: such rows see nothing, and are flagged
    for kw in (dict(window=50), dict(slopes=0.5 ** np.arange(1.0, H * G + 1))):
        check(pool, fmt, act, q, seqs, anything, H, D ** -0.5, want_status=2, **kw)
