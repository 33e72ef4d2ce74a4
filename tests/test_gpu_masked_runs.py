"""qkv_masked_attn's work list (GPU): runs of rows that begin anywhere, thousands of them, over the ends of the list's chunks;
tiles whose keys go to every team of SMs, some of them keys that only some rows see; and prompts that take the tcgen05 tiles
by the call's own rule.

Tables and pools are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

from masked_harness import Pool, Seqs, call, check, chunk_rows, dev16, query

pytestmark = pytest.mark.gpu


def _sampled(fmt, act, rng, seqs, pool, rows, H, G, D, pick, **kw):
    """The call over all rows, and the oracle at those picked."""
    qb = query(rng, len(rows), H * G, D, act)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, fmt, dev16(qb, act), seqs, rows, H, D ** -0.5, status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0
    sel = torch.from_numpy(pick).cuda()
    check(pool, fmt, act, qb[pick], seqs, rows[pick], H, D ** -0.5, got=(out[sel], lse[sel]),
          **{"max_row_end": int(rows[:, 2].max()), **kw})
    pad = torch.from_numpy(rows[:, 0] == -1).cuda()
    assert torch.isnan(out[pad]).all() and not torch.isnan(out[~pad]).any()


@pytest.mark.parametrize("fmt,act", [("int8_side", "bf16"), ("bf16", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("H,G,D", [(1, 16, 256), (2, 4, 128), (1, 48, 128)])
@pytest.mark.parametrize("longest", [1, 3, 40, 700])
def test_runs_of_any_length_begin_anywhere(monkeypatch, fmt, act, H, G, D, longest):
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", "tcgen05")
    rng = np.random.default_rng(longest + D + G)
    lengths = [900, 55, 1, 300]
    seqs = Seqs(rng, lengths, 16)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, H, D)
    runs = []
    while sum(map(len, runs)) < 2300:
        s = int(rng.integers(-1, 4))
        n = min(int(rng.integers(1, longest + 1)), lengths[max(s, 0)])
        first = int(rng.integers(0, lengths[max(s, 0)] - n + 1))
        end = np.arange(first, first + n) + 1
        # padding rows hold whatever the rows before left in their place
        runs.append(np.stack([np.full(n, s), np.maximum(end - 200, 0), end, end - 1], 1))
    rows = np.concatenate(runs).astype(np.int32)
    pick = np.unique(np.concatenate([rng.integers(0, len(rows), 150), [0, 1007, 1008, 1019, 1020, 1023, 1024, 2047, 2048, len(rows) - 1]]))
    _sampled(fmt, act, rng, seqs, pool, rows, H, G, D, pick)


@pytest.mark.parametrize("fmt,act", [("int8_side", "bf16"), ("bf16", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("G,D,n", [(16, 256, 5), (16, 256, 16), (8, 128, 12), (8, 128, 32)])
def test_a_tile_that_every_team_shares(monkeypatch, fmt, act, G, D, n):
    """Rows whose ranges chain together over the sequence: most teams' parts hold no key of most rows."""
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", "tcgen05")
    rng = np.random.default_rng(n + D)
    length = 30011
    seqs = Seqs(rng, [length], 16)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, 1, D)
    cuts = np.linspace(0, length, n + 1).astype(np.int32)
    rows = np.stack([np.zeros(n), np.maximum(cuts[:-1] - 1, 0), cuts[1:], cuts[1:] - 1], 1).astype(np.int32)
    rows[n // 2, 1:3] = 0, length
    check(pool, fmt, act, query(rng, n, G, D, act), seqs, rows, 1, D ** -0.5)


@pytest.mark.parametrize("fmt,act,H,G,D", [("int8_side", "bf16", 1, 16, 256), ("bf16", "bf16", 4, 8, 128), ("f16", "f16", 2, 3, 128)])
@pytest.mark.parametrize("mask,window,cap", [("causal", 0, 30.0), ("docs", 500, 0.0), ("prefix", 0, 0.0)])
def test_prompts_by_the_rule(fmt, act, H, G, D, mask, window, cap):
    rng = np.random.default_rng(window + D)
    lengths, new = (2003, 1201), (2003, 700)
    seqs = Seqs(rng, lengths, 16)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, H, D)
    rows = chunk_rows(lengths, new, mask, doc=311)
    pick = np.unique(np.concatenate([rng.integers(0, len(rows), 120), [0, 1, 2002, 2003, len(rows) - 1]]))
    _sampled(fmt, act, rng, seqs, pool, rows, H, G, D, pick, window=window, softcap=cap)


@pytest.mark.parametrize("tiles", ["mma", "tcgen05"])
@pytest.mark.parametrize("fmt,act,G,D", [("int8_side", "bf16", 16, 256), ("bf16", "bf16", 8, 128)])
@pytest.mark.parametrize("new", [1, 50])
def test_slopes_of_either_sign_and_any_size(monkeypatch, tiles, fmt, act, G, D, new):
    """A negative slope prefers far keys, a large one leaves the nearest (or the farthest) alone."""
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", tiles)
    rng = np.random.default_rng(G + new)
    seqs = Seqs(rng, [700, 333], 16)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, 1, D)
    rows = chunk_rows([700, 333], [new, new])
    rows[::3, 3] = 350  # in the middle of what these rows see
    slopes = np.resize([0.0, -0.01, 0.5, -0.5, 300.0, -300.0, 1e-6, 0.03], G)
    check(pool, fmt, act, query(rng, len(rows), G, D, act), seqs, rows, 1, D ** -0.5, slopes=slopes, softcap=20.0)
