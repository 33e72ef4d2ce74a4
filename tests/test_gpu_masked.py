"""qkv_masked_attn against the oracle (GPU): ranges, windows, documents, prefixes, capped scores and distance bias over every
format, for single tokens, drafts and prompts' chunks; rows that see nothing, padding, invalid rows and blocks, values that
are not finite where a row does not look.

Pools, scales and block tables are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

from masked_harness import Pool, Seqs, call, check, chunk_rows, dev16, query

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["mma", "tcgen05"])
def tiles(request, monkeypatch):
    """Each kind of tiles, whatever the call would choose at these sizes."""
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", request.param)


FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_side", "f16"), ("int8_inline", "bf16"),
        ("e4m3", "f16"), ("e4m3", "bf16")]
SLOPES = lambda n: 2.0 ** (-8.0 * np.arange(1, n + 1) / n)  # noqa: E731


def setup(seed, fmt, act, lengths, block, H, D, **kw):
    rng = np.random.default_rng(seed)
    seqs = Seqs(rng, lengths, block)
    return rng, seqs, Pool(rng, fmt, act, seqs.live, seqs.num_slots, H, D, **kw)


# rows per sequence: single tokens, drafts, a chunk, whole prompts
NEW = [(1, 1, 1), (5, 5, 5), (37, 1, 100), (150, 90, 260)]


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,H,G", [(128, 2, 8), (256, 1, 16), (128, 1, 3)])
@pytest.mark.parametrize("new", NEW)
def test_capped_and_biased_causal_rows(fmt, act, D, H, G, new):
    lengths = (150, 90, 260)
    rng, seqs, pool = setup(D + G, fmt, act, lengths, 16, H, D)
    rows = chunk_rows(lengths, new)
    check(pool, fmt, act, query(rng, len(rows), H * G, D, act, 2.0), seqs, rows, H, D ** -0.5, softcap=30.0,
          slopes=SLOPES(H * G))


@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("int8_side", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("mask,window", [("causal", 0), ("causal", 1), ("causal", 40), ("docs", 0), ("docs", 33), ("prefix", 0),
                                         ("prefix", 70)])
@pytest.mark.parametrize("kind", ["plain", "cap", "bias"])
@pytest.mark.parametrize("new", [(1, 2, 1), (200, 137, 3)])
def test_masks(fmt, act, mask, window, kind, new):
    lengths, H, G, D = (200, 137, 64), 1, 12, 128
    rng, seqs, pool = setup(window, fmt, act, lengths, 7, H, D)
    rows = chunk_rows(lengths, new, mask)
    check(pool, fmt, act, query(rng, len(rows), H * G, D, act), seqs, rows, H, D ** -0.5, window=window,
          softcap=5.0 if kind == "cap" else 0.0, slopes=SLOPES(H * G) if kind == "bias" else None,
          use_start=mask == "docs", use_pos=mask == "prefix")


@pytest.mark.parametrize("G", [1, 2, 5, 8, 9, 16, 17, 64, 128])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new", [(1, 1), (4, 3), (90, 31)])
def test_groups(G, D, new):
    lengths, H = (90, 131), 2 if G < 64 else 1
    rng, seqs, pool = setup(G, "int8_side", "bf16", lengths, 16, H, D)
    rows = chunk_rows(lengths, new)
    check(pool, "int8_side", "bf16", query(rng, len(rows), H * G, D, "bf16"), seqs, rows, H, D ** -0.5, window=50, softcap=20.0)


@pytest.mark.parametrize("block", [1, 5, 16, 100, 128])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_lengths_and_blocks(block, length):
    rng, seqs, pool = setup(length, "e4m3", "bf16", (length, length), block, 1, 128)
    for new in (1, length):
        rows = chunk_rows((length, length), (new, 1))
        check(pool, "e4m3", "bf16", query(rng, len(rows), 8, 128, "bf16"), seqs, rows, 1, 0.09, slopes=SLOPES(8))


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("n", [8, 120])
def test_rows_that_see_nothing_padding_and_invalid_rows(fmt, act, n):
    lengths, H, G, D = (130, 140), 1, 8, 128
    rng, seqs, pool = setup(n, fmt, act, lengths, 16, H, D)
    good = chunk_rows(lengths, (n, n))
    for bad in (False, True):
        rows = good.copy()
        rows[1] = (0, 0, 0, 0)                  # nothing
        rows[3] = (0, 9, 9, 9)                  # start = end
        rows[4] = (0, 30, 9, 9)                 # start > end
        rows[5, 0] = -1                         # padding
        rows[-1, 0] = -1
        rows[6] = (0, 0, 20, 100)               # all keys outside its window
        if bad:
            rows[7] = (0, 0, -1, 5)
            rows[n] = (2, 0, 10, 5)             # no such sequence
            rows[n + 1] = (-2, 0, 10, 5)
            rows[n + 2] = (1, -1, 10, 5)
            rows[n + 3] = (1, 0, 141, 5)        # past max_row_end
            rows[n + 4] = (1, 0, 10, -3)
            rows[n + 5] = (1, 0, 10, (1 << 30) + 1)
        check(pool, fmt, act, query(rng, len(rows), G * H, D, act), seqs, rows, H, 0.1, window=60, max_row_end=140,
              slopes=SLOPES(G * H), want_status=2 if bad else 0)


@pytest.mark.parametrize("n", [1, 100])
def test_no_keys_at_all(n):
    rng, seqs, pool = setup(0, "bf16", "bf16", (16,), 16, 1, 128)
    rows = np.zeros((n, 4), dtype=np.int32)
    check(pool, "bf16", "bf16", query(rng, n, 4, 128, "bf16"), seqs, rows, 1, 0.1, max_row_end=0)


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("n", [1, 4, 130])
def test_blocks_that_no_row_sees_may_be_anything(fmt, act, n):
    """Behind a window blocks are given back: their table entries are -1 or past the pool, and nothing is flagged."""
    lengths, H, G, D = (400, 390), 1, 8, 128
    rng, seqs, pool = setup(n, fmt, act, lengths, 16, H, D)
    rows = chunk_rows(lengths, (n, n))
    table = seqs.table.copy()
    for i in range(2):
        first = rows[rows[:, 0] == i][0, 3] - 50 + 1
        table[i, :max(0, first) // 16] = (-1, 1 << 29)[i]
    check(pool, fmt, act, query(rng, len(rows), G * H, D, act), seqs, rows, H, 0.1, window=50, table=table, want_status=0)


@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("n", [2, 100])
def test_missing_blocks_are_masked_and_flagged(fmt, act, n):
    lengths, H, G, D = (300, 290), 1, 8, 128
    rng, seqs, pool = setup(n, fmt, act, lengths, 16, H, D)
    rows = chunk_rows(lengths, (n, n))
    table = seqs.table.copy()
    table[0, 3], table[1, 9] = -7, 1 << 29
    check(pool, fmt, act, query(rng, len(rows), G * H, D, act), seqs, rows, H, 0.1, table=table, want_status=2)


@pytest.mark.parametrize("n", [3, 60])
def test_ranges_apart_with_blocks_missing_between(n):
    """Rows next to each other whose ranges lie far apart: what lies between is seen by none of them."""
    rng, seqs, pool = setup(n, "int8_side", "bf16", (900,), 16, 1, 128)
    table = seqs.table.copy()
    table[0, 5:40] = -1
    rows = np.array([(0, 0, 70, 70) if i % 2 else (0, 660, 800 + i, 800 + i) for i in range(n)], dtype=np.int32)
    check(pool, "int8_side", "bf16", query(rng, n, 8, 128, "bf16"), seqs, rows, 1, 0.1, table=table, want_status=0)


def poison(pool, fmt, slot, what, H):
    """NaN or infinity into one dim of a slot's V, or all of its K (the pool and the oracle's copy)."""
    D = pool.V.shape[-1]
    bits = {"bf16": {"nan": 0x7FC0, "inf": 0x7F80, "-inf": 0xFF80}, "f16": {"nan": 0x7E00, "inf": 0x7C00, "-inf": 0xFC00}}
    val = float(what)
    d = 5 if what == "nan" else D - 3
    if fmt == "e4m3":
        pool.cache[1][slot, :, d] = 0x7F
        pool.cache[0][slot] = 0xFF
        pool.V[slot, :, d], pool.K[slot] = np.nan, np.nan
    elif fmt in bits:
        b = np.array(bits[fmt][what], dtype=np.uint16).view(np.int16).item()
        pool.cache[1].view(torch.int16)[slot, :, d] = b
        pool.cache[0].view(torch.int16)[slot] = b
        pool.V[slot, :, d], pool.K[slot] = val, val
    elif fmt == "int8_side":
        pool.kw["k_scale_tok"][slot] = val
        pool.kw["v_scale_tok"][slot] = val
        pool.K[slot], pool.V[slot] = val, val
    else:
        rec = torch.tensor([val], dtype=torch.float32).view(torch.uint8).cuda()
        for x in (0, 1):
            pool.cache[x].view(torch.uint8)[slot, :, D:] = rec
        pool.K[slot], pool.V[slot] = val, val


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("n,D,G", [(2, 128, 8), (5, 128, 3), (130, 128, 8), (130, 256, 16), (300, 128, 1), (40, 256, 7)])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(fmt, act, what, n, D, G):
    """A token in the middle of the new ones holds NaN or infinities in V: the rows before it are as if it did not."""
    lengths, H = (350,), 1
    rng, seqs, pool = setup(n, fmt, act, lengths, 16, H, D)
    at = 350 - (n + 1) // 2
    k_was = pool.K.copy()
    poison(pool, fmt, int(seqs.table[0, at // 16]) * 16 + at % 16, what, H)
    rows = chunk_rows(lengths, (n,))
    for window in (0, 64):
        lo, hi = np.maximum(0, rows[:, 2] - window) if window else 0 * rows[:, 2], rows[:, 2]
        blind = ~((lo <= at) & (at < hi))
        q = query(rng, n, G * H, D, act)
        got = call(pool, fmt, dev16(q, act), seqs, rows, H, D ** -0.5, window=window)
        torch.cuda.synchronize()
        assert got[0][torch.from_numpy(blind).cuda()].isfinite().all() and got[1][torch.from_numpy(blind).cuda()].isfinite().all()
        assert not got[0][torch.from_numpy(~blind).cuda()].isfinite().all()
        # the rows that do not see it, against the oracle; the others are checked with finite keys below
        sub = np.where(blind[:, None], rows, np.array([-1, 0, 0, 0], dtype=np.int32))
        go, gl = got[0].clone(), got[1].clone()
        go[torch.from_numpy(~blind).cuda()] = float("nan")
        gl[torch.from_numpy(~blind).cuda()] = float("nan")
        check(pool, fmt, act, q, seqs, sub, H, D ** -0.5, window=window, got=(go, gl), max_row_end=350, want_status=0)
    if fmt in ("bf16", "f16", "e4m3"):  # K finite again: only the one dim of V of the rows that see it
        pool.K = k_was
        slot = int(seqs.table[0, at // 16]) * 16 + at % 16
        width = pool.cache[0].view(torch.int16 if fmt != "e4m3" else torch.uint8)
        width[slot] = 0
        pool.K[slot] = 0.0
        check(pool, fmt, act, query(rng, n, G * H, D, act), seqs, rows, H, D ** -0.5)
        check(pool, fmt, act, query(rng, n, G * H, D, act), seqs, rows, H, D ** -0.5, window=64)


@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("int8_side", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("n", [1, 90])
def test_rows_far_from_their_keys_keep_their_bias(fmt, act, n):
    """Positions 10^9 past the keys, or before them: the weights are those of the differences."""
    rng, seqs, pool = setup(n, fmt, act, (500,), 16, 1, 128)
    rows = chunk_rows((500,), (n,))
    rows[:, 3] = 1 << 30
    check(pool, fmt, act, query(rng, n, 8, 128, act), seqs, rows, 1, 0.1, slopes=SLOPES(8))
    rows[:, 1], rows[:, 3] = 300, np.arange(n) % 290
    check(pool, fmt, act, query(rng, n, 8, 128, act), seqs, rows, 1, 0.1, slopes=SLOPES(8))


@pytest.mark.parametrize("cap", [2.0 ** -20, 0.01, 1.0, 50.0, 2.0 ** 20])
@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("D", [128, 256])
def test_caps_from_the_smallest_to_the_largest(cap, n, D):
    rng, seqs, pool = setup(3, "int8_side", "bf16", (300,), 16, 1, D)
    rows = chunk_rows((300,), (n,))
    check(pool, "int8_side", "bf16", query(rng, n, 8, D, "bf16", 6.0), seqs, rows, 1, D ** -0.5, softcap=cap)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
@pytest.mark.parametrize("n", [2, 80])
def test_scales(scale, n):
    rng, seqs, pool = setup(5, "e4m3", "bf16", (200,), 16, 1, 128)
    rows = chunk_rows((200,), (n,))
    for cap in (0.0, 10.0):
        check(pool, "e4m3", "bf16", query(rng, n, 4, 128, "bf16"), seqs, rows, 1, scale, softcap=cap)


@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("int8_side", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D,H,G", [(128, 2, 8), (256, 1, 16)])
def test_long_keys_split_over_the_gpu(fmt, act, D, H, G):
    lengths = (5000, 3, 9001)
    rng, seqs, pool = setup(D, fmt, act, lengths, 64, H, D)
    for new in ((1, 1, 1), (9, 3, 20)):
        rows = chunk_rows(lengths, new)
        check(pool, fmt, act, query(rng, len(rows), H * G, D, act), seqs, rows, H, D ** -0.5, softcap=50.0)
        check(pool, fmt, act, query(rng, len(rows), H * G, D, act), seqs, rows, H, D ** -0.5, window=3000, slopes=SLOPES(H * G) / 50)


@pytest.mark.parametrize("n", [1, 70])
def test_rows_in_any_order(n):
    """Rows of sequences that take turns, and the same row twice."""
    lengths = (100, 220, 150)
    rng, seqs, pool = setup(n, "int8_side", "bf16", lengths, 16, 1, 128)
    rows = chunk_rows(lengths, (n, n, n))
    rows = np.concatenate([rows[rng.permutation(len(rows))], rows[:2], rows[:2]])
    check(pool, "int8_side", "bf16", query(rng, len(rows), 8, 128, "bf16"), seqs, rows, 1, 0.1, window=90, slopes=SLOPES(8))


@pytest.mark.parametrize("n", [1, 60])
def test_strided_queries(n):
    import quantized_kv_cache_write_gb300 as qkv
    rng, seqs, pool = setup(n, "e4m3", "bf16", (200,), 16, 1, 128)
    rows = chunk_rows((200,), (n,))
    qb = query(rng, n, 8, 128, "bf16")
    packed = torch.zeros((n, 12, 128), dtype=torch.bfloat16, device="cuda")
    packed[:, 2:10] = dev16(qb, "bf16")
    out = torch.full((n, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = call(pool, "e4m3", packed[:, 2:10], seqs, rows, 1, 0.1, out=out)
    assert qkv.QKV_E4M3 == 3
    check(pool, "e4m3", "bf16", qb, seqs, rows, 1, 0.1, got=got, want_status=0)


@pytest.mark.parametrize("seed", range(40))
def test_seeded_random_batches(seed):
    rng = np.random.default_rng(900 + seed)
    fmt, act = FMTS[seed % len(FMTS)]
    D, H, G = int(rng.choice([128, 256])), int(rng.choice([1, 2, 3])), int(rng.choice([1, 4, 7, 8, 16, 24]))
    block, count = int(rng.choice([1, 3, 16, 64])), int(rng.integers(1, 5))
    lengths = rng.integers(1, 400, count)
    new = [int(min(n, rng.choice([1, 2, 5, 30, 400]))) for n in lengths]
    seqs = Seqs(rng, lengths, block)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, H, D)
    mask = str(rng.choice(["causal", "docs", "prefix"]))
    rows = chunk_rows(lengths, new, mask, int(rng.integers(1, 60)))
    rows[rng.random(len(rows)) < 0.1, 0] = -1
    rows[rng.random(len(rows)) < 0.1, 2] = 0
    check(pool, fmt, act, query(rng, len(rows), H * G, D, act, float(rng.choice([0.3, 1.0, 4.0]))), seqs, rows, H, D ** -0.5,
          window=int(rng.choice([0, 1, 20, 130])), softcap=float(rng.choice([0.0, 8.0, 50.0])),
          slopes=SLOPES(H * G) if rng.random() < 0.5 else None)
