"""qkv_masked_attn where a key that a row sees holds values that are not finite, row by row and head by head (GPU): NaN in K
or in its scale, NaN and infinities in V or in its scale, infinite scores with and without a cap.

One KV head of one token is touched; the other head, and the rows that do not see the token, are as if it were not. Pools,
scales and block tables are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

from dense_harness import assert_within
from masked_harness import Pool, Seqs, bounds, call, check, chunk_rows, dev16, query
from oracle import dense
from oracle.quant import act_bits_to_f32

pytestmark = pytest.mark.gpu

FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16")]
SHAPES = [(3, 128, 3), (130, 128, 8), (70, 256, 16)]
H, DIM, LENGTH, BLOCK = 2, 5, 350, 16
BITS = {"bf16": {"nan": 0x7FC0, "inf": 0x7F80, "-inf": 0xFF80}, "f16": {"nan": 0x7E00, "inf": 0x7C00, "-inf": 0xFC00}}


@pytest.fixture(autouse=True, params=["mma", "tcgen05"])
def tiles(request, monkeypatch):
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", request.param)


def _setup(fmt, act, n, D, G):
    rng = np.random.default_rng(n + D)
    seqs = Seqs(rng, (LENGTH,), BLOCK)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, H, D)
    rows = chunk_rows((LENGTH,), (n,))
    at = LENGTH - (n + 1) // 2  # a token in the middle of the new ones
    slot = int(seqs.table[0, at // BLOCK]) * BLOCK + at % BLOCK
    return rng, seqs, pool, rows, at, slot


def _touch(pool, fmt, which, slot, what):
    """KV head 1 of `slot` in K (0) or V (1): one dim, or the head's scale. The values that it then holds."""
    D = pool.V.shape[-1]
    val = float(what)
    ref = (pool.K, pool.V)[which]
    if fmt in BITS:
        pool.cache[which].view(torch.int16)[slot, 1, DIM] = np.array(BITS[fmt][what], dtype=np.uint16).view(np.int16).item()
        ref[slot, 1, DIM] = val
    elif fmt == "e4m3":
        pool.cache[which][slot, 1, DIM] = 0x7F
        ref[slot, 1, DIM] = np.nan
    else:
        if fmt == "int8_side":
            pool.kw[("k_scale_tok", "v_scale_tok")[which]][slot, 1] = val
        else:
            pool.cache[which].view(torch.uint8)[slot, 1, D:] = torch.tensor([val], dtype=torch.float32).view(torch.uint8).cuda()
        with np.errstate(invalid="ignore"):
            ref[slot, 1] = ref[slot, 1] * val  # code * scale, the scale being positive before
    return val


def _kinds(G):
    return [dict(), dict(window=64), dict(softcap=20.0, slopes=2.0 ** -np.arange(1.0, H * G + 1))]


def _sees(rows, at, window=0, **_):
    lo = np.maximum(0, rows[:, 2] - window) if window else 0 * rows[:, 2]
    return (lo <= at) & (at < rows[:, 2])


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("n,D,G", SHAPES)
def test_nan_in_k(fmt, act, n, D, G):
    """Every output and the log-sum-exp of each row and head that sees it are NaN."""
    rng, seqs, pool, rows, at, slot = _setup(fmt, act, n, D, G)
    _touch(pool, fmt, 0, slot, "nan")
    for kw in _kinds(G):
        q = query(rng, n, H * G, D, act)
        out, lse = check(pool, fmt, act, q, seqs, rows, H, D ** -0.5, **kw)
        sees = torch.from_numpy(_sees(rows, at, **kw)).cuda()
        assert sees.any() and out[sees][:, G:].isnan().all() and lse[sees][:, G:].isnan().all()
        assert out[~sees].isfinite().all() and out[:, :G].isfinite().all()


@pytest.mark.parametrize("fmt,act,what", [(f, a, w) for f, a in FMTS for w in ("nan", "inf", "-inf") if f != "e4m3" or w == "nan"])
@pytest.mark.parametrize("n,D,G", SHAPES)
def test_values_of_v(fmt, act, what, n, D, G):
    """The dim (of an int8 pool: every dim) of each row and head that sees it; the log-sum-exp does not know."""
    rng, seqs, pool, rows, at, slot = _setup(fmt, act, n, D, G)
    _touch(pool, fmt, 1, slot, what)
    value = torch.from_numpy(pool.V[slot, 1]).cuda()
    odd = ~value.isfinite()
    assert odd.any()
    for kw in _kinds(G):
        q = query(rng, n, H * G, D, act)
        out, lse = check(pool, fmt, act, q, seqs, rows, H, D ** -0.5, **kw)
        sees = torch.from_numpy(_sees(rows, at, **kw)).cuda()
        got = out[sees][:, G:].double()
        # infinity times a weight below the smallest number is NaN
        assert (got.isnan() | (got == value))[..., odd].all() and got[..., value.isnan()].isnan().all()
        assert got[..., ~odd].isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("fmt,act", [x for x in FMTS if x[0] != "e4m3"])  # E4M3 has no infinity
@pytest.mark.parametrize("what", ["inf", "-inf"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("n,D,G", SHAPES)
def test_infinite_scores(fmt, act, what, softcap, n, D, G):
    """A key whose score is -infinity has no weight, +infinity makes the row's output and log-sum-exp NaN; under a cap they are
    -softcap and softcap. An int8 key's scale multiplies its codes' product with the query, so that only the product's
    sign is left of it."""
    rng, seqs, pool, rows, at, slot = _setup(fmt, act, n, D, G)
    scale, huge = D ** -0.5, 1e30  # as good as infinite in 64 bits
    clean = pool.K.copy()
    _touch(pool, fmt, 0, slot, what)
    pool.K = clean.copy()
    sign = 1.0 if what == "inf" else -1.0
    if fmt in BITS:
        pool.K[slot, 1, DIM] = sign * huge
    else:
        pool.K[slot, 1] *= sign * huge
    qb = query(rng, n, H * G, D, act)
    widen = act_bits_to_f32(qb, act).astype(np.float64)
    dot, terms = np.einsum("rgd,d->rg", widen, pool.K[slot, 1]), np.einsum("rgd,d->rg", np.abs(widen), np.abs(pool.K[slot, 1]))
    # a sign may be a rounding's where a sum of D products in fp32 is next to 0 (one infinite product has its own sign)
    unsure = np.abs(dot) <= (0 if fmt in BITS else D * 2.0 ** -23 * terms)
    unsure[:, :G] = False
    assert unsure.mean() < 0.01
    up = dot > 0
    up[:, :G] = False
    up &= _sees(rows, at)[:, None]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, fmt, dev16(qb, act), seqs, rows, H, scale, softcap=softcap, status=status)
    torch.cuda.synchronize()
    go, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    lo, hi, pos, pad, _ = dense.masked_rows(rows[:, 0], rows[:, 1], rows[:, 2], rows[:, 3], 0, 1, LENGTH)
    args = (rows[:, 0], lo, hi, pos, pad, seqs.table, BLOCK, scale, softcap, None, act)
    ref = list(dense.masked_attention(qb, pool.K, pool.V, *args))
    # the finite keys' magnitudes bound the errors of their scores; a capped score's own is at most the cap's
    ref[3] = np.maximum(dense.masked_attention(qb, clean, pool.V, *args)[3], softcap)
    o_tol, l_tol = bounds(pool, fmt, act, np.stack([rows[:, 0], lo, hi, pos], 1), ref, softcap, D)
    lost = up & ~unsure if softcap == 0.0 else np.zeros_like(up)
    assert up.any() and np.isnan(go[lost]).all() and np.isnan(gl[lost]).all()
    skip = lost | unsure
    assert_within(np.where(skip[..., None], 0.0, go), np.where(skip[..., None], 0.0, ref[0]), np.where(skip[..., None], 1.0, o_tol), "out")
    assert_within(np.where(skip, 0.0, gl), np.where(skip, 0.0, ref[1]), np.where(skip, 1.0, l_tol), "lse")
    assert int(status.item()) == 0
