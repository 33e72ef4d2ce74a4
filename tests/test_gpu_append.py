"""qkv_append_rope against the oracle (GPU): stored bytes bit for bit, the rotated query within one
rounding, through slot ids and block tables, every format, partial rotations, strides, skipped tokens.

The stored forms are those of "int8 per-(token,head) KV cache for the Qwen3.8-Flash-Next QSA path" §The
finding worth upstreaming and "Qwen3.8 Flash Next NVFP4 QSA FP8 E4M3 KV Scales" §Calibration."""

import numpy as np
import pytest
import torch

from dense_harness import ACT, bits16, dev16
from oracle import dense
from oracle import quant as oq

pytestmark = pytest.mark.gpu

FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_side", "f16"), ("int8_inline", "bf16"),
        ("int8_inline", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")]
KS, VS = np.float32(0.037), np.float32(0.051)


def table(positions, n):
    half = n // 2
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def empty(fmt, S, H, D, fill=0x5A):
    width, dt = (D + 4, np.uint8) if fmt == "int8_inline" else (D, np.uint16 if fmt in ACT else np.uint8)
    return np.frombuffer(bytes([fill]) * (S * H * width * np.dtype(dt).itemsize), dtype=dt).reshape(S, H, width).copy()


def stored(fmt, act, x, pool, scales, slots, layer):
    """Write fp32 rows x [n, H, D] at slots, as the oracle's quantisers store them."""
    if fmt in ACT:
        pool[slots] = bits16(x, fmt)
    elif fmt == "e4m3":
        pool[slots] = oq.e4m3_quantize(x, layer).view(np.uint8)
    else:
        codes, s = oq.int8_quantize(x)
        if fmt == "int8_side":
            pool[slots] = codes.view(np.uint8)
            scales[slots] = s
        else:
            pool[slots] = oq.int8_inline_records(codes, s)


def widen(bits, act):
    return oq.act_bits_to_f32(bits, act)


def run(fmt, act, kb, vb, qb, cs, pos, S, *, pairs=False, slots=None, seq=None, tab=None, block=1, status=None,
        kv=None, inplace=False, stream=None):
    import quantized_kv_cache_write_gb300 as qkv
    T, H, D = kb.shape
    kc, vc = empty(fmt, S, H, D), empty(fmt, S, H, D)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "int8_side": torch.int8}.get(fmt, torch.uint8)
    up = lambda c: torch.from_numpy(c.view(np.int16) if fmt in ACT else c).view(dt).cuda()
    kd, vd = up(kc), up(vc)
    sc = dict(k_scale=torch.full((S, H), -7.0, device="cuda"), v_scale=torch.full((S, H), -7.0, device="cuda")) \
        if fmt == "int8_side" else {}
    k, v = (dev16(kb, act), dev16(vb, act)) if kv is None else kv
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    q = q_out = None
    if qb is not None:
        q = dev16(qb, act)
        q_out = q if inplace else torch.full_like(q, float("nan"))
    qkv.qkv_append_rope(k, v, qkv.FORMATS[fmt], kd, vd, dev(cs), dev(pos), q=q, q_out=q_out, slot_mapping=dev(slots),
                        token_seq=dev(seq), block_table=dev(tab), block_size=block, interleaved=pairs,
                        k_scale_layer=float(KS) if fmt == "e4m3" else 1.0, v_scale_layer=float(VS) if fmt == "e4m3" else 1.0,
                        dev_status=status, stream=stream, **sc)
    torch.cuda.synchronize()
    back = lambda t: t.view(torch.int16 if fmt in ACT else torch.uint8).cpu().numpy()
    return back(kd), back(vd), {n: t.cpu().numpy() for n, t in sc.items()}, q_out


def expect(fmt, act, kb, vb, cs, pos, S, slots, pairs):
    """The pool after the oracle's append of tokens whose slot is >= 0."""
    T, H, D = kb.shape
    kc, vc = empty(fmt, S, H, D), empty(fmt, S, H, D)
    ks, vs = np.full((S, H), -7, np.float32), np.full((S, H), -7, np.float32)
    ok = slots >= 0
    kr = dense.rotate_f32(widen(kb, act), np.maximum(pos, 0), cs, pairs)
    stored(fmt, act, kr[ok], kc, ks, slots[ok], KS)
    stored(fmt, act, widen(vb, act)[ok], vc, vs, slots[ok], VS)
    view = (lambda c: c.view(np.int16)) if fmt in ACT else (lambda c: c)
    return view(kc), view(vc), {"k_scale": ks, "v_scale": vs}


def same(got, want, fmt):
    gk, gv, gs, _ = got
    wk, wv, ws = want
    assert np.array_equal(gk, wk), (fmt, "k", int((gk != wk).sum()))
    assert np.array_equal(gv, wv), (fmt, "v", int((gv != wv).sum()))
    for n in gs:
        assert np.array_equal(gs[n], ws[n]), (fmt, n)


def q_close(q_out, qb, act, cs, pos, pairs, live):
    ref = bits16(dense.rotate_f32(widen(qb, act), np.maximum(pos, 0), cs, pairs), act)
    got = q_out.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(got[live], ref[live])  # fp32 steps and one rounding: the same bits
    return got


def tokens(rng, T, H, D, act):
    x = rng.standard_normal((T, H, D)) * np.where(rng.random((T, 1, 1)) < 0.1, 20.0, 1.0)
    x[rng.random((T, H)) < 0.03] = 0.0  # all-zero heads: scale 0
    return bits16(x, act)


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 16), (128, 96), (256, 256), (256, 64), (256, 240)])
@pytest.mark.parametrize("pairs", [False, True])
def test_formats_and_rotations(fmt, act, D, rot, pairs):
    rng = np.random.default_rng(D + rot)
    T, H, Hq, S = 37, 2, 6, 64
    kb, vb, qb = tokens(rng, T, H, D, act), tokens(rng, T, H, D, act), tokens(rng, T, Hq, D, act)
    cs, pos = table(5000, rot), rng.integers(0, 5000, T).astype(np.int32)
    slots = rng.permutation(S)[:T].astype(np.int64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(fmt, act, kb, vb, qb, cs, pos, S, pairs=pairs, slots=slots, status=status)
    same(got, expect(fmt, act, kb, vb, cs, pos, S, slots, pairs), fmt)
    q_close(got[3], qb, act, cs, pos, pairs, slice(None))
    assert int(status.item()) == 0


@pytest.mark.parametrize("T,Hq,H", [(1, 16, 1), (1, 1, 1), (2, 7, 3), (700, 16, 1), (3001, 5, 2), (1500, 0, 4), (600, 32, 8)])
@pytest.mark.parametrize("D", [128, 256])
def test_sizes_on_both_sides_of_the_rows_per_warp_rule(T, Hq, H, D):
    rng = np.random.default_rng(T + Hq)
    kb, vb = tokens(rng, T, H, D, "bf16"), tokens(rng, T, H, D, "bf16")
    qb = tokens(rng, T, Hq, D, "bf16") if Hq else None
    cs, pos = table(900, 64), rng.integers(0, 900, T).astype(np.int32)
    slots = rng.permutation(T + 5)[:T].astype(np.int64)
    got = run("int8_side", "bf16", kb, vb, qb, cs, pos, T + 5, slots=slots)
    same(got, expect("int8_side", "bf16", kb, vb, cs, pos, T + 5, slots, False), "int8_side")
    if Hq:
        q_close(got[3], qb, "bf16", cs, pos, False, slice(None))


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("block", [1, 7, 16])
def test_paged_with_skipped_and_bad_tokens(fmt, act, block):
    rng = np.random.default_rng(block)
    T, H, Hq, D, seqs, wide = 60, 2, 4, 128, 3, 20
    kb, vb, qb = tokens(rng, T, H, D, act), tokens(rng, T, H, D, act), tokens(rng, T, Hq, D, act)
    S = seqs * wide * block
    tab = rng.permutation(seqs * wide).reshape(seqs, wide).astype(np.int32)
    seq = rng.integers(0, seqs, T).astype(np.int32)
    where = np.stack([rng.permutation(wide * block)[:T] if wide * block >= T else np.arange(T) % (wide * block) for _ in range(seqs)])
    pos = np.array([where[s][t % where.shape[1]] for t, s in enumerate(seq)], dtype=np.int32)
    # every (sequence, position) once
    _, first = np.unique(seq.astype(np.int64) * 10**6 + pos, return_index=True)
    dup = np.setdiff1d(np.arange(T), first)
    pos[dup] = -1
    live_q = pos >= 0
    slots = np.where(pos >= 0, tab[seq, np.maximum(pos, 0) // block].astype(np.int64) * block + np.maximum(pos, 0) % block, -1)
    i = np.flatnonzero(live_q)
    seq[i[0]] = seqs          # no such sequence: q is rotated all the same
    seq[i[1]] = -1
    slots[i[0]] = slots[i[1]] = -1
    # an unallocated block takes every token in it
    gone = (seq[i[2]], pos[i[2]] // block)
    tab[gone] = -3
    hit = (seq == gone[0]) & (pos >= 0) & (pos // block == gone[1])
    slots[hit] = -1
    pos[i[3]] = 900           # past the angle table: skipped whole
    slots[i[3]] = -1
    live_q[i[3]] = False
    pos[i[4]] = -2
    slots[i[4]] = -1
    live_q[i[4]] = False
    cs = table(900, 96)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(fmt, act, kb, vb, qb, cs, pos, S, seq=seq, tab=tab, block=block, status=status)
    same(got, expect(fmt, act, kb, vb, cs, np.where(live_q, pos, 0), S, slots, False), fmt)
    q = q_close(got[3], qb, act, cs, np.where(live_q, pos, 0), False, live_q)
    nan = np.uint16(dev16(bits16(np.full(1, np.nan), act), act).view(torch.int16).cpu().numpy().view(np.uint16)[0])
    assert np.isnan(widen(q[~live_q], act)).all(), nan  # left as they were
    assert int(status.item()) == 1


def test_slot_minus_one_rotates_q_only_and_bad_slots_are_flagged():
    rng = np.random.default_rng(3)
    T, H, Hq, D, S = 12, 1, 4, 256, 16
    kb, vb, qb = (tokens(rng, T, h, D, "bf16") for h in (H, H, Hq))
    cs, pos = table(50, 64), np.arange(T, dtype=np.int32)
    slots = np.arange(T, dtype=np.int64)
    slots[3] = -1
    for bad, want in ((-1, 0), (16, 1), (-2, 1), (1 << 40, 1)):
        slots[5] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run("e4m3", "bf16", kb, vb, qb, cs, pos, S, slots=slots, status=status)
        same(got, expect("e4m3", "bf16", kb, vb, cs, pos, S, np.where((slots >= 0) & (slots < S), slots, -1), False), "e4m3")
        q_close(got[3], qb, "bf16", cs, pos, False, slice(None))
        assert int(status.item()) == want


def test_packed_projection_in_place():
    """q, k and v as slices of one packed tensor; q rotated in place, its neighbours untouched."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(4)
    T, H, Hq, D = 300, 2, 8, 128
    packed_bits = tokens(rng, T, Hq + 2 * H, D, "bf16")
    packed = dev16(packed_bits, "bf16")
    cs, pos = table(700, 128), rng.integers(0, 700, T).astype(np.int32)
    slots = rng.permutation(T).astype(np.int64)
    kc = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v = packed[:, :Hq], packed[:, Hq:Hq + H], packed[:, Hq + H:]
    qkv.qkv_append_rope(k, v, qkv.QKV_BF16, kc, vc, torch.from_numpy(cs).cuda(), torch.from_numpy(pos).cuda(), q=q,
                        q_out=q, slot_mapping=torch.from_numpy(slots).cuda())
    got = packed.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = bits16(dense.rotate_f32(widen(packed_bits[:, :Hq], "bf16"), pos, cs, False), "bf16")
    assert np.array_equal(got[:, :Hq], ref)
    assert np.array_equal(got[:, Hq:], packed_bits[:, Hq:])
    kr = bits16(dense.rotate_f32(widen(packed_bits[:, Hq:Hq + H], "bf16"), pos, cs, False), "bf16")
    assert np.array_equal(kc.view(torch.int16).cpu().numpy().view(np.uint16)[slots], kr)
    assert np.array_equal(vc.view(torch.int16).cpu().numpy().view(np.uint16)[slots], packed_bits[:, Hq + H:])


def test_matches_a_write_of_tokens_that_need_no_rotation():
    """Angle 0 (position 0) leaves the keys as they are: the pool equals the plain write's, bit for bit."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(5)
    T, H, D = 64, 2, 256
    k, v = dev16(tokens(rng, T, H, D, "bf16"), "bf16"), dev16(tokens(rng, T, H, D, "bf16"), "bf16")
    slots = torch.from_numpy(rng.permutation(T).astype(np.int64)).cuda()
    cs = torch.from_numpy(table(4, 256)).cuda()
    a = [torch.zeros((T, H, D), dtype=torch.int8, device="cuda") for _ in range(4)]
    s = [torch.zeros((T, H), dtype=torch.float32, device="cuda") for _ in range(4)]
    qkv.qkv_write_int8(k, v, slots, a[0], a[1], s[0], s[1])
    qkv.qkv_append_rope(k, v, qkv.QKV_INT8_SIDE, a[2], a[3], cs, torch.zeros(T, dtype=torch.int32, device="cuda"),
                        slot_mapping=slots, k_scale=s[2], v_scale=s[3])
    for x, y in ((a[0], a[2]), (a[1], a[3]), (s[0], s[2]), (s[1], s[3])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("seed", range(16))
def test_seeded_random_appends(seed):
    rng = np.random.default_rng(500 + seed)
    fmt, act = FMTS[seed % len(FMTS)]
    D = int(rng.choice([128, 256]))
    H, Hq, T = int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 4, 15, 16, 33])), int(rng.integers(1, 900))
    rot = 16 * int(rng.integers(1, D // 16 + 1))
    pairs = bool(rng.integers(2))
    kb, vb, qb = tokens(rng, T, H, D, act), tokens(rng, T, H, D, act), tokens(rng, T, Hq, D, act)
    cs, pos = table(4000, rot), rng.integers(-1, 4000, T).astype(np.int32)
    slots = rng.permutation(T + 9)[:T].astype(np.int64)
    got = run(fmt, act, kb, vb, qb, cs, pos, T + 9, pairs=pairs, slots=slots, inplace=bool(rng.integers(2)))
    same(got, expect(fmt, act, kb, vb, cs, pos, T + 9, np.where(pos >= 0, slots, -1), pairs), fmt)
    q_close(got[3], qb, act, cs, pos, pairs, pos >= 0)
