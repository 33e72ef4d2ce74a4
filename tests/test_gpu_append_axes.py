"""qkv_append_axes against the oracle (GPU): every stored byte and the rotated query, with each pair turned by its own
axis's position: all formats, runs of pairs and axes in turn, both pairings, both addressings, skipped tokens."""

import numpy as np
import pytest
import torch

import test_gpu_append as base
from dense_harness import dev16

pytestmark = pytest.mark.gpu

FMTS = base.FMTS


def own_angles(cs, axis_pos, pair_axis):
    """A table with a row per token: its pairs' angles, each by its axis (skipped tokens: position 0's)."""
    half = cs.shape[1] // 2
    at = np.maximum(axis_pos[np.asarray(pair_axis)], 0).T  # [T, pairs]
    at = np.where(at < len(cs), at, 0)
    i = np.arange(half)
    return np.concatenate([cs[at, i], cs[at, half + i]], 1)


def run(fmt, act, kb, vb, qb, cs, axis_pos, pair_axis, S, *, pairs=False, slots=None, seq=None, pos=None, tab=None, block=1,
        status=None, inplace=False):
    import quantized_kv_cache_write_gb300 as qkv
    H, D = kb.shape[1:]
    kc, vc = base.empty(fmt, S, H, D), base.empty(fmt, S, H, D)
    is16 = fmt in ("bf16", "f16")
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "int8_side": torch.int8}.get(fmt, torch.uint8)
    kd, vd = (torch.from_numpy(c.view(np.int16) if is16 else c).view(dt).cuda() for c in (kc, vc))
    sc = dict(k_scale=torch.full((S, H), -7.0, device="cuda"), v_scale=torch.full((S, H), -7.0, device="cuda")) \
        if fmt == "int8_side" else {}
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q = q_out = None
    if qb is not None:
        q = dev16(qb, act)
        q_out = q if inplace else torch.full_like(q, float("nan"))
    qkv.qkv_append_axes(dev16(kb, act), dev16(vb, act), qkv.FORMATS[fmt], kd, vd, dev(cs), dev(axis_pos), pair_axis, q=q,
                        q_out=q_out, slot_mapping=dev(slots), token_seq=dev(seq), token_pos=dev(pos), block_table=dev(tab),
                        block_size=block, interleaved=pairs, k_scale_layer=float(base.KS) if fmt == "e4m3" else 1.0,
                        v_scale_layer=float(base.VS) if fmt == "e4m3" else 1.0, dev_status=status, **sc)
    torch.cuda.synchronize()
    back = lambda t: t.view(torch.int16 if is16 else torch.uint8).cpu().numpy()  # noqa: E731
    return back(kd), back(vd), {n: t.cpu().numpy() for n, t in sc.items()}, q_out


def layouts(rot, axes):
    half = rot // 2
    runs = [min(axes - 1, i * axes // half) for i in range(half)]
    return {"runs": runs, "turn": [i % axes for i in range(half)],
            "odd": [0 if i < 3 else (i * i) % axes for i in range(half)]}


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 48), (256, 240), (256, 16)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("layout,axes", [("runs", 3), ("turn", 3), ("odd", 4)])
def test_formats_pairings_and_layouts(fmt, act, D, rot, pairs, layout, axes):
    rng = np.random.default_rng(D + rot + axes)
    T, H, Hq, S = 37, 2, 6, 64
    kb, vb, qb = base.tokens(rng, T, H, D, act), base.tokens(rng, T, H, D, act), base.tokens(rng, T, Hq, D, act)
    cs, axis_pos = base.table(5000, rot), rng.integers(0, 5000, (axes, T)).astype(np.int32)
    pair_axis = layouts(rot, axes)[layout]
    slots = rng.permutation(S)[:T].astype(np.int64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(fmt, act, kb, vb, qb, cs, axis_pos, pair_axis, S, pairs=pairs, slots=slots, status=status)
    own, idx = own_angles(cs, axis_pos, pair_axis), np.arange(T, dtype=np.int32)
    base.same(got, base.expect(fmt, act, kb, vb, own, idx, S, slots, pairs), fmt)
    base.q_close(got[3], qb, act, own, idx, pairs, slice(None))
    assert int(status.item()) == 0


@pytest.mark.parametrize("T,Hq,H,D", [(1, 16, 1, 256), (700, 16, 1, 256), (3001, 5, 2, 128), (1500, 0, 4, 128), (600, 32, 8, 128)])
@pytest.mark.parametrize("axes", [1, 2, 3])
def test_sizes_on_both_sides_of_the_rows_per_warp_rule(T, Hq, H, D, axes):
    rng = np.random.default_rng(T + Hq)
    kb, vb = base.tokens(rng, T, H, D, "bf16"), base.tokens(rng, T, H, D, "bf16")
    qb = base.tokens(rng, T, Hq, D, "bf16") if Hq else None
    cs, axis_pos = base.table(900, 96), rng.integers(0, 900, (axes, T)).astype(np.int32)
    pair_axis = layouts(96, axes)["runs"]
    slots = rng.permutation(T + 5)[:T].astype(np.int64)
    got = run("int8_side", "bf16", kb, vb, qb, cs, axis_pos, None if axes == 1 else pair_axis, T + 5, slots=slots)
    own, idx = own_angles(cs, axis_pos, pair_axis), np.arange(T, dtype=np.int32)
    base.same(got, base.expect("int8_side", "bf16", kb, vb, own, idx, T + 5, slots, False), "int8_side")
    if Hq:
        base.q_close(got[3], qb, "bf16", own, idx, False, slice(None))


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("pairs", [False, True])
def test_axes_that_agree_equal_the_plain_append(fmt, act, pairs):
    """Bit for bit, whatever the pairs' axes."""
    rng = np.random.default_rng(7)
    T, H, Hq, D, S = 90, 2, 6, 128, 100
    kb, vb, qb = base.tokens(rng, T, H, D, act), base.tokens(rng, T, H, D, act), base.tokens(rng, T, Hq, D, act)
    cs, pos = base.table(700, 64), rng.integers(-1, 700, T).astype(np.int32)
    slots = rng.permutation(S)[:T].astype(np.int64)
    want = base.run(fmt, act, kb, vb, qb, cs, pos, S, pairs=pairs, slots=slots)
    got = run(fmt, act, kb, vb, qb, cs, np.stack([pos] * 3), layouts(64, 3)["turn"], S, pairs=pairs, slots=slots)
    for a, b in zip(got[:2], want[:2]):
        assert np.array_equal(a, b)
    assert all(np.array_equal(got[2][n], want[2][n]) for n in want[2])
    assert torch.equal(got[3].view(torch.int16), want[3].view(torch.int16))


@pytest.mark.parametrize("fmt,act", [("int8_inline", "f16"), ("e4m3", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("block", [1, 7, 16])
def test_paged_with_skipped_and_bad_tokens(fmt, act, block):
    rng = np.random.default_rng(block)
    T, H, Hq, D, seqs, wide = 50, 2, 4, 128, 3, 20
    kb, vb, qb = base.tokens(rng, T, H, D, act), base.tokens(rng, T, H, D, act), base.tokens(rng, T, Hq, D, act)
    S = seqs * wide * block
    tab = rng.permutation(seqs * wide).reshape(seqs, wide).astype(np.int32)
    seq, pos = (np.arange(T) % seqs).astype(np.int32), (np.arange(T) // seqs).astype(np.int32)
    axis_pos = rng.integers(0, 900, (3, T)).astype(np.int32)
    slots = tab[seq, pos // block].astype(np.int64) * block + pos % block
    live = np.ones(T, dtype=bool)
    for i, axis, bad in ((3, 0, -1), (4, 0, 900), (5, 1, -1), (6, 2, 1 << 30), (7, 1, -5)):  # skipped whole
        axis_pos[axis, i] = bad
        live[i], slots[i] = False, -1
    for i, name, bad in ((10, "seq", seqs), (11, "seq", -1), (12, "pos", -1), (13, "pos", wide * block), (14, "pos", -2)):
        {"seq": seq, "pos": pos}[name][i] = bad  # K and V are not stored, q is rotated
        slots[i] = -1
    gone = (seq[20], pos[20] // block)
    tab[gone] = -1
    slots[(seq == gone[0]) & (pos >= 0) & (pos // block == gone[1])] = -1
    cs, pair_axis = base.table(900, 96), layouts(96, 3)["turn"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(fmt, act, kb, vb, qb, cs, axis_pos, pair_axis, S, seq=seq, pos=pos, tab=tab, block=block, status=status)
    own, idx = own_angles(cs, axis_pos, pair_axis), np.arange(T, dtype=np.int32)
    base.same(got, base.expect(fmt, act, kb, vb, own, idx, S, slots, False), fmt)
    q = base.q_close(got[3], qb, act, own, idx, False, live)
    assert np.isnan(base.widen(q[~live], act)).all()  # left as they were
    assert int(status.item()) == 1


@pytest.mark.parametrize("axis,bad,flag", [(0, -1, 0), (0, -2, 1), (1, -1, 1), (1, 900, 1), (2, 1 << 30, 1)])
def test_what_is_flagged(axis, bad, flag):
    rng = np.random.default_rng(1)
    kb, vb = base.tokens(rng, 2, 1, 128, "bf16"), base.tokens(rng, 2, 1, 128, "bf16")
    axis_pos = np.full((3, 2), 5, dtype=np.int32)
    axis_pos[axis, 1] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs, pa = base.table(900, 32), layouts(32, 3)["runs"]
    slots = np.array([1, 0])
    got = run("int8_side", "bf16", kb, vb, None, cs, axis_pos, pa, 2, slots=slots, status=status)
    base.same(got, base.expect("int8_side", "bf16", kb, vb, own_angles(cs, axis_pos, pa), np.arange(2, dtype=np.int32), 2,
                               np.array([1, -1]), False), "int8_side")
    assert int(status.item()) == flag


def test_no_tokens():
    e = np.zeros((0, 1, 128), dtype=np.uint16)
    run("int8_side", "bf16", e, e, None, base.table(9, 32), np.zeros((3, 0), dtype=np.int32), layouts(32, 3)["runs"], 4,
        slots=np.zeros(0, dtype=np.int64))
