"""qkv_read against the oracle (GPU): every format into every type, through slot ids and block tables, K turned back by one
or more axes, skipped and invalid tokens, strides; and the round trip of a document to other positions."""

import numpy as np
import pytest
import torch

import test_gpu_append as base
from dense_harness import Pool, bits16
from oracle import dense
from test_gpu_append_axes import layouts, own_angles

pytestmark = pytest.mark.gpu

FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16")]
OUT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def read(pool, fmt, T, H, D, out, *, which="kv", stride=None, **kw):
    """k_out and v_out, filled with NaN before."""
    import quantized_kv_cache_write_gb300 as qkv
    got = {}
    for x in which:
        got[x + "_out"] = torch.full((T, stride or H * D), float("nan"), dtype=OUT[out], device="cuda")[:, :H * D].unflatten(1, (H, D))
    scales = {n.replace("_tok", ""): t for n, t in pool.kw.items()}
    qkv.qkv_read(qkv.FORMATS[fmt], *pool.cache, **got, **scales, **kw)
    torch.cuda.synchronize()
    return got


def rounded(x, out):
    """fp32 values as the output's type holds them."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(OUT[out])


def values(pool, x, slots):
    """The fp32 rows that the pool holds: a product of an exact code and an fp32 scale, rounded once."""
    return (pool.K if x == "k" else pool.V)[slots].astype(np.float32)


def equal(got, want):
    got = got.cpu()
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,H", [(128, 1), (128, 3), (256, 2)])
def test_formats_and_types(fmt, act, out, D, H):
    rng = np.random.default_rng(D + H)
    S, T = 70, 41
    pool = Pool(rng, fmt, act, np.arange(S), S, H, D)
    slots = rng.integers(0, S, T)  # some twice
    got = read(pool, fmt, T, H, D, out, slot_mapping=dev(slots))
    for x in "kv":
        equal(got[x + "_out"], rounded(values(pool, x, slots), out))


@pytest.mark.parametrize("T,H,D", [(1, 1, 256), (1, 8, 128), (5000, 1, 256), (3000, 5, 128), (9000, 1, 128)])
@pytest.mark.parametrize("which", ["kv", "k", "v"])
def test_sizes_on_both_sides_of_the_rows_per_warp_rule(T, H, D, which):
    rng = np.random.default_rng(T)
    pool = Pool(rng, "int8_side", "bf16", np.arange(T), T, H, D)
    slots = rng.permutation(T)
    got = read(pool, "int8_side", T, H, D, "bf16", which=which, stride=H * D + 8, slot_mapping=dev(slots))
    for x in which:
        equal(got[x + "_out"], rounded(values(pool, x, slots), "bf16"))


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot,axes", [(128, 128, 1), (128, 48, 3), (256, 240, 2), (256, 64, 1)])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_keys_turned_back(fmt, act, pairs, D, rot, axes, out):
    rng = np.random.default_rng(rot)
    S, T, H = 60, 33, 2
    pool = Pool(rng, fmt, act, np.arange(S), S, H, D)
    slots = rng.permutation(S)[:T]
    cs, axis_pos = base.table(3000, rot), rng.integers(0, 3000, (axes, T)).astype(np.int32)
    pair_axis = layouts(rot, axes)["turn"]
    got = read(pool, fmt, T, H, D, out, slot_mapping=dev(slots), cos_sin=dev(cs), axis_pos=dev(axis_pos),
               pair_axis=pair_axis if axes > 1 else None, interleaved=pairs)
    own = own_angles(cs, axis_pos, pair_axis)
    own[:, rot // 2:] *= -1
    equal(got["k_out"], rounded(dense.rotate_f32(values(pool, "k", slots), np.arange(T), own, pairs), out))
    equal(got["v_out"], rounded(values(pool, "v", slots), out))


@pytest.mark.parametrize("fmt,act", [("int8_side", "bf16"), ("int8_inline", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("block", [1, 7, 16])
@pytest.mark.parametrize("turned", [False, True])
def test_paged_with_skipped_and_bad_tokens(fmt, act, block, turned):
    rng = np.random.default_rng(block)
    T, H, D, seqs, wide = 50, 2, 128, 3, 20
    S = seqs * wide * block
    pool = Pool(rng, fmt, act, np.arange(S), S, H, D)
    tab = rng.permutation(seqs * wide).reshape(seqs, wide).astype(np.int32)
    seq, pos = (np.arange(T) % seqs).astype(np.int32), (np.arange(T) // seqs).astype(np.int32)
    slots = tab[seq, pos // block].astype(np.int64) * block + pos % block
    axis_pos = rng.integers(0, 900, (2, T)).astype(np.int32)
    for i, name, bad in ((10, "seq", seqs), (11, "seq", -1), (12, "pos", -1), (13, "pos", wide * block), (14, "pos", -2)):
        {"seq": seq, "pos": pos}[name][i] = bad
        slots[i] = -1
    for i, axis, bad in ((3, 0, -1), (4, 0, 900), (5, 1, -1)):
        axis_pos[axis, i] = bad
        if turned:
            slots[i] = -1
    tab[seq[20], pos[20] // block] = -1
    slots[(seq == seq[20]) & (pos >= 0) & (pos // block == pos[20] // block)] = -1
    tab[seq[31], pos[31] // block] = S  # past the pool
    slots[(seq == seq[31]) & (pos >= 0) & (pos // block == pos[31] // block)] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs, pair_axis = base.table(900, 96), layouts(96, 2)["runs"]
    kw = dict(cos_sin=dev(cs), axis_pos=dev(axis_pos), pair_axis=pair_axis) if turned else {}
    got = read(pool, fmt, T, H, D, "f32", token_seq=dev(seq), token_pos=dev(pos), block_table=dev(tab), block_size=block,
               dev_status=status, **kw)
    live = slots >= 0
    k = values(pool, "k", np.maximum(slots, 0))
    if turned:
        own = own_angles(cs, axis_pos, pair_axis)
        own[:, 48:] *= -1
        k = dense.rotate_f32(k, np.arange(T), own, False)
    nan = np.float32(np.nan)  # left as they were
    equal(got["k_out"], rounded(np.where(live[:, None, None], k, nan), "f32"))
    equal(got["v_out"], rounded(np.where(live[:, None, None], values(pool, "v", np.maximum(slots, 0)), nan), "f32"))
    assert int(status.item()) == 2


@pytest.mark.parametrize("bad,flag", [(-1, 0), (-2, 2), (9, 2), (1 << 40, 2)])
def test_what_is_flagged(bad, flag):
    pool = Pool(np.random.default_rng(0), "e4m3", "bf16", np.arange(9), 9, 1, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = read(pool, "e4m3", 2, 1, 128, "bf16", slot_mapping=dev(np.array([4, bad])), dev_status=status)
    equal(got["v_out"][0], rounded(values(pool, "v", 4), "bf16"))
    assert got["k_out"][1].isnan().all() and got["v_out"][1].isnan().all()
    assert int(status.item()) == flag


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_a_pool_of_16_bits_into_its_own_type_is_copied_bit_for_bit(fmt):
    """NaN payloads and infinities too."""
    import quantized_kv_cache_write_gb300 as qkv
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(256, 2, 128).cuda()
    pool = bits.view(OUT[fmt])
    k, v = torch.zeros_like(pool), torch.zeros_like(pool)
    qkv.qkv_read(qkv.FORMATS[fmt], pool, pool, k_out=k, v_out=v, slot_mapping=torch.arange(256, device="cuda"))
    assert torch.equal(k.view(torch.int16), bits) and torch.equal(v.view(torch.int16), bits)


def test_all_e4m3_codes():
    import quantized_kv_cache_write_gb300 as qkv
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(2, 1, 128).cuda()
    k = torch.zeros((2, 1, 128), device="cuda")
    qkv.qkv_read(qkv.QKV_E4M3, codes, codes, k_out=k, slot_mapping=torch.arange(2, device="cuda"), k_scale_layer=0.3)
    equal(k, (codes.cpu().view(torch.float8_e4m3fn).float() * torch.tensor(0.3)))


def test_a_document_moved_to_other_positions():
    """Appended, read back unturned, appended elsewhere: its keys are those of an append at the new positions, up to the
    roundings on the way: two of bf16 (the first append's and the read's) and the rotations' own, a few fp32 steps."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(9)
    T, H, D, S = 120, 2, 128, 300
    kb, vb = (bits16(rng.standard_normal((T, H, D)), "bf16") for _ in range(2))
    k, v = (dev(x.view(np.int16)).view(torch.bfloat16) for x in (kb, vb))
    cs = dev(base.table(4000, 128))
    old, new = np.arange(T, dtype=np.int32) + 1000, np.arange(T, dtype=np.int32) + 17
    kc, vc = (torch.zeros((S, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    first, second = dev(np.arange(T)), dev(np.arange(T) + 150)
    qkv.qkv_append_rope(k, v, qkv.QKV_BF16, kc, vc, cs, dev(old), slot_mapping=first)
    k1, v1 = torch.empty_like(k), torch.empty_like(v)
    qkv.qkv_read(qkv.QKV_BF16, kc, vc, k_out=k1, v_out=v1, slot_mapping=first, cos_sin=cs, axis_pos=dev(old[None]))
    qkv.qkv_append_rope(k1, v1, qkv.QKV_BF16, kc, vc, cs, dev(new), slot_mapping=second)
    assert torch.equal(vc[150:150 + T], v)
    x = base.widen(kb, "bf16").astype(np.float64)
    want = dense.rotate_f32(x.astype(np.float32), new, base.table(4000, 128), False).astype(np.float64)
    pair = np.sqrt(x[..., :64] ** 2 + x[..., 64:] ** 2)
    # each of the three bf16 roundings moves a pair by at most 2^-8 of its length; tables and rotations: 2^-18
    tol = np.concatenate([pair, pair], -1) * (3 * 2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -18)
    err = np.abs(kc[150:150 + T].float().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())
