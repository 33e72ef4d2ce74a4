"""The tiles of qkv_prefix_attn at their limits (GPU): long ranges of key blocks per tile, scales and values near the
ends of their ranges, and padding and flagged rows where no merge follows.

Compared with the fp64 oracle ("[Perf][SM70][FP8] Hoist QSA E4M3 KV scales" §Changes: hoisted scales; "[Model][SM70]
[FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope: paged storage, split-K workspace)."""

import numpy as np
import pytest
import torch

from dense_harness import ACT, Batch, Pool, bits16, dev16
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


def set_v(pool, codes, scale_bits):
    """V of an int8 pool: codes [S, H, D] and fp32 scales [S, H] into its layout, and their values into pool.V."""
    if pool.fmt == "int8_side":
        pool.cache[1].copy_(codes)
        pool.kw["v_scale_tok"].copy_(scale_bits)
    else:
        D = codes.shape[2]
        pool.cache[1][..., :D] = codes.view(torch.uint8)
        pool.cache[1][..., D:] = scale_bits.contiguous().view(torch.uint8).view(*scale_bits.shape, 4)
    pool.V = codes.cpu().numpy().astype(np.float64) * scale_bits.cpu().numpy().astype(np.float64)[..., None]


@pytest.mark.parametrize("fmt", ["int8_side", "int8_inline"])
@pytest.mark.parametrize("D,rows", [(128, 8), (128, 32), (256, 8), (256, 16)])
@pytest.mark.parametrize("low,high", [(0.0, 2.0 ** 50), (2.0 ** -80, 2.0 ** 98), (2.0 ** -140, 2.0 ** 40)])
def test_blocks_of_tiny_and_huge_v_scales_in_turn(fmt, D, rows, low, high):
    """tcgen05 tiles: runs of 1024 keys whose V scales lie more than 2^126 apart. The weights of the tiny ones' keys
    count in the sum all the same."""
    P = 70001
    rng = np.random.default_rng(41)
    b = Batch(rng, P, [1] * rows, 1, 64)
    pool = Pool(rng, fmt, "bf16", b.live, b.num_slots, 1, D)
    scale = torch.full((b.num_slots, 1), high, device="cuda")
    scale[torch.from_numpy(prefix_slots(b)[np.arange(P) // 1024 % 2 == 0]).cuda()] = low
    codes = torch.from_numpy(rng.integers(64, 128, (b.num_slots, 1, D)).astype(np.int8)).cuda()
    set_v(pool, codes, scale)
    q = bits16(rng.standard_normal((rows, 16, D)), "bf16")
    out, lse = call(pool, b, dev16(q, "bf16"), 1, 0.25 * D ** -0.5)
    check(pool, b, q, "bf16", 1, 0.25 * D ** -0.5, out, lse, what=f"{fmt} {D} {low} {high}")


@pytest.mark.parametrize("fmt", ["int8_side", "int8_inline"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("keys", [512, 4100])
@pytest.mark.parametrize("spare", [0, 900])
def test_sums_of_keys_with_the_largest_v_scales(fmt, D, keys, spare):
    """mma.sync tiles of 16 pairs and (with unused sequences in the table) of 8: V scales of 2^98, and weights that rise
    within the softmax's window. The outputs are 127 2^98, the sums on the way there are 2^30 times that."""
    rng = np.random.default_rng(42)
    rows, G = 420, 16 if spare == 0 else 8
    b = Batch(rng, 0, [keys], 1, 64)
    pool = Pool(rng, fmt, "bf16", b.live, b.num_slots, 1, D)
    b.row_seq, b.row_len = np.zeros(rows, np.int32), np.full(rows, keys, np.int32)
    b.table = np.concatenate([b.table, np.full((spare, b.table.shape[1]), -1, dtype=np.int32)])
    # K = the key's code in every dim, q = 1: logits of code D; the first 128 keys' 5.4 below the others'
    code = np.where(np.arange(keys) < 128, 1, 2)
    p = np.arange(keys)
    slots = torch.from_numpy(b.table[0, p // 64].astype(np.int64) * 64 + p % 64).cuda()
    k = torch.ones((b.num_slots, 1, D), dtype=torch.int8, device="cuda")
    k[slots] = torch.from_numpy(np.broadcast_to(code[:, None, None], (keys, 1, D)).astype(np.int8)).cuda()
    one = torch.ones((b.num_slots, 1), device="cuda")
    if fmt == "int8_side":
        pool.cache[0].copy_(k)
        pool.kw["k_scale_tok"].copy_(one)
    else:
        pool.cache[0][..., :D] = k.view(torch.uint8)
        pool.cache[0][..., D:] = one.view(torch.uint8).view(-1, 1, 4)
    pool.K = k.cpu().numpy().astype(np.float64)
    set_v(pool, torch.full((b.num_slots, 1, D), 127, dtype=torch.int8, device="cuda"), one * 2.0 ** 98)
    q = bits16(np.ones((rows, G, D)), "bf16")
    out, lse = call(pool, b, dev16(q, "bf16"), 1, 5.4 / D)
    check(pool, b, q, "bf16", 1, 5.4 / D, out, lse, what=f"{fmt} {D} {keys}")


@pytest.mark.parametrize("fmt,act", [("e4m3", "bf16"), ("int8_side", "f16"), ("int8_inline", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("prefix,own", [(200, [99, 100, 30]), (201, [100, 99, 3]), (0, [40, 1, 7]), (64, [0, 0, 0])])
@pytest.mark.parametrize("per,spare", [(1, 0), (1, 40), (3, 0), (3, 40)])
def test_both_tile_widths_with_and_without_a_prefix(fmt, act, prefix, own, per, spare):
    """Groups of 4 on mma.sync: prefixes of up to twice the rows' own keys and of more, exact tables and tall ones."""
    rng = np.random.default_rng(43)
    b = Batch(rng, prefix, [max(n, per) if n else 0 for n in own], per, 16)
    if 0 in own:
        b.row_len = np.full_like(b.row_len, prefix)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, 2, 128)
    b.table = np.concatenate([b.table, np.full((spare, b.table.shape[1]), -1, dtype=np.int32)])
    q = bits16(rng.standard_normal((3 * per, 8, 128)), act)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, act), 2, 128 ** -0.5, status=status)
    check(pool, b, q, act, 2, 128 ** -0.5, out, lse, what=f"{fmt} {prefix} {own} {per} {spare}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("D,G,spare", [(256, 16, 0), (128, 4, 0), (128, 4, 40)])
def test_padding_empty_and_bad_rows_without_a_merge(fmt, act, shared, D, G, spare):
    """One range of keys, of the prefix or of the rows' own: its tiles write the outputs themselves, and leave padding
    rows as they were."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(44)
    b = Batch(rng, 50 if shared else 0, [0] * 7 if shared else [50, 1, 49, 50, 7, 50, 33], 1, 16)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, 2, D)
    b.table = np.concatenate([b.table, np.full((spare, b.table.shape[1]), -1, dtype=np.int32)])
    q = bits16(rng.standard_normal((7, 2 * G, D)), act)
    assert qkv.qkv_prefix_attn_workspace(qkv.FORMATS[fmt], 7, 2 * G, 2, D, b.prefix, b.max_row_len) == 0
    seq, ln = b.row_seq.copy(), b.row_len.copy()
    seq[1] = seq[6] = -1     # padding
    seq[2] = 7 + spare       # no such sequence
    ln[3] = 0                # sees nothing
    ln[4] = 49 if shared else 51  # ends inside the prefix; longer than a row may be
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.full((7, 2 * G, D), 7.0, dtype=ACT[act], device="cuda"), torch.full((7, 2 * G), 7.0, device="cuda")
    call(pool, b, dev16(q, act), 2, D ** -0.5, row_seq=seq, row_len=ln, out=out, lse=lse, status=status)
    assert int(status.item()) == 2
    for r in (1, 6):
        assert (out[r] == 7).all() and (lse[r] == 7).all(), r
    for r in (2, 3, 4):
        assert (out[r] == 0).all() and torch.isneginf(lse[r]).all(), r
    check(pool, b, q, act, 2, D ** -0.5, out, lse, row_seq=seq, row_len=np.minimum(ln, b.max_row_len) * np.isin(np.arange(7), (0, 1, 5, 6)),
          what=f"{fmt} {shared} {D} {spare}")
    # without the bad rows nothing is flagged
    seq[2], ln[4] = 2, 0
    status.zero_()
    call(pool, b, dev16(q, act), 2, D ** -0.5, row_seq=seq, row_len=ln, out=out, lse=lse, status=status)
    assert int(status.item()) == 0


# (head dim, rows, groups, prefix): mma.sync tiles of 16 pairs and of 8 (rows alone), tcgen05 tiles on one SM and on two
KINDS = [(128, 6, 16, 90), (128, 6, 4, 0), (256, 6, 16, 0), (128, 8, 16, 70001), (128, 32, 16, 70001), (256, 8, 16, 70001), (256, 16, 16, 70001)]


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,rows,G,prefix", KINDS)
def test_a_query_that_is_not_finite_spoils_its_own_outputs_only(fmt, act, D, rows, G, prefix):
    rng = np.random.default_rng(45)
    b = Batch(rng, prefix, [30 + i for i in range(rows)], 1, 16)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, 1, D)
    q = bits16(rng.standard_normal((rows, G, D)), act)
    qd = dev16(q, act)
    qd[1, 2] = float("nan")
    qd[3, 0, 5] = float("inf")
    qd[4, G - 1, D - 1] = float("-inf")
    out, lse = call(pool, b, qd, 1, D ** -0.5)
    bad = np.zeros((rows, G), dtype=bool)
    bad[1, 2] = bad[3, 0] = bad[4, G - 1] = True
    at = torch.from_numpy(bad).cuda()
    assert not torch.isfinite(out.float()[at]).any() and not torch.isfinite(lse[at]).any()
    ref, ref_lse = call(pool, b, dev16(q, act), 1, D ** -0.5)  # the others as without them, in the last bits too
    assert torch.equal(out.view(torch.int16)[~at], ref.view(torch.int16)[~at]) and torch.equal(lse[~at], ref_lse[~at])
    check(pool, b, q, act, 1, D ** -0.5, ref, ref_lse, what=f"{fmt} {D} {rows}")


@pytest.mark.parametrize("D,rows,G,prefix", KINDS)
def test_values_of_a_bf16_pool_up_to_2_to_the_80(D, rows, G, prefix):
    rng = np.random.default_rng(46)
    b = Batch(rng, prefix, [700 + i for i in range(rows)], 1, 16)
    pool = Pool(rng, "bf16", "bf16", b.live, b.num_slots, 1, D)
    live = torch.from_numpy(b.live).cuda()
    pool.cache[1][live] = (pool.cache[1][live].float().sign() * 2.0 ** 80).to(torch.bfloat16)
    pool.V = np.sign(pool.V) * 2.0 ** 80
    q = bits16(rng.standard_normal((rows, G, D)), "bf16")
    out, lse = call(pool, b, dev16(q, "bf16"), 1, 2 * D ** -0.5)
    check(pool, b, q, "bf16", 1, 2 * D ** -0.5, out, lse, what=f"{D} {rows}")


@pytest.mark.parametrize("fmt", ["e4m3", "int8_side", "int8_inline", "bf16"])
@pytest.mark.parametrize("D,rows,G,prefix", KINDS)
@pytest.mark.parametrize("up", [40, -60])
def test_queries_of_any_magnitude(fmt, D, rows, G, prefix, up):
    """The query is scaled by a power of two into fp16 for byte pools: rows of other magnitudes, in one tile."""
    rng = np.random.default_rng(47)
    b = Batch(rng, prefix, [30 + i for i in range(rows)], 1, 16)
    pool = Pool(rng, fmt, "bf16", b.live, b.num_slots, 1, D)
    x = rng.standard_normal((rows, G, D)) * 2.0 ** -rng.integers(0, 12, (rows, G, 1)) * 2.0 ** -rng.integers(0, 12, (rows, G, D))
    x[0, 0] = 0.0
    x[2, 1, 1:] *= 2.0 ** -30
    q = bits16(x * 2.0 ** up, "bf16")
    scale = 4 * D ** -0.5 * 2.0 ** -up
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale)
    check(pool, b, q, "bf16", 1, scale, out, lse, what=f"{fmt} {D} {rows} {up}")


@pytest.mark.parametrize("fmt,act", [("e4m3", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("D,rows,G,prefix", KINDS)
def test_a_strided_query_and_no_lse(fmt, act, D, rows, G, prefix):
    """The query as a slice of a packed projection whose other columns hold NaN; the log-sum-exps are not asked for."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(48)
    b = Batch(rng, prefix, [30 + i for i in range(rows)], 1, 16)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, 1, D)
    q = bits16(rng.standard_normal((rows, G, D)), act)
    want, _ = call(pool, b, dev16(q, act), 1, D ** -0.5)
    wide = torch.full((rows, G + 5, D), float("nan"), dtype=ACT[act], device="cuda")
    wide[:, 3:3 + G] = dev16(q, act)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    out = torch.full((rows, G, D), float("nan"), dtype=ACT[act], device="cuda")
    need = qkv.qkv_prefix_attn_workspace(qkv.FORMATS[fmt], rows, G, 1, D, prefix, b.max_row_len, device="cuda:0")
    qkv.qkv_prefix_attn(wide[:, 3:3 + G], qkv.FORMATS[fmt], *pool.cache, dev(b.table), dev(b.row_seq), dev(b.row_len), 16,
                        D ** -0.5, max_row_len=b.max_row_len, num_kv_heads=1,
                        prefix_blocks=dev(b.prefix_blocks) if prefix else None, prefix_len=prefix, out=out,
                        workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"), **pool.kw)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("int8_side", "f16")])
@pytest.mark.parametrize("D,rows,G,prefix,at", [(*k, at) for k in KINDS for at in ("own", "prefix") if k[3] or at == "own"])
def test_a_value_that_is_not_finite_shows_though_its_weight_vanishes(fmt, act, D, rows, G, prefix, at):
    """A key that a row sees with a logit far below the others and a V of NaN: 0 x NaN is NaN, wherever the key falls in
    the split of the call into ranges and warps."""
    rng = np.random.default_rng(49)
    b = Batch(rng, prefix, [300 + i for i in range(rows)], 1, 16)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, 1, D)
    p = prefix + 5 if at == "own" else 40
    slots = [int((b.table[i] if at == "own" else b.prefix_blocks)[p // 16]) * 16 + p % 16 for i in range(rows)]
    for s in set(slots):
        if fmt == "int8_side":
            pool.cache[0][s], pool.kw["k_scale_tok"][s], pool.kw["v_scale_tok"][s] = -127, 10.0, float("nan")
        elif fmt == "e4m3":
            pool.cache[0][s], pool.cache[1][s] = 0xFE, 0x7F
        else:
            pool.cache[0][s], pool.cache[1][s] = -64.0, float("nan")
    q = dev16(bits16(np.abs(rng.standard_normal((rows, G, D))) + 0.5, act), act)
    out, lse = call(pool, b, q, 1, 1.0)
    assert torch.isnan(out.float()).all() and torch.isfinite(lse).all()
