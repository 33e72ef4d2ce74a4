"""qkv_prefix_attn against the fp64 oracle (GPU): formats, head dims and groups, one key to thousands,
odd block sizes, prefixes that end inside a block, rows that see nothing, leftovers in unused slots.

The shared prefix is read through its own block list and the rest through the block table ("[Model][SM70]
[FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope: paged storage, split-K workspace;
"[Perf][SM70][FP8] Hoist QSA E4M3 KV scales" §Changes: hoisted scales)."""

import numpy as np
import pytest
import torch

from dense_harness import ACT, Batch, Pool, assert_within, attention_bounds, bits16, dev16
from oracle import dense

pytestmark = pytest.mark.gpu

FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_side", "f16"), ("int8_inline", "bf16"),
        ("int8_inline", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")]


def call(pool, b, q, H, scale, *, row_seq=None, row_len=None, out=None, lse=None, status=None, max_row_len=None,
         ws_extra=0, stream=None, workspace=None):
    import quantized_kv_cache_write_gb300 as qkv
    R, Hq, D = q.shape
    fmt = qkv.FORMATS[pool.fmt]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    max_len = b.max_row_len if max_row_len is None else max_row_len
    need = qkv.qkv_prefix_attn_workspace(fmt, R, Hq, H, D, b.prefix, max_len)
    out = torch.full((R, Hq, D), float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((R, Hq), float("nan"), dtype=torch.float32, device="cuda") if lse is None else lse
    # whatever a workspace holds before the call must not matter
    ws = torch.full((need + ws_extra,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    qkv.qkv_prefix_attn(q, fmt, *pool.cache, dev(b.table), dev(b.row_seq if row_seq is None else row_seq),
                        dev(b.row_len if row_len is None else row_len), b.block, scale, max_row_len=max_len,
                        num_kv_heads=H, prefix_blocks=dev(b.prefix_blocks) if b.prefix else None, prefix_len=b.prefix,
                        out=out, lse=lse, workspace=ws, dev_status=status, stream=stream, **pool.kw)
    torch.cuda.synchronize()
    return out, lse


def check(pool, b, q_bits, act, H, scale, out, lse, row_seq=None, row_len=None, what=""):
    row_seq = b.row_seq if row_seq is None else row_seq
    row_len = b.row_len if row_len is None else row_len
    slots, _ = dense.row_slots(row_seq, row_len, b.prefix_blocks, b.prefix, b.table, b.block, pool.num_slots)
    ref, rlse, wabs, big = dense.prefix_attention(q_bits, pool.K, pool.V, slots, scale, act)
    live = np.array([s is not None for s in slots])
    vmax = float(np.abs(pool.V[b.live]).max()) if len(b.live) else 0.0
    n = max((len(s) for s in slots if s), default=0)
    tol, ltol = attention_bounds(ref, rlse, wabs, big, n, vmax, act, pool.fmt, q_bits.shape[2])
    assert_within(out.float().cpu().numpy()[live], ref[live], tol[live], what + " out")
    assert_within(lse.cpu().numpy()[live], rlse[live], ltol[live], what + " lse")
    return live


def case(seed, fmt, act, D, H, G, prefix, own, per, block, scale=None):
    rng = np.random.default_rng(seed)
    b = Batch(rng, prefix, own, per, block)
    pool = Pool(rng, fmt, act, b.live, b.num_slots, H, D)
    q_bits = bits16(rng.standard_normal((len(own) * per, H * G, D)), act)
    return b, pool, q_bits, (D ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D", [128, 256])
def test_formats(fmt, act, D):
    b, pool, q, scale = case(1, fmt, act, D, 2, 8, 333, [1, 200, 77, 0, 64], 1, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, act), 2, scale, status=status)
    check(pool, b, q, act, 2, scale, out, lse, what=f"{fmt} {act} {D}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 12, 16, 17, 33, 128])
@pytest.mark.parametrize("per", [1, 4])
def test_groups(G, per):
    b, pool, q, scale = case(2, "int8_side", "bf16", 128, 2, G, 150, [40, 9, 4], per, 16)
    out, lse = call(pool, b, dev16(q, "bf16"), 2, scale)
    check(pool, b, q, "bf16", 2, scale, out, lse, what=f"G {G} per {per}")


@pytest.mark.parametrize("prefix,own", [(0, [1]), (1, [0]), (1, [1]), (15, [2, 0]), (16, [16]), (17, [1, 31]), (0, [63, 64, 65]),
                                        (127, [1, 1]), (128, [129]), (129, [0, 0]), (255, [1]), (2049, [1, 700]),
                                        (0, [1, 3001]), (700, [1000, 1])])
@pytest.mark.parametrize("fmt", ["e4m3", "int8_side", "bf16"])
def test_lengths(prefix, own, fmt):
    b, pool, q, scale = case(3, fmt, "bf16", 128, 1, 8, prefix, own, 1, 16)
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale)
    check(pool, b, q, "bf16", 1, scale, out, lse, what=f"{fmt} {prefix} {own}")


@pytest.mark.parametrize("block", [1, 3, 7, 16, 100, 257])
def test_block_sizes(block):
    b, pool, q, scale = case(4, "e4m3", "f16", 256, 1, 16, 301, [5, 90, 260], 5, block)
    out, lse = call(pool, b, dev16(q, "f16"), 1, scale)
    check(pool, b, q, "f16", 1, scale, out, lse, what=f"block {block}")


@pytest.mark.parametrize("rows", [1, 2, 9, 33, 70])
@pytest.mark.parametrize("D,fmt,act", [(128, "e4m3", "bf16"), (256, "int8_side", "f16"), (128, "bf16", "bf16"), (256, "f16", "f16")])
def test_batches(rows, D, fmt, act):
    b, pool, q, scale = case(5, fmt, act, D, 2, 8, 600, [1 + i % 5 for i in range(rows)], 1, 32)
    out, lse = call(pool, b, dev16(q, act), 2, scale)
    check(pool, b, q, act, 2, scale, out, lse, what=f"rows {rows}")


@pytest.mark.parametrize("fmt,act", FMTS)
def test_draft_rows_of_one_sequence_with_leftovers_behind_the_shorter_ones(fmt, act):
    """Rows of one tile see different lengths; the key that only the last row sees holds infinities and
    NaN (a rejected draft's leftovers): the other rows must not notice."""
    b, pool, q, scale = case(6, fmt, act, 128, 1, 4, 40, [7, 30, 4], 4, 16)
    for i in range(3):
        n = int(b.row_len[4 * i + 3])
        slot = int(b.table[i, (n - 1) // 16]) * 16 + (n - 1) % 16
        raw = pool.cache[1].view(torch.uint8)
        raw[slot] = 0x7F if fmt != "int8_inline" else raw[slot]
        if fmt == "int8_side":
            pool.kw["v_scale_tok"][slot] = float("nan")
        if fmt == "int8_inline":
            raw[slot, :, 128:] = 0xFF  # a NaN scale
        if fmt == "bf16":
            pool.cache[1][slot] = float("inf")
        if fmt == "f16":
            pool.cache[1][slot] = float("-inf")
    out, lse = call(pool, b, dev16(q, act), 1, scale)
    first = np.arange(12) % 4 != 3
    seq, ln = b.row_seq[first], b.row_len[first]
    slots, _ = dense.row_slots(seq, ln, b.prefix_blocks, b.prefix, b.table, b.block, pool.num_slots)
    ref, rlse, wabs, big = dense.prefix_attention(q[first], pool.K, pool.V, slots, scale, act)
    vmax = float(np.abs(pool.V[b.live]).max())
    tol, ltol = attention_bounds(ref, rlse, wabs, big, 80, vmax, act, fmt, 128)
    assert_within(out.float().cpu().numpy()[first], ref, tol, "rows before the leftovers")
    assert_within(lse.cpu().numpy()[first], rlse, ltol, "lse before the leftovers")
    assert not torch.isfinite(out.float()[torch.from_numpy(~first).cuda()]).any()


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (256, 2)])
def test_draft_rows_in_a_large_table(fmt, act, D, G):
    """Few rows and many sequences (tiles of eight pairs): draft rows of one sequence share a tile, and the key that
    only the last of them sees holds a NaN of its own."""
    b, pool, q, scale = case(16, fmt, act, D, 2, G, 40, [7, 150, 4], 4, 16)
    b.table = np.concatenate([b.table, np.full((30, b.table.shape[1]), -1, dtype=np.int32)])
    for i in range(3):
        n = int(b.row_len[4 * i + 3])
        slot = int(b.table[i, (n - 1) // 16]) * 16 + (n - 1) % 16
        if fmt == "int8_side":
            pool.kw["v_scale_tok"][slot] = float("nan")
        elif fmt == "int8_inline":
            pool.cache[1].view(torch.uint8)[slot, :, D:] = 0xFF  # a NaN scale
        elif fmt == "e4m3":
            pool.cache[1].view(torch.uint8)[slot] = 0x7F
        else:
            pool.cache[1][slot] = float("nan")
    out, lse = call(pool, b, dev16(q, act), 2, scale)
    first = np.arange(12) % 4 != 3
    slots, _ = dense.row_slots(b.row_seq[first], b.row_len[first], b.prefix_blocks, b.prefix, b.table, b.block, pool.num_slots)
    ref, rlse, wabs, big = dense.prefix_attention(q[first], pool.K, pool.V, slots, scale, act)
    tol, ltol = attention_bounds(ref, rlse, wabs, big, 190, float(np.abs(pool.V[b.live]).max()), act, fmt, D)
    assert_within(out.float().cpu().numpy()[first], ref, tol, "rows before the leftovers")
    assert_within(lse.cpu().numpy()[first], rlse, ltol, "lse before the leftovers")
    assert torch.isnan(out.float()[torch.from_numpy(~first).cuda()]).all()


def test_empty_padding_and_bad_rows():
    b, pool, q, scale = case(7, "int8_side", "bf16", 256, 1, 16, 50, [20, 30, 10, 5, 8, 9], 1, 16)
    for max_parts in (False, True):  # with and without keys of their own
        seq, ln = b.row_seq.copy(), b.row_len.copy()
        ln[0] = 0            # sees nothing
        seq[1] = -1          # padding
        seq[2] = 6           # no such sequence
        ln[3] = 49           # ends inside the prefix
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((6, 16, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((6, 16), 7.0, dtype=torch.float32, device="cuda")
        call(pool, b, dev16(q, "bf16"), 1, scale, row_seq=seq, row_len=ln, out=out, lse=lse, status=status)
        assert int(status.item()) == 2
        for r in (0, 2, 3):
            assert (out[r] == 0).all() and torch.isneginf(lse[r]).all(), r
        assert (out[1] == 7).all() and (lse[1] == 7).all()
        keep = np.array([4, 5])
        slots, _ = dense.row_slots(seq[keep], ln[keep], b.prefix_blocks, b.prefix, b.table, b.block, pool.num_slots)
        ref, rlse, wabs, big = dense.prefix_attention(q[keep], pool.K, pool.V, slots, scale)
        tol, ltol = attention_bounds(ref, rlse, wabs, big, 100, float(np.abs(pool.V[b.live]).max()), "bf16", "int8_side", 256)
        assert_within(out.float().cpu().numpy()[keep], ref, tol, "out")
        assert_within(lse.cpu().numpy()[keep], rlse, ltol, "lse")


@pytest.mark.parametrize("prefix", [0, 40])
def test_every_row_empty(prefix):
    """max_row_len as small as it may be; one part of keys or none."""
    b, pool, q, scale = case(8, "e4m3", "bf16", 128, 1, 8, prefix, [1, 1], 1, 16)
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale, row_len=np.zeros(2, np.int32), max_row_len=prefix)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("own", [[0, 0], [3, 40]])
def test_unallocated_blocks_and_slots_past_the_pool_are_masked_and_flagged(own):
    b, pool, q, scale = case(9, "int8_side", "bf16", 128, 1, 16, 100, own, 1, 16)
    b.prefix_blocks[2] = -1
    b.prefix_blocks[4] = 1 << 26
    if own[1]:
        b.table[1, 100 // 16 + 1] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale, status=status)
    check(pool, b, q, "bf16", 1, scale, out, lse, what="bad blocks")
    assert int(status.item()) == 2


def test_every_block_of_the_prefix_unallocated():
    b, pool, q, scale = case(10, "bf16", "bf16", 128, 1, 8, 64, [0, 3], 1, 16)
    b.prefix_blocks[:] = -1
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale)
    check(pool, b, q, "bf16", 1, scale, out, lse, what="no prefix block")
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("scale", [-0.1, 0.0, 2.0])
@pytest.mark.parametrize("fmt,act", [("int8_side", "bf16"), ("e4m3", "f16"), ("bf16", "bf16"), ("f16", "f16")])
def test_scales_of_either_sign(scale, fmt, act):
    b, pool, q, _ = case(11, fmt, act, 128, 1, 16, 90, [4, 50], 1, 16)
    out, lse = call(pool, b, dev16(q, act), 1, scale)
    check(pool, b, q, act, 1, scale, out, lse, what=f"scale {scale}")


def test_strided_query_and_status_and_repeatability():
    b, pool, q, scale = case(12, "e4m3", "bf16", 256, 2, 4, 500, [10, 60, 3], 2, 32)
    wide = torch.zeros((6, 20, 256), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = dev16(q, "bf16")
    out, lse = call(pool, b, wide[:, 3:11], 2, scale)
    check(pool, b, q, "bf16", 2, scale, out, lse, what="strided")
    for _ in range(3):
        o2, l2 = call(pool, b, wide[:, 3:11], 2, scale)
        assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


def test_rows_in_any_order():
    """Rows of a sequence need not follow each other, nor be sorted by length."""
    b, pool, q, scale = case(13, "int8_side", "f16", 128, 1, 4, 70, [20, 30, 25], 4, 16)
    p = np.random.default_rng(0).permutation(12)
    out, lse = call(pool, b, dev16(q[p], "f16"), 1, scale, row_seq=b.row_seq[p], row_len=b.row_len[p])
    check(pool, b, q[p], "f16", 1, scale, out, lse, row_seq=b.row_seq[p], row_len=b.row_len[p], what="any order")


def test_tiny_and_huge_v_scales():
    """int8 V scales over many powers of two, rising and falling along the keys."""
    b, pool, q, scale = case(14, "int8_side", "bf16", 128, 1, 16, 260, [100, 3], 1, 16, scale=0.02)
    s = pool.kw["v_scale_tok"]
    e = torch.from_numpy(np.random.default_rng(1).integers(-40, 30, s.shape)).cuda().float()
    live = torch.from_numpy(b.live).cuda()
    s[live] = torch.exp2(e[live])
    pool.V = pool.cache[1].cpu().numpy().astype(np.float64) * s.double().cpu().numpy()[..., None]
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale)
    check(pool, b, q, "bf16", 1, scale, out, lse, what="scales")


def test_one_key_that_dominates_late():
    """A rising maximum: every tile raises the reference."""
    rng = np.random.default_rng(15)
    b = Batch(rng, 400, [50], 1, 16)
    pool = Pool(rng, "bf16", "bf16", b.live, b.num_slots, 1, 128)
    q = bits16(np.ones((1, 8, 128)), "bf16")
    kb = bits16(np.repeat(np.linspace(-4, 4, 450)[:, None, None], 128, 2), "bf16")
    from oracle import attention as oatt
    order = [int(b.prefix_blocks[p // 16]) * 16 + p % 16 if p < 400 else int(b.table[0, p // 16]) * 16 + p % 16 for p in range(450)]
    pool.cache[0][torch.tensor(order).cuda()] = dev16(kb, "bf16")
    full = np.zeros(pool.K.shape)
    full[order] = oatt.bf16_pool_fp64(kb)
    pool.K = full
    out, lse = call(pool, b, dev16(q, "bf16"), 1, 0.25)
    check(pool, b, q, "bf16", 1, 0.25, out, lse, what="rising")


def test_workspace_too_small_is_refused():
    import quantized_kv_cache_write_gb300 as qkv
    b, pool, q, scale = case(16, "e4m3", "bf16", 128, 1, 8, 600, [30, 3], 1, 16)
    need = qkv.qkv_prefix_attn_workspace(qkv.QKV_E4M3, 2, 8, 1, 128, 600, b.max_row_len)
    assert need > 0
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), None):
        with pytest.raises(qkv.QKVError):
            qkv.qkv_prefix_attn(dev16(q, "bf16"), qkv.QKV_E4M3, *pool.cache, torch.from_numpy(b.table).cuda(),
                                torch.from_numpy(b.row_seq).cuda(), torch.from_numpy(b.row_len).cuda(), 16, scale,
                                max_row_len=b.max_row_len, num_kv_heads=1,
                                prefix_blocks=torch.from_numpy(b.prefix_blocks).cuda(), prefix_len=600,
                                out=torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda"), workspace=ws,
                                **pool.kw)


def test_a_call_of_more_units_than_32_bits_number_is_refused():
    import quantized_kv_cache_write_gb300 as qkv
    with pytest.raises(qkv.QKVError) as e:
        qkv.qkv_prefix_attn_workspace(qkv.QKV_E4M3, 1 << 20, 64, 8, 128, 1 << 29, 1 << 29)
    assert e.value.status == qkv.QKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("seed", range(24))
def test_seeded_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    fmt, act = FMTS[seed % len(FMTS)]
    D, H = int(rng.choice([128, 256])), int(rng.choice([1, 2, 3]))
    G, per = int(rng.choice([1, 4, 6, 8, 16, 20])), int(rng.choice([1, 1, 2, 5]))
    prefix = int(rng.choice([0, 1, 30, 257, 900, 1800]))
    own = [int(rng.integers(per, 200)) for _ in range(int(rng.integers(1, 9)))]
    block = int(rng.choice([1, 8, 13, 16, 64]))
    b, pool, q, scale = case(2000 + seed, fmt, act, D, H, G, prefix, own, per, block)
    out, lse = call(pool, b, dev16(q, act), H, scale)
    check(pool, b, q, act, H, scale, out, lse, what=f"seed {seed}")


@pytest.mark.parametrize("fmt", ["int8_side", "int8_inline"])
@pytest.mark.parametrize("leftover", [float("inf"), 3e38, 1e30, -1e30, float("nan")])
@pytest.mark.parametrize("spare", [0, 30])
def test_a_huge_scale_behind_a_shorter_row_of_the_tile(fmt, leftover, spare):
    """The V scale of the key that only a sequence's last draft row sees bounds that row's weights alone: the others
    keep theirs (with 30 unused sequences in the table: tiles of eight pairs)."""
    b, pool, q, scale = case(17, fmt, "bf16", 128, 1, 4, 40, [7, 30, 4], 4, 16)
    b.table = np.concatenate([b.table, np.full((spare, b.table.shape[1]), -1, dtype=np.int32)])
    for i in range(3):
        n = int(b.row_len[4 * i + 3])
        slot = int(b.table[i, (n - 1) // 16]) * 16 + (n - 1) % 16
        if fmt == "int8_side":
            pool.kw["v_scale_tok"][slot] = leftover
        else:
            pool.cache[1].view(torch.uint8)[slot, :, 128:] = torch.tensor(np.array([leftover], np.float32).view(np.uint8)).cuda()
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale)
    first = np.arange(12) % 4 != 3
    slots, _ = dense.row_slots(b.row_seq[first], b.row_len[first], b.prefix_blocks, b.prefix, b.table, b.block, pool.num_slots)
    ref, rlse, wabs, big = dense.prefix_attention(q[first], pool.K, pool.V, slots, scale)
    tol, ltol = attention_bounds(ref, rlse, wabs, big, 70, float(np.abs(pool.V[b.live]).max()), "bf16", fmt, 128)
    assert_within(out.float().cpu().numpy()[first], ref, tol, "rows before the leftovers")
    assert_within(lse.cpu().numpy()[first], rlse, ltol, "lse before the leftovers")


# Batches behind long prefixes: several ranges of keys, tiles whose last pairs do not exist.
@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,rows,G,H", [(128, 9, 8, 1), (128, 70, 8, 2), (256, 21, 16, 1), (128, 13, 12, 3)])
def test_many_pairs_behind_a_long_prefix(fmt, act, D, rows, G, H):
    b, pool, q, scale = case(20, fmt, act, D, H, G, 9001, [1 + 3 * (i % 4) for i in range(rows)], 1, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, act), H, scale, status=status)
    check(pool, b, q, act, H, scale, out, lse, what=f"{fmt} {act} {D} {rows}")
    assert int(status.item()) == 0
    for _ in range(2):
        o2, l2 = call(pool, b, dev16(q, act), H, scale)
        assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


# The tcgen05 tiles: one SM or two per tile, tiles with few pairs, many tiles of one block, more tiles than SMs.
@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,rows,G,H,prefix", [(128, 9, 8, 1, 33001), (128, 70, 8, 2, 2401), (256, 21, 16, 1, 4001), (128, 13, 12, 3, 5601),
                                               (128, 40, 128, 8, 65), (256, 8, 16, 1, 10301), (128, 300, 1, 2, 4401), (256, 64, 128, 1, 161)])
def test_tcgen05_tiles(fmt, act, D, rows, G, H, prefix):
    assert -(-rows * G // 16) * H * prefix * D > 20 << 20  # of one byte each: K bytes that mma.sync tiles would read
    b, pool, q, scale = case(30, fmt, act, D, H, G, prefix, [1 + 3 * (i % 4) for i in range(rows)], 1, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, act), H, scale, status=status)
    check(pool, b, q, act, H, scale, out, lse, what=f"{fmt} {act} {D} {rows}")
    assert int(status.item()) == 0
    o2, l2 = call(pool, b, dev16(q, act), H, scale)
    assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


@pytest.mark.parametrize("seed", range(24))
def test_seeded_random_tcgen05_shapes(seed):
    rng = np.random.default_rng(3000 + seed)
    fmt, act = FMTS[seed % len(FMTS)]
    D, H, per = int(rng.choice([128, 256])), int(rng.choice([1, 2, 4])), int(rng.choice([1, 1, 2, 5]))
    G, seqs = int(rng.choice([1, 3, 8, 12, 16, 32, 128])), int(rng.integers(1, 40))
    tiles = -(-seqs * per * G // 16) * H
    prefix = (20 << 20) // (tiles * D) + int(rng.integers(1, 300))  # just past the rule, for one byte per value
    if prefix * seqs * per * G * H > 1 << 25:
        prefix = max(1, (1 << 25) // (seqs * per * G * H))
    own = [int(rng.integers(per, 60)) for _ in range(seqs)]
    b, pool, q, scale = case(4000 + seed, fmt, act, D, H, G, prefix, own, per, int(rng.choice([1, 7, 16, 64, 128])))
    seq, ln = b.row_seq.copy(), b.row_len.copy()
    idle = rng.random(len(seq)) < 0.1
    seq[idle] = -1
    out, lse = torch.full((len(seq), H * G, D), 7.0, dtype=ACT[act], device="cuda"), torch.full((len(seq), H * G), 7.0, device="cuda")
    call(pool, b, dev16(q, act), H, scale, row_seq=seq, row_len=ln, out=out, lse=lse)
    check(pool, b, q, act, H, scale, out, lse, row_seq=seq, row_len=ln, what=f"seed {seed}")
    assert (out[torch.from_numpy(idle).cuda()] == 7).all() and (lse[torch.from_numpy(idle).cuda()] == 7).all()


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D", [128, 256])
def test_tcgen05_tiles_with_bad_blocks_empty_rows_and_padding(fmt, act, D):
    b, pool, q, scale = case(31, fmt, act, D, 2, 8, 7001, [1 + i % 3 for i in range(24)], 1, 16)
    b.prefix_blocks[5], b.prefix_blocks[100:140], b.prefix_blocks[-1] = 1 << 26, -1, -7
    seq, ln = b.row_seq.copy(), b.row_len.copy()
    seq[3], seq[23], ln[5], ln[6] = -1, -1, 0, 6999  # padding twice, nothing, and a length inside the prefix: bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.full((24, 16, D), 7.0, dtype=ACT[act], device="cuda"), torch.full((24, 16), 7.0, device="cuda")
    call(pool, b, dev16(q, act), 2, scale, row_seq=seq, row_len=ln, out=out, lse=lse, status=status)
    assert int(status.item()) == 2
    for r in (3, 23):
        assert (out[r] == 7).all() and (lse[r] == 7).all()
    for r in (5, 6):
        assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    keep = np.array([r for r in range(24) if r not in (3, 5, 6, 23)])
    slots, _ = dense.row_slots(seq[keep], ln[keep], b.prefix_blocks, b.prefix, b.table, b.block, pool.num_slots)
    ref, rlse, wabs, big = dense.prefix_attention(q[keep], pool.K, pool.V, slots, scale, act)
    tol, ltol = attention_bounds(ref, rlse, wabs, big, 7004, float(np.abs(pool.V[b.live]).max()), act, fmt, D)
    assert_within(out.float().cpu().numpy()[keep], ref, tol, "out")
    assert_within(lse.cpu().numpy()[keep], rlse, ltol, "lse")
    # no block at all: the rows see their own keys alone
    b.prefix_blocks[:] = -1
    out, lse = call(pool, b, dev16(q, act), 2, scale)
    check(pool, b, q, act, 2, scale, out, lse, what="no prefix block")


@pytest.mark.parametrize("prefix", [20000, 20001, 40000])
@pytest.mark.parametrize("D,fmt", [(128, "e4m3"), (256, "int8_side"), (128, "bf16")])
def test_blocks_of_many_ctas(prefix, D, fmt):
    b, pool, q, scale = case(21, fmt, "bf16", D, 1, 8, prefix, [2] * 17, 1, 64)
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale)
    check(pool, b, q, "bf16", 1, scale, out, lse, what=f"{prefix} {D} {fmt}")


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("falling", [False, True])
def test_rising_and_falling_logits_and_scales_over_many_blocks(D, falling):
    """The row maximum and the int8 V scales grow (or fall) block after block, so that the reference
    is raised again and again, by the logits and by the scales."""
    rng = np.random.default_rng(22)
    P, rows, G = 30000, 12, 16
    b = Batch(rng, P, [1] * rows, 1, 16)
    pool = Pool(rng, "int8_side", "bf16", b.live, b.num_slots, 1, D)
    order = torch.tensor([int(b.prefix_blocks[p // 16]) * 16 + p % 16 for p in range(P)]).cuda()
    ramp = torch.linspace(0, 1, P, device="cuda")
    if falling:
        ramp = ramp.flip(0)
    pool.kw["k_scale_tok"][order] = 0.002 + 0.05 * ramp[:, None]
    pool.kw["v_scale_tok"][order] = torch.exp2(-20 + 24 * ramp)[:, None]
    pool.cache[0][order] = torch.randint(100, 128, (P, 1, D), device="cuda", dtype=torch.int8)
    for c, x, name in ((0, "K", "k_scale_tok"), (1, "V", "v_scale_tok")):
        setattr(pool, x, pool.cache[c].cpu().numpy().astype(np.float64) * pool.kw[name].double().cpu().numpy()[..., None])
    q = bits16(np.abs(rng.standard_normal((rows, G, D))), "bf16")
    out, lse = call(pool, b, dev16(q, "bf16"), 1, D ** -0.5)
    check(pool, b, q, "bf16", 1, D ** -0.5, out, lse, what="ramp")


def test_blocks_without_any_valid_key_among_many():
    """Whole 128-key blocks masked at the start, in the middle and at the end of the prefix."""
    b, pool, q, scale = case(23, "e4m3", "bf16", 128, 1, 16, 12000, [3] * 20, 1, 32)
    for lo, hi in ((0, 30), (100, 140), (360, 375)):
        b.prefix_blocks[lo:hi] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pool, b, dev16(q, "bf16"), 1, scale, status=status)
    check(pool, b, q, "bf16", 1, scale, out, lse, what="masked blocks")
    assert int(status.item()) == 2


@pytest.mark.parametrize("fmt,act", [("int8_side", "bf16"), ("e4m3", "f16"), ("bf16", "bf16"), ("int8_inline", "f16")])
@pytest.mark.parametrize("D,rows,G", [(128, 40, 16), (256, 40, 16), (256, 7, 16), (128, 7, 16)])
def test_each_row_has_one_heavy_key_somewhere(fmt, act, D, rows, G):
    """One key of the prefix carries most of a row's weight, at another place for every row (the last
    key of a range among them): a block whose contribution is dropped or counted twice shows."""
    P, H = 30001, 1
    b, pool, _, _ = case(24, fmt, act, D, H, G, P, [2] * rows, 1, 16)
    rng = np.random.default_rng(25)
    q = rng.standard_normal((rows, G, D))
    order = np.array([int(b.prefix_blocks[p // 16]) * 16 + p % 16 for p in range(P)])
    heavy = np.linspace(0, P - 1, rows).astype(int)
    heavy[1::3] = np.minimum(heavy[1::3] // 128 * 128 + 127, P - 1)
    K = pool.K[order[heavy], 0]
    q = 0.25 * q + 6.0 * (K / np.linalg.norm(K, axis=1, keepdims=True))[:, None]
    q = bits16(q, act)
    out, lse = call(pool, b, dev16(q, act), H, 1.0 if D == 128 else 0.7)
    check(pool, b, q, act, H, 1.0 if D == 128 else 0.7, out, lse, what=f"heavy {fmt} {D}")


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("rows", [1, 20])
def test_empty_pool(fmt, act, rows):
    """num_slots = 0 (through the C ABI): every key is masked and flagged, nothing of the pool is read."""
    import ctypes
    import quantized_kv_cache_write_gb300 as qkv
    b, pool, q, scale = case(26, fmt, act, 128, 1, 16, 40, [2] * rows, 1, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = dev16(q, act)
    out, lse = torch.full_like(qd, 7.0), torch.full((rows, 16), 7.0, device="cuda")
    ws = torch.empty(qkv.qkv_prefix_attn_workspace(qkv.FORMATS[fmt], rows, 16, 1, 128, 40, 42), dtype=torch.uint8, device="cuda")
    keep = [torch.from_numpy(x).cuda() for x in (b.prefix_blocks, b.table, b.row_seq, b.row_len)]
    ptr = lambda n: pool.kw[n].data_ptr() if torch.is_tensor(pool.kw.get(n)) else None
    d = qkv.PrefixDesc(size=ctypes.sizeof(qkv.PrefixDesc), fmt=qkv.FORMATS[fmt], q_fp16=int(act == "f16"), q=qd.data_ptr(),
                       q_stride=16 * 128, rows=rows, num_q_heads=16, num_kv_heads=1, head_dim=128,
                       k_cache=pool.cache[0].data_ptr(), v_cache=pool.cache[1].data_ptr(), k_scale_tok=ptr("k_scale_tok"),
                       v_scale_tok=ptr("v_scale_tok"), k_scale_layer=1.0, v_scale_layer=1.0, num_slots=0,
                       prefix_blocks=keep[0].data_ptr(), prefix_len=40, block_table=keep[1].data_ptr(), num_seqs=rows,
                       max_blocks=b.table.shape[1], block_size=16, row_seq=keep[2].data_ptr(), row_len=keep[3].data_ptr(),
                       max_row_len=42, softmax_scale=scale, out=out.data_ptr(), lse=lse.data_ptr(),
                       workspace=ws.data_ptr(), workspace_bytes=ws.numel(), dev_status=status.data_ptr())
    assert qkv.lib.qkv_prefix_attn(ctypes.byref(d), torch.cuda.current_stream().cuda_stream) == qkv.QKV_OK
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all() and int(status.item()) == 2
