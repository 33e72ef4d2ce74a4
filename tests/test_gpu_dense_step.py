"""qkv_append_rope and qkv_prefix_attn as a decode or draft step uses them, one after the other (GPU): the prompt and
every step's tokens are appended with their rotation, and the step's rotated queries attend over the pool that holds
them. Eager, captured and replayed, on other streams, with padding rows, in pools past 4 GB.

The references are computed in fp64 from the pool's own bytes ("[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache"
§Implementation scope: paged storage)."""

import numpy as np
import pytest
import torch

from dense_harness import ACT, assert_within, attention_bounds, bits16, dev16
from oracle import attention as oatt
from oracle import dense
from test_gpu_append import KS, VS, table

pytestmark = pytest.mark.gpu

FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16")]
BLOCK = 16


class Engine:
    """Sequences behind a shared prompt whose step is an append and an attention call."""

    def __init__(self, seed, fmt, act, D, H, G, prefix, seqs, per, steps, pad=0):
        import quantized_kv_cache_write_gb300 as qkv
        self.qkv, self.fmt, self.act, self.D, self.H, self.G = qkv, fmt, act, D, H, G
        self.prefix, self.seqs, self.per, self.steps, self.pad = prefix, seqs, per, steps, pad
        self.rng = np.random.default_rng(seed)
        self.start = [prefix + 3 * i % 7 for i in range(seqs)]  # first positions differ; the tokens between are appended first
        most = max(self.start) + steps * per
        wide, first = -(-most // BLOCK), prefix // BLOCK
        shared = -(-prefix // BLOCK)
        ids = self.rng.permutation(shared + seqs * (wide - first)).astype(np.int32)
        self.prefix_blocks = ids[:shared].copy()
        self.table = np.full((seqs + 1, max(wide, shared)), -1, dtype=np.int32)  # the last row: the prompt's own
        self.table[:seqs, first:wide] = ids[shared:].reshape(seqs, wide - first)
        self.table[seqs, :shared] = self.prefix_blocks
        self.S, self.most = len(ids) * BLOCK, most
        self.max_row_len = most
        width, dt = (D + 4, torch.uint8) if fmt == "int8_inline" else (D, ACT.get(fmt, torch.int8 if fmt == "int8_side" else torch.uint8))
        self.cache = [torch.zeros((self.S, H, width), dtype=dt, device="cuda") for _ in "kv"]
        self.scales = [torch.zeros((self.S, H), device="cuda") for _ in "kv"] if fmt == "int8_side" else [None, None]
        self.layer = (float(KS), float(VS)) if fmt == "e4m3" else (1.0, 1.0)
        self.cs = torch.from_numpy(table(most + 1, D)).cuda()
        self.tab, self.pb = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.prefix_blocks).cuda()
        R = self.R = seqs * per + pad
        self.q, self.k, self.v = (torch.zeros((R, n, D), dtype=ACT[act], device="cuda") for n in (H * G, H, H))
        self.q_out, self.out = torch.full_like(self.q, 7.0), torch.full_like(self.q, 7.0)
        self.lse = torch.full((R, H * G), 7.0, device="cuda")
        self.row_seq = torch.from_numpy(np.concatenate([np.repeat(np.arange(seqs), per), np.full(pad, -1)]).astype(np.int32)).cuda()
        self.pos, self.row_len = (torch.full((R,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        need = qkv.qkv_prefix_attn_workspace(qkv.FORMATS[fmt], R, H * G, H, D, prefix, self.max_row_len)
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if prefix:
            self.append(self.bits(prefix, H), self.bits(prefix, H), np.arange(prefix), np.full(prefix, seqs))
        for i, n in enumerate(self.start):
            if n > prefix:
                self.append(self.bits(n - prefix, H), self.bits(n - prefix, H), np.arange(prefix, n), np.full(n - prefix, i))

    def bits(self, *shape):
        return bits16(self.rng.standard_normal((shape[0], shape[1], self.D)), self.act)

    def append(self, kb, vb, pos, seq):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).cuda()
        self.qkv.qkv_append_rope(dev16(kb, self.act), dev16(vb, self.act), self.qkv.FORMATS[self.fmt], *self.cache, self.cs,
                                 dev(pos), token_seq=dev(seq), block_table=self.tab, block_size=BLOCK,
                                 k_scale=self.scales[0], v_scale=self.scales[1], k_scale_layer=self.layer[0],
                                 v_scale_layer=self.layer[1], dev_status=self.status)

    def load(self, step):
        """A step's inputs into the tensors that its calls read."""
        pos = np.concatenate([[n + step * self.per + j for n in self.start for j in range(self.per)], np.full(self.pad, -1)])
        self.np_pos = pos.astype(np.int32)
        for t, n in ((self.q, self.H * self.G), (self.k, self.H), (self.v, self.H)):
            b = self.bits(self.R, n)
            t.copy_(dev16(b, self.act))
            if t is self.q:
                self.qb = b
        self.pos.copy_(torch.from_numpy(self.np_pos))
        self.row_len.copy_(torch.from_numpy(np.where(pos >= 0, pos + 1, 0).astype(np.int32)))

    def step(self, stream=None):
        f = self.qkv.FORMATS[self.fmt]
        self.qkv.qkv_append_rope(self.k, self.v, f, *self.cache, self.cs, self.pos, q=self.q, q_out=self.q_out,
                                 token_seq=self.row_seq, block_table=self.tab, block_size=BLOCK, k_scale=self.scales[0],
                                 v_scale=self.scales[1], k_scale_layer=self.layer[0], v_scale_layer=self.layer[1],
                                 dev_status=self.status, stream=stream)
        self.qkv.qkv_prefix_attn(self.q_out, f, *self.cache, self.tab, self.row_seq, self.row_len, BLOCK, self.D ** -0.5,
                                 max_row_len=self.max_row_len, num_kv_heads=self.H, prefix_blocks=self.pb if self.prefix else None,
                                 prefix_len=self.prefix, k_scale_tok=self.scales[0], v_scale_tok=self.scales[1],
                                 k_scale_layer=self.layer[0], v_scale_layer=self.layer[1], out=self.out, lse=self.lse,
                                 workspace=self.ws, dev_status=self.status, stream=stream)

    def values(self):
        raw = [c.cpu() for c in self.cache]
        if self.fmt in ACT:
            widen = oatt.f16_pool_fp64 if self.fmt == "f16" else oatt.bf16_pool_fp64
            return [widen(c.view(torch.int16).numpy().view(np.uint16)) for c in raw]
        if self.fmt == "int8_side":
            return [oatt.int8_side_pool_fp64(c.numpy(), s.cpu().numpy()) for c, s in zip(raw, self.scales)]
        if self.fmt == "int8_inline":
            return [oatt.int8_inline_pool_fp64(c.numpy()) for c in raw]
        return [oatt.e4m3_pool_fp64(c.numpy(), np.float32(s)) for c, s in zip(raw, self.layer)]

    def check(self, what):
        n = self.R - self.pad
        rot = bits16(dense.rotate_f32(oatt_f32(self.qb[:n], self.act), self.np_pos[:n], self.cs.cpu().numpy(), False), self.act)
        got = self.q_out.view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.array_equal(got[:n], rot), what
        K, V = self.values()
        seq, ln = self.row_seq.cpu().numpy()[:n], self.np_pos[:n] + 1
        slots, _ = dense.row_slots(seq, ln, self.prefix_blocks, self.prefix, self.table, BLOCK, self.S)
        ref, rlse, wabs, big = dense.prefix_attention(rot, K, V, slots, self.D ** -0.5, self.act)
        tol, ltol = attention_bounds(ref, rlse, wabs, big, int(ln.max()), float(np.abs(V).max()), self.act, self.fmt, self.D)
        assert_within(self.out.float().cpu().numpy()[:n], ref, tol, what + " out")
        assert_within(self.lse.cpu().numpy()[:n], rlse, ltol, what + " lse")
        for t in (self.out, self.q_out, self.lse):  # rows behind the last sequence: as they were
            assert (t[n:] == 7.0).all(), what
        assert int(self.status.item()) == 0


def oatt_f32(bits, act):
    from oracle import quant as oq
    return oq.act_bits_to_f32(bits, act)


# (head_dim, KV heads, group, prompt, sequences, rows per sequence): single tokens, drafts, no shared prompt, and a
# prompt of more K bytes than the mma.sync tiles take
SHAPES = [(128, 2, 4, 100, 3, 1), (256, 1, 16, 70, 2, 5), (128, 1, 8, 0, 4, 2), (128, 8, 16, 700, 9, 4), (256, 1, 16, 3003, 16, 2)]


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_steps_in_a_row(fmt, act, shape):
    e = Engine(1, fmt, act, *shape, steps=3)
    for s in range(3):
        e.load(s)
        e.step()
        torch.cuda.synchronize()
        e.check(f"{fmt} {shape} step {s}")


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_captured_steps_with_padding_rows(fmt, act, shape):
    """One graph, captured before the pool holds the step's tokens, replayed for three steps: lengths, positions and
    tokens are read from their tensors each time. The last rows of the batch are padding."""
    e, plain = Engine(2, fmt, act, *shape, steps=4, pad=3), Engine(2, fmt, act, *shape, steps=4, pad=3)
    s = torch.cuda.Stream()
    e.load(0), plain.load(0)
    with torch.cuda.stream(s):
        e.step()  # a first call may set kernel attributes
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        e.step()
    plain.step()
    for i in range(1, 4):
        e.load(i), plain.load(i)
        g.replay()
        plain.step()
        torch.cuda.synchronize()
        e.check(f"{fmt} {shape} replay {i}")
        for a, b in ((e.out, plain.out), (e.q_out, plain.q_out)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(e.lse, plain.lse)
        for a, b in zip(e.cache, plain.cache):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_engines_on_two_streams():
    """Steps of two engines, each with its own pool and workspace, in flight at the same time."""
    shapes = [("int8_side", "bf16", 256, 1, 16, 3003, 16, 2), ("e4m3", "bf16", 128, 8, 16, 700, 9, 4)]
    alone, both = ([Engine(3 + i, *s, steps=6) for i, s in enumerate(shapes)] for _ in range(2))
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for i in range(6):
        for e in alone + both:
            e.load(i)
        torch.cuda.synchronize()
        for e, s in zip(both, streams):
            e.step(stream=s)
        torch.cuda.synchronize()
        for e in alone:
            e.step()
            torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16)) and torch.equal(a.lse, b.lse)
    for e in both:
        e.check("two streams")


def test_two_graphs_that_share_a_workspace():
    """A workspace holds nothing between calls: graphs that are replayed one after the other may share it."""
    e = [Engine(5 + i, "e4m3", "bf16", 128, 8, 16, 700, 9, 4, steps=3) for i in range(2)]
    e[1].ws = e[0].ws
    s = torch.cuda.Stream()
    graphs = []
    for x in e:
        x.load(0)
        with torch.cuda.stream(s):
            x.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.step()
        graphs.append(g)
    for i in (1, 2):
        for x, g in zip(e, graphs):
            x.load(i)
            torch.cuda.synchronize()
            g.replay()
        torch.cuda.synchronize()
        for x in e:
            x.check(f"shared workspace, replay {i}")


@pytest.mark.parametrize("fmt,slots", [("bf16", 1_100_000), ("e4m3", 2_200_000)])
@pytest.mark.parametrize("rows", [2, 40])
def test_pools_past_4_gb(fmt, slots, rows):
    """Records past the 4 GB mark of each pool (offsets of more than 32 bits), by both kinds of tile."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(7)
    H, G, D, P, own = 8, 16, 256, 300, 20
    dt = ACT.get(fmt, torch.uint8)
    cache = [torch.zeros((slots, H, D), dtype=dt, device="cuda") for _ in "kv"]
    assert cache[0].numel() * cache[0].element_size() > 1 << 32
    nblk = slots // BLOCK
    shared, first = -(-P // BLOCK), P // BLOCK
    ids = (nblk - 1 - rng.permutation(2000)[:shared + 3 * rows]).astype(np.int32)  # the pool's last blocks
    tab = np.full((rows + 1, first + 3), -1, dtype=np.int32)
    tab[:rows, first:] = ids[shared:].reshape(rows, 3)
    tab[rows, :shared] = ids[:shared]
    n = P + rows * own
    pos = np.concatenate([np.arange(P)] + [np.arange(P, P + own)] * rows).astype(np.int32)
    seq = np.concatenate([np.full(P, rows)] + [np.full(own, i) for i in range(rows)]).astype(np.int32)
    kb, vb = (bits16(rng.standard_normal((n, H, D)), "bf16") for _ in "kv")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    layer = (float(KS), float(VS)) if fmt == "e4m3" else (1.0, 1.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = table(P + own, D)
    qkv.qkv_append_rope(dev16(kb, "bf16"), dev16(vb, "bf16"), qkv.FORMATS[fmt], *cache, dev(cs), dev(pos), token_seq=dev(seq),
                        block_table=dev(tab), block_size=BLOCK, k_scale_layer=layer[0], v_scale_layer=layer[1], dev_status=status)
    qb = bits16(rng.standard_normal((rows, H * G, D)), "bf16")
    out, lse = torch.empty((rows, H * G, D), dtype=torch.bfloat16, device="cuda"), torch.empty((rows, H * G), device="cuda")
    ws = torch.empty(qkv.qkv_prefix_attn_workspace(qkv.FORMATS[fmt], rows, H * G, H, D, P, P + own), dtype=torch.uint8, device="cuda")
    row_seq, row_len = np.arange(rows, dtype=np.int32), np.full(rows, P + own, dtype=np.int32)
    qkv.qkv_prefix_attn(dev16(qb, "bf16"), qkv.FORMATS[fmt], *cache, dev(tab), dev(row_seq), dev(row_len), BLOCK, D ** -0.5,
                        max_row_len=P + own, num_kv_heads=H, prefix_blocks=dev(ids[:shared]), prefix_len=P,
                        k_scale_layer=layer[0], v_scale_layer=layer[1], out=out, lse=lse, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    slot_lists, _ = dense.row_slots(row_seq, row_len, ids[:shared], P, tab, BLOCK, slots)
    used = np.unique(np.concatenate([np.asarray(s) for s in slot_lists]))
    small = [c[torch.from_numpy(used).cuda()].cpu() for c in cache]
    if fmt == "bf16":
        K, V = (oatt.bf16_pool_fp64(c.view(torch.int16).numpy().view(np.uint16)) for c in small)
    else:
        K, V = (oatt.e4m3_pool_fp64(c.numpy(), np.float32(s)) for c, s in zip(small, layer))
    assert np.abs(K).sum(-1).min() > 0  # every record was written
    ref, rlse, wabs, big = dense.prefix_attention(qb, K, V, [np.searchsorted(used, s).tolist() for s in slot_lists], D ** -0.5, "bf16")
    tol, ltol = attention_bounds(ref, rlse, wabs, big, P + own, float(np.abs(V).max()), "bf16", fmt, D)
    assert_within(out.float().cpu().numpy(), ref, tol, "out")
    assert_within(lse.cpu().numpy(), rlse, ltol, "lse")
