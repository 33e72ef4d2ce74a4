"""qkv_append_axes, qkv_masked_attn and qkv_read as a model's steps use them, one after the other (GPU): a prompt of text
and image tokens is appended and attends in one chunk, single tokens follow, a document is read back, turned back and
appended elsewhere. Eager, captured and replayed with padding rows, on two streams, in pools past 4 GB; both kinds of tiles.

The references are computed in fp64 from the pool's own bytes ("[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache"
§Implementation scope: paged storage)."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from dense_harness import ACT, dev16
from masked_harness import Pool, Seqs, call, check, chunk_rows, query
from oracle import attention as oatt
from test_gpu_append import KS, VS, table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["mma", "tcgen05"])
def tiles(request, monkeypatch):
    """Each kind of tiles, whatever the call would choose at these sizes."""
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", request.param)


FMTS = [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16")]
BLOCK = 16


class Held:
    """An empty pool that the operators fill; K, V: its values in fp64, read from its bytes."""

    def __init__(self, fmt, S, H, D):
        self.fmt, self.num_slots = fmt, S
        width, dt = (D + 4, torch.uint8) if fmt == "int8_inline" else (D, ACT.get(fmt, torch.int8 if fmt == "int8_side" else torch.uint8))
        self.cache = [torch.zeros((S, H, width), dtype=dt, device="cuda") for _ in "kv"]
        self.scales = [torch.zeros((S, H), device="cuda") for _ in "kv"] if fmt == "int8_side" else [None, None]
        self.kw = dict(k_scale_tok=self.scales[0], v_scale_tok=self.scales[1]) if fmt == "int8_side" else {}
        self.layer = {}
        if fmt == "e4m3":
            self.kw = self.layer = dict(k_scale_layer=float(KS), v_scale_layer=float(VS))

    def _values(self, i):
        c = self.cache[i]
        if self.fmt in ACT:
            bits = c.view(torch.int16).cpu().numpy().view(np.uint16)
            return (oatt.f16_pool_fp64 if self.fmt == "f16" else oatt.bf16_pool_fp64)(bits)
        c = c.cpu().numpy()
        if self.fmt == "int8_side":
            return oatt.int8_side_pool_fp64(c, self.scales[i].cpu().numpy())
        return oatt.int8_inline_pool_fp64(c) if self.fmt == "int8_inline" else oatt.e4m3_pool_fp64(c, (KS, VS)[i])

    K = property(lambda self: self._values(0))
    V = property(lambda self: self._values(1))


class Step:
    """One sequence's tokens into the pool by several axes, and the rotated queries."""

    def __init__(self, seed, fmt, act, H, G, D, length):
        import quantized_kv_cache_write_gb300 as qkv
        self.qkv, self.fmt, self.act, self.H, self.G, self.D = qkv, fmt, act, H, G, D
        self.rng = np.random.default_rng(seed)
        self.seqs = Seqs(self.rng, (length, length), BLOCK)
        self.pool = Held(fmt, self.seqs.num_slots, H, D)
        self.cs = torch.from_numpy(table(4096, D)).cuda()
        self.table = torch.from_numpy(self.seqs.table).cuda()
        self.pair_axis = [i % 3 if i < 3 * (D // 8) else 0 for i in range(D // 2)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, seq, pos, axis_pos):
        T = len(pos)
        q, k, v = (dev16(query(self.rng, T, n, self.D, self.act), self.act) for n in (self.H * self.G, self.H, self.H))
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        self.qkv.qkv_append_axes(k, v, self.qkv.FORMATS[self.fmt], *self.pool.cache, self.cs, dev(axis_pos), self.pair_axis, q=q,
                                 q_out=q, token_seq=dev(np.full(T, seq)), token_pos=dev(pos), block_table=self.table,
                                 block_size=BLOCK, k_scale=self.pool.scales[0], v_scale=self.pool.scales[1],
                                 dev_status=self.status, **self.pool.layer)
        return q

    def attend(self, q, rows, **kw):
        got = call(self.pool, self.fmt, q, self.seqs, rows, self.H, self.D ** -0.5, status=self.status, **kw)
        bits = q.view(torch.int16).cpu().numpy().view(np.uint16)
        check(self.pool, self.fmt, self.act, bits, self.seqs, rows, self.H, self.D ** -0.5, got=got, want_status=0,
              **{k: v for k, v in kw.items() if k in ("window", "softcap", "slopes", "max_row_end")})
        assert int(self.status.item()) == 0
        return got


def image_positions(n, first=0):
    """Text tokens, then a grid of 7 columns: three axes."""
    t = np.arange(n)
    text = n // 3
    grid = np.stack([np.zeros(n, int), (t - text) // 7, (t - text) % 7]) + text
    return first + np.where(t < text, t, grid)


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,H,G,n", [(128, 2, 8, 90), (256, 1, 16, 200), (128, 1, 4, 700)])
def test_prompt_tokens_and_a_document_moved(fmt, act, D, H, G, n):
    e = Step(D + n, fmt, act, H, G, D, n + 80)
    q = e.append(0, np.arange(n), image_positions(n))
    rows = np.stack([np.zeros(n), np.zeros(n), np.maximum(np.arange(n) + 1, n // 4), np.arange(n)], 1).astype(np.int32)
    e.attend(q, rows, softcap=30.0)          # the prompt: its first quarter sees itself
    for i in range(3):                       # single tokens, in a window
        q = e.append(0, [n + i], image_positions(1, n + i))
        e.attend(q, np.array([(0, 0, n + i + 1, n + i)], np.int32), window=50, slopes=2.0 ** -np.arange(1, H * G + 1) if i else None)
    # tokens 10 to 50 read back, turned back, and appended to the other sequence at positions of its own
    m = 41
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    k, v = (torch.zeros((m, H, D), dtype=ACT[act], device="cuda") for _ in "kv")
    sc = dict(k_scale=e.pool.scales[0], v_scale=e.pool.scales[1], **e.pool.layer)
    e.qkv.qkv_read(e.qkv.FORMATS[fmt], *e.pool.cache, k_out=k, v_out=v, token_seq=dev(np.zeros(m)), token_pos=dev(np.arange(10, 51)),
                   block_table=e.table, block_size=BLOCK, cos_sin=e.cs, axis_pos=dev(image_positions(n)[:, 10:51]),
                   pair_axis=e.pair_axis, dev_status=e.status, **sc)
    e.qkv.qkv_append_axes(k, v, e.qkv.FORMATS[fmt], *e.pool.cache, e.cs, dev(image_positions(m, 300)), e.pair_axis,
                          token_seq=dev(np.ones(m)), token_pos=dev(np.arange(m)), block_table=e.table, block_size=BLOCK,
                          dev_status=e.status, **sc)
    assert torch.isfinite(k).all() and (k != 0).any()
    q = dev16(query(e.rng, m, H * G, D, act), act)
    e.attend(q, np.array([(1, 0, i + 1, i) for i in range(m)], np.int32))


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("D,G,new,length", [(128, 8, 2, 400), (256, 16, 160, 1700), (128, 4, 640, 2000)])
def test_captured_and_replayed_with_other_rows_and_padding(fmt, act, D, G, new, length):
    """One graph serves batches of any rows up to its sizes: tables, ranges and queries are read when it runs."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(D + new)
    seqs = Seqs(rng, (length, length), BLOCK)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, 1, D)
    R = 2 * new
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q = torch.zeros((R, G, D), dtype=ACT[act], device="cuda")
    cols = [torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(4)]
    out, lse = torch.zeros_like(q), torch.zeros((R, G), device="cuda")
    ws = torch.full((qkv.qkv_masked_attn_workspace(qkv.FORMATS[fmt], R, 2, G, 1, D, length),), 0xFF, dtype=torch.uint8, device="cuda")
    slopes, status, tab = dev(np.float32(2.0) ** -np.arange(1, G + 1, dtype=np.float32)), torch.zeros(1, dtype=torch.int32, device="cuda"), dev(seqs.table)

    def step():
        qkv.qkv_masked_attn(q, qkv.FORMATS[fmt], *pool.cache, tab, cols[0], cols[2], BLOCK, D ** -0.5, max_row_end=length,
                            row_start=cols[1], row_pos=cols[3], softcap=20.0, slopes=slopes, out=out, lse=lse, workspace=ws,
                            dev_status=status, **pool.kw)

    def load(rows, bits):
        for c, x in zip(cols, rows.T):
            c.copy_(dev(np.ascontiguousarray(x)))
        q.copy_(dev16(bits, act))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))

    rows = chunk_rows((length, length), (new, new))
    load(rows, query(rng, R, G, D, act))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for kind in range(3):
        rows = chunk_rows((length, length), (new, new), ("causal", "docs", "prefix")[kind], doc=90)
        if kind:
            rows[rng.random(R) < 0.2, 0] = -1
            rows[-R // 4:, 0] = -1   # a batch smaller than the graph's
        bits = query(rng, R, G, D, act)
        load(rows, bits)
        graph.replay()
        torch.cuda.synchronize()
        got = (out.clone(), lse.clone())
        check(pool, fmt, act, bits, seqs, rows, 1, D ** -0.5, softcap=20.0, slopes=2.0 ** -np.arange(1, G + 1), got=got,
              want_status=0, max_row_end=length)
        assert int(status.item()) == 0
        load(rows, bits)
        step()  # eager: the same bits
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), got[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), got[1].view(torch.int32))


@pytest.mark.parametrize("D,G,new", [(128, 8, 3), (256, 16, 150)])
def test_two_streams_at_once(D, G, new):
    """Each with its own workspace: neither disturbs the other."""
    rng = np.random.default_rng(new)
    lengths = (1500, 1200)
    seqs = Seqs(rng, lengths, BLOCK)
    pool = Pool(rng, "int8_side", "bf16", seqs.live, seqs.num_slots, 1, D)
    rows = [chunk_rows(lengths, (new, new)), chunk_rows(lengths, (new, new), "docs")]
    bits = [query(rng, 2 * new, G, D, "bf16") for _ in range(2)]
    alone = [call(pool, "int8_side", dev16(b, "bf16"), seqs, r, 1, 0.08, softcap=9.0) for b, r in zip(bits, rows)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    dev = [dev16(b, "bf16") for b in bits]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, d, r in zip(streams, dev, rows):
            with torch.cuda.stream(s):
                got.append(call(pool, "int8_side", d, seqs, r, 1, 0.08, softcap=9.0))
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            assert torch.equal(a[0].view(torch.int16), g[0].view(torch.int16)) and torch.equal(a[1], g[1])


@pytest.mark.parametrize("n", [2, 150])
def test_workspaces_and_outputs(n):
    """One byte too few is refused; without lse the outputs are the same; a stream given by hand."""
    import quantized_kv_cache_write_gb300 as qkv
    rng = np.random.default_rng(n)
    seqs = Seqs(rng, (1300,), BLOCK)
    pool = Pool(rng, "e4m3", "bf16", seqs.live, seqs.num_slots, 1, 128)
    rows = chunk_rows((1300,), (n,))
    q = dev16(query(rng, n, 16, 128, "bf16"), "bf16")
    want = call(pool, "e4m3", q, seqs, rows, 1, 0.1)
    need = qkv.qkv_masked_attn_workspace(qkv.QKV_E4M3, n, 1, 16, 1, 128, 1300)
    assert need > 0
    with pytest.raises(qkv.QKVError):
        call(pool, "e4m3", q, seqs, rows, 1, 0.1, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    args = (dev(seqs.table), dev(rows[:, 0]), dev(rows[:, 2]))
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.zeros_like(q)
    torch.cuda.synchronize()
    qkv.qkv_masked_attn(q, qkv.QKV_E4M3, *pool.cache, *args, BLOCK, 0.1, max_row_end=1300, out=out, workspace=ws, stream=s, **pool.kw)
    s.synchronize()
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("fmt,act", FMTS)
@pytest.mark.parametrize("n,D,G", [(2, 128, 8), (150, 128, 8), (150, 256, 16)])
def test_queries_that_are_not_finite_stay_in_their_rows(fmt, act, n, D, G):
    rng = np.random.default_rng(n)
    seqs = Seqs(rng, (1300,), BLOCK)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, 1, D)
    rows = chunk_rows((1300,), (n,))
    bits = query(rng, n, G, D, act)
    clean = call(pool, fmt, dev16(bits, act), seqs, rows, 1, 0.1, softcap=30.0)
    bits[n // 2, 1, 3] = 0x7FC0 if act == "bf16" else 0x7E00
    bits[n // 2, 2, 5] = 0x7F80 if act == "bf16" else 0x7C00
    got = call(pool, fmt, dev16(bits, act), seqs, rows, 1, 0.1, softcap=30.0)
    torch.cuda.synchronize()
    assert got[0][n // 2, 1].isnan().all()
    keep = torch.ones((n, G), dtype=torch.bool)
    keep[n // 2, 1:3] = False
    assert torch.equal(got[0].cpu()[keep].view(torch.int16), clean[0].cpu()[keep].view(torch.int16))
    assert torch.equal(got[1].cpu()[keep], clean[1].cpu()[keep])


@pytest.mark.parametrize("fmt", ["bf16", "int8_side"])
def test_pools_past_4_gb(fmt):
    """Blocks at the end of a pool of 4.5 GB per tensor: appended, attended to by both kinds of tiles and read back."""
    import quantized_kv_cache_write_gb300 as qkv
    H, D, G, n = 4, 256, 4, 300
    S = (9 << 29) // (H * D * (2 if fmt == "bf16" else 1)) // BLOCK * BLOCK
    rng = np.random.default_rng(1)
    pool = Held(fmt, S, H, D)
    blocks = np.arange(S // BLOCK - 40, S // BLOCK, dtype=np.int32)[rng.permutation(40)]
    tab = blocks[None, :20].copy()
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    k, v = (dev16(query(rng, n, H, D, "bf16"), "bf16") for _ in "kv")
    pos, seq = dev(np.arange(n, dtype=np.int32)), dev(np.zeros(n, np.int32))
    cs, status = torch.from_numpy(table(400, 64)).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    qkv.qkv_append_axes(k, v, qkv.FORMATS[fmt], *pool.cache, cs, pos[None].contiguous(), token_seq=seq, token_pos=pos, block_table=dev(tab),
                        block_size=BLOCK, k_scale=pool.scales[0], v_scale=pool.scales[1], dev_status=status)
    ko, vo = (torch.zeros((n, H, D), device="cuda") for _ in "kv")
    qkv.qkv_read(qkv.FORMATS[fmt], *pool.cache, k_out=ko, v_out=vo, token_seq=seq, token_pos=pos, block_table=dev(tab), block_size=BLOCK,
                 k_scale=pool.scales[0], v_scale=pool.scales[1], dev_status=status)
    assert (vo - v.float()).abs().max() <= v.float().abs().max() / 127
    for m in (2, n):
        q = dev16(query(rng, m, H * G, D, "bf16"), "bf16")
        got = []
        # the same keys as the first blocks of a small pool of the same values
        small = Held(fmt, 20 * BLOCK, H, D)
        for i in range(2):
            for b in range(20):
                small.cache[i][b * BLOCK:(b + 1) * BLOCK] = pool.cache[i][int(tab[0, b]) * BLOCK:(int(tab[0, b]) + 1) * BLOCK]
                if fmt == "int8_side":
                    small.scales[i][b * BLOCK:(b + 1) * BLOCK] = pool.scales[i][int(tab[0, b]) * BLOCK:(int(tab[0, b]) + 1) * BLOCK]
        ends = dev(np.arange(n - m + 1, n + 1, dtype=np.int32))
        for p, t in ((pool, tab), (small, np.arange(20, dtype=np.int32)[None])):
            out, lse = torch.zeros_like(q), torch.zeros((m, H * G), device="cuda")
            ws = torch.empty(qkv.qkv_masked_attn_workspace(qkv.FORMATS[fmt], m, 1, H * G, H, D, n), dtype=torch.uint8, device="cuda")
            qkv.qkv_masked_attn(q, qkv.FORMATS[fmt], *p.cache, dev(t), dev(np.zeros(m, np.int32)), ends, BLOCK, D ** -0.5, max_row_end=n,
                                num_kv_heads=H, out=out, lse=lse, workspace=ws, dev_status=status, **p.kw)
            got.append((out, lse))
        torch.cuda.synchronize()
        assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])
    assert int(status.item()) == 0


@pytest.mark.parametrize("D,n", [(128, 3), (128, 150), (256, 150)])
def test_v_scales_far_apart_and_unseen(D, n):
    """int8 V scales from 2^-60 to 2^60 along the keys, ascending and descending; a row whose keys' scales are all small keeps
    their bits, whatever the scales that other rows of its tile see."""
    rng = np.random.default_rng(D)
    seqs = Seqs(rng, (600,), BLOCK)
    for up in (1, -1):
        pool = Pool(rng, "int8_side", "bf16", seqs.live, seqs.num_slots, 1, D)
        j = np.arange(600)
        slot = seqs.table[0, j // BLOCK].astype(np.int64) * BLOCK + j % BLOCK
        scale = np.float32(2.0) ** np.linspace(-60, 60, 600).astype(np.float32)[::up]
        codes = pool.cache[1].cpu().numpy()
        vs = pool.kw["v_scale_tok"].cpu().numpy()
        vs[slot, 0] = scale
        pool.kw["v_scale_tok"] = torch.from_numpy(vs).cuda()
        pool.V[slot] = codes[slot].astype(np.float64) * scale[:, None, None].astype(np.float64)
        # documents of 40 keys: a row's largest V scale is at most 2^8 of its smallest
        rows = chunk_rows((600,), (n,), "docs", doc=20)
        q = query(rng, n, 8, D, "bf16")
        got = call(pool, "int8_side", dev16(q, "bf16"), seqs, rows, 1, 0.1)
        torch.cuda.synchronize()
        for r in rng.permutation(n)[:20]:  # each row against its own keys' magnitudes
            one = rows[r:r + 1]
            lo, hi = int(one[0, 1]), int(one[0, 2])
            sub = SimpleNamespace(cache=pool.cache, kw=pool.kw, K=pool.K, V=np.zeros_like(pool.V))
            sub.V[slot[lo:hi]] = pool.V[slot[lo:hi]]
            check(sub, "int8_side", "bf16", q[r:r + 1], seqs, one, 1, 0.1, got=(got[0][r:r + 1], got[1][r:r + 1]), want_status=0)
