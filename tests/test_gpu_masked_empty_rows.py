"""qkv_masked_attn's rows that see nothing, among rows that do (GPU): they are empty whatever the others' keys hold, and the
others take no longer for them.

Pools and block tables are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

from masked_harness import Pool, Seqs, call, chunk_rows, dev16, query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tiles", ["mma", "tcgen05"])
@pytest.mark.parametrize("fmt,act", [("bf16", "bf16"), ("f16", "f16"), ("int8_side", "bf16"), ("int8_inline", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("n,D,G,length", [(4, 128, 3, 900), (130, 128, 8, 900), (9, 256, 16, 9001), (150, 256, 4, 400)])
def test_they_are_empty_whatever_the_others_see(monkeypatch, tiles, fmt, act, n, D, G, length):
    """NaN in K and in V of the first token, which all rows that see anything see: those are NaN, the empty ones 0 and -infinity."""
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", tiles)
    rng = np.random.default_rng(n + D)
    seqs = Seqs(rng, (length,), 16)
    pool = Pool(rng, fmt, act, seqs.live, seqs.num_slots, 1, D)
    rows = chunk_rows((length,), (n,))
    empty = np.zeros(n, dtype=bool)
    empty[1::3] = True
    rows[empty, 2] = 0
    q = dev16(query(rng, n, G, D, act), act)
    clean = call(pool, fmt, q, seqs, rows, 1, D ** -0.5, max_row_end=length)
    slot = int(seqs.table[0, 0]) * 16
    for x in range(2):
        if fmt == "int8_side":
            pool.kw[("k_scale_tok", "v_scale_tok")[x]][slot] = float("nan")
        elif fmt == "int8_inline":
            pool.cache[x].view(torch.uint8)[slot, :, D:] = torch.tensor([float("nan")]).view(torch.uint8).cuda()
        elif fmt == "e4m3":
            pool.cache[x][slot] = 0x7F
        else:
            pool.cache[x][slot] = float("nan")
    odd = call(pool, fmt, q, seqs, rows, 1, D ** -0.5, max_row_end=length)
    torch.cuda.synchronize()
    e = torch.from_numpy(empty).cuda()
    for out, lse in (clean, odd):
        assert not out[e].float().abs().max() > 0 and out[e].isfinite().all()
        assert (lse[e] == -float("inf")).all()
    assert clean[0][~e].isfinite().all() and clean[1][~e].isfinite().all()
    assert odd[0][~e].isnan().all() and odd[1][~e].isnan().all()


@pytest.mark.parametrize("fmt,seqs_n,rows_n,ctx,H,G,D,every", [("int8_side", 1, 2048, 8000, 4, 8, 128, 29), ("e4m3", 8, 5, 2000, 8, 2, 128, 3)])
def test_the_others_take_no_longer(fmt, seqs_n, rows_n, ctx, H, G, D, every):
    """A chunk on the tcgen05 tiles and drafts on the mma.sync tiles, replayed in turn with and without empty rows (1.40 and 1.5
    times the time while every block was masked for them)."""
    import quantized_kv_cache_write_gb300 as qkv
    gen = torch.Generator(device="cuda").manual_seed(1)
    length, block = ctx + rows_n, 16
    wide = -(-length // block)
    S = seqs_n * wide * block
    table = torch.arange(seqs_n * wide, device="cuda").int().view(seqs_n, wide)
    seq = torch.arange(seqs_n, device="cuda").int().repeat_interleave(rows_n)
    full = (ctx + 1 + torch.arange(rows_n, device="cuda")).int().repeat(seqs_n)
    some = full.clone()
    some[every - 1::every] = 0
    kw = {}
    if fmt == "e4m3":
        k, v = (torch.randn((S, H, D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8) for _ in "kv")
    else:
        k, v = (torch.randint(-127, 128, (S, H, D), device="cuda", generator=gen, dtype=torch.int8) for _ in "kv")
        kw = {x: torch.full((S, H), 0.02, device="cuda") for x in ("k_scale_tok", "v_scale_tok")}
    q = torch.randn((len(seq), H * G, D), device="cuda", generator=gen).to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(qkv.qkv_masked_attn_workspace(qkv.FORMATS[fmt], len(seq), seqs_n, H * G, H, D, length), dtype=torch.uint8, device="cuda")
    graphs = []
    for end in (full, some):
        step = lambda: qkv.qkv_masked_attn(q, qkv.FORMATS[fmt], k, v, table, seq, end, block, D ** -0.5, max_row_end=length,  # noqa: E731, B023
                                           num_kv_heads=H, out=out, workspace=ws, **kw)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                step()
        graphs.append(g)
    times = [[], []]
    for _ in range(25):
        for i, g in enumerate(graphs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            times[i].append(a.elapsed_time(b))
    assert min(times[1]) <= 1.15 * min(times[0]), (min(times[0]), min(times[1]))
