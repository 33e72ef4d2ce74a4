"""One named case of the library's kernels, launched a few times: the command a profiler wraps.

    python -m quantized_kv_cache_write_gb300.profile_cases <case> [--launches N]

Each case builds its slot pool with the library's own write kernels from the seeded
generator's inputs (the append and prefix cases: from seeded random values on the device), then launches
the case's call N times (default 3), each after an L2
flush (a 256 MiB write), and synchronises. Profile the last launch with
`-k regex:<kernel> -s <N - 1> -c 1`. Cases:

  page1_<fmt>        2048 rows x top-k 1024 over 262144 slots, fmt = int8_side, int8_inline,
                     e4m3 or bf16 ("int8 per-(token,head) KV cache for the Qwen3.8-Flash-Next
                     QSA path", §The finding worth upstreaming)
  page1_tcgen05      the same, int8 side, QSA_ENGINE_TCGEN05
  page1_gqa32        the same, int8 side, 32 query heads on one KV head
  page1_hd128        the same, int8 side, head_dim 128 (128 B of codes per head row)
  e4m3_layer         one calibrated E4M3 layer: 64 rows x top-k 2051 over 131072 slots, fused
                     split-K at qsa_suggest_num_splits' count ("[Perf][SM70][FP8] Hoist QSA
                     E4M3 KV scales", §Combined SM70 validation provenance)
  long_context       40 rows x top-k 2048 of 8 x 131072-token sequences, int8 side, fused at
                     the suggested split count
  mixed_<engine>     the 49-row catch-up/decode batch, E4M3, varlen, fused, 8 splits, engine =
                     default or persistent ("[Model][SM70][FP8] Add calibrated E4M3 QSA KV
                     cache", §Targeted mixed-batch scheduler regression)
  chunked_prefill    8192 causal rows (row i attends min(1024, i) of the 8192 tokens just
                     written into a 524288-slot int8 side pool), varlen
  write_<fmt>_fill   the page-1 pool fill: 262144 bf16 tokens written into a 262144-slot pool,
                     fmt = int8 (side tensors) or e4m3 (calibrated scales)
  merge_e4m3_layer   qsa_splitk_merge of the E4M3 layer's split partials (64 rows, 16 heads, P
                     from qsa_suggest_num_splits), the separate-merge path
  append_<fmt>       qkv_append_rope of an 8192-token chunk: int8 (16 + 1 heads of 256, side scales,
                     524288-slot pool) or bf16 (32 + 8 heads of 128)
  prefix_<fmt>       qkv_prefix_attn of a batch behind a shared prefix: int8 (64 rows x 16 heads of 256
                     behind 65536 keys), e4m3 (64 rows x 64 heads of 128, 8 KV heads, 32768 keys) or
                     bf16 (128 rows x 32 heads of 128, 4 KV heads, 8191 keys, up to 2048 of their own)
  dense_e4m3         the same call without a prefix: 64 rows x 64 heads of 128, up to 8192 keys each
  append_axes        qkv_append_axes of 8192 patches with three axes: 32 + 8 heads of 128, bf16
  read_int8          qkv_read of 131072 tokens of an int8 side pool (one head of 256) to bf16
  masked_<what>      qkv_masked_attn: prompt (4096 causal rows x 16 heads of 256, int8 side, capped), documents (8192
                     packed rows x 32 heads of 128, 4 KV heads, bf16) or decode (64 rows x 64 heads of 128, 8 KV heads,
                     up to 8192 e4m3 keys each, capped)
"""

from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_kv_cache_write_gb300 as q  # noqa: E402
from gen import (chunked_prefill, e4m3_splitk_layer, long_context_decode, mixed_catchup_decode,  # noqa: E402
                 page1_shape, small_random)

CASES = ["page1_int8_side", "page1_int8_inline", "page1_e4m3", "page1_bf16", "page1_tcgen05", "page1_gqa32",
         "page1_hd128", "e4m3_layer", "long_context", "mixed_default", "mixed_persistent", "chunked_prefill",
         "write_int8_fill", "write_e4m3_fill", "merge_e4m3_layer", "append_int8", "append_bf16", "prefix_int8",
         "prefix_e4m3", "prefix_bf16", "dense_e4m3", "append_axes", "read_int8", "masked_prompt", "masked_documents",
         "masked_decode"]


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _pool(wl, fmt):
    """The workload's tokens written by the library: caches and the gather's scale arguments."""
    S, H, D = wl.num_slots, wl.num_kv_heads, wl.head_dim
    k, v, slots = _dev(wl.k_tokens), _dev(wl.v_tokens), torch.from_numpy(wl.slot_mapping).cuda()
    if fmt == "bf16":
        kc = torch.zeros((S, H, D), dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        kc[slots], vc[slots] = k, v
        return kc, vc, {}
    if fmt in ("int8_side", "int8_inline"):
        side = fmt == "int8_side"
        kc = torch.zeros((S, H, D if side else D + 4), dtype=torch.int8 if side else torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        if side:
            ks = torch.zeros((S, H), dtype=torch.float32, device="cuda")
            vs = torch.zeros_like(ks)
            q.qkv_write_int8(k, v, slots, kc, vc, ks, vs)
            return kc, vc, dict(k_scale_tok=ks, v_scale_tok=vs)
        q.qkv_write_int8(k, v, slots, kc, vc, layout=q.QKV_INT8_INLINE)
        return kc, vc, {}
    amax = torch.zeros(1, dtype=torch.int32, device="cuda")
    sc = torch.zeros(2, dtype=torch.float32, device="cuda")
    q.qkv_e4m3_calibrate(k, amax, sc[0:1])
    q.qkv_e4m3_calibrate(v, amax, sc[1:2])
    ksl, vsl = sc.tolist()
    kc = torch.zeros((S, H, D), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    q.qkv_write_e4m3(k, v, slots, kc, vc, ksl, vsl)
    return kc, vc, dict(k_scale_layer=ksl, v_scale_layer=vsl)


def _append(case: str):
    fmt, Hq, H, D, S = ("int8_side", 16, 1, 256, 524288) if case == "append_int8" else ("bf16", 32, 8, 128, 65536)
    T, gen = 8192, torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randn((T, Hq + 2 * H, D), device="cuda", generator=gen).to(torch.bfloat16)
    ang = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
        -torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, 131072, (T,), device="cuda", generator=gen).int()
    slots = torch.randperm(S, device="cuda", generator=gen)[:T]
    kc = torch.zeros((S, H, D), dtype=torch.bfloat16 if fmt == "bf16" else torch.int8, device="cuda")
    vc, q_out = torch.zeros_like(kc), torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    kw = {} if fmt == "bf16" else {n: torch.zeros((S, H), device="cuda") for n in ("k_scale", "v_scale")}
    return lambda: q.qkv_append_rope(packed[:, Hq:Hq + H], packed[:, Hq + H:], q.FORMATS[fmt], kc, vc, cs, pos,
                                     q=packed[:, :Hq], q_out=q_out, slot_mapping=slots, **kw)


def _prefix(case: str):
    fmt, rows, Hq, H, D, P, own, block = {
        "prefix_int8": ("int8_side", 64, 16, 1, 256, 65536, 64, 16),
        "prefix_e4m3": ("e4m3", 64, 64, 8, 128, 32768, 512, 64),
        "prefix_bf16": ("bf16", 128, 32, 4, 128, 8191, 2048, 32),
        "dense_e4m3": ("e4m3", 64, 64, 8, 128, 0, 8192, 64)}[case]
    gen = torch.Generator(device="cuda").manual_seed(2)
    lens = [P + 1 + (own - 1) * i // (rows - 1) for i in range(rows)]
    wide = -(-max(lens) // block)
    shared, mine = -(-P // block), wide - P // block
    S = (shared + rows * mine) * block
    ids = torch.randperm(shared + rows * mine, device="cuda", generator=gen).int()
    table = torch.full((rows, wide), -1, dtype=torch.int32, device="cuda")
    table[:, P // block:] = ids[shared:].view(rows, mine)
    kw = {}
    if fmt == "bf16":
        kc, vc = (torch.randn((S, H, D), device="cuda", generator=gen).to(torch.bfloat16) for _ in "kv")
    elif fmt == "e4m3":
        kc, vc = (torch.randn((S, H, D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8)
                  for _ in "kv")
    else:
        kc, vc = (torch.randint(-127, 128, (S, H, D), device="cuda", generator=gen, dtype=torch.int8) for _ in "kv")
        kw = {n: torch.full((S, H), 0.02, device="cuda") for n in ("k_scale_tok", "v_scale_tok")}
    qd = torch.randn((rows, Hq, D), device="cuda", generator=gen).to(torch.bfloat16)
    out = torch.empty_like(qd)
    seq, ln = torch.arange(rows, device="cuda").int(), torch.tensor(lens, device="cuda").int()
    ws = torch.empty(q.qkv_prefix_attn_workspace(q.FORMATS[fmt], rows, Hq, H, D, P, max(lens)), dtype=torch.uint8,
                     device="cuda")
    return lambda: q.qkv_prefix_attn(qd, q.FORMATS[fmt], kc, vc, table, seq, ln, block, D ** -0.5, max_row_len=max(lens),
                                     num_kv_heads=H, prefix_blocks=ids[:shared], prefix_len=P, out=out, workspace=ws,
                                     **kw)


def _append_axes():
    T, Hq, H, D, S = 8192, 32, 8, 128, 65536
    gen = torch.Generator(device="cuda").manual_seed(3)
    packed = torch.randn((T, Hq + 2 * H, D), device="cuda", generator=gen).to(torch.bfloat16)
    ang = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
        -torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    t = torch.arange(T, device="cuda")
    axis_pos = torch.stack([t // 1024, t // 32 % 32, t % 32]).int()  # frames of 32 x 32 patches
    slots = torch.randperm(S, device="cuda", generator=gen)[:T]
    kc = torch.zeros((S, H, D), dtype=torch.bfloat16, device="cuda")
    vc, q_out = torch.zeros_like(kc), torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    pair_axis = [0] * 16 + [1] * 24 + [2] * 24
    return lambda: q.qkv_append_axes(packed[:, Hq:Hq + H], packed[:, Hq + H:], q.QKV_BF16, kc, vc, cs, axis_pos, pair_axis,
                                     q=packed[:, :Hq], q_out=q_out, slot_mapping=slots)


def _read_int8():
    T, H, D, S = 131072, 1, 256, 262144
    gen = torch.Generator(device="cuda").manual_seed(4)
    kc, vc = (torch.randint(-127, 128, (S, H, D), device="cuda", generator=gen, dtype=torch.int8) for _ in "kv")
    ks, vs = (torch.rand((S, H), device="cuda", generator=gen) * 0.02 for _ in "kv")
    slots = torch.randperm(S, device="cuda", generator=gen)[:T]
    k_out, v_out = (torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    return lambda: q.qkv_read(q.QKV_INT8_SIDE, kc, vc, k_out=k_out, v_out=v_out, slot_mapping=slots, k_scale=ks, v_scale=vs)


def _masked(case: str):
    fmt, seqs, rows, keys, Hq, H, D, block, cap = {
        "masked_prompt": ("int8_side", 1, 4096, 4096, 16, 1, 256, 16, 30.0),
        "masked_documents": ("bf16", 4, 2048, 2048, 32, 4, 128, 16, 0.0),
        "masked_decode": ("e4m3", 64, 1, 8192, 64, 8, 128, 16, 50.0)}[case]
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = keys // block
    S = seqs * wide * block
    table = torch.randperm(seqs * wide, device="cuda", generator=gen).int().view(seqs, wide)
    row_seq = torch.arange(seqs, device="cuda").int().repeat_interleave(rows)
    row_end = torch.arange(1, rows + 1, device="cuda").int().repeat(seqs)
    start = None
    if case == "masked_documents":
        start = (row_end - 1) // 256 * 256
    if rows == 1:
        row_end = torch.randint(1, keys + 1, (seqs,), device="cuda", generator=gen).int()
    kw = {}
    if fmt == "bf16":
        kc, vc = (torch.randn((S, H, D), device="cuda", generator=gen).to(torch.bfloat16) for _ in "kv")
    elif fmt == "e4m3":
        kc, vc = (torch.randn((S, H, D), device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8)
                  for _ in "kv")
    else:
        kc, vc = (torch.randint(-127, 128, (S, H, D), device="cuda", generator=gen, dtype=torch.int8) for _ in "kv")
        kw = {n: torch.full((S, H), 0.02, device="cuda") for n in ("k_scale_tok", "v_scale_tok")}
    qd = torch.randn((seqs * rows, Hq, D), device="cuda", generator=gen).to(torch.bfloat16)
    out = torch.empty_like(qd)
    ws = torch.empty(q.qkv_masked_attn_workspace(q.FORMATS[fmt], seqs * rows, seqs, Hq, H, D, keys), dtype=torch.uint8,
                     device="cuda")
    return lambda: q.qkv_masked_attn(qd, q.FORMATS[fmt], kc, vc, table, row_seq, row_end, block, D ** -0.5,
                                     max_row_end=keys, num_kv_heads=H, row_start=start, softcap=cap, out=out, workspace=ws,
                                     **kw)


def build(case: str):
    """The case's launch as a closure (inputs resident on the device)."""
    if case.startswith("page1_"):
        what = case[len("page1_"):]
        if what == "gqa32":
            wl, fmt = small_random(11, num_slots=262144, rows=2048, topk=1024, outlier_frac=0.01, num_q_heads=32), \
                "int8_side"
        elif what == "hd128":
            wl, fmt = small_random(11, num_slots=262144, rows=2048, topk=1024, outlier_frac=0.01, head_dim=128), \
                "int8_side"
        else:
            wl, fmt = page1_shape(1, with_step=False), ("int8_side" if what == "tcgen05" else what)
        kc, vc, kw = _pool(wl, fmt)
        qd, idx = _dev(wl.q), torch.from_numpy(np.ascontiguousarray(wl.topk, dtype=np.int32)).cuda()
        out = torch.empty((wl.rows, wl.num_q_heads, wl.head_dim), dtype=torch.float32, device="cuda")
        engine = q.QSA_ENGINE_TCGEN05 if what == "tcgen05" else q.QSA_ENGINE_DEFAULT
        return lambda: q.qsa_gather_attn_ex(qd, q.FORMATS[fmt], kc, vc, idx, wl.softmax_scale, out=out,
                                            engine=engine, **kw)
    if case in ("e4m3_layer", "long_context"):
        wl, fmt = (e4m3_splitk_layer(0), "e4m3") if case == "e4m3_layer" else (long_context_decode(3), "int8_side")
        kc, vc, kw = _pool(wl, fmt)
        qd, idx = _dev(wl.q), torch.from_numpy(np.ascontiguousarray(wl.topk, dtype=np.int32)).cuda()
        R, Hq, D = wl.rows, wl.num_q_heads, wl.head_dim
        P = q.qsa_suggest_num_splits(q.FORMATS[fmt], R, Hq, wl.num_kv_heads, wl.topk.shape[1])
        out = torch.empty((R, Hq, D), dtype=torch.float32, device="cuda")
        o_part = torch.empty((R, P, Hq, D), dtype=torch.float32, device="cuda")
        lse_part = torch.empty((R, P, Hq), dtype=torch.float32, device="cuda")
        counters = torch.zeros((R, wl.num_kv_heads, 1), dtype=torch.int32, device="cuda")
        return lambda: q.qsa_gather_attn_splitk_fused(qd, q.FORMATS[fmt], kc, vc, idx, wl.softmax_scale, num_splits=P,
                                                      out=out, o_part=o_part, lse_part=lse_part, counters=counters,
                                                      **kw)
    if case in ("mixed_default", "mixed_persistent"):
        wl = mixed_catchup_decode(6)
        kc, vc, kw = _pool(wl, "e4m3")
        qd, idx = _dev(wl.q), torch.from_numpy(np.ascontiguousarray(wl.topk, dtype=np.int32)).cuda()
        lens = torch.from_numpy(wl.row_len).cuda()
        R, Hq, D, P = wl.rows, wl.num_q_heads, wl.head_dim, wl.num_splits
        out = torch.empty((R, Hq, D), dtype=torch.float32, device="cuda")
        o_part = torch.empty((R, P, Hq, D), dtype=torch.float32, device="cuda")
        lse_part = torch.empty((R, P, Hq), dtype=torch.float32, device="cuda")
        counters = torch.zeros((R, 1, 1), dtype=torch.int32, device="cuda")
        sched = torch.zeros(2, dtype=torch.int32, device="cuda")
        engine = q.QSA_ENGINE_PERSISTENT if case == "mixed_persistent" else q.QSA_ENGINE_DEFAULT
        return lambda: q.qsa_gather_attn_ex(qd, q.QKV_E4M3, kc, vc, idx, wl.softmax_scale, num_splits=P, out=out,
                                            o_part=o_part, lse_part=lse_part, counters=counters, topk_len=lens,
                                            engine=engine, sched=sched if engine == q.QSA_ENGINE_PERSISTENT else None,
                                            **kw)
    if case == "chunked_prefill":
        wl = chunked_prefill(4)
        kc, vc, kw = _pool(wl, "int8_side")
        qd, idx = _dev(wl.q), torch.from_numpy(np.ascontiguousarray(wl.topk, dtype=np.int32)).cuda()
        lens = torch.from_numpy(np.minimum(np.arange(wl.rows), wl.topk.shape[1]).astype(np.int32)).cuda()
        out = torch.empty((wl.rows, wl.num_q_heads, wl.head_dim), dtype=torch.float32, device="cuda")
        return lambda: q.qsa_gather_attn_varlen(qd, q.QKV_INT8_SIDE, kc, vc, idx, lens, wl.softmax_scale, out=out,
                                                **kw)
    if case in ("write_int8_fill", "write_e4m3_fill"):
        wl = page1_shape(1, with_step=False)
        S, H, D = wl.num_slots, wl.num_kv_heads, wl.head_dim
        k, v, slots = _dev(wl.k_tokens), _dev(wl.v_tokens), torch.from_numpy(wl.slot_mapping).cuda()
        kc = torch.zeros((S, H, D), dtype=torch.int8 if case == "write_int8_fill" else torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        if case == "write_int8_fill":
            ks = torch.zeros((S, H), dtype=torch.float32, device="cuda")
            vs = torch.zeros_like(ks)
            return lambda: q.qkv_write_int8(k, v, slots, kc, vc, ks, vs)
        amax = torch.zeros(1, dtype=torch.int32, device="cuda")
        sc = torch.zeros(2, dtype=torch.float32, device="cuda")
        q.qkv_e4m3_calibrate(k, amax, sc[0:1])
        q.qkv_e4m3_calibrate(v, amax, sc[1:2])
        ksl, vsl = sc.tolist()
        return lambda: q.qkv_write_e4m3(k, v, slots, kc, vc, ksl, vsl)
    if case == "merge_e4m3_layer":
        wl = e4m3_splitk_layer(0)
        kc, vc, kw = _pool(wl, "e4m3")
        qd, idx = _dev(wl.q), torch.from_numpy(np.ascontiguousarray(wl.topk, dtype=np.int32)).cuda()
        R, Hq, D = wl.rows, wl.num_q_heads, wl.head_dim
        P = q.qsa_suggest_num_splits(q.QKV_E4M3, R, Hq, wl.num_kv_heads, wl.topk.shape[1])
        o_part = torch.empty((R, P, Hq, D), dtype=torch.float32, device="cuda")
        lse_part = torch.empty((R, P, Hq), dtype=torch.float32, device="cuda")
        q.qsa_gather_attn(qd, q.QKV_E4M3, kc, vc, idx, wl.softmax_scale, num_splits=P, o_part=o_part,
                          lse_part=lse_part, **kw)
        out = torch.empty((R, Hq, D), dtype=torch.float32, device="cuda")
        lse = torch.empty((R, Hq), dtype=torch.float32, device="cuda")
        return lambda: q.qsa_splitk_merge(o_part, lse_part, out, lse, v_scale_post=float(kw["v_scale_layer"]))
    if case in ("append_int8", "append_bf16"):
        return _append(case)
    if case in ("prefix_int8", "prefix_e4m3", "prefix_bf16", "dense_e4m3"):
        return _prefix(case)
    if case == "append_axes":
        return _append_axes()
    if case == "read_int8":
        return _read_int8()
    if case in ("masked_prompt", "masked_documents", "masked_decode"):
        return _masked(case)
    raise SystemExit(f"unknown case {case!r}; one of {', '.join(CASES)}")


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("case", choices=CASES)
    ap.add_argument("--launches", type=int, default=3)
    args = ap.parse_args()
    if not torch.cuda.is_available():
        raise SystemExit("profile_cases needs a CUDA device")
    run = build(args.case)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for i in range(args.launches):
        flush.fill_(i & 0xFF)
        run()
    torch.cuda.synchronize()
    print(f"{args.case}: {args.launches} launches done")


if __name__ == "__main__":
    main()
