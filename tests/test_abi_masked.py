"""Refusals of qkv_masked_attn without a GPU: the C ABI's checks come before any CUDA call, the binding's before the
library's; and the descriptor matches the header."""

import ctypes

import pytest
import torch

from test_abi_axes_read import header_fields
from test_abi_dense import FAKE, lib  # noqa: F401  (the built library)


def masked(lib, **over):
    d = lib.MaskedDesc()
    a = dict(size=ctypes.sizeof(lib.MaskedDesc), fmt=lib.QKV_INT8_SIDE, q_fp16=0, q=FAKE, q_stride=1024, rows=4,
             num_q_heads=8, num_kv_heads=2, head_dim=128, k_cache=FAKE, v_cache=FAKE, k_scale_tok=FAKE, v_scale_tok=FAKE,
             k_scale_layer=1.0, v_scale_layer=1.0, num_slots=64, block_table=FAKE, num_seqs=2, max_blocks=4, block_size=16,
             row_seq=FAKE, row_start=FAKE, row_end=FAKE, row_pos=FAKE, max_row_end=40, window=8, softmax_scale=0.1,
             softcap=30.0, slopes=FAKE, out=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(over)
    for n, x in a.items():
        setattr(d, n, x)
    return lib.lib.qkv_masked_attn(ctypes.byref(d), None)


def test_masked_refusals(lib):  # noqa: F811
    E = lib
    assert lib.lib.qkv_masked_attn(None, None) == E.QKV_ERR_ARG
    assert masked(lib, size=8) == E.QKV_ERR_ARG
    assert masked(lib, rows=0) == E.QKV_OK
    assert masked(lib, rows=-1) == E.QKV_ERR_ARG
    assert masked(lib, rows=1 << 29) == E.QKV_ERR_ARG  # (row, head) pairs are numbered in 32 bits
    assert masked(lib, head_dim=96) == E.QKV_ERR_UNSUPPORTED
    assert masked(lib, num_q_heads=9) == E.QKV_ERR_ARG
    assert masked(lib, num_q_heads=260, q_stride=1 << 16) == E.QKV_ERR_UNSUPPORTED
    assert masked(lib, num_kv_heads=0) == E.QKV_ERR_ARG
    assert masked(lib, fmt=5) == E.QKV_ERR_ARG
    assert masked(lib, q_fp16=3) == E.QKV_ERR_ARG
    kw = dict(k_scale_tok=None, v_scale_tok=None)
    assert masked(lib, fmt=E.QKV_BF16, q_fp16=1, **kw) == E.QKV_ERR_ARG
    assert masked(lib, fmt=E.QKV_F16, **kw) == E.QKV_ERR_ARG
    assert masked(lib, v_scale_tok=None) == E.QKV_ERR_ARG
    assert masked(lib, fmt=E.QKV_E4M3) == E.QKV_ERR_ARG
    for bad in (float("nan"), float("inf")):
        assert masked(lib, softmax_scale=bad) == E.QKV_ERR_ARG
    for bad in (float("nan"), float("inf"), -1.0, 1e-7, 2e6):
        assert masked(lib, softcap=bad) == E.QKV_ERR_ARG, bad
    for bad in (-1.0, 0.0, float("nan"), float("inf")):
        assert masked(lib, fmt=E.QKV_E4M3, k_scale_layer=bad, **kw) == E.QKV_ERR_SCALE
        assert masked(lib, fmt=E.QKV_E4M3, v_scale_layer=bad, **kw) == E.QKV_ERR_SCALE
    assert masked(lib, window=-1) == E.QKV_ERR_ARG
    assert masked(lib, max_row_end=-1) == E.QKV_ERR_ARG
    assert masked(lib, max_row_end=65) == E.QKV_ERR_ARG  # past the table
    assert masked(lib, max_row_end=(1 << 30) + 1, max_blocks=1 << 28, block_size=7) == E.QKV_ERR_ARG
    for name in ("num_seqs", "max_blocks", "block_size"):
        assert masked(lib, **{name: 0}) == E.QKV_ERR_ARG, name
    assert masked(lib, block_size=1 << 30) == E.QKV_ERR_ARG
    assert masked(lib, num_slots=1 << 30) == E.QKV_ERR_UNSUPPORTED
    assert masked(lib, num_slots=-1) == E.QKV_ERR_ARG
    for name in ("q", "out", "k_cache", "v_cache", "block_table", "row_seq", "row_end"):
        assert masked(lib, **{name: None}) == E.QKV_ERR_ARG, name
    for name in ("q", "out", "k_cache", "v_cache", "workspace"):
        assert masked(lib, **{name: FAKE + 8}) == E.QKV_ERR_ALIGN, name
    for name in ("block_table", "row_seq", "row_start", "row_end", "row_pos", "slopes", "lse", "dev_status", "k_scale_tok"):
        assert masked(lib, **{name: FAKE + 2}) == E.QKV_ERR_ALIGN, name
    assert masked(lib, q_stride=1016) == E.QKV_ERR_ARG
    assert masked(lib, q_stride=1028) == E.QKV_ERR_ALIGN


def test_workspace_refusals(lib):  # noqa: F811
    E, n = lib, ctypes.c_size_t(0)
    f = lambda *a: lib.lib.qkv_masked_attn_workspace(*a, ctypes.byref(n))  # noqa: E731
    assert f(E.QKV_E4M3, 4, 1, 8, 3, 128, 10, 0) == E.QKV_ERR_ARG
    assert f(E.QKV_E4M3, 4, 1, 8, 2, 100, 10, 0) == E.QKV_ERR_UNSUPPORTED
    assert f(E.QKV_E4M3, 4, 0, 8, 2, 128, 10, 0) == E.QKV_ERR_ARG
    assert f(E.QKV_E4M3, 4, 1, 8, 2, 128, -1, 0) == E.QKV_ERR_ARG
    assert f(E.QKV_E4M3, 4, 1, 8, 2, 128, 10, -1) == E.QKV_ERR_ARG
    assert f(7, 4, 1, 8, 2, 128, 10, 0) == E.QKV_ERR_ARG
    assert lib.lib.qkv_masked_attn_workspace(E.QKV_E4M3, 4, 1, 8, 2, 128, 10, 0, None) == E.QKV_ERR_ARG


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros((4, 8, 128))), "q must"),
    (dict(q=torch.zeros((4, 8 * 128), dtype=torch.bfloat16)), "q must"),
    (dict(num_kv_heads=1), "k_cache"),
    (dict(v_cache=torch.zeros((8, 2, 128), dtype=torch.int8)), "slots"),
    (dict(fmt=2), "k_cache"),
    (dict(block_table=torch.zeros(8, dtype=torch.int32)), "block_table"),
    (dict(block_table=torch.zeros((2, 4), dtype=torch.int64)), "block_table"),
    (dict(row_seq=torch.zeros(3, dtype=torch.int32)), "row_seq"),
    (dict(row_end=torch.zeros(4)), "row_end"),
    (dict(row_start=torch.zeros(5, dtype=torch.int32)), "row_start"),
    (dict(row_pos=torch.zeros(4, dtype=torch.int64)), "row_pos"),
    (dict(slopes=torch.zeros(4)), "slopes"),
    (dict(slopes=torch.zeros(8, dtype=torch.float64)), "slopes"),
    (dict(out=torch.zeros((4, 8, 128))), "out"),
    (dict(lse=torch.zeros((4, 4))), "lse"),
    (dict(k_scale_tok=torch.zeros((9, 1))), "k_scale_tok"),
    (dict(workspace=torch.zeros((4, 8)).t()), "workspace"),
    (dict(), "CUDA device"),
])
def test_masked_binding_refuses(lib, change, match):  # noqa: F811
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kw = dict(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16), fmt=1, k_cache=torch.zeros((9, 2, 128), dtype=torch.int8),
              v_cache=torch.zeros((9, 2, 128), dtype=torch.int8), block_table=i32(2, 4), row_seq=i32(4), row_end=i32(4),
              block_size=16, softmax_scale=0.1, max_row_end=40, num_kv_heads=2, k_scale_tok=torch.zeros((9, 2)),
              v_scale_tok=torch.zeros((9, 2)), out=torch.zeros((4, 8, 128), dtype=torch.bfloat16))
    kw.update(change)
    with pytest.raises(ValueError, match=match):
        lib.qkv_masked_attn(kw.pop("q"), kw.pop("fmt"), kw.pop("k_cache"), kw.pop("v_cache"), kw.pop("block_table"),
                            kw.pop("row_seq"), kw.pop("row_end"), kw.pop("block_size"), kw.pop("softmax_scale"), **kw)


def test_descriptor_matches_the_header_and_is_packed_alike(lib):  # noqa: F811
    assert [(n, t) for n, t in lib.MaskedDesc._fields_] == header_fields("qkv_masked_desc")
    pack = next(c.cell_contents for c in lib._call_masked.__closure__ if getattr(c.cell_contents, "__name__", "") == "pack")
    values = [float(i) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(lib.MaskedDesc._fields_)]
    assert pack(*values) == bytes(lib.MaskedDesc(*values))
