"""Refusals of the dense cache operators without a GPU: the host-side validation of the C ABI returns
before any CUDA call, and the binding refuses tensors that disagree before it calls the library.

The fail-closed scale gate follows "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Non-obvious
design decisions."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import quantized_kv_cache_write_gb300 as q
    return q


FAKE = 0x10000  # never dereferenced: the calls fail first


def append(lib, **over):
    d = lib.AppendDesc()
    a = dict(size=ctypes.sizeof(lib.AppendDesc), fmt=lib.QKV_INT8_SIDE, act_fp16=0, q=FAKE, q_out=FAKE, k=FAKE, v=FAKE,
             num_tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=128, q_stride=1024, q_out_stride=1024, kv_stride=256,
             cos_sin=FAKE, num_positions=100, rotary_dim=64, interleaved=0, token_pos=FAKE, slot_mapping=FAKE,
             k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, k_scale_layer=1.0, v_scale_layer=1.0, num_slots=64)
    a.update(over)
    for n, x in a.items():
        setattr(d, n, x)
    return lib.lib.qkv_append_rope(ctypes.byref(d), None)


def test_append_refusals(lib):
    E = lib
    assert lib.lib.qkv_append_rope(None, None) == E.QKV_ERR_ARG
    assert append(lib, size=8) == E.QKV_ERR_ARG
    assert append(lib, num_tokens=0) == E.QKV_OK
    assert append(lib, num_tokens=-1) == E.QKV_ERR_ARG
    assert append(lib, head_dim=64) == E.QKV_ERR_UNSUPPORTED
    assert append(lib, fmt=9) == E.QKV_ERR_ARG
    assert append(lib, act_fp16=2) == E.QKV_ERR_ARG
    for fmt, f16 in ((E.QKV_BF16, 1), (E.QKV_F16, 0)):  # a 16-bit pool takes its own type
        assert append(lib, fmt=fmt, act_fp16=f16, k_scale=None, v_scale=None) == E.QKV_ERR_ARG
    for rot in (0, 8, 24, 130, 144, -16):
        assert append(lib, rotary_dim=rot) == E.QKV_ERR_ARG, rot
    assert append(lib, interleaved=2) == E.QKV_ERR_ARG
    assert append(lib, num_positions=-1) == E.QKV_ERR_ARG
    assert append(lib, q=None) == E.QKV_ERR_ARG  # q without q_out
    assert append(lib, num_q_heads=0) == E.QKV_ERR_ARG
    assert append(lib, q_stride=1016) == E.QKV_ERR_ARG
    assert append(lib, q_out_stride=1028) == E.QKV_ERR_ALIGN
    assert append(lib, kv_stride=248) == E.QKV_ERR_ARG
    assert append(lib, kv_stride=260) == E.QKV_ERR_ALIGN
    for name in ("k", "v", "k_cache", "v_cache", "token_pos", "cos_sin"):
        assert append(lib, **{name: None}) == E.QKV_ERR_ARG, name
    for name in ("q", "q_out", "k", "v", "k_cache", "v_cache", "cos_sin"):
        assert append(lib, **{name: FAKE + 8}) == E.QKV_ERR_ALIGN, name
    for name in ("token_pos", "k_scale", "dev_status"):
        assert append(lib, **{name: FAKE + 2}) == E.QKV_ERR_ALIGN, name
    assert append(lib, k_scale=None) == E.QKV_ERR_ARG
    assert append(lib, fmt=E.QKV_E4M3) == E.QKV_ERR_ARG  # per-token scales belong to the side layout
    assert append(lib, num_tokens=1 << 31) == E.QKV_ERR_ARG  # more rows than one launch's grid holds
    # addressing: one of the two
    assert append(lib, token_seq=FAKE) == E.QKV_ERR_ARG
    paged = dict(slot_mapping=None, token_seq=FAKE, block_table=FAKE, num_seqs=2, max_blocks=4, block_size=16)
    for name, x in (("token_seq", None), ("block_table", None), ("num_seqs", 0), ("max_blocks", 0), ("block_size", 0),
                    ("block_size", 1 << 30)):
        assert append(lib, **{**paged, name: x}) == E.QKV_ERR_ARG, name
    assert append(lib, **{**paged, "block_table": FAKE + 2}) == E.QKV_ERR_ALIGN


@pytest.mark.parametrize("bad", [-1.0, 0.0, float("nan"), float("inf")])
def test_append_scale_gate_fails_closed(lib, bad):
    kw = dict(fmt=lib.QKV_E4M3, k_scale=None, v_scale=None)
    assert append(lib, k_scale_layer=bad, **kw) == lib.QKV_ERR_SCALE
    assert append(lib, v_scale_layer=bad, **kw) == lib.QKV_ERR_SCALE


def prefix(lib, **over):
    d = lib.PrefixDesc()
    a = dict(size=ctypes.sizeof(lib.PrefixDesc), fmt=lib.QKV_INT8_SIDE, q_fp16=0, q=FAKE, q_stride=1024, rows=4,
             num_q_heads=8, num_kv_heads=2, head_dim=128, k_cache=FAKE, v_cache=FAKE, k_scale_tok=FAKE, v_scale_tok=FAKE,
             k_scale_layer=1.0, v_scale_layer=1.0, num_slots=64, prefix_blocks=FAKE, prefix_len=20, block_table=FAKE,
             num_seqs=2, max_blocks=4, block_size=16, row_seq=FAKE, row_len=FAKE, max_row_len=40, softmax_scale=0.1,
             out=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(over)
    for n, x in a.items():
        setattr(d, n, x)
    return lib.lib.qkv_prefix_attn(ctypes.byref(d), None)


def test_prefix_refusals(lib):
    E = lib
    assert lib.lib.qkv_prefix_attn(None, None) == E.QKV_ERR_ARG
    assert prefix(lib, size=8) == E.QKV_ERR_ARG
    assert prefix(lib, rows=0) == E.QKV_OK
    assert prefix(lib, rows=-1) == E.QKV_ERR_ARG
    assert prefix(lib, rows=1 << 29) == E.QKV_ERR_ARG  # (row, head) pairs are numbered in 32 bits
    assert prefix(lib, head_dim=96) == E.QKV_ERR_UNSUPPORTED
    assert prefix(lib, num_q_heads=9) == E.QKV_ERR_ARG
    assert prefix(lib, num_q_heads=260, q_stride=1 << 16) == E.QKV_ERR_UNSUPPORTED  # a group of 130
    assert prefix(lib, num_kv_heads=0) == E.QKV_ERR_ARG
    assert prefix(lib, fmt=5) == E.QKV_ERR_ARG
    assert prefix(lib, q_fp16=3) == E.QKV_ERR_ARG
    kw = dict(k_scale_tok=None, v_scale_tok=None)
    assert prefix(lib, fmt=E.QKV_BF16, q_fp16=1, **kw) == E.QKV_ERR_ARG
    assert prefix(lib, fmt=E.QKV_F16, **kw) == E.QKV_ERR_ARG
    assert prefix(lib, k_scale_tok=None) == E.QKV_ERR_ARG
    assert prefix(lib, fmt=E.QKV_E4M3) == E.QKV_ERR_ARG
    for bad in (float("nan"), float("inf")):
        assert prefix(lib, softmax_scale=bad) == E.QKV_ERR_ARG
    for bad in (-1.0, 0.0, float("nan"), float("inf")):
        assert prefix(lib, fmt=E.QKV_E4M3, k_scale_layer=bad, **kw) == E.QKV_ERR_SCALE
        assert prefix(lib, fmt=E.QKV_E4M3, v_scale_layer=bad, **kw) == E.QKV_ERR_SCALE
    assert prefix(lib, prefix_len=-1) == E.QKV_ERR_ARG
    assert prefix(lib, max_row_len=19) == E.QKV_ERR_ARG  # below the prefix
    assert prefix(lib, max_row_len=65) == E.QKV_ERR_ARG  # past the table
    assert prefix(lib, max_row_len=(1 << 30) + 1, max_blocks=1 << 28, block_size=7) == E.QKV_ERR_ARG
    for name in ("num_seqs", "max_blocks", "block_size"):
        assert prefix(lib, **{name: 0}) == E.QKV_ERR_ARG, name
    assert prefix(lib, block_size=1 << 30) == E.QKV_ERR_ARG
    assert prefix(lib, num_slots=1 << 30) == E.QKV_ERR_UNSUPPORTED
    assert prefix(lib, num_slots=-1) == E.QKV_ERR_ARG
    for name in ("q", "out", "k_cache", "v_cache", "block_table", "row_seq", "row_len", "prefix_blocks"):
        assert prefix(lib, **{name: None}) == E.QKV_ERR_ARG, name
    for name in ("q", "out", "k_cache", "v_cache", "workspace"):
        assert prefix(lib, **{name: FAKE + 8}) == E.QKV_ERR_ALIGN, name
    for name in ("block_table", "row_seq", "row_len", "prefix_blocks", "lse", "dev_status", "k_scale_tok"):
        assert prefix(lib, **{name: FAKE + 2}) == E.QKV_ERR_ALIGN, name
    assert prefix(lib, q_stride=1016) == E.QKV_ERR_ARG
    assert prefix(lib, q_stride=1028) == E.QKV_ERR_ALIGN


def test_workspace_refusals(lib):
    E, n = lib, ctypes.c_size_t(0)
    f = lambda *a: lib.lib.qkv_prefix_attn_workspace(*a, ctypes.byref(n))
    assert f(E.QKV_E4M3, 4, 8, 3, 128, 0, 10) == E.QKV_ERR_ARG
    assert f(E.QKV_E4M3, 4, 8, 2, 100, 0, 10) == E.QKV_ERR_UNSUPPORTED
    assert f(E.QKV_E4M3, 4, 8, 2, 128, 11, 10) == E.QKV_ERR_ARG
    assert f(7, 4, 8, 2, 128, 0, 10) == E.QKV_ERR_ARG
    assert lib.lib.qkv_prefix_attn_workspace(E.QKV_E4M3, 4, 8, 2, 128, 0, 10, None) == E.QKV_ERR_ARG


def _append_kw():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(k=torch.zeros((4, 2, 128), dtype=torch.bfloat16), v=torch.zeros((4, 2, 128), dtype=torch.bfloat16),
                fmt=1, k_cache=torch.zeros((9, 2, 128), dtype=torch.int8), v_cache=torch.zeros((9, 2, 128), dtype=torch.int8),
                cos_sin=torch.zeros((50, 64)), token_pos=i32(4), slot_mapping=torch.zeros(4, dtype=torch.int64),
                k_scale=torch.zeros((9, 2)), v_scale=torch.zeros((9, 2)))


@pytest.mark.parametrize("change,match", [
    (dict(k_cache=torch.zeros((9, 1, 128), dtype=torch.int8)), "k_cache"),
    (dict(v_cache=torch.zeros((8, 2, 128), dtype=torch.int8)), "slots"),
    (dict(v_cache=torch.zeros((9, 2, 128), dtype=torch.bfloat16)), "v_cache"),
    (dict(fmt=2), "k_cache"),
    (dict(fmt=12), "format"),
    (dict(cos_sin=torch.zeros(50)), "cos_sin"),
    (dict(cos_sin=torch.zeros((50, 64), dtype=torch.float64)), "cos_sin"),
    (dict(token_pos=torch.zeros(4, dtype=torch.int64)), "token_pos"),
    (dict(token_pos=torch.zeros(5, dtype=torch.int32)), "token_pos"),
    (dict(slot_mapping=torch.zeros(4, dtype=torch.int32)), "slot_mapping"),
    (dict(k_scale=torch.zeros((8, 2))), "k_scale"),
    (dict(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16)), "together"),
    (dict(q=torch.zeros((4, 8, 128), dtype=torch.float16), q_out=torch.zeros((4, 8, 128), dtype=torch.float16)), "q and q_out"),
    (dict(q=torch.zeros((3, 8, 128), dtype=torch.bfloat16), q_out=torch.zeros((3, 8, 128), dtype=torch.bfloat16)), "q must"),
    (dict(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16), q_out=torch.zeros((4, 7, 128), dtype=torch.bfloat16)), "q_out must"),
    (dict(q=torch.zeros((8, 4, 128), dtype=torch.bfloat16).transpose(0, 1), q_out=torch.zeros((4, 8, 128), dtype=torch.bfloat16)),
     "contiguous heads"),
    (dict(), "CUDA device"),
])
def test_append_binding_refuses(lib, change, match):
    with pytest.raises(ValueError, match=match):
        kw = {**_append_kw(), **change}
        lib.qkv_append_rope(kw.pop("k"), kw.pop("v"), kw.pop("fmt"), kw.pop("k_cache"), kw.pop("v_cache"), kw.pop("cos_sin"),
                            kw.pop("token_pos"), **kw)


def _prefix_kw():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16), fmt=1, k_cache=torch.zeros((9, 2, 128), dtype=torch.int8),
                v_cache=torch.zeros((9, 2, 128), dtype=torch.int8), block_table=i32(2, 4), row_seq=i32(4), row_len=i32(4),
                block_size=16, softmax_scale=0.1, max_row_len=40, num_kv_heads=2, prefix_blocks=i32(2), prefix_len=20,
                k_scale_tok=torch.zeros((9, 2)), v_scale_tok=torch.zeros((9, 2)),
                out=torch.zeros((4, 8, 128), dtype=torch.bfloat16))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros((4, 8, 128))), "q must"),
    (dict(q=torch.zeros((4, 8 * 128), dtype=torch.bfloat16)), "q must"),
    (dict(num_kv_heads=1), "k_cache"),
    (dict(v_cache=torch.zeros((8, 2, 128), dtype=torch.int8)), "slots"),
    (dict(block_table=torch.zeros(8, dtype=torch.int32)), "block_table"),
    (dict(block_table=torch.zeros((2, 4), dtype=torch.int64)), "block_table"),
    (dict(row_seq=torch.zeros(3, dtype=torch.int32)), "row_seq"),
    (dict(row_len=torch.zeros(4)), "row_len"),
    (dict(out=torch.zeros((4, 8, 128))), "out"),
    (dict(out=torch.zeros((3, 8, 128), dtype=torch.bfloat16)), "out"),
    (dict(lse=torch.zeros((4, 4))), "lse"),
    (dict(prefix_blocks=None), "prefix_blocks"),
    (dict(prefix_blocks=torch.zeros(1, dtype=torch.int32)), "cover"),
    (dict(k_scale_tok=torch.zeros((9, 1))), "k_scale_tok"),
    (dict(workspace=torch.zeros((4, 8)).t()), "workspace"),
    (dict(), "CUDA device"),
])
def test_prefix_binding_refuses(lib, change, match):
    kw = {**_prefix_kw(), **change}
    with pytest.raises(ValueError, match=match):
        lib.qkv_prefix_attn(kw.pop("q"), kw.pop("fmt"), kw.pop("k_cache"), kw.pop("v_cache"), kw.pop("block_table"),
                            kw.pop("row_seq"), kw.pop("row_len"), kw.pop("block_size"), kw.pop("softmax_scale"), **kw)


def test_descriptors_match_the_header(lib):
    """Field names, order and C types of the two descriptors, read from the header."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qkv.h")).read()
    for struct, name in ((lib.AppendDesc, "qkv_append_desc"), (lib.PrefixDesc, "qkv_prefix_desc")):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        c = {"size_t": ctypes.c_size_t, "qkv_format": ctypes.c_int, "int": ctypes.c_int, "int64_t": ctypes.c_int64,
             "float": ctypes.c_float}
        want = []
        for line in body.strip().splitlines():
            t, n = re.match(r"\s*((?:const )?\w+\*?)\s+(\w+);", line).groups()
            want.append((n, ctypes.c_void_p if t.endswith("*") else c[t]))
        assert [(n, t) for n, t in struct._fields_] == want


@pytest.mark.parametrize("field,value", [("max_row_len", 1 << 31), ("max_blocks", -(1 << 40)), ("softmax_scale", 1e300),
                                         ("workspace_bytes", -1), ("q", 1 << 64), ("head_dim", 128.5)])
def test_scalars_that_do_not_fit_the_descriptor_are_refused(lib, field, value):
    """Before anything is called: a size is never cut to its field's width."""
    import quantized_kv_cache_write_gb300 as qkv
    fields = [value if name == field else 0 for name, _ in qkv.PrefixDesc._fields_]
    with pytest.raises(ValueError, match="out of range"):
        qkv._call_prefix(0, None, *fields)


def test_packed_descriptors_equal_the_structures(lib):
    """The bytes that the binding passes are those of the structure, field for field."""
    import ctypes
    import struct
    import quantized_kv_cache_write_gb300 as qkv
    for desc, call in ((qkv.AppendDesc, qkv._call_append), (qkv.PrefixDesc, qkv._call_prefix)):
        pack = next(c.cell_contents for c in call.__closure__ if getattr(c.cell_contents, "__name__", "") == "pack")
        values = [float(i) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(desc._fields_)]
        assert pack(*values) == bytes(desc(*values)) and isinstance(pack.__self__, struct.Struct)
