"""Refusals of qkv_append_axes and qkv_read without a GPU: the C ABI's checks come before any CUDA call, the binding's
before the library's; and the descriptors match the header."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from test_abi_dense import FAKE, _append_kw, lib  # noqa: F401  (lib: the built library)


def axes(lib, pair_axis=None, **over):
    d = lib.AppendAxesDesc()
    a = dict(size=ctypes.sizeof(lib.AppendAxesDesc), fmt=lib.QKV_INT8_SIDE, act_fp16=0, q=FAKE, q_out=FAKE, k=FAKE, v=FAKE,
             num_tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=128, q_stride=1024, q_out_stride=1024, kv_stride=256,
             cos_sin=FAKE, num_positions=100, rotary_dim=64, interleaved=0, slot_mapping=FAKE, k_cache=FAKE, v_cache=FAKE,
             k_scale=FAKE, v_scale=FAKE, k_scale_layer=1.0, v_scale_layer=1.0, num_slots=64, axis_pos=FAKE, num_axes=3)
    a.update(over)
    for n, x in a.items():
        setattr(d, n, x)
    if pair_axis is not None:
        held = (ctypes.c_uint8 * len(pair_axis))(*pair_axis)
        d.pair_axis = ctypes.addressof(held)
    return lib.lib.qkv_append_axes(ctypes.byref(d), None)


def test_axes_refusals(lib):  # noqa: F811
    E = lib
    assert lib.lib.qkv_append_axes(None, None) == E.QKV_ERR_ARG
    assert axes(lib, size=ctypes.sizeof(lib.AppendDesc)) == E.QKV_ERR_ARG
    assert axes(lib, num_tokens=0) == E.QKV_OK
    assert axes(lib, num_tokens=0, axis_pos=None) == E.QKV_OK
    assert axes(lib, num_tokens=-1) == E.QKV_ERR_ARG
    assert axes(lib, head_dim=64) == E.QKV_ERR_UNSUPPORTED
    assert axes(lib, act_fp16=2) == E.QKV_ERR_ARG
    assert axes(lib, fmt=E.QKV_BF16, act_fp16=1, k_scale=None, v_scale=None) == E.QKV_ERR_ARG
    for rot in (0, 8, 24, 144, -16):
        assert axes(lib, rotary_dim=rot) == E.QKV_ERR_ARG, rot
    for n in (0, -1, 5):
        assert axes(lib, num_axes=n) == E.QKV_ERR_ARG, n
    assert axes(lib, axis_pos=None) == E.QKV_ERR_ARG
    assert axes(lib, axis_pos=FAKE + 2) == E.QKV_ERR_ALIGN
    assert axes(lib, [0] * 31 + [3]) == E.QKV_ERR_ARG  # an axis that there is not
    assert axes(lib, [255] + [0] * 31) == E.QKV_ERR_ARG
    assert axes(lib, token_pos=FAKE) == E.QKV_ERR_ARG  # belongs to the paged addressing
    assert axes(lib, token_seq=FAKE) == E.QKV_ERR_ARG
    paged = dict(slot_mapping=None, token_seq=FAKE, token_pos=FAKE, block_table=FAKE, num_seqs=2, max_blocks=4, block_size=16)
    for name in ("token_seq", "token_pos", "block_table"):
        assert axes(lib, **{**paged, name: None}) == E.QKV_ERR_ARG, name
        assert axes(lib, **{**paged, name: FAKE + 2}) == E.QKV_ERR_ALIGN, name
    for bad in (-1.0, 0.0, float("nan"), float("inf")):
        assert axes(lib, fmt=E.QKV_E4M3, k_scale=None, v_scale=None, v_scale_layer=bad) == E.QKV_ERR_SCALE


def read(lib, pair_axis=None, **over):
    d = lib.ReadDesc()
    a = dict(size=ctypes.sizeof(lib.ReadDesc), fmt=lib.QKV_INT8_SIDE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE,
             k_scale_layer=1.0, v_scale_layer=1.0, num_slots=64, num_kv_heads=2, head_dim=128, num_tokens=4, slot_mapping=FAKE,
             out_type=0, k_out=FAKE, v_out=FAKE, out_stride=256, cos_sin=FAKE, num_positions=100, rotary_dim=64,
             axis_pos=FAKE, num_axes=2)
    a.update(over)
    for n, x in a.items():
        setattr(d, n, x)
    if pair_axis is not None:
        held = (ctypes.c_uint8 * len(pair_axis))(*pair_axis)
        d.pair_axis = ctypes.addressof(held)
    return lib.lib.qkv_read(ctypes.byref(d), None)


def test_read_refusals(lib):  # noqa: F811
    E = lib
    assert lib.lib.qkv_read(None, None) == E.QKV_ERR_ARG
    assert read(lib, size=8) == E.QKV_ERR_ARG
    assert read(lib, num_tokens=0) == E.QKV_OK
    for name in ("num_tokens", "num_slots"):
        assert read(lib, **{name: -1}) == E.QKV_ERR_ARG, name
    assert read(lib, num_tokens=(1 << 31) + 1) == E.QKV_ERR_ARG
    assert read(lib, num_kv_heads=0) == E.QKV_ERR_ARG
    assert read(lib, head_dim=64) == E.QKV_ERR_UNSUPPORTED
    assert read(lib, fmt=5) == E.QKV_ERR_ARG
    for t in (-1, 3):
        assert read(lib, out_type=t) == E.QKV_ERR_ARG
    assert read(lib, k_scale=None) == E.QKV_ERR_ARG
    assert read(lib, fmt=E.QKV_E4M3) == E.QKV_ERR_ARG
    for bad in (-1.0, 0.0, float("nan"), float("inf")):
        assert read(lib, fmt=E.QKV_E4M3, k_scale=None, v_scale=None, k_scale_layer=bad) == E.QKV_ERR_SCALE
    assert read(lib, k_out=None, v_out=None) == E.QKV_ERR_ARG
    for name in ("k_cache", "v_cache", "axis_pos", "slot_mapping"):
        assert read(lib, **{name: None}) == E.QKV_ERR_ARG, name
    assert read(lib, cos_sin=None) == E.QKV_ERR_ARG  # positions without a table
    for rot in (0, 8, 24, 144):
        assert read(lib, rotary_dim=rot) == E.QKV_ERR_ARG, rot
    assert read(lib, interleaved=2) == E.QKV_ERR_ARG
    assert read(lib, num_axes=5) == E.QKV_ERR_ARG
    assert read(lib, [0] * 31 + [2]) == E.QKV_ERR_ARG
    assert read(lib, out_stride=248) == E.QKV_ERR_ARG
    assert read(lib, out_stride=260) == E.QKV_ERR_ALIGN
    for name in ("k_cache", "v_cache", "k_out", "v_out", "cos_sin"):
        assert read(lib, **{name: FAKE + 8}) == E.QKV_ERR_ALIGN, name
    for name in ("axis_pos", "k_scale", "dev_status"):
        assert read(lib, **{name: FAKE + 2}) == E.QKV_ERR_ALIGN, name
    assert read(lib, slot_mapping=FAKE + 4) == E.QKV_ERR_ALIGN
    for name in ("token_seq", "token_pos", "block_table"):
        assert read(lib, **{name: FAKE}) == E.QKV_ERR_ARG, name  # one addressing only
    paged = dict(slot_mapping=None, token_seq=FAKE, token_pos=FAKE, block_table=FAKE, num_seqs=2, max_blocks=4, block_size=16)
    for name, x in (("token_seq", None), ("token_pos", None), ("block_table", None), ("num_seqs", 0), ("max_blocks", 0),
                    ("block_size", 0), ("block_size", 1 << 30)):
        assert read(lib, **{**paged, name: x}) == E.QKV_ERR_ARG, name


@pytest.mark.parametrize("change,match", [
    (dict(axis_pos=torch.zeros((3, 5), dtype=torch.int32)), "axis_pos"),
    (dict(axis_pos=torch.zeros((3, 4), dtype=torch.int64)), "axis_pos"),
    (dict(axis_pos=torch.zeros(4, dtype=torch.int32)), "axis_pos"),
    (dict(pair_axis=[0] * 31), "pair_axis"),
    (dict(pair_axis=[]), "pair_axis"),
    (dict(pair_axis=[256] * 32), "range"),
    (dict(cos_sin=torch.zeros(50)), "cos_sin"),
    (dict(token_pos=torch.zeros(4, dtype=torch.int64)), "token_pos"),
    (dict(), "CUDA device"),
])
def test_axes_binding_refuses(lib, change, match):  # noqa: F811
    kw = _append_kw()
    kw.pop("token_pos")
    kw = {**kw, "axis_pos": torch.zeros((3, 4), dtype=torch.int32), "pair_axis": [0] * 32, **change}
    with pytest.raises(ValueError, match=match):
        lib.qkv_append_axes(kw.pop("k"), kw.pop("v"), kw.pop("fmt"), kw.pop("k_cache"), kw.pop("v_cache"), kw.pop("cos_sin"),
                            kw.pop("axis_pos"), kw.pop("pair_axis"), **kw)


@pytest.mark.parametrize("change,match", [
    (dict(k_out=None, v_out=None), "k_out or v_out"),
    (dict(k_out=torch.zeros((4, 2, 128), dtype=torch.float64)), "k_out"),
    (dict(k_out=torch.zeros((4, 256))), "k_out"),
    (dict(v_out=torch.zeros((4, 2, 128), dtype=torch.float16)), "one type"),
    (dict(v_out=torch.zeros((5, 2, 128))), "v_out"),
    (dict(v_out=torch.zeros((4, 264))[:, :256].unflatten(1, (2, 128))), "stride"),
    (dict(k_out=torch.zeros((2, 4, 128)).transpose(0, 1)), "contiguous heads"),
    (dict(k_cache=torch.zeros((9, 1, 128), dtype=torch.int8)), "k_cache"),
    (dict(fmt=9), "format"),
    (dict(k_scale=torch.zeros((8, 2))), "k_scale"),
    (dict(slot_mapping=torch.zeros(4, dtype=torch.int32)), "slot_mapping"),
    (dict(cos_sin=None), "together"),
    (dict(axis_pos=None), "together"),
    (dict(pair_axis=[0] * 5), "pair_axis"),
    (dict(), "CUDA device"),
])
def test_read_binding_refuses(lib, change, match):  # noqa: F811
    kw = dict(fmt=1, k_cache=torch.zeros((9, 2, 128), dtype=torch.int8), v_cache=torch.zeros((9, 2, 128), dtype=torch.int8),
              k_out=torch.zeros((4, 2, 128)), v_out=torch.zeros((4, 2, 128)), slot_mapping=torch.zeros(4, dtype=torch.int64),
              k_scale=torch.zeros((9, 2)), v_scale=torch.zeros((9, 2)), cos_sin=torch.zeros((50, 64)),
              axis_pos=torch.zeros((1, 4), dtype=torch.int32))
    kw.update(change)
    with pytest.raises(ValueError, match=match):
        lib.qkv_read(kw.pop("fmt"), kw.pop("k_cache"), kw.pop("v_cache"), **kw)


def test_pair_axis_is_a_sequence_and_needs_angles(lib):  # noqa: F811
    axis_pos = torch.zeros((3, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        lib._axes(axis_pos, 32, 64, 4)  # a number of pairs is no list of axes
    want = bytes([i % 3 for i in range(32)])
    for given in (list(want), want, torch.tensor(list(want)), np.array(list(want))):
        assert bytes(lib._axes(axis_pos, given, 64, 4)[3]) == want
    with pytest.raises(ValueError, match="pair_axis"):
        lib.qkv_read(1, torch.zeros((9, 2, 128), dtype=torch.int8), torch.zeros((9, 2, 128), dtype=torch.int8),
                     k_out=torch.zeros((4, 2, 128)), slot_mapping=torch.zeros(4, dtype=torch.int64), k_scale=torch.zeros((9, 2)),
                     v_scale=torch.zeros((9, 2)), pair_axis=[0] * 32)


def header_fields(name):
    """Field names and C types of a descriptor in the header, a nested descriptor's in place."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qkv.h")).read()
    c = {"size_t": ctypes.c_size_t, "qkv_format": ctypes.c_int, "qkv_out_type": ctypes.c_int, "int": ctypes.c_int,
         "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    want = []
    for line in re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1).strip().splitlines():
        t, n = re.match(r"\s*((?:const )?\w+\*?)\s+(\w+);", line).groups()
        want += header_fields(t) if t.endswith("_desc") else [(n, ctypes.c_void_p if t.endswith("*") else c[t])]
    return want


def test_descriptors_match_the_header(lib):  # noqa: F811
    for struct, name in ((lib.AppendAxesDesc, "qkv_append_axes_desc"), (lib.ReadDesc, "qkv_read_desc")):
        assert [(n, t) for n, t in struct._fields_] == header_fields(name)
    # the nested descriptor ends where its alignment does: its fields in place sit where C puts them
    assert ctypes.sizeof(lib.AppendDesc) == lib.AppendAxesDesc.axis_pos.offset


def test_packed_descriptors_equal_the_structures(lib):  # noqa: F811
    for desc, call in ((lib.AppendAxesDesc, lib._call_axes), (lib.ReadDesc, lib._call_read)):
        pack = next(c.cell_contents for c in call.__closure__ if getattr(c.cell_contents, "__name__", "") == "pack")
        values = [float(i) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(desc._fields_)]
        assert pack(*values) == bytes(desc(*values))
