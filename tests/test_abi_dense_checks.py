"""More of the dense cache operators' binding, without a GPU: pools whose tensors hold another type than the format's,
which the kernels would misread, and the device that a workspace is asked for."""

import pytest
import torch

from test_abi_dense import _append_kw, _prefix_kw, lib  # noqa: F401  (the built library)

BF16, F16, I8, U8 = torch.bfloat16, torch.float16, torch.int8, torch.uint8
# format code, the types that hold it, types of the same size that do not
POOLS = [(0, (BF16, torch.int16, torch.uint16), (F16,)),
         (4, (F16, torch.int16, torch.uint16), (BF16,)),
         (1, (I8, U8), (torch.bool, torch.float8_e4m3fn)),
         (2, (I8, U8), (torch.bool, torch.float8_e4m3fn)),
         (3, (torch.float8_e4m3fn, U8, I8), (torch.float8_e5m2, torch.bool))]


def _pool(fmt, dtype):
    return torch.zeros((9, 2, 132 if fmt == 2 else 128), dtype=torch.uint8 if dtype.itemsize == 1 else torch.int16).view(dtype)


def _calls(lib, fmt, k_cache, v_cache):
    act = F16 if fmt == 4 else BF16
    a = {**_append_kw(), "fmt": fmt, "k_cache": k_cache, "v_cache": v_cache}
    a["k"], a["v"] = a["k"].to(act), a["v"].to(act)
    p = {**_prefix_kw(), "fmt": fmt, "k_cache": k_cache, "v_cache": v_cache}
    p["q"], p["out"] = p["q"].to(act), p["out"].to(act)
    yield lambda: lib.qkv_append_rope(a.pop("k"), a.pop("v"), a.pop("fmt"), a.pop("k_cache"), a.pop("v_cache"), a.pop("cos_sin"),
                                      a.pop("token_pos"), **a)
    yield lambda: lib.qkv_prefix_attn(p.pop("q"), p.pop("fmt"), p.pop("k_cache"), p.pop("v_cache"), p.pop("block_table"),
                                      p.pop("row_seq"), p.pop("row_len"), p.pop("block_size"), p.pop("softmax_scale"), **p)


@pytest.mark.parametrize("fmt,held,others", POOLS)
def test_a_pool_of_another_type_is_refused(lib, fmt, held, others):  # noqa: F811
    right = _pool(fmt, held[0])
    for wrong in others:
        for k, v, name in ((_pool(fmt, wrong), right, "k_cache"), (right, _pool(fmt, wrong), "v_cache")):
            for f in _calls(lib, fmt, k, v):
                with pytest.raises(ValueError, match=name):
                    f()


@pytest.mark.parametrize("fmt,held,others", POOLS)
def test_every_type_that_holds_the_format_passes_the_check(lib, fmt, held, others):  # noqa: F811
    """They get as far as the device check: these tensors are on the CPU."""
    for dtype in held:
        for f in _calls(lib, fmt, _pool(fmt, dtype), _pool(fmt, held[0])):
            with pytest.raises(ValueError, match="CUDA device"):
                f()


def test_the_workspace_is_asked_for_on_the_given_device(lib, monkeypatch):  # noqa: F811
    """The size goes by the device's SMs, and the call runs on its tensors' device."""
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *exc):
            current[0] = self.before

    class Library:
        def qkv_prefix_attn_workspace(self, *args):
            seen.append(current[0])
            return lib.QKV_OK

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(lib, "lib", Library())
    shape = (lib.QKV_E4M3, 4, 8, 2, 128, 20, 40)
    lib.qkv_prefix_attn_workspace(*shape)
    lib.qkv_prefix_attn_workspace(*shape, device=3)
    assert seen == [0, 3] and current == [0]
