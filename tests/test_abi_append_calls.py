"""The host's part of an append, without a GPU: a step's append is bound by the host's time, so the binding makes no more
Python calls for one than its checks need, and the two appends pass the same fields."""

import sys

import pytest
import torch

from test_abi_dense import _append_kw, lib  # noqa: F401  (lib: the built library)


def _recorded(lib, monkeypatch):
    """The binding with its device check and its library calls replaced: what was passed, by entry point."""
    passed = {}
    monkeypatch.setattr(lib, "_on_cuda", lambda *tensors: 0)
    monkeypatch.setattr(lib, "_call_append", lambda dev, stream, *fields: passed.update(rope=fields))
    monkeypatch.setattr(lib, "_call_axes", lambda dev, stream, *fields: passed.update(axes=fields))
    return passed


def _args(paged):
    kw = _append_kw()
    kw.update(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16), q_out=torch.zeros((4, 8, 128), dtype=torch.bfloat16))
    if paged:
        kw.update(slot_mapping=None, token_seq=torch.zeros(4, dtype=torch.int32), block_size=3,
                  block_table=torch.zeros((2, 4), dtype=torch.int32))
    return [kw.pop(n) for n in ("k", "v", "fmt", "k_cache", "v_cache", "cos_sin")], kw


@pytest.mark.parametrize("paged", [False, True])
def test_an_append_makes_no_more_python_calls_than_its_checks(lib, monkeypatch, paged):  # noqa: F811
    passed = _recorded(lib, monkeypatch)
    args, kw = _args(paged)
    calls = []
    sys.setprofile(lambda frame, event, _: calls.append(frame.f_code.co_name) if event == "call" else None)
    try:
        lib.qkv_append_rope(*args, **kw)
    finally:
        sys.setprofile(None)
    assert "rope" in passed
    # the public call and its body, the tokens' and the pool's checks, two of q, one of each of the five small tensors that
    # are given (paged: six), the device's and the library call
    assert len(calls) <= (14 if paged else 13), calls


@pytest.mark.parametrize("paged", [False, True])
def test_the_two_appends_pass_the_same_fields(lib, monkeypatch, paged):  # noqa: F811
    passed = _recorded(lib, monkeypatch)
    args, kw = _args(paged)
    lib.qkv_append_rope(*args, **kw)
    axis_pos = torch.zeros((3, 4), dtype=torch.int32)
    if not paged:
        kw.pop("token_pos")
    lib.qkv_append_axes(*args, axis_pos, [0] * 32, **kw)
    want = list(passed["rope"])
    names = [n for n, _ in lib.AppendDesc._fields_]
    if not paged:
        want[names.index("token_pos")] = 0
    assert list(passed["axes"][1:len(names)]) == want[1:]  # all but the descriptor's size
    assert passed["axes"][len(names):][:2] == (axis_pos.data_ptr(), 3)
