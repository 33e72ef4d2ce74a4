"""The oracle of the dense cache operators, pinned on the CPU: the rotation against the complex product in
64 bits and its inverse, the attention against a textbook softmax and against differences."""

import numpy as np
import pytest

from gen.workloads import f32_to_bf16_bits
from oracle import dense
from oracle import quant as oq


def _table(positions, n):
    ang = np.arange(positions)[:, None] * 100.0 ** (-np.arange(n // 2) / (n // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("n", [16, 48, 128])
def test_rotation_is_the_complex_product(pairs, n):
    rng = np.random.default_rng(n)
    x = rng.standard_normal((9, 2, 128)).astype(np.float32)
    cs, pos = _table(40, n), rng.integers(0, 40, 9)
    y = dense.rotate_f32(x, pos, cs, pairs)
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if pairs else (x[..., :n // 2], x[..., n // 2:n])
    z = (a.astype(np.complex128) + 1j * b) * (cs[pos, :n // 2].astype(np.float64) + 1j * cs[pos, n // 2:])[:, None]
    ya, yb = (y[..., 0:n:2], y[..., 1:n:2]) if pairs else (y[..., :n // 2], y[..., n // 2:n])
    # three fp32 roundings, each half a step of a value not above |a| + |b|
    tol = 3 * 2.0 ** -24 * (np.abs(a) + np.abs(b))
    assert (np.abs(ya - z.real) <= tol).all() and (np.abs(yb - z.imag) <= tol).all()
    assert np.array_equal(y[..., n:], x[..., n:])


def test_rotation_at_position_zero_changes_nothing():
    x = np.random.default_rng(0).standard_normal((3, 1, 256)).astype(np.float32)
    assert np.array_equal(dense.rotate_f32(x, np.zeros(3, int), _table(2, 256), False), x)


def test_row_slots_by_hand():
    table = np.array([[-1, 5, 2], [-1, 7, -1]], dtype=np.int32)
    slots, flagged = dense.row_slots(np.array([0, 1, -1, 0]), np.array([9, 6, 3, 0]), np.array([3, 1]), 5, table, 4, 100)
    # the prefix of 5 ends inside its second block; position 5 onwards is the row's own
    assert slots[0] == [12, 13, 14, 15, 4, 21, 22, 23, 8]
    assert slots[1] == [12, 13, 14, 15, 4, 29]
    assert slots[2] is None and slots[3] == [] and not flagged
    for seq, n in ((2, 6), (0, 4), (0, 13), (1, 9)):  # no such sequence; inside the prefix; too long; unallocated
        assert dense.row_slots(np.array([seq]), np.array([n]), np.array([3, 1]), 5, table, 4, 100)[1]


def test_attention_is_a_textbook_softmax_and_lse_is_its_potential():
    rng = np.random.default_rng(1)
    q = f32_to_bf16_bits(rng.standard_normal((2, 4, 128)).astype(np.float32))
    K, V = rng.standard_normal((12, 2, 128)), rng.standard_normal((12, 2, 128))
    slots = [[3, 1, 7, 11], [0, 2]]
    out, lse, wabs, _ = dense.prefix_attention(q, K, V, slots, 0.1)
    qf = oq.bf16_bits_to_f32(q).astype(np.float64)
    for r in range(2):
        for g in range(4):
            s = np.exp(0.1 * K[slots[r], g // 2] @ qf[r, g])
            assert np.allclose(out[r, g], (s / s.sum()) @ V[slots[r], g // 2], rtol=0, atol=1e-13)
            assert abs(lse[r, g] - np.log(s.sum())) < 1e-13
            assert (wabs[r, g] >= np.abs(out[r, g]) - 1e-13).all()
    # the derivative of lse by a logit is that key's weight: a difference along K gives w scale q
    d = 1e-6
    K2 = K.copy()
    K2[7, 0, 5] += d
    _, lse2, _, _ = dense.prefix_attention(q, K2, V, slots, 0.1)
    s = np.exp(0.1 * K[slots[0], 0] @ qf[0, 0])
    assert abs((lse2[0, 0] - lse[0, 0]) / d - (s / s.sum())[2] * 0.1 * qf[0, 0, 5]) < 1e-5


def test_empty_and_padding_rows():
    q = f32_to_bf16_bits(np.ones((2, 1, 128), np.float32))
    out, lse, _, _ = dense.prefix_attention(q, np.ones((2, 1, 128)), np.ones((2, 1, 128)), [[], None], 1.0)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isnan(out[1]).all()
