"""The oracle of masked attention: its masks by hand, and its attention against sums written out key by key."""

import math

import numpy as np
import pytest

from oracle import dense
from oracle.quant import act_bits_to_f32


def _bits(x):
    return x.astype(np.float16).view(np.uint16)


def test_masked_rows_by_hand():
    #        whole  start  window  empty   pad    bad seq  bad end  bad start  bad pos  window leaves none
    seq = [0, 1, 0, 0, -1, 2, 0, 0, 0, 1]
    start = [0, 3, 0, 5, 0, 0, 0, -1, 0, 0]
    end = [7, 9, 9, 5, 4, 4, 11, 4, 4, 3]
    pos = [6, 8, 20, 4, 3, 3, 10, 3, -1, 30]
    lo, hi, p, pad, bad = dense.masked_rows(seq, start, end, pos, 15, 2, 10)
    assert list(zip(lo, hi, p)) == [(0, 7, 6), (3, 9, 8), (6, 9, 20), (0, 0, 0), (0, 0, 0), (0, 0, 0), (0, 0, 0), (0, 0, 0),
                                    (0, 0, 0), (0, 0, 0)]
    assert list(pad) == [s == -1 for s in seq] and bad
    # without row_start and row_pos: from 0 on, at the last position seen
    lo, hi, p, _, bad = dense.masked_rows([0, 0], None, [10, 2], None, 4, 1, 10)
    assert (list(lo), list(hi), list(p), bad) == ([6, 0], [10, 2], [9, 1], False)


def _case():
    rng = np.random.default_rng(5)
    S, H, G, D, block = 48, 2, 2, 8, 4
    K, V = rng.standard_normal((S, H, D)), rng.standard_normal((S, H, D))
    table = rng.permutation(S // block).reshape(2, -1)
    q = _bits(rng.standard_normal((4, H * G, D)) * 2)
    seq, lo, hi, pos = (np.array(x) for x in ([0, 1, 0, 1], [0, 3, 7, 0], [9, 23, 20, 0], [8, 30, 2, 0]))
    return K, V, table, block, q, seq, lo, hi, pos, np.array([0.5, 0.25, 0.0, 1.5]), 0.7, 3.0


def _by_hand(K, V, table, block, q, seq, lo, hi, pos, slopes, scale, cap, mistake=""):
    qf = act_bits_to_f32(q, "f16").astype(np.float64)
    R, Hq, D = qf.shape
    G = Hq // K.shape[1]
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf)
    for r in range(R):
        for g in range(Hq):
            s, v = [], []
            for j in range(lo[r], hi[r] + (mistake == "end")):
                slot = int(table[seq[r], j // block]) * block + j % block
                z = scale * math.fsum(qf[r, g] * K[slot, g // G if mistake != "head" else g % K.shape[1]])
                far = abs(pos[r] - j) if mistake != "sign" else pos[r] - j
                if mistake == "order":
                    s.append(cap * math.tanh((z - slopes[g] * far) / cap))
                else:
                    s.append(cap * math.tanh(z / cap) - slopes[g] * far)
                v.append(V[slot, g // G])
            if s:
                m = max(s)
                w = [math.exp(x - m) for x in s]
                lse[r, g] = m + math.log(math.fsum(w))
                out[r, g] = [math.fsum(w[i] * v[i][d] for i in range(len(w))) / math.fsum(w) for d in range(D)]
    return out, lse


def _agrees(got, want):
    seen = np.isfinite(want[1])
    return (np.allclose(got[0], want[0], rtol=1e-11, atol=1e-11) and np.allclose(got[1][seen], want[1][seen], rtol=1e-11) and
            (got[1][~seen] == -np.inf).all())


def test_masked_attention_is_the_sum_written_out():
    K, V, table, block, q, seq, lo, hi, pos, slopes, scale, cap = case = _case()
    got = dense.masked_attention(q, K, V, seq, lo, hi, pos, np.zeros(4, bool), table, block, scale, cap, slopes, "f16")
    assert _agrees(got, _by_hand(*case)) and not got[5]


@pytest.mark.parametrize("mistake", ["end", "head", "sign", "order"])
def test_a_planted_mistake_fails(mistake):
    K, V, table, block, q, seq, lo, hi, pos, slopes, scale, cap = case = _case()
    got = dense.masked_attention(q, K, V, seq, lo, hi, pos, np.zeros(4, bool), table, block, scale, cap, slopes, "f16")
    assert not _agrees(got, _by_hand(*case, mistake=mistake))


def test_keys_without_a_slot_are_masked_and_padding_rows_left():
    K, V, table, block, q, seq, lo, hi, pos, slopes, scale, cap = _case()
    table = table.copy()
    table[0, 1] = -1  # positions 4 to 7 of sequence 0
    got = dense.masked_attention(q, K, V, seq, lo, hi, pos, np.arange(4) == 3, table, block, scale, cap, slopes, "f16")
    assert got[5] and np.isnan(got[0][3]).all() and np.isnan(got[1][3]).all()
    without = dense.masked_attention(q[2:3], K, V, *np.array([[0], [8], [20], [2]]), np.zeros(1, bool), table, block, scale, cap, slopes, "f16")
    assert np.allclose(got[0][2], without[0][0]) and np.allclose(got[1][2], without[1][0])
