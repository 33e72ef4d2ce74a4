"""Oracle of the dense cache operators (test infrastructure; see the package docstring): the position
rotation of new tokens, attention of a batch over a shared prefix and its rows' own keys, and attention of rows
that each see a range of their sequence's keys, with capped scores and a distance bias.

Rotation, for a pair of head dims (a, b) with cosine c and sine s, all fp32:
    a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))
pair i is dims (i, i + n / 2) of the n rotated dims, or (2i, 2i + 1) when interleaved.

Attention of one row and query head over the keys j it sees, in fp64:
    s_j = scale q . K_j,  o = sum_j softmax(s)_j V_j,  lse = log sum_j exp(s_j)
"""

from __future__ import annotations

import numpy as np

from .quant import act_bits_to_f32


def rotate_f32(x: np.ndarray, pos: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x fp32 [T, H, D] rotated by the rows pos [T] of cos_sin fp32 [positions, n]."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    n = cos_sin.shape[1]
    out = x.copy()
    for i in range(n // 2):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n // 2)
        c = cos_sin[pos, i].astype(np.float32)[:, None]
        s = cos_sin[pos, n // 2 + i].astype(np.float32)[:, None]
        a, b = x[:, :, ia], x[:, :, ib]
        out[:, :, ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        out[:, :, ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return out


def row_slots(row_seq, row_len, prefix_blocks, prefix_len, block_table, block_size, num_slots):
    """Per row the slots of the keys it sees, in order, without the invalid ones (unallocated blocks,
    slots past the pool); None for a padding row. Also whether anything had to be flagged."""
    flagged = False
    got = []
    num_seqs, max_blocks = block_table.shape
    for seq, n in zip(row_seq.tolist(), row_len.tolist()):
        if seq == -1:
            got.append(None)
            continue
        if not 0 <= seq < num_seqs or n < 0 or n > max_blocks * block_size or 0 < n < prefix_len:
            flagged = True
            got.append([])
            continue
        p = np.arange(n)
        blk = np.empty(n, dtype=np.int64)
        blk[:prefix_len] = np.asarray(prefix_blocks)[p[:prefix_len] // block_size] if prefix_len else 0
        blk[prefix_len:] = block_table[seq, p[prefix_len:] // block_size]
        slot = blk * block_size + p % block_size
        ok = (blk >= 0) & (slot < num_slots)
        flagged |= not ok.all()
        got.append(slot[ok].tolist())
    return got, flagged


def prefix_attention(q_bits: np.ndarray, K: np.ndarray, V: np.ndarray, slots, scale: float, q_dtype: str = "bf16"):
    """fp64 attention of rows q_bits [R, Hq, D] over pools K, V [S, Hkv, D] at each row's slots.

    Returns out [R, Hq, D], lse [R, Hq] and, for error bounds, sum_j w_j |V_j| [R, Hq, D],
    max_j |scale| sum_d |q_d K_jd| [R, Hq]. Padding rows (None) give NaN."""
    q = act_bits_to_f32(q_bits, q_dtype).astype(np.float64)
    R, Hq, D = q.shape
    G = Hq // K.shape[1]
    out, wabs = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    lse, big = np.full((R, Hq), -np.inf), np.zeros((R, Hq))
    for r, sl in enumerate(slots):
        if sl is None:
            out[r], lse[r] = np.nan, np.nan
    rows = [r for r, sl in enumerate(slots) if sl]
    if not rows:
        return out, lse, wabs, big
    # the keys that all rows see first, gathered once
    n = min(len(slots[r]) for r in rows)
    lists = np.array([slots[r][:n] for r in rows])
    differ = np.flatnonzero((lists != lists[0]).any(0))
    n = int(differ[0]) if len(differ) else n
    for h in range(K.shape[1]):
        heads = slice(h * G, (h + 1) * G)
        k0, v0 = K[slots[rows[0]][:n], h], V[slots[rows[0]][:n], h]
        ak0, av0 = np.abs(k0), np.abs(v0)
        for r in rows:
            k1, v1 = K[slots[r][n:], h], V[slots[r][n:], h]
            qr = q[r, heads]
            s = scale * np.concatenate([qr @ k0.T, qr @ k1.T], 1)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            total = e.sum(1, keepdims=True)
            w = e / total
            out[r, heads] = w[:, :n] @ v0 + w[:, n:] @ v1
            wabs[r, heads] = w[:, :n] @ av0 + w[:, n:] @ np.abs(v1)
            lse[r, heads] = (m + np.log(total))[:, 0]
            mags = np.concatenate([np.abs(qr) @ ak0.T, np.abs(qr) @ np.abs(k1).T], 1)
            big[r, heads] = abs(scale) * mags.max(1)
    return out, lse, wabs, big


def masked_rows(row_seq, row_start, row_end, row_pos, window, num_seqs, max_row_end):
    """Per row the range [lo, hi) of positions it sees and its position p ([0, 0), 0: none), whether it is a padding row,
    and whether any row is invalid (it sees nothing)."""
    n = len(row_seq)
    lo, hi, pos = np.zeros(n, np.int64), np.zeros(n, np.int64), np.zeros(n, np.int64)
    pad, flagged = np.asarray(row_seq) == -1, False
    for r in range(n):
        a, e = (0 if row_start is None else int(row_start[r])), int(row_end[r])
        p = e - 1 if row_pos is None else int(row_pos[r])
        if pad[r]:
            continue
        if not 0 <= row_seq[r] < num_seqs or not 0 <= e <= max_row_end or a < 0 or (a < e and not 0 <= p <= 1 << 30):
            flagged = True
        elif a < e:
            a = max(a, p - window + 1) if window else a
            if a < e:
                lo[r], hi[r], pos[r] = a, e, p
    return lo, hi, pos, pad, flagged


def masked_attention(q_bits, K, V, row_seq, lo, hi, pos, pad, block_table, block_size, scale, softcap=0.0, slopes=None,
                     q_dtype: str = "bf16"):
    """fp64 attention of rows q_bits [R, Hq, D] over the positions [lo, hi) of their sequences in pools K, V [S, Hkv, D]:
    scores softcap tanh(scale q . K / softcap) - slopes |pos - j|; keys without a slot are masked.

    Returns out, lse and, for error bounds, sum_j w_j |V_j|, max_j |scale| sum_d |q_d K_jd|, the largest |slope| times
    distance from the nearest seen key, and whether a row sees a key without a slot. Values that are not finite reach only
    the rows that see their key. Padding rows give NaN."""
    q = act_bits_to_f32(q_bits, q_dtype).astype(np.float64)
    R, Hq, D = q.shape
    S, H, _ = K.shape
    G = Hq // H
    out, wabs = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    lse, big, far = np.full((R, Hq), -np.inf), np.zeros((R, Hq)), np.zeros((R, Hq))
    out[pad], lse[pad] = np.nan, np.nan
    flagged = False
    sl = np.zeros(Hq) if slopes is None else np.asarray(slopes, np.float64)
    live = [r for r in range(R) if lo[r] < hi[r]]
    for seq in sorted({int(row_seq[r]) for r in live}):
        rows = np.array([r for r in live if row_seq[r] == seq])
        a, e = int(lo[rows].min()), int(hi[rows].max())
        j = np.arange(a, e)
        blk = block_table[seq, j // block_size].astype(np.int64)
        slot = blk * block_size + j % block_size
        ok = (blk >= 0) & (slot < S)
        inside = (j >= lo[rows, None]) & (j < hi[rows, None])
        flagged |= bool((inside & ~ok).any())
        j, slot, sees = j[ok], slot[ok], (inside & ok)[:, ok]
        seen = sees.any(0)
        j, slot, sees = j[seen], slot[seen], sees[:, seen]
        if not len(j):
            continue
        near = np.minimum(np.maximum(pos[rows], lo[rows]), hi[rows] - 1)
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            k, v = K[slot, h], V[slot, h]
            qr = q[rows, heads]  # [r, G, D]
            with np.errstate(invalid="ignore", over="ignore"):
                z = scale * np.einsum("rgd,jd->rgj", qr, k)
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                dist = np.abs(pos[rows, None] - j).astype(np.float64)
                z = z - sl[heads][None, :, None] * dist[:, None]
                z = np.where(sees[:, None], z, -np.inf)
                m = z.max(-1, keepdims=True)
                ex = np.where(sees[:, None], np.exp(z - np.where(np.isfinite(m), m, 0.0)), 0.0)
                total = ex.sum(-1, keepdims=True)
                w = ex / np.where(total > 0, total, 1.0)
                w = np.where(np.isnan(total), np.nan, w)
                fin = np.isfinite(v)
                v0 = np.where(fin, v, 0.0)
                o = w @ v0
                bad = np.flatnonzero(~fin.all(1))
                for b in bad:
                    rr = np.flatnonzero(sees[:, b])
                    o[rr] += np.where(fin[b], 0.0, v[b])
                out[rows, heads] = o
                wabs[rows, heads] = w @ np.abs(v0)
                lse[rows, heads] = np.where(total[..., 0] > 0, (m + np.log(total))[..., 0], np.where(np.isnan(total[..., 0]), np.nan, -np.inf))
                mags = np.einsum("rgd,jd->rgj", np.abs(qr), np.abs(np.where(np.isfinite(k), k, 0.0)))
                big[rows, heads] = abs(scale) * np.where(sees[:, None], mags, 0.0).max(-1)
                reach = np.where(sees, np.abs(near[:, None] - j), 0).max(-1)
                far[rows, heads] = np.abs(sl[heads])[None] * reach[:, None]
    return out, lse, wabs, big, far, flagged
