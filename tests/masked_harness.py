"""Test-side helpers of qkv_masked_attn: batches of rows with masks over paged sequences, the call, and its comparison with
the oracle."""

from __future__ import annotations

import numpy as np
import torch

from dense_harness import HALF_STEP, Pool, assert_within, attention_bounds, bits16, dev16
from oracle import dense


class Seqs:
    """Block tables of sequences of these lengths, their blocks scattered over the pool, with spare blocks of leftovers."""

    def __init__(self, rng, lengths, block, spare=2):
        need = [-(-n // block) for n in lengths]
        ids = rng.permutation(sum(need) + spare).astype(np.int32)
        self.block, self.lengths = block, list(lengths)
        self.table = np.full((len(lengths), max(1, max(need)) + 1), -1, dtype=np.int32)
        at, live = 0, []
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
            p = np.arange(lengths[i])
            live.append(self.table[i, p // block].astype(np.int64) * block + p % block)
        self.live = np.concatenate(live) if live else np.zeros(0, np.int64)
        self.num_slots = max(1, len(ids) * block)


def chunk_rows(lengths, new, mask="causal", doc=50):
    """(seq, start, end, pos) of the last new[i] tokens of every sequence; documents of doc, doc + 1, ... tokens; prefix:
    the first half of the sequence sees itself."""
    rows = []
    for i, (n, m) in enumerate(zip(lengths, new)):
        starts, at, k = [], 0, 0
        while at <= n:
            starts.append(at)
            at, k = at + doc + k, k + 1
        for p in range(n - m, n):
            start = max(x for x in starts if x <= p) if mask == "docs" else 0
            rows.append((i, start, max(p + 1, n // 2) if mask == "prefix" else p + 1, p))
    return np.array(rows, dtype=np.int32).reshape(-1, 4)


def call(pool, fmt, q, seqs, rows, H, scale, *, use_start=True, use_pos=True, window=0, softcap=0.0, slopes=None, max_row_end=None,
         status=None, workspace=None, out=None, lse=None, stream=None, table=None):
    """The public call; rows (seq, start, end, pos). Returns out, lse (NaN where not written)."""
    import quantized_kv_cache_write_gb300 as qkv
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    R, Hq, D = q.shape
    table = seqs.table if table is None else table
    top = int(max([0, *rows[:, 2]])) if max_row_end is None else max_row_end
    out = torch.full_like(q, float("nan")) if out is None else out
    lse = torch.full((R, Hq), float("nan"), dtype=torch.float32, device="cuda") if lse is None else lse
    if workspace is None:
        need = qkv.qkv_masked_attn_workspace(qkv.FORMATS[fmt], R, len(table), Hq, H, D, top, window)
        workspace = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN as any type
    qkv.qkv_masked_attn(q, qkv.FORMATS[fmt], *pool.cache, dev(table), dev(rows[:, 0]), dev(rows[:, 2]), seqs.block, scale,
                        max_row_end=top, num_kv_heads=H, row_start=dev(rows[:, 1]) if use_start else None,
                        row_pos=dev(rows[:, 3]) if use_pos else None, window=window, softcap=softcap,
                        slopes=None if slopes is None else dev(np.asarray(slopes, np.float32)), out=out, lse=lse,
                        workspace=workspace, dev_status=status, stream=stream, **pool.kw)
    return out, lse


def bounds(pool, fmt, act, rows, ref, softcap, D):
    """attention_bounds with the scores' further errors: a capped score's 2^-19 of itself (tanh is off by less than 2^-20 of
    itself, and its product and argument round), and it is no larger than softcap or the logit; a bias's 2^-22 of slope
    times distance. Each moves a weight by as much twice (it is a quotient), and the log-sum-exp once. The bias that the
    log-sum-exp gets back at the end rounds once more."""
    out, lse, wabs, big, far, _ = ref
    n = np.maximum(rows[:, 2] - np.maximum(rows[:, 1], 0), 0)
    vmax = float(np.nanmax(np.where(np.isfinite(pool.V), np.abs(pool.V), 0.0)))
    o_tol, l_tol = attention_bounds(out, lse, wabs, big, n[:, None, None], vmax, act, fmt, D)
    extra = np.minimum(softcap, big) * 2.0 ** -19 + far * 2.0 ** -22
    return o_tol + 2 * extra[..., None] * wabs, np.broadcast_to(l_tol[0] if l_tol.ndim == 3 else l_tol, lse.shape) + extra


def check(pool, fmt, act, qb, seqs, rows, H, scale, *, window=0, softcap=0.0, slopes=None, use_start=True, use_pos=True,
          max_row_end=None, table=None, want_status=None, got=None, **kw):
    """The call (or what it gave: got) against the oracle, padding rows left as they were and the status word."""
    q = dev16(qb, act)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = seqs.table if table is None else table
    top = int(max([0, *rows[:, 2]])) if max_row_end is None else max_row_end
    if got is None:
        got = call(pool, fmt, q, seqs, rows, H, scale, window=window, softcap=softcap, slopes=slopes, use_start=use_start,
                   use_pos=use_pos, max_row_end=top, status=status, table=table, **kw)
        torch.cuda.synchronize()
    lo, hi, pos, pad, bad = dense.masked_rows(rows[:, 0], rows[:, 1] if use_start else None, rows[:, 2],
                                              rows[:, 3] if use_pos else None, window, len(table), top)
    ref = dense.masked_attention(qb, pool.K, pool.V, rows[:, 0], lo, hi, pos, pad, table, seqs.block, scale, softcap, slopes, act)
    D = qb.shape[-1]
    span = np.stack([rows[:, 0], lo, hi, pos], 1)
    o_tol, l_tol = bounds(pool, fmt, act, span, ref, softcap, D)
    go, gl = got[0].float().cpu().numpy().astype(np.float64), got[1].cpu().numpy().astype(np.float64)
    assert np.isnan(go[pad]).all() and np.isnan(gl[pad]).all(), "padding rows were written"
    # rows that see something not finite have the oracle's NaN and infinities (an infinite value may have become NaN
    # where its weight is below the smallest number)
    live = ~pad
    odd = live[:, None, None] & ~np.isfinite(ref[0])
    assert not np.isfinite(go[odd]).any(), "a value that is not finite was lost"
    fine = live[:, None, None] & np.isfinite(ref[0])
    assert_within(np.where(fine, go, 0.0), np.where(fine, ref[0], 0.0), np.where(fine, o_tol, 1.0), "out")
    lf = live[:, None] & ~np.isnan(ref[1])
    assert_within(np.where(lf, gl, 0.0), np.where(lf, ref[1], 0.0), np.where(lf, l_tol, 1.0), "lse")
    assert np.isnan(gl[live[:, None] & np.isnan(ref[1])]).all()
    flagged = bad or ref[5]
    assert int(status.item()) == (2 if flagged else 0) if want_status is None else int(status.item()) == want_status
    return got


def query(rng, R, Hq, D, act, spread=1.0):
    return bits16(rng.standard_normal((R, Hq, D)) * spread, act)


__all__ = ["HALF_STEP", "Pool", "Seqs", "bits16", "call", "check", "chunk_rows", "dev16", "query"]
