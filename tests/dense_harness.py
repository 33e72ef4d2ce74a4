"""Test-side helpers of the dense cache operators: seeded pools with anything in their unused places,
block tables, and the error bounds that the comparisons use."""

from __future__ import annotations

import numpy as np
import torch

from gen.workloads import f32_to_bf16_bits, f32_to_f16_bits
from oracle import attention as oatt
from oracle import quant as oq

# A rounding is off by at most half a step, relative to the value.
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
ACT = {"bf16": torch.bfloat16, "f16": torch.float16}


def bits16(x: np.ndarray, act: str) -> np.ndarray:
    return f32_to_bf16_bits(x.astype(np.float32)) if act == "bf16" else f32_to_f16_bits(x.astype(np.float32))


def dev16(bits: np.ndarray, act: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(ACT[act]).cuda()


class Pool:
    """A pool of `fmt` whose live slots hold random tokens and whose other slots hold NaN, infinities
    and other leftovers. K, V: its values in fp64 (NaN in unused slots)."""

    def __init__(self, rng, fmt, act, live, num_slots, H, D, outliers=0.02):
        n = len(live)
        k = rng.standard_normal((n, H, D)) * np.where(rng.random((n, 1, 1)) < outliers, 6.0, 1.0)
        v = rng.standard_normal((n, H, D)) * np.where(rng.random((n, 1, 1)) < outliers, 20.0, 1.0)
        kb, vb = bits16(k, act), bits16(v, act)
        S = max(num_slots, 1)
        dead = np.setdiff1d(np.arange(S), live)
        slots = np.asarray(live, dtype=np.int64)
        self.fmt, self.kw = fmt, {}
        if fmt in ("bf16", "f16"):
            kc, vc = oq.write_bf16(kb, vb, slots, S)
            for c in (kc, vc):
                c[dead] = rng.choice(np.array([0x7FFF, 0xFFC1, 0x7F80 if fmt == "bf16" else 0x7C00], dtype=np.uint16),
                                     c[dead].shape)
            widen = oatt.f16_pool_fp64 if fmt == "f16" else oatt.bf16_pool_fp64
            self.K, self.V = widen(kc), widen(vc)
            self.cache = [dev16(c, fmt) for c in (kc, vc)]
        elif fmt == "int8_side":
            kc, vc, ks, vs = oq.write_int8(kb, vb, slots, S, "side", dtype=act)
            for s in (ks, vs):
                s[dead] = rng.choice(np.array([np.nan, np.inf, 3e38], dtype=np.float32), s[dead].shape)
            kc[dead], vc[dead] = 127, -127
            self.K, self.V = oatt.int8_side_pool_fp64(kc, ks), oatt.int8_side_pool_fp64(vc, vs)
            self.cache = [torch.from_numpy(c).cuda() for c in (kc, vc)]
            self.kw = dict(k_scale_tok=torch.from_numpy(ks).cuda(), v_scale_tok=torch.from_numpy(vs).cuda())
        elif fmt == "int8_inline":
            kc, vc = oq.write_int8(kb, vb, slots, S, "inline", dtype=act)
            kc[dead], vc[dead] = 0xFF, 0x7F
            self.K, self.V = oatt.int8_inline_pool_fp64(kc), oatt.int8_inline_pool_fp64(vc)
            self.cache = [torch.from_numpy(c).cuda() for c in (kc, vc)]
        else:
            ks, vs = oq.e4m3_calibrated_scale(kb, dtype=act), oq.e4m3_calibrated_scale(vb, dtype=act)
            kc, vc = oq.write_e4m3(kb, vb, slots, S, ks, vs, dtype=act)
            kc[dead], vc[dead] = 0x7F, 0xFF
            self.K, self.V = oatt.e4m3_pool_fp64(kc, ks), oatt.e4m3_pool_fp64(vc, vs)
            self.cache = [torch.from_numpy(c).cuda() for c in (kc, vc)]
            self.kw = dict(k_scale_layer=float(ks), v_scale_layer=float(vs))
        self.num_slots = S


class Batch:
    """Block tables of sequences that share `prefix` tokens and have own[i] more, `per` query rows each."""

    def __init__(self, rng, prefix, own, per, block, spare_blocks=2):
        total = [prefix + n for n in own]
        shared = -(-prefix // block)
        mine = [max(0, -(-n // block) - prefix // block) for n in total]
        ids = rng.permutation(shared + sum(mine) + spare_blocks).astype(np.int32)
        self.block, self.prefix = block, prefix
        self.prefix_blocks = ids[:shared].copy()
        self.max_row_len = max(total)
        wide = max(1, -(-self.max_row_len // block)) + 1
        self.table = np.full((len(own), wide), -1, dtype=np.int32)
        at = shared
        live = [self.prefix_blocks[p // block] * block + p % block for p in range(prefix)]
        for i, n in enumerate(mine):
            self.table[i, prefix // block:prefix // block + n] = ids[at:at + n]
            at += n
            live += [self.table[i, p // block] * block + p % block for p in range(prefix, total[i])]
        self.live = np.array(live, dtype=np.int64)
        self.num_slots = len(ids) * block
        self.row_seq = np.repeat(np.arange(len(own)), per).astype(np.int32)
        self.row_len = np.array([n - per + 1 + i for n in total for i in range(per)], dtype=np.int32)


def attention_bounds(ref, lse, wabs, big, n_keys, vmax, act, fmt, D):
    """Elementwise bounds of |out - ref| and |lse - ref|.

    out: half a step of its own type; one rounding of every p to the MMA's 16-bit operand (bf16
    pools: bf16, others fp16), so at most that share of sum w |V|; the logits' fp32 sums of D products
    (each step off by at most 2^-23 of the magnitudes' sum, twice because w is a quotient), the
    exponentials and sums (2^-18 together); and, for p below fp16's normal range, 2^-28 of the largest V per key.
    lse: the logits' error, 2^-21 of the values that are added and n steps of the fp32 sum."""
    u_p = HALF_STEP["bf16" if fmt == "bf16" else "f16"]
    logit = D * 2.0 ** -23 * big
    out = HALF_STEP[act] * np.abs(ref) + (u_p + 2 * logit + 2.0 ** -18)[..., None] * wabs + n_keys * 2.0 ** -28 * vmax
    with np.errstate(invalid="ignore"):
        l_tol = logit + 2.0 ** -21 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 16) + n_keys * 2.0 ** -24
    if act == "f16":
        out = out + 2.0 ** -25  # an output below fp16's normal range
    return out, l_tol


def assert_within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same_inf = np.isinf(ref) & (got == ref)
    with np.errstate(invalid="ignore"):
        err = np.where(same_inf, 0.0, np.abs(got - ref))
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(err, nan=np.inf), -1)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; worst at {i}: got {got[i]!r} "
                             f"ref {ref[i]!r} tol {np.broadcast_to(tol, err.shape)[i]:.3e}")
