"""The error of qkv_masked_attn's distance bias alone (GPU): queries of zeros, so that the scores are the bias, and slopes that
prefer far keys, so that the log-sum-exp is that of the farthest ones.

Pools and block tables are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

from dense_harness import assert_within

pytestmark = pytest.mark.gpu

BLOCK, NEAR = 16, 4  # blocks at the sequence's end that there are


@pytest.mark.parametrize("tiles", ["mma", "tcgen05"])
@pytest.mark.parametrize("D,G", [(128, 8), (256, 16)])
@pytest.mark.parametrize("length", [64, 1008, 20000, 200000])
@pytest.mark.parametrize("n", [1, 40])
def test_a_bias_is_off_by_no_more_than_stated(monkeypatch, tiles, D, G, length, n):
    """2^-21 |slope| max(d, 32) for a key at distance d from the nearest one that the row sees. Only the first block of the
    sequence and its last ones are there, so that few weights are added: the log-sum-exp adds the part's logarithm, its product
    with log 2, a join and the nearest key's bias, six roundings of itself, and 2^-18 of the exponentials and their sum."""
    import quantized_kv_cache_write_gb300 as qkv
    monkeypatch.setenv("QKV_TEST_MASKED_TILES", tiles)
    rng = np.random.default_rng(length + n)
    table = np.full((1, length // BLOCK), -1, dtype=np.int32)
    table[0, -NEAR:], table[0, 0] = 1 + np.arange(NEAR), 0
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    kc, vc = (dev(rng.standard_normal((BLOCK * (1 + NEAR), 1, D)).astype(np.float32)).to(torch.bfloat16) for _ in "kv")
    q = torch.zeros((n, G, D), dtype=torch.bfloat16, device="cuda")
    slopes = -(2.0 ** rng.uniform(-14, 3, G)).astype(np.float32)
    end = np.arange(length - n + 1, length + 1, dtype=np.int32)
    need = qkv.qkv_masked_attn_workspace(qkv.QKV_BF16, n, 1, G, 1, D, length)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    there = np.repeat(table[0] >= 0, BLOCK).nonzero()[0]
    for pos in (end - 1, np.zeros(n, np.int32)):  # behind the keys, before them
        out, lse = torch.empty_like(q), torch.empty((n, G), dtype=torch.float32, device="cuda")
        qkv.qkv_masked_attn(q, qkv.QKV_BF16, kc, vc, dev(table), dev(np.zeros(n, np.int32)), dev(end), BLOCK, 0.1, max_row_end=length,
                            row_pos=dev(pos.astype(np.int32)), slopes=dev(slopes), out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        d = np.abs(pos[:, None] - there).astype(np.float64)
        s = np.where(there < end[:, None], -slopes.astype(np.float64)[:, None, None] * d, -np.inf)  # [G, n, keys]
        m = s.max(-1)
        ref = (m + np.log(np.exp(s - m[..., None]).sum(-1))).T
        far = np.where(there < end[:, None], d, 0).max(-1)
        tol = 2.0 ** -21 * np.abs(slopes) * np.maximum(far, 32)[:, None] + 6 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -18
        assert_within(lse.cpu().numpy(), ref, tol, "lse")
        assert out.isfinite().all()
