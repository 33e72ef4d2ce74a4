"""qkv_masked_attn under block tables with rows that no token belongs to (GPU): no more sequences than rows have a part in a
batch, so a few rows run alike whatever the table's height.

Tables and pools are those of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

KEYS, BLOCK = 60000, 64


@pytest.mark.parametrize("fmt,rows,H,G,D", [("e4m3", 1, 8, 8, 128), ("e4m3", 1, 4, 1, 128), ("bf16", 4, 1, 32, 128), ("int8_side", 1, 1, 16, 256),
                                            ("int8_side", 3, 1, 16, 256), ("f16", 2, 2, 128, 256)])
def test_a_few_rows_run_alike_under_a_taller_table(fmt, rows, H, G, D):
    import quantized_kv_cache_write_gb300 as qkv
    gen = torch.Generator(device="cuda").manual_seed(rows + D)
    blocks = -(-KEYS // BLOCK)
    shape = (blocks * BLOCK, H, D)
    kw = {}
    if fmt in ("bf16", "f16"):
        act = torch.bfloat16 if fmt == "bf16" else torch.float16
        k, v = (torch.randn(shape, device="cuda", generator=gen).to(act) for _ in "kv")
    else:
        act = torch.bfloat16
        if fmt == "e4m3":
            k, v = (torch.randn(shape, device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8) for _ in "kv")
        else:
            k, v = (torch.randint(-127, 128, shape, device="cuda", generator=gen, dtype=torch.int8) for _ in "kv")
            kw = {n: torch.full(shape[:2], 0.02, device="cuda") for n in ("k_scale_tok", "v_scale_tok")}
    q = torch.randn((rows, H * G, D), device="cuda", generator=gen).to(act)
    table = torch.full((1000, blocks), -1, dtype=torch.int32, device="cuda")
    table[:rows] = torch.arange(blocks, device="cuda").int()
    seq = torch.arange(rows, device="cuda").int()
    end = KEYS - 7 * seq
    got, needs = [], []
    for seqs in (rows, 4 * rows, 1000):
        need = qkv.qkv_masked_attn_workspace(qkv.FORMATS[fmt], rows, seqs, H * G, H, D, KEYS)
        out, lse = torch.zeros_like(q), torch.zeros((rows, H * G), device="cuda")
        qkv.qkv_masked_attn(q, qkv.FORMATS[fmt], k, v, table[:seqs], seq, end, BLOCK, D ** -0.5, max_row_end=KEYS, num_kv_heads=H,
                            out=out, lse=lse, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), **kw)
        torch.cuda.synchronize()
        got.append((out, lse)), needs.append(need)
    assert needs[0] == needs[1] == needs[2], needs
    assert np.isfinite(got[0][1].cpu().numpy()).all()
    for out, lse in got[1:]:
        assert torch.equal(out.view(torch.int16), got[0][0].view(torch.int16)) and torch.equal(lse, got[0][1])
