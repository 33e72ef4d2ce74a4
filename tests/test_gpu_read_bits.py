"""qkv_read of a 16-bit pool into its own type, K turned back (GPU): what is not turned is copied bit for bit, NaNs with their
payloads and all.

The pool is that of "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Implementation scope, unquantised."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 32), (256, 96), (256, 16), (128, 112)])
def test_dims_that_are_not_turned_are_copied(fmt, pairs, D, rot):
    import quantized_kv_cache_write_gb300 as qkv
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float16
    gen = torch.Generator(device="cuda").manual_seed(D + rot)
    T, H = 40, 3
    bits = [torch.randint(-(1 << 15), 1 << 15, (T, H, D), device="cuda", generator=gen, dtype=torch.int32).to(torch.int16) for _ in "kv"]
    one = torch.ones((1, rot // 2), device="cuda")
    out = [torch.zeros((T, H, D), dtype=dtype, device="cuda") for _ in "kv"]
    qkv.qkv_read(qkv.FORMATS[fmt], *bits, k_out=out[0], v_out=out[1], slot_mapping=torch.arange(T, device="cuda"),
                 cos_sin=torch.cat([0.6 * one, 0.8 * one], 1).contiguous(), axis_pos=torch.zeros((1, T), dtype=torch.int32, device="cuda"),
                 interleaved=pairs)
    torch.cuda.synchronize()
    assert torch.equal(out[0].view(torch.int16)[..., rot:], bits[0][..., rot:])
    assert torch.equal(out[1].view(torch.int16), bits[1])
