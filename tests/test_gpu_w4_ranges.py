"""4-bit products over the range of scales and activations, on each of the dense layer's kernels (up to 8, up to 16 and
more tokens), against the definition in 64 bits.  Tolerances as in test_gpu_w4.py."""
import pytest
import torch

from moe_decode_block_b200 import w4
from test_gpu_w4 import _check_linear, _x
from w4_reference import random_w4

pytestmark = pytest.mark.gpu

BATCHES = [3, 8, 9, 16, 17, 64]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,lo,hi", [(torch.bfloat16, -60, 26), (torch.float16, -20, 11)])
@pytest.mark.parametrize("b", BATCHES)
def test_scales_of_many_magnitudes(b, dtype, lo, hi, zeros):
    """Outputs whose scales are about 2^lo .. 2^hi: in fp16 from subnormal ones to weights near 65,504 (4,094 times up to
    16), in bf16 to just below 2^27."""
    n, k = 96, 256
    codes, scales, z = random_w4(n, k, 64, zeros, dtype, seed=b)
    mantissa = 1 + torch.rand(n, k // 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(b))
    scales = (mantissa.clamp_(max=1.99) * torch.exp2(torch.linspace(lo, hi, n, device="cuda").round())[:, None]).to(dtype)
    x = (_x(b, k, torch.float32, seed=b) / (256.0 if dtype is torch.float16 else 1.0)).to(dtype)
    out = torch.full((b, n), float("nan"), dtype=dtype, device="cuda")
    w4.linear(x, w4.pack(codes, scales, z), out, 64, zeros=zeros)
    assert bool(out.isfinite().all())
    _check_linear(x, codes, scales, z, None, out)
