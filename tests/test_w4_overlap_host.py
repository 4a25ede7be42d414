"""moe_w4_linear refuses an output on its input (no GPU needed), and takes both as columns of one buffer."""
import ctypes

import pytest
import torch

import moe_decode_block_b200 as mdb
from moe_decode_block_b200 import build as mbuild
from moe_decode_block_b200 import w4

BAD = mdb.MOE_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses: for a machine without a GPU")
def test_rows_that_share_bytes_are_refused():
    mbuild.build_library()
    lib = mdb.load_library()
    buf = ctypes.create_string_buffer(1 << 15)
    mem = (ctypes.addressof(buf) + 63) // 64 * 64

    def call(x, out, b=3, k=64, n=32, xs=64, os=32):
        return lib.moe_w4_linear(x, mem + 16384, None, out, b, k, n, 64, 0, xs, os, 0, None)

    free = mdb.MOE_ERR_NO_DEVICE
    assert call(mem, mem) == BAD
    assert call(mem, mem + 2 * (3 * 64 - 1)) == BAD  # the last element of x
    assert call(mem, mem + 2 * 3 * 64) == free
    assert call(mem + 2 * 96, mem + 2) == BAD  # the first element of x
    assert call(mem + 2 * 96, mem) == free
    # columns of one buffer of 96, either way round
    assert call(mem, mem + 2 * 64, xs=96, os=96) == free
    assert call(mem + 2 * 32, mem, xs=96, os=96) == free
    assert call(mem, mem + 2 * 63, xs=96, os=96) == BAD
    assert call(mem, mem + 2 * 65, xs=96, os=96) == BAD  # into the next row of x
    # one row of x for all tokens, between rows of out
    assert call(mem + 2 * 32, mem, xs=0, os=96) == free
    assert call(mem + 2 * 24, mem, xs=0, os=96) == BAD
    # one token: strides do not count
    assert call(mem, mem + 2 * 64, b=1, xs=5, os=5) == free
    assert call(mem, mem + 2 * 63, b=1, xs=5, os=5) == BAD
    assert call(mem, mem, b=0) == mdb.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("b", [1, 7, 16, 40])
def test_columns_of_one_buffer(b):
    from test_gpu_w4 import _check_linear, _x
    from w4_reference import random_w4
    codes, scales, _ = random_w4(48, 128, 64, False, torch.bfloat16, seed=b)
    packed = w4.pack(codes, scales)
    both = torch.zeros(b, 176, dtype=torch.bfloat16, device="cuda")
    both[:, :128] = _x(b, 128, torch.bfloat16, seed=b)
    x, out = both[:, :128], both[:, 128:]
    w4.linear(x, packed, out, 64)
    torch.cuda.synchronize()
    _check_linear(x.contiguous(), codes, scales, None, None, out.contiguous())
    keep = both.clone()
    with pytest.raises(mdb.MoEDecodeError):
        w4.linear(x, packed, both[:, 120:168], 64)
    with pytest.raises(mdb.MoEDecodeError):
        w4.linear(x, packed, both[:, :48], 64)
    torch.cuda.synchronize()
    assert torch.equal(both, keep)
