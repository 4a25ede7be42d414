"""The bounded waits of the tcgen05 4-bit kernels run out, without faulting or hanging the GPU: moe_w4_test_hold keeps the
first CTA's first step from being handed over, a short limit ends the waits for it, the status says so, and what comes
after is right."""
import pytest
import torch

from gpu_helpers import margin_x
from moe_decode_block_b200 import MOE_ERR_DEVICE_TIMEOUT, MOE_OK, w4
from test_gpu_w4 import TINY_W4, W4Block, _check_linear, _x
from w4_reference import random_w4

pytestmark = pytest.mark.gpu

LIMIT = 1 << 9  # probes: 10 ms


@pytest.fixture(autouse=True)
def back_to_normal():
    yield
    w4.test_hold(0)
    w4.set_wait_limit(0)


@pytest.mark.parametrize("b,n,k", [(17, 256, 64), (40, 300, 1024), (64, 5000, 2048)])
def test_linear_reports_a_wait_that_ran_out(b, n, k):
    codes, scales, z = random_w4(n, k, 64, True, torch.bfloat16, seed=n)
    packed, x = w4.pack(codes, scales, z), _x(b, k, torch.bfloat16, seed=b)
    out = torch.empty(b, n, dtype=torch.bfloat16, device="cuda")
    assert w4.linear_status() == MOE_OK
    w4.set_wait_limit(LIMIT)
    w4.linear(x, packed, out, 64, zeros=True)  # the limit alone does no harm
    assert w4.linear_status() == MOE_OK
    _check_linear(x, codes, scales, z, None, out)
    w4.test_hold(1)
    w4.linear(x, packed, out, 64, zeros=True)
    assert w4.linear_status() == MOE_ERR_DEVICE_TIMEOUT
    assert w4.linear_status() == MOE_OK  # reading cleared it
    w4.set_wait_limit(0)
    for _ in range(2):
        out.fill_(float("nan"))
        w4.linear(x, packed, out, 64, zeros=True)
        assert w4.linear_status() == MOE_OK
        _check_linear(x, codes, scales, z, None, out)


def test_linear_calls_behind_and_beside_one_that_ran_out():
    """The next calls are launched while the one that waits is ending, on its stream and on another."""
    b, n, k = 33, 700, 1024
    codes, scales, z = random_w4(n, k, 128, False, torch.float16, seed=1)
    packed, x = w4.pack(codes, scales, z), _x(b, k, torch.float16, seed=2)
    outs = [torch.full((b, n), float("nan"), dtype=torch.float16, device="cuda") for _ in range(5)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    w4.set_wait_limit(LIMIT)
    w4.test_hold(1)
    for i, o in enumerate(outs):
        w4.linear(x, packed, o, 128, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert w4.linear_status() == MOE_ERR_DEVICE_TIMEOUT
    for o in outs[1:]:
        _check_linear(x, codes, scales, z, None, o)
    assert w4.linear_status() == MOE_OK


@pytest.mark.parametrize("b,held", [(9, 1), (40, 1), (40, 2), (64, 2)])
def test_block_reports_a_wait_that_ran_out(b, held):
    m = W4Block(TINY_W4, 64, True, seed=100 + b)
    blk = m.handle(64)
    try:
        x = margin_x(b, TINY_W4.hidden, m, 2, seed=1000 + b)
        blk.set_wait_limit(1 << 12)
        out, ids, w = m.forward(blk, x)
        assert blk.status() == MOE_OK  # the limit alone does no harm
        m.check(x, out, ids, w)
        w4.test_hold(held)
        m.forward(blk, x)
        assert blk.status() == MOE_ERR_DEVICE_TIMEOUT
        t = torch.arange(1024, device="cuda", dtype=torch.float32)
        assert float(t.sum()) == 1023 * 1024 / 2
        blk.set_wait_limit(0)
        for _ in range(2):
            out, ids, w = m.forward(blk, x)
            torch.cuda.synchronize()
            m.check(x, out, ids, w)
            assert blk.status() == MOE_OK
    finally:
        blk.close()
