"""The first forward of a handle, and the first call without one, on a stream that does not wait for the default stream
while that is busy: the zeroed state must be there before, whatever the memory held."""
import os
import subprocess
import sys

import pytest
import torch

from gpu_helpers import Run, margin_x, oracle_check
from moe_decode_block_b200 import MOE_ERR_DEVICE_TIMEOUT, MOE_OK, synth, w4
from test_gpu_w4 import TINY_W4, W4Block, _x
from w4_reference import random_w4

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _fill_free_memory():
    t = [torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del t
    torch.cuda.empty_cache()


@pytest.mark.parametrize("b", [1, 8, 40])
def test_new_4bit_handle_beside_a_busy_default_stream(b):
    m = W4Block(TINY_W4, 64, False, seed=400 + b)
    x = margin_x(b, TINY_W4.hidden, m, 2, seed=4000 + b)
    side = torch.cuda.Stream()
    for _ in range(2):
        _fill_free_memory()
        out = torch.full_like(x, float("nan"))
        ids, w = torch.full((b, 2), -1, dtype=torch.int32, device="cuda"), torch.full((b, 2), float("nan"), device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # 50 ms on the default stream
        blk = m.handle(b)
        try:
            blk.forward_w4(x, m.router_w, *m.packed, out, ids, w, 64, stream=side)
            side.synchronize()
            got = [t.clone() for t in (out, ids, w)]
            torch.cuda.synchronize()
            m.check(x, *got)
            m.check(x, out, ids, w)
            assert blk.status() == MOE_OK
        finally:
            blk.close()


@pytest.mark.parametrize("b", [1, 8, 40])
def test_new_handle_beside_a_busy_default_stream(b):
    s = synth.TINY
    wts = synth.make_weights(s, seed=0, device="cuda")
    x = margin_x(b, s.hidden, wts, s.top_k, seed=b)
    out = torch.full_like(x, float("nan"))
    ids, w = torch.empty(b, s.top_k, dtype=torch.int32, device="cuda"), torch.empty(b, s.top_k, device="cuda")
    side = torch.cuda.Stream()
    _fill_free_memory()
    torch.cuda._sleep(100_000_000)
    run = Run(s, wts, max_batch=b)
    try:
        run.blk.forward(x, wts.router_w, wts.w13, wts.w2, wts.shared_w13, wts.shared_w2, out, ids, w, stream_main=side,
                        stream_aux=side)
        side.synchronize()
        oracle_check(wts, s.top_k, x, out, ids, w)
        assert run.blk.status() == MOE_OK
    finally:
        run.blk.close()


NO_HANDLE = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from moe_decode_block_b200 import router_topk_noalloc, router_topk_noalloc_status
x = torch.randn(64, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
rw = torch.randn(512, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(torch.bfloat16)
ids, w = torch.empty(64, 4, dtype=torch.int32, device="cuda"), torch.empty(64, 4, device="cuda")
side = torch.cuda.Stream()
torch.cuda.synchronize()
torch.cuda._sleep(100_000_000)
for _ in range(20):
    router_topk_noalloc(x, rw, ids, w, 4, stream=side)
side.synchronize()
got = ids.long()
torch.cuda.synchronize()
logits = x.double() @ rw.double()
best = logits.topk(4, dim=1).values
assert float((torch.gather(logits, 1, got) - best).abs().max()) < 1e-2
assert router_topk_noalloc_status(side) == 0
print("right")
"""


def test_first_call_without_a_handle_beside_a_busy_default_stream():
    code = NO_HANDLE.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "right" in r.stdout, r.stderr[-3000:]


def test_a_status_that_was_cleared_stays_cleared_and_the_next_is_not():
    codes, scales, _ = random_w4(300, 256, 64, False, torch.bfloat16, seed=5)
    packed, x = w4.pack(codes, scales), _x(20, 256, torch.bfloat16, seed=6)
    out = torch.empty(20, 300, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    w4.set_wait_limit(64)
    try:
        for _ in range(3):
            w4.test_hold(1)
            w4.linear(x, packed, out, 64, stream=side)
            assert w4.linear_status(side) == MOE_ERR_DEVICE_TIMEOUT
            assert w4.linear_status(side) == MOE_OK
    finally:
        w4.test_hold(0)
        w4.set_wait_limit(0)
