"""4-bit products and the balance loss where a caller may take them: buffers rewritten between calls that overlap, two
handles at once, first calls inside a capture, offsets beyond 32 bits, the smallest and the largest sizes."""
import os
import subprocess
import sys

import pytest
import torch

from gpu_helpers import margin_x
from moe_decode_block_b200 import MOE_OK, balance, synth, w4
from test_gpu_balance import _check as _check_balance
from test_gpu_balance import _run as _run_balance
from test_gpu_w4 import MANY, TINY_W4, W4Block, _check_linear, _x
from w4_reference import U, assert_within, random_w4

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("b,n,k", [(1, 2048, 1024), (8, 700, 2048), (16, 1500, 1024), (40, 700, 1024), (64, 4096, 512)])
def test_linear_on_a_buffer_rewritten_between_calls(b, n, k):
    """Each call must see the x that was written right before it, and the next writer must not come too early."""
    codes, scales, z = random_w4(n, k, 64, False, torch.bfloat16, seed=b)
    packed = w4.pack(codes, scales)
    xs = [_x(b, k, torch.bfloat16, seed=100 * b + i) for i in range(24)]
    x = torch.empty_like(xs[0])
    outs = [torch.full((b, n), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for src, out in zip(xs, outs):
        x.copy_(src)
        w4.linear(x, packed, out, 64)
    torch.cuda.synchronize()
    for src, out in zip(xs, outs):
        _check_linear(src, codes, scales, None, None, out)
    # the output of one call the input of the next, in two buffers by turns
    if n >= k:
        return
    sq, ss, _ = random_w4(k, k, 64, False, torch.bfloat16, seed=b + 1)
    ps, bufs, seen = w4.pack(sq, ss), [x, torch.empty_like(x)], []
    x.copy_(xs[0])
    for i in range(6):
        w4.linear(bufs[i % 2], ps, bufs[1 - i % 2], 64)
        seen.append(bufs[1 - i % 2].clone())
    torch.cuda.synchronize()
    for before, after in zip([xs[0]] + seen, seen):
        _check_linear(before, sq, ss, None, None, after)


@pytest.mark.parametrize("shape,b", [(TINY_W4, 3), (TINY_W4, 8), (TINY_W4, 9), (MANY, 24), (MANY, 64)])
def test_block_on_a_buffer_rewritten_between_forwards_two_handles(shape, b):
    m = W4Block(shape, 64, True, seed=200 + b)
    handles, streams = [m.handle(b), m.handle(b)], [torch.cuda.Stream(), torch.cuda.Stream()]
    try:
        xs = [margin_x(b, shape.hidden, m, shape.top_k, seed=2000 + 10 * b + i) for i in range(6)]
        results = []
        torch.cuda.synchronize()
        for blk, st in zip(handles, streams):
            with torch.cuda.stream(st):
                x = torch.empty_like(xs[0])
                for src in xs + xs[::-1]:
                    x.copy_(src)
                    results.append((src, *m.forward(blk, x, stream=st)))
        torch.cuda.synchronize()
        for src, out, ids, w in results:
            m.check(src, out, ids, w)
        assert all(h.status() == MOE_OK for h in handles)
    finally:
        for h in handles:
            h.close()


SHAPES = [synth.BlockShape(64, 8, 1, 64, 64), synth.BlockShape(64, 8, 8, 64, 0, n_shared=0), synth.BlockShape(128, 8, 3, 64, 192),
          synth.BlockShape(16384, 8, 2, 64, 64), synth.BlockShape(64, 1024, 32, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("b", [1, 8, 9, 64])
def test_smallest_and_largest_blocks(shape, b):
    m = W4Block(shape, 32 if shape.hidden < 128 else 64, False, seed=300 + b)
    blk = m.handle(b)
    try:
        x = torch.randn(b, shape.hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(b)).to(torch.bfloat16)
        for _ in range(2):
            out, ids, w = m.forward(blk, x)
            torch.cuda.synchronize()
            y, tol = m.expected(x, ids, w)  # (for the routing that it returned: margins are not asked for here)
            want = x.double() + y
            assert_within(out, want, tol + U[torch.bfloat16] * (want.abs() + tol) + 2.0 ** -24 * x.double().abs())
            logits = x.double() @ m.router_w.double()
            best = logits.topk(shape.top_k, dim=1).values
            assert float((torch.gather(logits, 1, ids.long()) - best).abs().max()) <= 1e-3
        assert blk.status() == MOE_OK
    finally:
        blk.close()


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from moe_decode_block_b200 import MoEDecode, balance, w4
from w4_reference import random_w4
torch.cuda.init()
what = {what!r}
g = torch.cuda.CUDAGraph()
if what.startswith("linear"):
    b = int(what[6:])
    packed = torch.randint(0, 100, (w4.packed_bytes(256, 256, 64),), dtype=torch.uint8, device="cuda")
    x, out, again = torch.ones(b, 256, dtype=torch.float16, device="cuda"), *(torch.zeros(b, 256, dtype=torch.float16, device="cuda") for _ in range(2))
    packed.view(16, -1)[:, 2048:] = torch.full((16, 64), 0.01, dtype=torch.float16, device="cuda").view(torch.uint8)
    call = lambda o: w4.linear(x, packed, o, 64)
elif what.startswith("balance"):
    t = int(what[7:])
    z, ids = torch.randn(t, 64, device="cuda"), torch.zeros(t, 2, dtype=torch.int32, device="cuda")
    out, again = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    counts, ws = torch.zeros(65, dtype=torch.int32, device="cuda"), torch.zeros(balance.workspace_bytes(64), dtype=torch.uint8, device="cuda")
    call = lambda o: balance.balance_loss(z, ids, o, counts, workspace=ws)
else:
    b = int(what[5:])
    mk = lambda n, k, lead=(): w4.pack(*random_w4(n, k, 64, False, torch.bfloat16, 1, lead=lead))
    ws = [mk(256, 128, (8,)), mk(128, 128, (8,)), mk(256, 128), mk(128, 128)]
    rw = torch.randn(128, 8, device="cuda").to(torch.bfloat16)
    x = torch.randn(b, 128, device="cuda").to(torch.bfloat16)
    out, again = torch.zeros_like(x), torch.zeros_like(x)
    ids, w = torch.zeros(b, 2, dtype=torch.int32, device="cuda"), torch.zeros(b, 2, device="cuda")
    blk = MoEDecode(128, 8, 2, 128, 128, max_batch=64, w4=True)
    call = lambda o: blk.forward_w4(x, rw, *ws, o, ids, w, 64)
torch.cuda.synchronize()
with torch.cuda.graph(g):
    call(out)
g.replay()
torch.cuda.synchronize()
call(again)
torch.cuda.synchronize()
assert bool(out.isfinite().all()) and bool((out != 0).any())
assert float((out.float() - again.float()).abs().max()) <= 0.02 * float(out.float().abs().max())
print("same")
"""


@pytest.mark.parametrize("what", ["linear1", "linear9", "linear17", "balance64", "balance600", "block3", "block20"])
def test_first_call_of_a_process_inside_a_capture(what):
    code = FIRST.format(root=ROOT, tests=os.path.join(ROOT, "tests"), what=what)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-3000:]


@pytest.mark.parametrize("b", [8, 16, 64])
def test_linear_rows_further_apart_than_32_bits(b):
    n, k, pitch = 100, 128, (1 << 33) // b // 2 + 8  # elements: the last row begins near 2^32
    codes, scales, _ = random_w4(n, k, 64, False, torch.bfloat16, seed=b)
    packed = w4.pack(codes, scales)
    store = torch.empty(b * pitch, dtype=torch.bfloat16, device="cuda").view(b, pitch)
    x, out = store[:, :k], store[:, 1024:1024 + n]
    src = _x(b, k, torch.bfloat16, seed=b)
    x.copy_(src)
    w4.linear(x, packed, out, 64)
    _check_linear(src, codes, scales, None, None, out.contiguous())
    del store, x, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("b", [1, 16, 64])
def test_linear_matrix_larger_than_32_bits(b):
    """524,288 outputs of 17,408 inputs: 4.6 GB of codes; the first rows, some inside and the last against 64 bits."""
    n, k = 524288, 17408
    g = torch.Generator(device="cuda").manual_seed(b)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = ((torch.rand(n, k // 128, device="cuda", generator=g) + 0.5) * 0.005).to(torch.bfloat16)
    packed = w4.pack(codes, scales)
    x = _x(b, k, torch.bfloat16, seed=b)
    out = torch.full((b, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.linear(x, packed, out, 128)
    torch.cuda.synchronize()
    assert bool(out.isfinite().all())
    for r in (0, 123456, 493448, n - 64):  # (byte 2^32 of the packed matrix lies in row 484,000)
        _check_linear(x, codes[r:r + 64], scales[r:r + 64], None, None, out[:, r:r + 64].contiguous())
    del codes, scales, packed, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("grad", [False, True])
def test_balance_most_tokens(grad):
    t, e, k = 1 << 24, 8, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = (torch.randn(t, e, device="cuda", generator=g) * 2).clamp_(-8, 8).to(torch.float32 if grad else torch.bfloat16)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    loss, counts, d = _run_balance(logits, ids, dlogits="new" if grad else None)
    _check_balance(logits, ids, None, None, 0.5, None, loss, counts, d)
    del logits, ids, d
    torch.cuda.empty_cache()


def test_balance_rows_further_apart_than_32_bits():
    t, e = 1100, 64
    store = torch.empty(t, 1 << 22, dtype=torch.bfloat16, device="cuda")  # 9 GB
    logits = store[:, 8:8 + e]
    g = torch.Generator(device="cuda").manual_seed(2)
    src = (torch.randn(t, e, device="cuda", generator=g) * 2).clamp_(-8, 8).to(torch.bfloat16)
    logits.copy_(src)
    ids = torch.topk(src.float(), 4, dim=1).indices.to(torch.int32)
    loss, counts, d = _run_balance(logits, ids, dlogits=store[:, 1000:1000 + e])
    _check_balance(src, ids, None, None, 0.5, None, loss, counts, d.contiguous())
    del store, logits, d
    torch.cuda.empty_cache()
