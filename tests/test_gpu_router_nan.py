"""Logits that are NaN: a token's ids stay distinct and in range, whatever the number of experts that can be compared,
so no expert gets more assignments than there are tokens (what the 4-bit kernels' lists are sized by)."""
import pytest
import torch

from moe_decode_block_b200 import (MOE_ERR_DEVICE_PLAN, MOE_OK, MoEDecode, router_topk_noalloc, router_topk_noalloc_status,
                                   synth)
from test_gpu_w4 import W4Block
from w4_reference import U, assert_within

pytestmark = pytest.mark.gpu

E8 = synth.BlockShape(hidden=192, n_experts=8, top_k=8, inter=64, shared_inter=64)


def _distinct(ids, e):
    s = ids.long().sort(dim=1).values
    return bool((s >= 0).all()) and bool((s < e).all()) and bool((s[:, 1:] != s[:, :-1]).all())


@pytest.mark.parametrize("e,k,nan", [(8, 8, 1), (8, 8, 8), (8, 4, 6), (16, 8, 9), (16, 12, 6), (16, 16, 5), (64, 20, 60), (384, 8, 380),
                                     (384, 32, 200), (1024, 8, 1020), (1024, 32, 1000)])
@pytest.mark.parametrize("b", [1, 5, 64])
def test_router_ids_are_distinct(b, e, k, nan):
    g = torch.Generator(device="cuda").manual_seed(b + e + k)
    x = torch.randn(b, 256, device="cuda", generator=g).to(torch.bfloat16)
    rw = (torch.randn(256, e, device="cuda", generator=g) * 0.05).to(torch.bfloat16)
    cols = torch.randperm(e, device="cuda", generator=g)[:nan]
    rw[:, cols] = float("nan")
    ids, w = torch.full((b, k), -1, dtype=torch.int32, device="cuda"), torch.empty(b, k, device="cuda")
    router_topk_noalloc(x, rw, ids, w, k)
    torch.cuda.synchronize()
    assert _distinct(ids, e)
    st = router_topk_noalloc_status()
    if k <= 8:  # the comparable experts first, in their order; then whatever is left
        assert st == (MOE_ERR_DEVICE_PLAN if e - nan < k else MOE_OK)
        logits = x.double() @ rw.double()
        logits[:, cols] = -float("inf")
        n = min(k, e - nan)
        best = logits.topk(n, dim=1).values if n else logits[:, :0]
        assert_within(torch.gather(logits, 1, ids[:, :n].long()), best, torch.full_like(best, 1e-4))
    router_topk_noalloc(torch.zeros_like(x), torch.zeros_like(rw), ids, w, k)  # the next call is as ever
    assert router_topk_noalloc_status() == MOE_OK
    assert torch.equal(ids, torch.arange(k, dtype=torch.int32, device="cuda").expand(b, k))


@pytest.mark.parametrize("b", [1, 3, 8, 9, 40, 64])
def test_4bit_block_with_an_expert_of_nan_logits(b):
    """Seven of eight experts can be compared where eight are asked for: the eighth takes weight 0, the rest is the formula's."""
    m = W4Block(E8, 32, True, seed=90 + b)
    m.router_w = m.router_w.clone()
    m.router_w[:, 3] = float("nan")
    blk = m.handle(64)
    try:
        x = torch.randn(b, 192, device="cuda", generator=torch.Generator(device="cuda").manual_seed(b)).to(torch.bfloat16)
        for _ in range(2):
            out, ids, w = m.forward(blk, x)
            torch.cuda.synchronize()
            assert blk.status() == MOE_ERR_DEVICE_PLAN
            assert _distinct(ids, 8) and bool((ids[:, 7] == 3).all()) and not bool(w[:, 7].any())
            y, tol = m.expected(x, ids, w)
            want = x.double() + y
            assert_within(out, want, tol + U[torch.bfloat16] * (want.abs() + tol) + 2.0 ** -24 * x.double().abs())
    finally:
        blk.close()


@pytest.mark.parametrize("b", [8, 64])
def test_4bit_block_with_infinite_activations_stays_in_its_rows(b):
    """Two infinities in every second token make about half of its logits NaN: those tokens' outputs are not finite, the others' are right."""
    m = W4Block(E8, 64, False, seed=99)
    blk = m.handle(64)
    try:
        x = torch.randn(b, 192, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).to(torch.bfloat16)
        x[::2, 5] = float("inf")
        x[::2, 100] = -float("inf")
        out, ids, w = m.forward(blk, x)
        torch.cuda.synchronize()
        assert blk.status() == MOE_ERR_DEVICE_PLAN
        assert _distinct(ids, 8)
        assert not bool(out[::2].isfinite().all(dim=1).any())
        rows = torch.arange(1, b, 2, device="cuda")
        # (weights are rounded for the shared expert's and for heavy experts' whole lists: all b tokens choose all 8 experts)
        xs = x.clone()
        xs[::2] = 0
        y, tol = m.expected(xs, ids, torch.where(torch.arange(b, device="cuda")[:, None] % 2 == 1, w, torch.zeros_like(w)))
        want = x.double() + y
        assert_within(out[rows], want[rows], (tol + U[torch.bfloat16] * (want.abs() + tol) + 2.0 ** -24 * x.double().abs())[rows])
    finally:
        blk.close()


@pytest.mark.parametrize("b", [1, 8, 64])
def test_bf16_block_with_an_expert_of_nan_logits(b):
    s = synth.BlockShape(hidden=256, n_experts=8, top_k=8, inter=128, shared_inter=128)
    wts = synth.make_weights(s, seed=3, device="cuda")
    blk = MoEDecode(s.hidden, 8, 8, s.inter, s.shared_inter, max_batch=64)
    try:
        rw = wts.router_w.clone()
        rw[:, 3] = float("nan")
        x = torch.randn(b, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(b)).to(torch.bfloat16)
        out, ids, w = torch.empty_like(x), torch.empty(b, 8, dtype=torch.int32, device="cuda"), torch.empty(b, 8, device="cuda")
        blk.forward(x, rw, wts.w13, wts.w2, wts.shared_w13, wts.shared_w2, out, ids, w)
        torch.cuda.synchronize()
        assert blk.status() == MOE_ERR_DEVICE_PLAN
        assert _distinct(ids, 8) and bool((ids[:, 7] == 3).all()) and not bool(w[:, 7].any()) and bool(out.isfinite().all())
    finally:
        blk.close()
