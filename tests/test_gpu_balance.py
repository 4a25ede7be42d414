"""The router's balance loss, its gradient and the counts on a B200
(moe_balance_loss) against the 64-bit formulas and against differences.

Tolerance: an exponential is off by 2^-22 (two steps) plus its argument's
roundings -- the bias's addition and the product with log2(e), at most 2^-24 of
|z| <= 16 and of |z - max| log2(e) <= 48 -- 5e-6 in all; a row's sums of 1,024
such terms add 2^-24 * 42 (32 terms a lane, ten steps of adding up): under 1e-5
for a probability, REL.  A gradient p (c - s) is then off by 2 REL of p |c - s|
and REL of p sum p |c - c0|; with c0 within one of the mean count, |c - c0| is
|c - s| + |s - c0|."""
import pytest
import torch

from moe_decode_block_b200 import balance
from w4_reference import TINY, U, assert_within, balance64

pytestmark = pytest.mark.gpu
REL = 1e-5


def _inputs(t, e, k, dtype, seed, live=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(t, e, device="cuda", generator=g) * 2).clamp_(-8, 8).to(dtype)
    bias = torch.randn(e, device="cuda", generator=g).clamp_(-4, 4)
    ids = torch.topk(logits.float() + bias, k, dim=1).indices.to(torch.int32) if t else torch.zeros(0, k, dtype=torch.int32, device="cuda")
    mask = None if live is None else torch.rand(t, device="cuda", generator=g) < live
    return logits, bias, ids, mask


def _run(logits, ids, mask=None, bias=None, coef=0.5, grad=None, dlogits="new", **kw):
    e = logits.shape[1]
    loss = torch.full((1,), float("nan"), device="cuda")
    counts = torch.full((e + 1,), -7, dtype=torch.int32, device="cuda")
    if isinstance(dlogits, str):
        dlogits = torch.full_like(logits, float("nan"))
    balance.balance_loss(logits, ids, loss, counts, token_mask=mask, router_bias=bias, coef=coef, dlogits=dlogits, grad_loss=grad, **kw)
    torch.cuda.synchronize()
    return loss, counts, dlogits


def _check(logits, ids, mask, bias, coef, grad, loss, counts, dlogits):
    g = 1.0 if grad is None else float(grad)
    l64, c64, d64, spread, p, c, f = balance64(logits, ids, mask, bias, coef, g)
    assert torch.equal(counts, c64)
    s = (p * c).sum(dim=1, keepdim=True)
    c0 = int(c64[-1]) * ids.shape[1] // logits.shape[1]
    off = spread + (s - c0).abs() * p.sum(dim=1, keepdim=True)
    assert_within(loss, l64.view(1), f * 3 * REL * off.sum() + 2.0 ** -23 * l64.abs() + 2.0 ** -149, "loss")
    if dlogits is not None:
        u = U[logits.dtype]
        tol = abs(g) * f * REL * p * (2 * (c - s).abs() + 3 * off) + 2.0 ** -22 * d64.abs()
        # the formula's own 64-bit roundings: p c and s each off by under 2^-48 of s (up to 1,024 terms, the softmax's
        # exponential and quotient 2^-50), where c - s cancels to nothing (every expert chosen alike: the gradient is 0)
        tol = tol + 2.0 ** -47 * abs(g) * f * p * (c + s)
        assert_within(dlogits, d64, tol + u * (d64.abs() + tol) + TINY[logits.dtype], "dlogits")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e,k", [(8, 1), (8, 8), (24, 3), (128, 4), (136, 2), (256, 8), (384, 8), (512, 6), (1000, 32), (1024, 2)])
@pytest.mark.parametrize("t", [1, 7, 64, 513, 1500])
def test_sizes_and_types(t, e, k, dtype):
    logits, bias, ids, mask = _inputs(t, e, k, dtype, seed=t + e, live=0.7 if t % 2 else None)
    grad = torch.full((1,), 3.0e3 if dtype is torch.float16 else 1.25, device="cuda")
    loss, counts, d = _run(logits, ids, mask, bias, grad=grad)
    _check(logits, ids, mask, bias, 0.5, grad, loss, counts, d)


@pytest.mark.parametrize("t", [20000, 70001])
def test_long(t):
    logits, bias, ids, mask = _inputs(t, 384, 8, torch.float32, seed=t, live=0.9)
    loss, counts, d = _run(logits, ids, mask, None)
    _check(logits, ids, mask, None, 0.5, None, loss, counts, d)


@pytest.mark.parametrize("t", [0, 1, 300, 2000])
def test_no_live_token(t):
    logits, bias, ids, _ = _inputs(t, 40, 4, torch.float32, seed=t)
    mask = torch.zeros(t, dtype=torch.uint8, device="cuda")
    loss, counts, d = _run(logits, ids, mask, bias)
    assert float(loss) == 0.0 and not bool(counts.any()) and not bool(d.any())


def test_masked_rows_may_hold_anything():
    t, e = 900, 64
    logits, bias, ids, _ = _inputs(t, e, 4, torch.bfloat16, seed=5)
    mask = torch.arange(t, device="cuda") % 3 != 1
    clean = _run(logits, ids, mask, bias)
    logits[~mask] = float("nan")
    ids[~mask] = 1 << 30
    dirty = _run(logits, ids, mask, bias)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    assert not bool(dirty[2][~mask].any())


@pytest.mark.parametrize("t", [50, 1200])
def test_experts_that_cannot_be_chosen_and_empty_rows(t):
    """-inf and the type's lowest value; a row of -inf alone counts its ids and has no gradient."""
    logits, bias, ids, _ = _inputs(t, 48, 3, torch.float32, seed=9)
    logits[:, 5] = -float("inf")
    logits[:, 6] = torch.finfo(torch.float32).min
    logits[4] = -float("inf")
    logits[t - 1] = torch.finfo(torch.float32).min  # all alike: a uniform row
    ids[2, 1] = -1
    ids[3, 0] = 48
    loss, counts, d = _run(logits, ids)
    assert bool(d.isfinite().all()) and not bool(d[4].any()) and not bool(d[:t - 1, 5:7].any())
    _check(logits, ids, None, None, 0.5, None, loss, counts, d)


@pytest.mark.parametrize("t", [50, 1200])
def test_nan_is_not_hidden(t):
    logits, bias, ids, _ = _inputs(t, 48, 3, torch.float32, seed=10)
    logits[7, 7] = float("nan")
    loss, counts, d = _run(logits, ids)
    assert bool(loss.isnan()) and bool(d[7].isnan().all()) and bool(d[8].isfinite().all())


def test_repeated_ids_count_each_time():
    logits, _, ids, _ = _inputs(700, 16, 4, torch.float32, seed=11)
    ids[:] = 3
    loss, counts, d = _run(logits, ids)
    assert int(counts[3]) == 2800
    _check(logits, ids, None, None, 0.5, None, loss, counts, d)


@pytest.mark.parametrize("t", [60, 1700])
def test_strided_rows_in_place_and_no_gradient(t):
    wide, bias, _, _ = _inputs(t, 96, 4, torch.float32, seed=12)
    logits = wide[:, 8:72]
    ids = torch.topk(logits, 4, dim=1).indices.to(torch.int32)
    keep = wide.clone()
    loss, counts, d = _run(logits, ids, dlogits=torch.full((t, 80), 5.0, device="cuda")[:, 4:68])
    _check(logits, ids, None, None, 0.5, None, loss, counts, d)
    assert bool((d._base[:, :4] == 5).all()) and bool((d._base[:, 68:] == 5).all())
    loss2, counts2, _ = _run(logits, ids, dlogits=None)
    assert torch.equal(loss, loss2) and torch.equal(counts, counts2) and torch.equal(wide, keep)
    loss3, _, d3 = _run(logits, ids, dlogits=logits)  # the logits' own buffer
    assert torch.equal(loss, loss3) and torch.equal(d3, d)
    assert torch.equal(wide[:, :8], keep[:, :8]) and torch.equal(wide[:, 72:], keep[:, 72:])


@pytest.mark.parametrize("t", [40, 600])
def test_gradient_against_differences(t):
    """The kernel's loss itself, in two directions: (L(z + h v) - L(z - h v)) / 2 h with the counts held (the ids stay).
    Off by h^2 / 6 of the third derivative along v (|v| <= 1: under 16 f sum p |c - s|) and the two losses' roundings / h."""
    logits, bias, ids, _ = _inputs(t, 32, 2, torch.float32, seed=13)
    loss, counts, d = _run(logits, ids, None, bias, coef=100.0)
    _, _, _, spread, p, c, f = balance64(logits, ids, None, bias, 100.0)
    h = 2.0 ** -6
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        v = torch.rand(t, 32, device="cuda", generator=g).sub_(0.5).mul_(2).mul_(64).round_().div_(64)
        up = float(_run(logits + h * v, ids, None, bias, coef=100.0)[0])
        dn = float(_run(logits - h * v, ids, None, bias, coef=100.0)[0])
        want = float((d.double() * v.double()).sum())
        tol = h * h / 6 * 16 * f * float(spread.sum()) + (2.0 ** -22 * abs(up) + 6 * REL * f * float(spread.sum())) / h
        assert abs((up - dn) / (2 * h) - want) <= tol


def test_same_bits_graph_streams_and_workspaces():
    t, e, k = 5000, 256, 4
    logits, bias, ids, mask = _inputs(t, e, k, torch.bfloat16, seed=14, live=0.8)
    first = _run(logits, ids, mask, bias)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for i in range(6):
        loss, counts = torch.empty(1, device="cuda"), torch.empty(e + 1, dtype=torch.int32, device="cuda")
        d, ws = torch.empty_like(logits), torch.full((balance.workspace_bytes(e),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        balance.balance_loss(logits, ids, loss, counts, token_mask=mask, router_bias=bias, coef=0.5, dlogits=d, workspace=ws,
                             stream=streams[i % 2])
        results.append((loss, counts, d))
    torch.cuda.synchronize()
    for r in results:
        for a, b in zip(first, r):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):  # another stream needs its own workspace
        balance.balance_loss(logits, ids, loss, counts, stream=streams[0])
    lg, ig = logits.clone(), ids.clone()
    loss, counts, d = torch.empty(1, device="cuda"), torch.empty(e + 1, dtype=torch.int32, device="cuda"), torch.empty_like(logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        balance.balance_loss(lg, ig, loss, counts, token_mask=mask, router_bias=bias, coef=0.5, dlogits=d)
    other = _inputs(t, e, k, torch.bfloat16, seed=15)
    lg.copy_(other[0])
    ig.copy_(other[2])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    _check(lg, ig, mask, bias, 0.5, None, loss, counts, d)
