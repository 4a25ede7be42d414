"""Layers, routers, blocks and the balance loss one behind the other on a stream and in a graph, each started while the
one before it ends: every result against 64 bits and the oracle's routing, whatever the routers chose."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import MIN_MARGIN, W_ATOL
from moe_decode_block_b200 import MOE_OK, balance, router_topk_noalloc, synth, w4
from test_gpu_balance import _check as _check_balance
from test_gpu_w4 import MANY, TINY_W4, W4Block, _check_linear, _x
from w4_reference import random_w4

pytestmark = pytest.mark.gpu


def _margins(x, m, k):
    logits, _, _ = oracle.router(synth.bf16_bits(x), synth.bf16_bits(m.router_w), k, None)
    return torch.from_numpy(np.asarray(oracle.topk_margin(logits, k)) >= MIN_MARGIN)


class Chain:
    """x0 -> layer -> x1 -> router alone and block -> x2 -> layer -> x3 -> router alone -> loss on its ids."""

    def __init__(self, shape, b, seed):
        self.m, self.b, self.k = W4Block(shape, 64, False, seed=seed), b, shape.top_k
        H, E = shape.hidden, shape.n_experts
        self.la, self.lb = (random_w4(H, H, 64, True, torch.bfloat16, seed=seed + i) for i in (1, 2))
        self.pa, self.pb = w4.pack(*self.la), w4.pack(*self.lb)
        self.blk = self.m.handle(b)
        self.logits = _x(b, E, torch.float32, seed=seed + 3)
        # tokens whose routing after the first layer does not hang on the order of a sum
        keep, i = [], 0
        while sum(len(t) for t in keep) < b:
            x0, x1 = _x(b, H, torch.bfloat16, seed=seed * 1000 + i), torch.empty(b, H, dtype=torch.bfloat16, device="cuda")
            w4.linear(x0, self.pa, x1, 64, zeros=True)
            keep.append(x0[_margins(x1, self.m, self.k).cuda()])
            i += 1
            assert i < 200
        self.x0 = torch.cat(keep)[:b].contiguous()
        new = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.x1, self.x2, self.x3 = (torch.empty_like(self.x0) for _ in range(3))
        self.ids = [torch.empty(b, self.k, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.w = [new(b, self.k) for _ in range(3)]
        self.loss, self.counts, self.d = new(1), torch.empty(E + 1, dtype=torch.int32, device="cuda"), new(b, E)

    def poison(self):
        for t in (self.x1, self.x2, self.x3, *self.w, self.loss, self.d):
            t.fill_(float("nan"))
        for t in (*self.ids, self.counts):
            t.fill_(-1)

    def run(self):
        m = self.m
        w4.linear(self.x0, self.pa, self.x1, 64, zeros=True)
        router_topk_noalloc(self.x1, m.router_w, self.ids[1], self.w[1], self.k)
        w4.linear(self.x0, self.pa, self.x1, 64, zeros=True)  # the same again, right before the block
        self.blk.forward_w4(self.x1, m.router_w, *m.packed, self.x2, self.ids[0], self.w[0], 64)
        w4.linear(self.x2, self.pb, self.x3, 64, zeros=True)
        router_topk_noalloc(self.x3, m.router_w, self.ids[2], self.w[2], self.k)
        balance.balance_loss(self.logits, self.ids[2], self.loss, self.counts, coef=0.5, dlogits=self.d)

    def check(self):
        _check_linear(self.x0, *self.la, None, self.x1)
        assert bool(_margins(self.x1, self.m, self.k).all())
        self.m.check(self.x1, self.x2, self.ids[0], self.w[0])  # (the oracle's ids too)
        assert torch.equal(self.ids[0], self.ids[1])
        assert float((self.w[0] - self.w[1]).abs().max()) <= 2 * W_ATOL
        _check_linear(self.x2, *self.lb, None, self.x3)
        _, ids, w = oracle.router(synth.bf16_bits(self.x3), synth.bf16_bits(self.m.router_w), self.k, None)
        clear = _margins(self.x3, self.m, self.k).numpy()
        assert clear.mean() > 0.5
        np.testing.assert_array_equal(self.ids[2].cpu().numpy()[clear], ids[clear])
        assert np.abs(self.w[2].cpu().numpy()[clear].astype(np.float64) - w[clear]).max() <= W_ATOL
        _check_balance(self.logits, self.ids[2], None, None, 0.5, None, self.loss, self.counts, self.d)


@pytest.mark.parametrize("shape,b", [(TINY_W4, 1), (TINY_W4, 8), (TINY_W4, 12), (TINY_W4, 40), (MANY, 5), (MANY, 64)])
def test_chain_on_a_stream_and_in_a_graph(shape, b):
    c = Chain(shape, b, seed=11 * b)
    try:
        for _ in range(3):
            c.poison()
            c.run()
            torch.cuda.synchronize()
            c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
            c.run()
        for _ in range(2):
            c.poison()
            graph.replay()
            torch.cuda.synchronize()
            c.check()
        assert c.blk.status() == MOE_OK and w4.linear_status() == MOE_OK
    finally:
        c.blk.close()
