"""4-bit weight products on a B200: moe_w4_pack, moe_w4_linear and the block on
4-bit expert weights (moe_decode_forward_w4), against plain 64-bit forms on
every element.

Tolerances count roundings: one to the output's type, the fp32 sums as
product_tolerance says, and in the block one bf16 rounding of each expert's
activation before the down projection."""
import numpy as np
import pytest
import torch

import oracle
from moe_decode_block_b200 import (MOE_ERR_DEVICE_TIMEOUT, MOE_OK, MoEDecode, MoEDecodeError, reduce_residual,
                                   router_topk_noalloc, synth, w4)
from gpu_helpers import W_ATOL, margin_x
from w4_reference import TINY as TINY_STEP
from w4_reference import U, assert_within, dequant64, product_magnitude, product_tolerance, random_w4

pytestmark = pytest.mark.gpu


def _x(b, k, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(b, k, device="cuda", generator=g).to(dtype)


def _weights(codes, scales, zeros, tokens, exact=16):
    """The weights as the products take them: exact up to `exact` tokens, above rounded once to the scales' type."""
    w = dequant64(codes, scales, zeros)
    return w if tokens <= exact else w.to(scales.dtype).double()  # (12 to 15 bits: exact in the fp32 between)


def _fp32_error(x, codes, scales, zeros, w, exact=16):
    """What the fp32 sums may be off by, in 64 bits."""
    if len(x) <= exact:
        return product_tolerance(x.shape[1], x.dtype) * product_magnitude(x, codes, scales, zeros)
    # one chain of K / 16 instructions (each under 2^-23 of the sum of magnitudes), 8 CTAs, bias
    return (x.shape[1] / 16 + 10) * 2.0 ** -23 * (x.double().abs() @ w.abs().T)


def _check_linear(x, codes, scales, zeros, bias, out):
    w = _weights(codes, scales, zeros, len(x))
    y = x.double() @ w.T
    off = _fp32_error(x, codes, scales, zeros, w)
    if bias is not None:
        y, off = y + bias.double(), off + 2.0 ** -23 * bias.double().abs()
    assert_within(out, y, U[x.dtype] * (y.abs() + off) + off + TINY_STEP[x.dtype])


def _packed_by_definition(codes, scales, zeros, n, k, group):
    """The packed bytes, element by element from the layout's definition."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).cpu().numpy()
    s = scales.cpu().view(torch.int16).numpy().view(np.uint16)
    z = None if zeros is None else zeros.cpu().to(scales.dtype).view(torch.int16).numpy().view(np.uint16)
    panels, tiles, groups = -(-n // 16), k // 64, k // group
    width = 64 if zeros is not None else 32
    out = np.zeros((panels, tiles * 512 + groups * width), dtype=np.uint8)
    for p in range(panels):
        words = np.zeros((tiles, 32, 4), dtype=np.uint32)
        for tile in range(tiles):
            for lane in range(32):
                g, t = lane // 4, lane % 4
                for sw in range(4):
                    for j in range(4):
                        row = p * 16 + g + 8 * (j & 1)
                        col = tile * 64 + 32 * (sw >> 1) + 8 * t + 4 * (sw & 1) + 2 * (j >> 1)
                        if row < n:
                            words[tile, lane, sw] |= np.uint32(int(q[row, col]) << (4 * j) | int(q[row, col + 1]) << (16 + 4 * j))
        ent = np.zeros((groups, 8, width // 16), dtype=np.uint16)
        for hi in range(2):
            for g in range(8):
                row = p * 16 + g + 8 * hi
                if row < n:
                    ent[:, g, hi] = s[row]
                    if z is not None:
                        ent[:, g, 2 + hi] = z[row]
        out[p] = np.concatenate([words.reshape(-1).view(np.uint8), ent.reshape(-1).view(np.uint8)])
    return out


@pytest.mark.parametrize("n,k,group,zeros,dtype", [(16, 64, 64, False, torch.bfloat16), (37, 256, 32, True, torch.float16),
                                                    (5, 128, 128, True, torch.bfloat16)])
def test_pack_follows_the_layout(n, k, group, zeros, dtype):
    codes, scales, z = random_w4(n, k, group, zeros, dtype, seed=n)
    got = w4.pack(codes, scales, z)
    assert got.numel() == w4.packed_bytes(n, k, group, zeros)
    np.testing.assert_array_equal(got.cpu().numpy(), _packed_by_definition(codes, scales, z, n, k, group))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("b", [1, 2, 8, 9, 16, 17, 33, 64])
def test_linear_tokens_groups_types(b, group, zeros, dtype):
    n, k = 200, 640
    codes, scales, z = random_w4(n, k, group, zeros, dtype, seed=7 * b)
    x = _x(b, k, dtype, seed=b)
    out = torch.full((b, n), float("nan"), dtype=dtype, device="cuda")
    w4.linear(x, w4.pack(codes, scales, z), out, group, zeros=zeros)
    _check_linear(x, codes, scales, z, None, out)


@pytest.mark.parametrize("b", [1, 11, 40])
@pytest.mark.parametrize("n,k", [(1, 64), (15, 64), (17, 128), (63, 7168), (64, 448), (65, 576), (1003, 1600), (4096, 2048),
                                 (16, 32768), (5000, 192)])
def test_linear_sizes(n, k, b):
    codes, scales, z = random_w4(n, k, 64, True, torch.bfloat16, seed=n + k)
    x = _x(b, k, torch.bfloat16, seed=n)
    bias = _x(1, n, torch.bfloat16, seed=k)[0].contiguous()
    out = torch.full((b, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.linear(x, w4.pack(codes, scales, z), out, 64, zeros=True, bias=bias)
    _check_linear(x, codes, scales, z, bias, out)


def test_linear_strided_rows_and_untouched_neighbours():
    b, n, k = 6, 100, 320
    codes, scales, z = random_w4(n, k, 32, False, torch.float16, seed=1)
    wide = _x(b, k + 24, torch.float16, seed=2)
    x = wide[:, 8:8 + k]  # 16-byte aligned rows
    store = torch.full((b + 2, n + 30), 7.0, dtype=torch.float16, device="cuda")
    out = store[1:b + 1, 3:3 + n]
    w4.linear(x, w4.pack(codes, scales, z), out, 32)
    _check_linear(x, codes, scales, z, None, out)
    store[1:b + 1, 3:3 + n] = 7.0
    assert bool((store == 7.0).all())
    # one token's x seen by every row
    x1 = x[:1].expand(b, k)
    w4.linear(x1, w4.pack(codes, scales, z), out, 32)
    _check_linear(x1, codes, scales, z, None, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear_infinities_and_nan_stay_with_their_token(dtype):
    """NaN, and an infinity (infinity minus infinity), make their token NaN and no other."""
    b, n, k = 5, 48, 256
    codes, scales, z = random_w4(n, k, 128, False, dtype, seed=3)
    x = _x(b, k, dtype, seed=4)
    packed = w4.pack(codes, scales, z)
    clean = torch.empty(b, n, dtype=dtype, device="cuda")
    w4.linear(x, packed, clean, 128)
    x[1, 10] = float("nan")
    x[3, 77] = float("inf")
    out = torch.empty_like(clean)
    w4.linear(x, packed, out, 128)
    for t in (0, 2, 4):
        assert torch.equal(out[t], clean[t])
    assert bool(out[1].isnan().all()) and bool(out[3].isnan().all())


@pytest.mark.parametrize("dtype,lo,hi", [(torch.bfloat16, -50, 50), (torch.float16, -20, 8)])
def test_linear_activations_of_many_magnitudes(dtype, lo, hi):
    """Rows of |x| about 2^lo .. 2^hi, and one row that mixes them."""
    n, k = 40, 512
    codes, scales, z = random_w4(n, k, 64, True, dtype, seed=13)
    x = _x(17, k, torch.float32, seed=14)
    e = torch.linspace(lo, hi, 16, device="cuda").round()
    x[:16] *= torch.exp2(e)[:, None]
    x[16] *= torch.exp2(e.repeat(k // 16) - hi)
    x = x.to(dtype)
    out = torch.empty(17, n, dtype=dtype, device="cuda")
    w4.linear(x, w4.pack(codes, scales, z), out, 64, zeros=True)
    _check_linear(x, codes, scales, z, None, out)


def test_linear_same_bits_graph_streams_and_empty_batch():
    b, n, k = 9, 1536, 2048
    codes, scales, z = random_w4(n, k, 128, True, torch.bfloat16, seed=5)
    packed = w4.pack(codes, scales, z)
    x = _x(b, k, torch.bfloat16, seed=6)
    first = torch.empty(b, n, dtype=torch.bfloat16, device="cuda")
    w4.linear(x, packed, first, 128, zeros=True)
    torch.cuda.synchronize()
    # calls on two streams at once
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(first) for _ in range(8)]
    for i, o in enumerate(outs):
        w4.linear(x, packed, o, 128, zeros=True, stream=side[i % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    # captured, replayed on new inputs
    xg, og = x.clone(), torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.linear(xg, packed, og, 128, zeros=True)
    xg.copy_(_x(b, k, torch.bfloat16, seed=8))
    graph.replay()
    torch.cuda.synchronize()
    _check_linear(xg, codes, scales, z, None, og)
    w4.linear(x[:0], packed, first[:0], 128, zeros=True)  # nothing to do


@pytest.mark.parametrize("b,n,k", [(17, 256, 64), (64, 1536, 2048), (40, 300, 7168)])
def test_linear_many_tokens_two_streams_two_graphs_and_status(b, n, k):
    """Above 16 tokens: calls that overlap, on streams and in graphs, give the bits of one alone; no wait gives up."""
    codes, scales, z = random_w4(n, k, 64, True, torch.float16, seed=25)
    packed = w4.pack(codes, scales, z)
    x = _x(b, k, torch.float16, seed=26)
    first = torch.empty(b, n, dtype=torch.float16, device="cuda")
    w4.linear(x, packed, first, 64, zeros=True)
    assert w4.linear_status() == MOE_OK
    _check_linear(x, codes, scales, z, None, first)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.full_like(first, float("nan")) for _ in range(10)]
    for i, o in enumerate(outs):
        w4.linear(x, packed, o, 64, zeros=True, stream=side[i % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
        o.fill_(float("nan"))
    graphs = []
    for i in range(2):  # calls one behind the other, each started while the one before it ends
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            for o in outs[5 * i:5 * i + 5]:
                w4.linear(x, packed, o, 64, zeros=True)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, side):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    assert w4.linear_status() == MOE_OK


def test_linear_many_tokens_rows_apart_at_odd_addresses():
    """Above 16 tokens: rows that start at any 16-bit element; what lies between them stays."""
    b, n, k = 33, 261, 448
    codes, scales, z = random_w4(n, k, 32, False, torch.bfloat16, seed=27)
    packed = w4.pack(codes, scales, z)
    x = _x(b, k, torch.bfloat16, seed=28)
    bias = _x(1, n, torch.bfloat16, seed=29)[0]
    for pitch, off in ((n, 0), (n + 3, 1), (n + 7, 4), (n + 7, 2)):  # the third: rows on 8-byte boundaries
        buf = torch.full((b * pitch + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[off:off + b * pitch].view(b, pitch)[:, :n]
        w4.linear(x, packed, out, 32, bias=bias)
        torch.cuda.synchronize()
        _check_linear(x, codes, scales, z, bias, out.contiguous())
        out.fill_(7.0)
        assert bool((buf == 7.0).all())


# ------------------------------------------------------------------ the block
class W4Block:
    """Plain and packed weights of one block."""

    def __init__(self, shape, group, zeros, seed, bias=None):
        self.s, self.group, self.zeros = shape, group, zeros
        H, I, Is, E = shape.hidden, shape.inter, shape.shared_inter, shape.n_experts
        self.router_w = synth._normal_bf16((H, E), synth.WEIGHT_STD, synth.seed_for(seed, "router_w"), "cuda")
        self.router_bias = bias
        mk = lambda n, k, i, lead=(): random_w4(n, k, group, zeros, torch.bfloat16, seed * 10 + i, lead=lead)  # noqa: E731
        self.w13, self.w2 = mk(2 * I, H, 1, (E,)), mk(H, I, 2, (E,))
        self.s13, self.s2 = (mk(2 * Is, H, 3), mk(H, Is, 4)) if shape.n_shared else (None, None)
        self.packed = [None if w is None else w4.pack(*w) for w in (self.w13, self.w2, self.s13, self.s2)]

    def handle(self, max_batch, **kw):
        s = self.s
        return MoEDecode(s.hidden, s.n_experts, s.top_k, s.inter, s.shared_inter, n_shared=s.n_shared, max_batch=max_batch,
                         router_bias=self.router_bias, w4=True, **kw)

    def forward(self, blk, x, out=None, stream=None):
        b, k = x.shape[0], self.s.top_k
        out = torch.full_like(x, float("nan")) if out is None else out
        ids = torch.full((b, k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((b, k), float("nan"), dtype=torch.float32, device="cuda")
        blk.forward_w4(x, self.router_w, *self.packed, out, ids, w, self.group, zeros=self.zeros, stream=stream)
        return out, ids, w

    def expected(self, x, ids, w):
        """(sum of the experts' outputs, its tolerance) in 64 bits, for the routing given."""
        xd = x.double()
        y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
        H, I = self.s.hidden, self.s.inter

        def add(rows, weight, w13, w2, inter):
            xr = xd[rows]
            # an expert with more than 8 tokens takes weights rounded to bf16
            a13, a2 = _weights(*w13, len(xr), exact=8), _weights(*w2, len(xr), exact=8)
            h = xr @ a13.T
            dh = _fp32_error(xr, *w13, a13, exact=8)
            g, u, dg, du = h[:, :inter], h[:, inter:], dh[:, :inter], dh[:, inter:]
            sig = torch.sigmoid(g)
            a = g * sig * u
            # |silu'| <= 1.1; silu and the product in fp32: 2^-20 covers expf, the division and two products
            da = 1.1 * dg * (u.abs() + du) + (g * sig).abs() * du + 2.0 ** -20 * a.abs()
            da = da + U[torch.bfloat16] * (a.abs() + da)  # stored in bf16
            y[rows] += weight * (a @ a2.T)
            most = a.abs() + da
            tol[rows] += weight * (da @ a2.abs().T + _fp32_error(most, *w2, a2, exact=8) + 2.0 ** -23 * product_magnitude(most, *w2))

        for e in torch.unique(ids).tolist():
            t, j = (ids == e).nonzero(as_tuple=True)
            pick = lambda ws: tuple(None if v is None else v[e] for v in ws)  # noqa: E731
            add(t, w[t, j].double()[:, None], pick(self.w13), pick(self.w2), I)
        if self.s.n_shared:
            add(torch.arange(len(x), device="cuda"), 1.0, self.s13, self.s2, self.s.shared_inter)
        return y, tol + (self.s.top_k + 2) * 2.0 ** -24 * (y.abs() + tol)

    def check(self, x, out, ids, w):
        bias = None if self.router_bias is None else self.router_bias.cpu().numpy()
        _, o_ids, o_w = oracle.router(synth.bf16_bits(x), synth.bf16_bits(self.router_w), self.s.top_k, bias)
        np.testing.assert_array_equal(ids.cpu().numpy(), o_ids)
        assert np.max(np.abs(w.cpu().numpy().astype(np.float64) - o_w)) <= W_ATOL
        y, tol = self.expected(x, ids, w)
        if out.dtype is torch.float32:  # partial sum
            assert_within(out, y, tol + 2.0 ** -24 * y.abs())
        else:
            want = x.double() + y
            assert_within(out, want, tol + U[torch.bfloat16] * (want.abs() + tol) + 2.0 ** -24 * x.double().abs())


TINY_W4 = synth.BlockShape(hidden=256, n_experts=16, top_k=2, inter=128, shared_inter=192)
NO_SHARED = synth.BlockShape(hidden=192, n_experts=8, top_k=8, inter=64, shared_inter=0, n_shared=0)
MANY = synth.BlockShape(hidden=1024, n_experts=40, top_k=3, inter=320, shared_inter=64)


@pytest.mark.parametrize("b", [1, 2, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("shape,group,zeros", [(TINY_W4, 64, False), (TINY_W4, 32, True), (NO_SHARED, 32, False),
                                               (MANY, 64, True)])
def test_block_every_element(shape, group, zeros, b):
    m = W4Block(shape, group, zeros, seed=20 + b)
    blk = m.handle(64)
    try:
        x = margin_x(b, shape.hidden, m, shape.top_k, seed=400 + b)
        out, ids, w = m.forward(blk, x)
        torch.cuda.synchronize()
        m.check(x, out, ids, w)
        assert blk.status() == MOE_OK
        assert blk.stats()["last_kernels"] == (4 if b <= 8 else 7)
    finally:
        blk.close()


def test_block_one_expert_takes_every_token():
    """A router bias sends all 64 tokens to expert 5 first: two units of one expert, the others' few tokens beside them."""
    bias = torch.zeros(16, device="cuda")
    bias[5] = 50.0
    m = W4Block(TINY_W4, 64, True, seed=31, bias=bias)
    blk = m.handle(64)
    try:
        x = margin_x(64, TINY_W4.hidden, m, 2, seed=431)
        out, ids, w = m.forward(blk, x)
        torch.cuda.synchronize()
        assert bool((ids[:, 0] == 5).all())
        m.check(x, out, ids, w)
    finally:
        blk.close()


def test_block_full_size_experts():
    """16 experts of the full size (hidden 7168, inter 2048), groups of 128, batch 1, 8 and 40."""
    m = W4Block(synth.PROF, 128, False, seed=40)
    blk = m.handle(40)
    try:
        for b in (1, 8, 40):
            x = margin_x(b, synth.PROF.hidden, m, synth.PROF.top_k, seed=440 + b)
            out, ids, w = m.forward(blk, x)
            torch.cuda.synchronize()
            m.check(x, out, ids, w)
    finally:
        blk.close()
        del m
        torch.cuda.empty_cache()


def test_block_short_wait_limit_is_reported_and_the_handle_recovers():
    """One probe for each wait: a forward either ends in time and is right, or says that it did not."""
    m = W4Block(synth.PROF, 128, False, seed=41)
    blk = m.handle(40)
    try:
        x = margin_x(40, synth.PROF.hidden, m, synth.PROF.top_k, seed=445)
        blk.set_wait_limit(1)
        out, ids, w = m.forward(blk, x)
        torch.cuda.synchronize()
        st = blk.status()
        assert st in (MOE_OK, MOE_ERR_DEVICE_TIMEOUT)
        if st == MOE_OK:
            m.check(x, out, ids, w)
        blk.set_wait_limit(0)
        out, ids, w = m.forward(blk, x)
        torch.cuda.synchronize()
        assert blk.status() == MOE_OK
        m.check(x, out, ids, w)
    finally:
        blk.close()
        del m
        torch.cuda.empty_cache()


def test_block_partial_sums_of_two_ranks():
    """The tensor-parallel form: each rank's slice of every expert, the fp32 sums added by reduce_residual."""
    shape, b = synth.BlockShape(256, 16, 2, 128, 128), 13
    m = W4Block(shape, 64, True, seed=50)
    x = margin_x(b, 256, m, 2, seed=450)
    c, parts = 64, []
    half = synth.BlockShape(256, 16, 2, c, c)
    for r in range(2):
        rank = W4Block.__new__(W4Block)
        rank.s, rank.group, rank.zeros, rank.router_w, rank.router_bias = half, 64, True, m.router_w, None
        rows = torch.cat([torch.arange(r * c, (r + 1) * c), 128 + torch.arange(r * c, (r + 1) * c)]).cuda()
        up = lambda ws: tuple(v[..., rows, :].contiguous() for v in ws)  # noqa: E731
        # 64 inputs of the down projection: 32 bytes of codes and one group
        dn = lambda ws: tuple(v.unflatten(-1, (2, -1))[..., r, :].contiguous() for v in ws)  # noqa: E731
        rank.w13, rank.w2, rank.s13, rank.s2 = up(m.w13), dn(m.w2), up(m.s13), dn(m.s2)
        rank.packed = [w4.pack(*ws) for ws in (rank.w13, rank.w2, rank.s13, rank.s2)]
        blk = rank.handle(16, partial=True)
        try:
            out, ids, w = rank.forward(blk, x, out=torch.full((b, 256), float("nan"), device="cuda"))
            torch.cuda.synchronize()
            rank.check(x, out, ids, w)
            parts.append(out)
        finally:
            blk.close()
    out = torch.empty_like(x)
    reduce_residual(parts, x, out)
    torch.cuda.synchronize()
    m.check(x, out, ids, w)


def test_block_graph_replay_two_handles_and_smaller_batches():
    m = W4Block(TINY_W4, 64, False, seed=60)
    a, b2 = m.handle(16), m.handle(16)
    try:
        x = margin_x(12, 256, m, 2, seed=460)
        xg, og = x.clone(), torch.empty_like(x)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m.forward(a, xg, out=og, stream=s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, ids, w = m.forward(a, xg, out=og)
        xg.copy_(margin_x(12, 256, m, 2, seed=461))
        # the other handle's eager calls run beside the replay
        with torch.cuda.stream(s):
            results = [(xb, *m.forward(b2, xb, stream=s)) for xb in (x[:1], x[:7], x)]
        graph.replay()
        torch.cuda.synchronize()
        m.check(xg, og, ids, w)
        for xb, out, i, ww in results:
            m.check(xb, out, i, ww)
        # the eager call of a handle that was captured, back to back with replays
        graph.replay()
        out, i2, w2 = m.forward(a, x[:3])
        torch.cuda.synchronize()
        m.check(x[:3], out, i2, w2)
        empty = m.forward(a, x[:0])
        assert empty[0].shape[0] == 0
    finally:
        a.close()
        b2.close()


def test_entry_points_reject_the_other_handles_and_groups():
    m = W4Block(TINY_W4, 64, False, seed=70)
    h4 = m.handle(4)
    h16 = MoEDecode(256, 16, 2, 128, 192, max_batch=4)
    try:
        x = _x(2, 256, torch.bfloat16, seed=1)
        out, ids, w = torch.empty_like(x), torch.empty(2, 2, dtype=torch.int32, device="cuda"), torch.empty(2, 2, device="cuda")
        with pytest.raises(MoEDecodeError):
            h16.forward_w4(x, m.router_w, *m.packed, out, ids, w, 64)
        with pytest.raises(MoEDecodeError):
            h4.forward(x, m.router_w, m.packed[0], m.packed[1], m.packed[2], m.packed[3], out, ids, w)
        with pytest.raises(ValueError):  # packed in groups of 64
            h4.forward_w4(x, m.router_w, *m.packed, out, ids, w, 32)
        with pytest.raises(MoEDecodeError):
            h4.forward_w4(x, m.router_w, *m.packed, out, ids, w, 48)
        with pytest.raises(MoEDecodeError):
            h4.forward_w4(x, m.router_w, *m.packed, x, ids, w, 64)
    finally:
        h4.close()
        h16.close()


def test_router_layer_and_counts_together():
    """The pieces beside each other: the router alone, a dense 4-bit layer on its tokens, the block on the result."""
    from moe_decode_block_b200 import balance
    m = W4Block(TINY_W4, 64, False, seed=80)
    codes, scales, z = random_w4(256, 256, 64, False, torch.bfloat16, seed=81)
    packed = w4.pack(codes, scales, z)
    blk = m.handle(8)
    try:
        x0 = _x(8, 256, torch.bfloat16, seed=82)
        x = torch.empty_like(x0)
        w4.linear(x0, packed, x, 64)
        out, ids, w = m.forward(blk, x)
        ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
        router_topk_noalloc(x, m.router_w, ids2, w2, 2)
        loss, counts = torch.empty(1, device="cuda"), torch.empty(17, dtype=torch.int32, device="cuda")
        balance.balance_loss(x.float() @ m.router_w.float(), ids, loss, counts)
        torch.cuda.synchronize()
        _check_linear(x0, codes, scales, z, None, x)
        assert torch.equal(counts[:16].cpu(), torch.bincount(ids.reshape(-1).cpu(), minlength=16).int()) and int(counts[16]) == 8
        if torch.equal(ids, ids2):  # (a near tie may fall either way between two runs of the router)
            y, tol = m.expected(x, ids, w)
            want = x.double() + y
            assert_within(out, want, tol + U[torch.bfloat16] * (want.abs() + tol) + 2.0 ** -24 * x.double().abs())
    finally:
        blk.close()
