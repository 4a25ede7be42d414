"""4-bit products over the range of scales and activations, on each of the dense layer's kernels (up to 8, up to 16 and
more tokens), and the distance of the rounded weights from the definition.  Tolerances as in test_gpu_w4.py, and where
weights are rounded, half a step of each."""
import pytest
import torch

from moe_decode_block_b200 import MoEDecodeError, w4
from gpu_helpers import margin_x
from test_gpu_w4 import MANY, TINY_W4, W4Block, _check_linear, _x
from w4_reference import TINY, U, assert_within, dequant64, product_magnitude, product_tolerance, random_w4

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


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,lo,hi", [(torch.bfloat16, -57, 62), (torch.float16, -24, 11)])
@pytest.mark.parametrize("b", BATCHES)
def test_activations_of_many_magnitudes(b, dtype, lo, hi, zeros):
    """Tokens whose |x| are 2^lo .. 2^hi (bf16: the ends of what the small kernels hold; fp16: from the smallest subnormal),
    and one that mixes them.  A mix whose large part cancels in a group would show there."""
    n, k = 72, 512
    codes, scales, z = random_w4(n, k, 64, zeros, dtype, seed=40 + b)
    g = torch.Generator(device="cuda").manual_seed(b)
    x = (1 + 0.99 * torch.rand(b, k, device="cuda", generator=g)) * torch.where(torch.rand(b, k, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    e = torch.linspace(lo, hi, max(2, b - 1), device="cuda").round()
    x[:b - 1] *= torch.exp2(e[:b - 1])[:, None]
    x[b - 1] *= torch.exp2(torch.linspace(lo, hi, k, device="cuda").round())
    x = x.to(dtype)
    out = torch.full((b, n), float("nan"), dtype=dtype, device="cuda")
    w4.linear(x, w4.pack(codes, scales, z), out, 64, zeros=zeros)
    assert bool(out.isfinite().all())
    _check_linear(x, codes, scales, z, None, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b", [1, 5, 8, 13, 16, 33, 64])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_values_that_are_not_finite_stay_with_their_token(b, dtype, bad):
    """In the first token (whose row also stands for those that do not exist), in one inside and in the last."""
    n, k = 48, 256
    codes, scales, z = random_w4(n, k, 128, False, dtype, seed=3)
    packed = w4.pack(codes, scales, z)
    x = _x(b, k, dtype, seed=4)
    clean = torch.empty(b, n, dtype=dtype, device="cuda")
    w4.linear(x, packed, clean, 128)
    for rows in ([0], [b - 1], [0, b // 2]):
        xb = x.clone()
        for r in rows:
            xb[r, (17 * r + 10) % k] = float(bad)
        out = torch.zeros_like(clean)
        w4.linear(xb, packed, out, 128)
        hit = torch.zeros(b, dtype=torch.bool, device="cuda")
        hit[rows] = True
        assert not bool(out[hit].isfinite().any())
        if bad == "nan":
            assert bool(out[hit].isnan().all())
        assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("b", [17, 32, 64])
def test_many_tokens_from_the_definition(b, group, zeros, dtype):
    """Above 16 tokens, against the weights as defined: half a step of each weight besides the sums' own error, and the mean
    square a third of what independent roundings at half a step would give."""
    n, k = 500, 2048
    codes, scales, z = random_w4(n, k, group, zeros, dtype, seed=50 + b)
    x = _x(b, k, dtype, seed=b)
    out = torch.full((b, n), float("nan"), dtype=dtype, device="cuda")
    w4.linear(x, w4.pack(codes, scales, z), out, group, zeros=zeros)
    w = dequant64(codes, scales, z)
    y = x.double() @ w.T
    mag = x.double().abs() @ w.abs().T
    # weights: U each; sums: one chain of K / 16 instructions (each under 2^-23 of the magnitudes) and 8 CTAs
    off = U[dtype] * mag + (k / 16 + 10) * 2.0 ** -23 * (1 + U[dtype]) * mag
    assert_within(out, y, off + U[dtype] * (y.abs() + off) + TINY[dtype])
    # the roundings of the weights and of the outputs are each uniform within half a step at most, so their variance is
    # at most a third of its square; 1.2 covers the spread of the sum over 8,500 or more outputs
    var = (U[dtype] ** 2 / 3) * (x.double() ** 2 @ (w ** 2).T + y ** 2)
    assert float(((out.double() - y) ** 2).mean()) <= 1.2 * float(var.mean())


class _Defined(W4Block):
    """expected() from the weights as defined; experts of more than 8 tokens may have each weight off by half a step."""

    def expected(self, x, ids, w):
        xd = x.double()
        y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
        half = U[torch.bfloat16]

        def product(v, dv, ws):
            """(v W^T, what it may be off by) for inputs v that are off by dv."""
            a, most = dequant64(*ws), v.abs() + dv
            mag = most @ a.abs().T
            off = dv @ a.abs().T + product_tolerance(v.shape[1]) * product_magnitude(most, *ws)
            if len(v) > 8:
                off = dv @ a.abs().T + half * mag + (v.shape[1] / 16 + 10) * 2.0 ** -23 * (1 + half) * mag
            return v @ a.T, off

        def add(rows, weight, w13, w2, inter):
            h, dh = product(xd[rows], torch.zeros_like(xd[rows]), w13)
            g, u, dg, du = h[:, :inter], h[:, inter:], dh[:, :inter], dh[:, inter:]
            sig = torch.sigmoid(g)
            a = g * sig * u
            da = 1.1 * dg * (u.abs() + du) + (g * sig).abs() * du + 2.0 ** -20 * a.abs()
            da = da + half * (a.abs() + da)
            v, dv = product(a, da, w2)
            y[rows] += weight * v
            tol[rows] += weight * (dv + 2.0 ** -23 * product_magnitude(a.abs() + da, *w2))

        for e in torch.unique(ids).tolist():
            t, j = (ids == e).nonzero(as_tuple=True)
            pick = lambda ws: tuple(None if v is None else v[e] for v in ws)  # noqa: E731
            add(t, w[t, j].double()[:, None], pick(self.w13), pick(self.w2), self.s.inter)
        if self.s.n_shared:
            add(torch.arange(len(x), device="cuda"), 1.0, self.s13, self.s2, self.s.shared_inter)
        return y, tol + (self.s.top_k + 2) * 2.0 ** -24 * (y.abs() + tol)


@pytest.mark.parametrize("shape,group,zeros", [(TINY_W4, 64, False), (TINY_W4, 32, True), (MANY, 64, True)])
@pytest.mark.parametrize("b", [3, 9, 33, 64])
def test_block_from_the_definition(b, shape, group, zeros):
    m = _Defined(shape, group, zeros, seed=70 + b)
    blk = m.handle(64)
    try:
        x = margin_x(b, shape.hidden, m, shape.top_k, seed=700 + b)
        out, ids, w = m.forward(blk, x)
        torch.cuda.synchronize()
        m.check(x, out, ids, w)
    finally:
        blk.close()


def test_a_number_of_tokens_beyond_32_bits_is_refused():
    codes, scales, _ = random_w4(1, 64, 64, False, torch.bfloat16, seed=1)
    packed, row = w4.pack(codes, scales), _x(1, 64, torch.bfloat16, seed=1)
    out = torch.empty(2 ** 32 + 1, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(MoEDecodeError):
        w4.linear(row.expand(2 ** 32 + 1, 64), packed, out, 64)
    del out
    torch.cuda.empty_cache()
