"""Plain 64-bit forms of the 4-bit weight products and of the router's balance
loss, from their definitions (no code of the package)."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}  # one subnormal step


def random_w4(n, k, group, zeros, dtype, seed, device="cuda", lead=()):
    """Plain codes [*, n, k / 2], scales [*, n, k / group] and zero points (or None) of random matrices."""
    g = torch.Generator(device=device).manual_seed(seed)
    codes = torch.randint(0, 256, (*lead, n, k // 2), dtype=torch.uint8, device=device, generator=g)
    scales = ((torch.rand(*lead, n, k // group, device=device, generator=g) + 0.5) * 0.005).to(dtype)
    z = torch.randint(0, 16, (*lead, n, k // group), dtype=torch.uint8, device=device, generator=g) if zeros else None
    return codes, scales, z


def dequant64(codes, scales, zeros=None):
    """float64 [..., n, k] of plain codes."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
    group = q.shape[-1] // scales.shape[-1]
    s = scales.double().repeat_interleave(group, dim=-1)
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, dim=-1)
    return (q - z) * s


def product_tolerance(k, dtype=torch.bfloat16):
    """Relative to sum s (q + z) |x| (product_magnitude): s sum q x and s z sum x are taken apart.  A tensor-core instruction on
    subnormal codes is off by under 2^-24 of its sum of |q x| in bf16 and 2^-20 in fp16 (measured, worst of 25,600: 4.9e-8 and
    5.8e-7; four times that allowed, in fp16 for the chain as a whole, whose
    errors are relative to its largest product); eight are chained to a group, two more roundings scale it; then the adds of
    K / 64 tiles at most, 8 warps, 8 CTAs, bias."""
    return 10 * (2.0 ** -18 / 8 if dtype is torch.float16 else 2.0 ** -22) + (k / 64 + 8 + 8 + 1) * 2.0 ** -24


def product_magnitude(x, codes, scales, zeros=None):
    """sum s (q + z) |x| in 64 bits."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
    group = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, dim=-1)
    return x.double().abs() @ ((q + z) * scales.double().repeat_interleave(group, dim=-1)).transpose(-1, -2)


def assert_within(got, want, tol, what=""):
    """|got - want| <= tol element by element (64 bits)."""
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).nan_to_num(float('inf')).max()):.3g} "
                                 f"over its tolerance, first at {bad.nonzero()[0].tolist()}")


def balance64(logits, ids, mask=None, bias=None, coef=1.0, grad=1.0):
    """(loss, counts [E + 1], dlogits, spread): spread[t] = sum_e p_te |c_e - S_t| scales the tolerance."""
    t, e = logits.shape
    k = ids.shape[1]
    z = logits.double() + (0.0 if bias is None else bias.double())
    live = torch.ones(t, dtype=torch.bool, device=z.device) if mask is None else mask.bool()
    chosen = ids[live].reshape(-1).long()
    chosen = chosen[(chosen >= 0) & (chosen < e)]
    c = torch.bincount(chosen, minlength=e).double()
    n = int(live.sum())
    f = coef * e / (k * n * n) if n else 0.0
    p = torch.softmax(z, dim=1) if t else z
    p = torch.where((z == -torch.inf).all(dim=1, keepdim=True) | ~live[:, None], torch.zeros_like(p), p)
    s = (p * c).sum(dim=1, keepdim=True)
    d = grad * f * p * (c - s)
    counts = torch.cat([c.long(), torch.tensor([n], device=z.device)]).to(torch.int32)
    return f * s.sum(), counts, d, (p * (c - s).abs()).sum(dim=1, keepdim=True), p, c, f
