"""Products with 4-bit weights (a scale, and optionally a zero point, per group
of inputs): argument marshalling of moe_w4_pack and moe_w4_linear.

    packed = w4.pack(codes, scales, zeros)          # once, at load time
    w4.linear(x, packed, out, group=128, zeros=True)

The block's experts take the same packed matrices: MoEDecode(..., w4=True)
and its forward_w4.
"""
from __future__ import annotations

from contextlib import nullcontext

from . import (MOE_DTYPE_BF16, MOE_DTYPE_FP16, _check, _current_device, _current_stream, _stream_handle,
               load_library)

MAX_BATCH = 64       # of linear()
MAX_SIZE = 1 << 20   # above MOE_W4_MAX_IN and MOE_W4_MAX_OUT
_CODES = {}


def _codes() -> dict:
    """torch dtype -> MOE_DTYPE_* of the products."""
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_FP16})
    return _CODES


def _dtype_code(t) -> int:
    code = _codes().get(t.dtype)
    if code is None:
        raise ValueError(f"expected bfloat16 or float16, got {t.dtype}")
    return code


def _on(device):
    """Make `device` current where it is not (the library launches on the
    current device)."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {device}")
    return nullcontext() if device.index == _current_device() else torch.cuda.device(device)


def packed_bytes(out_features: int, in_features: int, group: int, zeros: bool = False) -> int:
    """Bytes of a packed [out_features, in_features] matrix."""
    n = 0
    if 0 < out_features <= MAX_SIZE and 0 < in_features <= MAX_SIZE and 0 < group <= 128:  # (32 bits)
        n = load_library().moe_w4_packed_bytes(int(out_features), int(in_features), int(group), int(bool(zeros)))
    if n == 0:
        raise ValueError(f"no packed form for [{out_features}, {in_features}] in groups of {group}")
    return n


def pack(codes, scales, zeros=None, out=None, stream=None):
    """Lay matrices out for the products: codes [..., N, K / 2] uint8 (input
    2 j in the low half of byte j), scales [..., N, K / group] bfloat16 or
    float16, zeros [..., N, K / group] uint8 or None -> uint8
    [..., ceil(N / 16), panel bytes].  Leading axes (experts) are packed one
    matrix at a time.  Scales are kept as they are (linear() says which range
    its products hold); zero points 0..15, the low four bits count."""
    import torch
    lib = load_library()
    if codes.dtype is not torch.uint8 or codes.dim() < 2 or not codes.is_cuda:
        raise ValueError("codes: expected a uint8 [..., N, K / 2] tensor on the GPU")
    n, k = codes.shape[-2], codes.shape[-1] * 2
    if scales.shape[:-1] != codes.shape[:-1] or scales.shape[-1] < 1 or k % scales.shape[-1]:
        raise ValueError(f"scales {tuple(scales.shape)} do not fit codes {tuple(codes.shape)}")
    group = k // scales.shape[-1]
    if zeros is not None and (zeros.dtype is not torch.uint8 or zeros.shape != scales.shape):
        raise ValueError("zeros: expected uint8 of the scales' shape")
    for name, t in (("codes", codes), ("scales", scales), ("zeros", zeros)):
        if t is not None and (not t.is_contiguous() or t.device != codes.device):
            raise ValueError(f"{name}: expected a contiguous tensor on {codes.device}")
    code = _dtype_code(scales)
    one = packed_bytes(n, k, group, zeros is not None)
    shape = (*codes.shape[:-2], -(-n // 16), one // -(-n // 16))
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=codes.device)
    elif out.shape != shape or out.dtype is not torch.uint8 or not out.is_contiguous() or out.device != codes.device:
        raise ValueError(f"out: expected a contiguous uint8 {shape} tensor on {codes.device}")
    with _on(codes.device):
        sm = _stream_handle(stream) if stream is not None else _current_stream(codes.get_device())
        for m in range(codes[..., 0, 0].numel()):
            z = None if zeros is None else zeros.data_ptr() + m * n * (k // group)
            rc = lib.moe_w4_pack(codes.data_ptr() + m * n * (k // 2), scales.data_ptr() + m * n * (k // group) * 2, z,
                                 out.data_ptr() + m * one, n, k, group, code, sm)
            _check(rc, "moe_w4_pack")
    return out


def _refuse_linear(x, packed, out, group, zeros, bias):
    """Say what is wrong with linear()'s arguments."""
    if x.dim() != 2 or out.dim() != 2 or out.shape[0] != x.shape[0]:
        raise ValueError(f"x {tuple(x.shape)} and out {tuple(out.shape)}: expected [B, K] and [B, N]")
    _dtype_code(x)
    for name, t in (("x", x), ("packed", packed), ("out", out), ("bias", bias)):
        if t is not None and (t.device.type != "cuda" or t.device != x.device):
            raise ValueError(f"{name}: on {t.device}, expected one GPU (x is on {x.device})")
    if out.dtype != x.dtype:
        raise ValueError(f"out: {out.dtype}, x is {x.dtype}")
    if x.stride(1) != 1 or out.stride(1) != 1:
        raise ValueError("x and out: elements of a row must be contiguous")
    N = out.shape[1]
    if bias is not None and (bias.dtype != x.dtype or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError(f"bias: expected {N} contiguous elements of {x.dtype}")
    raise ValueError(f"packed: expected {packed_bytes(N, x.shape[1], group, zeros)} contiguous bytes (uint8), got "
                     f"{packed.numel()} of {packed.dtype}")


def linear(x, packed, out, group: int, zeros: bool = False, bias=None, stream=None):
    """out[b, n] = bias[n] + sum_k x[b, k] W[n, k]: x [B, K], out [B, N] (rows
    may be strided, elements not), packed the [N, K] matrix from pack(), bias
    [N] or None; all of one 16-bit type; no row of out on a row of x.  `stream`
    belongs to x's device.

    Sums in fp32.  Up to 16 tokens no weight is rounded; in bfloat16 |x| is
    held from 2^-57 to 2^63 and a sum to within 2^-72, if not better, and an
    infinite activation gives NaN.  Above 16
    each weight s (q - z) is rounded once to x's type, which has to hold it;
    scales in bfloat16 are then below 2^27 (2^122 with zero points)."""
    B, K = x.shape
    Bo, N = out.shape
    sx, so = x.stride(), out.stride()
    dtype, dev = x.dtype, x.get_device()
    code = _codes().get(dtype)
    # a packed matrix's size; a shape that the library refuses is its to refuse
    need = (N + 15) // 16 * (K // 64 * 512 + (K // group * (64 if zeros else 32) if group > 0 else 0))
    if (code is None or dev < 0 or Bo != B or sx[1] != 1 or so[1] != 1 or out.dtype is not dtype
            or out.get_device() != dev or packed.get_device() != dev or packed.numel() != need
            or packed.element_size() != 1 or not packed.is_contiguous()
            or (bias is not None and (bias.dtype is not dtype or bias.numel() != N or bias.get_device() != dev
                                      or not bias.is_contiguous()))):
        _refuse_linear(x, packed, out, group, zeros, bias)
    call = load_library().moe_w4_linear
    # (numbers beyond 32 bits must not come around to small ones: the library refuses these)
    if B > MAX_BATCH or K > MAX_SIZE or N > MAX_SIZE or not 0 < group <= 128:
        B, K, N, group = MAX_BATCH + 1, 64, 1, 0
    args = (x.data_ptr(), packed.data_ptr(), None if bias is None else bias.data_ptr(), out.data_ptr(), B, K, N, group,
            1 if zeros else 0, sx[0], so[0], code)
    if dev == _current_device():
        rc = call(*args, _current_stream(dev) if stream is None else _stream_handle(stream))
    else:
        with _on(x.device):
            rc = call(*args, _current_stream(dev) if stream is None else _stream_handle(stream))
    if rc:
        _check(rc, "moe_w4_linear")
    return out


def linear_status(stream=None) -> int:
    """Synchronise `stream` and return the device status of the linear() calls
    on the current device (MOE_OK or an MOE_ERR_* code); clears it."""
    dev = _current_device()
    return load_library().moe_w4_linear_status(_current_stream(dev) if stream is None else _stream_handle(stream))


def set_wait_limit(probes: int = 0):
    """Bound of the device-side waits of later linear() calls of this process
    in probes of up to 20 us (0: the default, 2/3 s)."""
    _check(load_library().moe_w4_linear_set_wait_limit(int(probes)), "moe_w4_linear_set_wait_limit")


def test_hold(launches: int):
    """Testing only: the first CTA of each of the next `launches` tcgen05
    kernels never hands over its first step, so its waits run out."""
    _check(load_library().moe_w4_test_hold(int(launches)), "moe_w4_test_hold")


test_hold.__test__ = False  # (not a test itself, where it is imported into one)
