"""The router's balance loss, its gradient and the choices per expert:
argument marshalling of moe_balance_loss.

    balance.balance_loss(logits, topk_ids, loss, counts)                     # serving: the load
    balance.balance_loss(logits, topk_ids, loss, counts, dlogits=dlogits)    # training: in the same pass
"""
from __future__ import annotations

from . import (MOE_DTYPE_BF16, MOE_DTYPE_FP16, MOE_DTYPE_FP32, _check, _current_device, _current_stream,
               _stream_handle, load_library)
from .w4 import _on

ONE_LAUNCH = 512  # tokens up to which no workspace is needed
MAX_TOKENS = 1 << 24
_TYPES = {}
_WORKSPACE = {}


def _types() -> dict:
    """torch dtype -> MOE_DTYPE_* of the logits, and the types of the other tensors."""
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: MOE_DTYPE_FP32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_FP16,
                       "i32": torch.int32, "f32": torch.float32})
    return _TYPES


def _workspace(n_experts: int) -> int:
    """workspace_bytes, or 1 for numbers of experts that the library refuses."""
    n = _WORKSPACE.get(n_experts)
    if n is None:
        n = _WORKSPACE[n_experts] = max(1, load_library().moe_balance_workspace_bytes(n_experts))
    return n


def workspace_bytes(n_experts: int) -> int:
    n = load_library().moe_balance_workspace_bytes(int(n_experts))
    if n == 0:
        raise ValueError(f"no balance loss for {n_experts} experts")
    return n


def balance_loss(logits, topk_ids, loss, counts, token_mask=None, router_bias=None, coef: float = 1.0, dlogits=None,
                 grad_loss=None, workspace=None, stream=None):
    """loss [1] float32 and counts [E + 1] int32 (the choices of each expert,
    then the live tokens) of logits [T, E] (float32, bfloat16 or float16; rows
    may be strided) and topk_ids [T, k] int32; with dlogits [T, E] also the
    gradient, times grad_loss [1].  token_mask [T] bool or uint8: 0 is a padded
    token.  workspace (above ONE_LAUNCH tokens): a uint8 tensor of
    workspace_bytes(E), by default a new one (torch's allocator ties it to the
    current stream, so pass one when `stream` is another).  Autograd does not
    see the call: dlogits is the gradient."""
    T, E = logits.shape
    Ti, k = topk_ids.shape
    dev = logits.get_device()
    types = _types()
    code = types.get(logits.dtype)
    zs = logits.stride()
    ds = (0, 1) if dlogits is None else dlogits.stride()
    i32, f32 = types["i32"], types["f32"]
    if (code is None or dev < 0 or Ti != T or (zs[1] != 1 and T) or (ds[1] != 1 and T) or topk_ids.dtype is not i32
            or counts.dtype is not i32 or loss.dtype is not f32 or loss.numel() != 1 or counts.numel() != E + 1
            or not topk_ids.is_contiguous() or not counts.is_contiguous() or topk_ids.get_device() != dev
            or loss.get_device() != dev or counts.get_device() != dev or token_mask is not None
            or (router_bias is not None and (router_bias.dtype is not f32 or router_bias.numel() != E
                                             or not router_bias.is_contiguous() or router_bias.get_device() != dev))
            or (dlogits is not None and (dlogits.dtype is not logits.dtype or dlogits.shape != logits.shape
                                         or dlogits.get_device() != dev))
            or (grad_loss is not None and (grad_loss.dtype is not f32 or grad_loss.numel() != 1
                                           or grad_loss.get_device() != dev))
            or workspace is not None):
        _look_closer(logits, topk_ids, loss, counts, token_mask, router_bias, dlogits, grad_loss, workspace)
    if workspace is None and T > ONE_LAUNCH:
        if stream is not None and _stream_handle(stream) != _current_stream(dev):
            raise ValueError("workspace: needed with a stream that is not the current one")
        import torch
        workspace = torch.empty(_workspace(E), dtype=torch.uint8, device=logits.device)
    call = load_library().moe_balance_loss
    args = (logits.data_ptr(), None if router_bias is None else router_bias.data_ptr(), topk_ids.data_ptr(),
            None if token_mask is None else token_mask.data_ptr(), loss.data_ptr(), counts.data_ptr(),
            None if dlogits is None else dlogits.data_ptr(), None if grad_loss is None else grad_loss.data_ptr(),
            min(T, MAX_TOKENS + 1), E, k, zs[0], ds[0], coef, code, None if workspace is None else workspace.data_ptr())  # (T: 32 bits there)
    if dev == _current_device():
        rc = call(*args, _current_stream(dev) if stream is None else _stream_handle(stream))
    else:
        with _on(logits.device):
            rc = call(*args, _current_stream(dev) if stream is None else _stream_handle(stream))
    if rc:
        _check(rc, "moe_balance_loss")
    return loss


def _look_closer(logits, topk_ids, loss, counts, token_mask, router_bias, dlogits, grad_loss, workspace):
    """Raise ValueError for a tensor that does not fit the call."""
    import torch
    T, E = logits.shape
    if _types().get(logits.dtype) is None:
        raise ValueError(f"logits: expected float32, bfloat16 or float16, got {logits.dtype}")
    if topk_ids.shape[0] != T or topk_ids.dtype is not torch.int32 or not topk_ids.is_contiguous():
        raise ValueError(f"topk_ids: expected contiguous int32 [{T}, k]")
    if T and logits.stride(1) != 1:
        raise ValueError("logits: elements of a row must be contiguous")
    if loss.dtype is not torch.float32 or loss.numel() != 1:
        raise ValueError("loss: expected one float32")
    if counts.dtype is not torch.int32 or counts.numel() != E + 1 or not counts.is_contiguous():
        raise ValueError(f"counts: expected contiguous int32 [{E + 1}]")
    if token_mask is not None and (token_mask.dtype not in (torch.bool, torch.uint8) or token_mask.numel() != T
                                   or not token_mask.is_contiguous()):
        raise ValueError(f"token_mask: expected contiguous bool or uint8 [{T}]")
    if router_bias is not None and (router_bias.dtype is not torch.float32 or router_bias.numel() != E
                                    or not router_bias.is_contiguous()):
        raise ValueError(f"router_bias: expected contiguous float32 [{E}]")
    if dlogits is not None and (dlogits.dtype != logits.dtype or dlogits.shape != logits.shape
                                or (T and dlogits.stride(1) != 1)):
        raise ValueError("dlogits: expected the logits' shape and type, elements of a row contiguous")
    if grad_loss is not None and (grad_loss.dtype is not torch.float32 or grad_loss.numel() != 1):
        raise ValueError("grad_loss: expected one float32")
    for name, t in (("logits", logits), ("topk_ids", topk_ids), ("loss", loss), ("counts", counts),
                    ("token_mask", token_mask), ("router_bias", router_bias), ("dlogits", dlogits),
                    ("grad_loss", grad_loss), ("workspace", workspace)):
        if t is not None and (t.device.type != "cuda" or t.device != logits.device):
            raise ValueError(f"{name}: on {t.device}, expected one GPU (the logits are on {logits.device})")
    if workspace is not None and (not workspace.is_contiguous()
                                  or workspace.numel() * workspace.element_size() < workspace_bytes(E)):
        raise ValueError(f"workspace: expected {workspace_bytes(E)} contiguous bytes")
