"""The router's balance loss, its gradient and the choices per expert:
argument marshalling of moe_balance_loss.

    balance.balance_loss(logits, topk_ids, loss, counts)                     # serving: the load
    balance.balance_loss(logits, topk_ids, loss, counts, dlogits=dlogits)    # training: in the same pass
"""
from __future__ import annotations

from typing import Optional

from . import MOE_DTYPE_BF16, MOE_DTYPE_FP16, MOE_DTYPE_FP32, _check, _current_stream, _ptr, _stream_handle, load_library
from .w4 import _on


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
    token.  workspace: a uint8 tensor of workspace_bytes(E), by default a new
    one (torch's allocator ties it to the current stream, so pass one when
    `stream` is another)."""
    import torch
    lib = load_library()
    T, E = logits.shape
    k = topk_ids.shape[1]
    codes = {torch.float32: MOE_DTYPE_FP32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_FP16}
    code = codes.get(logits.dtype)
    if code is None:
        raise ValueError(f"logits: expected float32, bfloat16 or float16, got {logits.dtype}")
    if topk_ids.shape[0] != T or topk_ids.dtype is not torch.int32 or not topk_ids.is_contiguous():
        raise ValueError(f"topk_ids: expected contiguous int32 [{T}, k]")
    if E and T and logits.stride(1) != 1:
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
    for name, t in (("topk_ids", topk_ids), ("loss", loss), ("counts", counts), ("token_mask", token_mask),
                    ("router_bias", router_bias), ("dlogits", dlogits), ("grad_loss", grad_loss),
                    ("workspace", workspace)):
        if t is not None and t.device != logits.device:
            raise ValueError(f"{name}: on {t.device}, the logits on {logits.device}")
    if workspace is not None and (not workspace.is_contiguous()
                                  or workspace.numel() * workspace.element_size() < workspace_bytes(E)):
        raise ValueError(f"workspace: expected {workspace_bytes(E)} contiguous bytes")
    with _on(logits.device):
        if workspace is None:
            if stream is not None and _stream_handle(stream) != _current_stream():
                raise ValueError("workspace: needed with a stream that is not the current one")
            workspace = torch.empty(max(1, lib.moe_balance_workspace_bytes(E)), dtype=torch.uint8, device=logits.device)
        sm = _stream_handle(stream) if stream is not None else _current_stream()
        rc = lib.moe_balance_loss(logits.data_ptr(), _ptr(router_bias), topk_ids.data_ptr(), _ptr(token_mask),
                                  loss.data_ptr(), counts.data_ptr(), _ptr(dlogits), _ptr(grad_loss), T, E, k,
                                  logits.stride(0), dlogits.stride(0) if dlogits is not None else 0, float(coef), code,
                                  workspace.data_ptr(), sm)
    _check(rc, "moe_balance_loss")
    return loss
