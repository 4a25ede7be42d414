"""Measured cases of the 4-bit weight products and of the router's balance loss.

Three operators:
  linear   y = x W^T (+ bias) for 1..64 tokens, W in 4 bits with a scale (and optionally a zero point) per group of inputs
  block    the whole decode block -- router, top-k, the experts' SwiGLU products and the shared expert's, residual -- with
           4-bit expert weights
  balance  the balance loss of the router and the tokens per expert; with "grad", the gradient with respect to the logits

`own` false: the plain forms in elementary torch operations; `own` true: the library's entry points.

The packed 4-bit matrix (W [N, K], groups of G inputs): panels of 16 outputs, uint8 [ceil(N / 16), panel bytes].  A panel
holds K / 64 tiles of 512 bytes, then K / G entries of scales (and zero points).  A tile is 32 lanes (g, t) of four 32-bit words
s; bits 4j and 16 + 4j of a word are the codes of output g + 8 (j & 1) and of the inputs
32 (s >> 1) + 8 t + 4 (s & 1) + 2 (j >> 1) and the next.  An entry is, for each g, the scales of outputs g and g + 8, and with
zero points those two after them, all in the activations' type.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest call, one token through a tiny block's width: what a launch costs
        {"name": "linear_tiny_b1", "op": "linear", "b": 1, "k": 256, "n": 256, "g": 64, "zeros": False, "bias": False, "dtype": "bf16"},
        # the full-size block's gate and up projection as a dense layer, one token
        {"name": "linear_up_b1", "op": "linear", "b": 1, "k": 7168, "n": 4096, "g": 128, "zeros": False, "bias": False, "dtype": "bf16"},
        # its down projection, a small batch, zero points and half the group
        {"name": "linear_down_b8_zeros", "op": "linear", "b": 8, "k": 2048, "n": 7168, "g": 64, "zeros": True, "bias": False, "dtype": "fp16"},
        # sizes that fill no tile: 13 tokens, 1,003 outputs, the smallest group
        {"name": "linear_ragged_b13", "op": "linear", "b": 13, "k": 1600, "n": 1003, "g": 32, "zeros": True, "bias": True, "dtype": "bf16"},
        # the widest dense layer at the largest batch
        {"name": "linear_wide_b64", "op": "linear", "b": 64, "k": 7168, "n": 16384, "g": 128, "zeros": False, "bias": True, "dtype": "bf16"},
        # a tiny block: launches again
        {"name": "block_tiny_b3", "op": "block", "b": 3, "h": 256, "e": 16, "top_k": 2, "i": 128, "shared": True, "g": 64, "zeros": False},
        # the full-size block, one token
        {"name": "block_full_b1", "op": "block", "b": 1, "h": 7168, "e": 384, "top_k": 8, "i": 2048, "shared": True, "g": 128, "zeros": False},
        # the full-size block, a small batch, zero points
        {"name": "block_full_b8_zeros", "op": "block", "b": 8, "h": 7168, "e": 384, "top_k": 8, "i": 2048, "shared": True, "g": 128, "zeros": True},
        # 16 experts of full size at the largest batch: about 32 tokens for each
        {"name": "block_16_experts_b64", "op": "block", "b": 64, "h": 7168, "e": 16, "top_k": 8, "i": 2048, "shared": True, "g": 128, "zeros": False},
        # the load of one decode batch, as a server watches it
        {"name": "balance_decode_64", "op": "balance", "t": 64, "e": 384, "top_k": 8, "dtype": "fp32", "live": 1.0, "bias": True, "grad": False},
        # a training batch, loss and gradient
        {"name": "balance_train_65536", "op": "balance", "t": 65536, "e": 384, "top_k": 8, "dtype": "fp32", "live": 1.0, "bias": False, "grad": True},
        # an odd number of padded tokens in 16 bits
        {"name": "balance_train_masked_16383", "op": "balance", "t": 16383, "e": 256, "top_k": 4, "dtype": "bf16", "live": 0.8, "bias": True, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "block", "balance"])
    if op == "linear":
        g = rng.choice([32, 64, 128])
        step = max(g, 64)
        return {"op": op, "b": _log(rng, 1, 64), "k": step * max(1, _log(rng, 256, 7168) // step), "n": _log(rng, 16, 16384), "g": g,
                "zeros": rng.random() < 0.5, "bias": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "block":
        g = rng.choice([32, 64, 128])
        h, i = 128 * max(1, _log(rng, 256, 7168) // 128), 128 * max(1, _log(rng, 128, 2048) // 128)
        e = 8 * max(1, _log(rng, 8, 384) // 8)
        c = {"op": op, "b": _log(rng, 1, 64), "h": h, "e": e, "top_k": min(e, rng.randint(1, 8)), "i": i, "shared": rng.random() < 0.7, "g": g,
             "zeros": rng.random() < 0.4}
        while work(c)["bytes"] > 1.4e9:  # no more than the full-size block at a batch of 8
            c["b"] = (c["b"] + 1) // 2
        return c
    return {"op": op, "t": _log(rng, 1, 65536), "e": 8 * max(1, _log(rng, 8, 384) // 8), "top_k": rng.randint(1, 8), "dtype": rng.choice(["fp32", "bf16"]),
            "live": rng.choice([1.0, 1.0, 0.7]), "bias": rng.random() < 0.5, "grad": rng.random() < 0.7}


# ------------------------------------------------------- packed 4-bit matrices
def _panel_bytes(k, g, zeros):
    return k // 64 * 512 + k // g * (64 if zeros else 32)


def _random_packed(count, n, k, g, zeros, dtype, gen):
    """`count` packed matrices: codes as a quantiser leaves normal weights of deviation 0.02 (a group's largest magnitude is near the code range's end)."""
    p = -(-n // 16)
    out = torch.empty(count, p, _panel_bytes(k, g, zeros), dtype=torch.uint8, device=DEV)
    for c in range(count):
        v = torch.randn(p, k // 64 * 512, 2, device=DEV, generator=gen).mul_(2.6).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        out[c, :, : k // 64 * 512] = v[..., 0] | (v[..., 1] << 4)
        e = torch.empty(p, k // g, 8, 2, 2 if zeros else 1, device=DEV)
        e[..., 0] = (torch.rand(p, k // g, 8, 2, device=DEV, generator=gen) + 0.5) * (0.02 / 2.6)
        if zeros:
            e[..., 1] = torch.randint(5, 11, (p, k // g, 8, 2), device=DEV, generator=gen)
        out[c, :, k // 64 * 512:] = e.transpose(-1, -2).contiguous().to(dtype).view(torch.uint8).reshape(p, -1)
    return out


def _unpack(w, n, k, g, zeros, dtype):
    """fp32 [..., n, k] of packed matrices [..., panels, panel bytes]."""
    m, p, tiles = w.shape[:-2], w.shape[-2], k // 64
    words = w[..., : tiles * 512].contiguous().view(torch.int32).view(-1, p, tiles, 8, 4, 2, 2)  # matrix, panel, tile, g, t, s >> 1, s & 1
    sh = torch.tensor([[[0, 16], [4, 20]], [[8, 24], [12, 28]]], dtype=torch.int32, device=w.device)  # j >> 1, j & 1, pair
    q = (words[..., None, None, None] >> sh) & 15
    q = q.permute(0, 1, 8, 3, 2, 5, 4, 6, 7, 9).reshape(-1, p * 16, k // g, g)  # (panel, j & 1, g), (tile, s >> 1, t, s & 1, j >> 1, pair)
    e = w[..., tiles * 512:].contiguous().view(dtype).view(-1, p, k // g, 8, 2 if zeros else 1, 2).float()  # matrix, panel, group, g, which, j & 1
    e = e.permute(4, 0, 1, 5, 3, 2).reshape(2 if zeros else 1, -1, p * 16, k // g, 1)
    return ((q.float() - (e[1] if zeros else 8.0)) * e[0]).view(*m, p * 16, k)[..., :n, :]


# ------------------------------------------------------------------- prepare
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "linear":
        dt = DT[case["dtype"]]
        s["x"] = torch.randn(case["b"], case["k"], device=DEV, generator=gen).to(dt)
        s["w"] = _random_packed(1, case["n"], case["k"], case["g"], case["zeros"], dt, gen)[0]
        s["bias"] = torch.randn(case["n"], device=DEV, generator=gen).to(dt) if case["bias"] else None
        s["out"] = torch.empty(case["b"], case["n"], device=DEV, dtype=dt)
        return s
    if case["op"] == "block":
        b, h, e, i, g, zs = case["b"], case["h"], case["e"], case["i"], case["g"], case["zeros"]
        s["router_w"] = (torch.randn(h, e, device=DEV, generator=gen) * 0.02).to(torch.bfloat16)
        s["w13"] = _random_packed(e, 2 * i, h, g, zs, torch.bfloat16, gen)
        s["w2"] = _random_packed(e, h, i, g, zs, torch.bfloat16, gen)
        s["s13"] = _random_packed(1, 2 * i, h, g, zs, torch.bfloat16, gen)[0] if case["shared"] else None
        s["s2"] = _random_packed(1, h, i, g, zs, torch.bfloat16, gen)[0] if case["shared"] else None
        # tokens whose selected logits stand apart, so that the selection does not hang on the order of a sum
        x = torch.randn(16 * b, h, device=DEV, generator=gen).to(torch.bfloat16)
        top = (x.double() @ s["router_w"].double()).topk(min(e, case["top_k"] + 1), dim=1).values
        gap = (top[:, :-1] - top[:, 1:]).amin(dim=1) if top.shape[1] > 1 else torch.ones(len(x), device=DEV)
        s["x"] = x[torch.argsort((gap < 1e-3).to(torch.int8), stable=True)[:b]].contiguous()
        s["out"] = torch.empty_like(s["x"])
        s["ids"] = torch.empty(b, case["top_k"], dtype=torch.int32, device=DEV)
        s["wts"] = torch.empty(b, case["top_k"], dtype=torch.float32, device=DEV)
        if own:  # the handle of this block
            from moe_decode_block_b200 import MoEDecode
            s["block"] = MoEDecode(h, e, case["top_k"], i, i, n_shared=int(case["shared"]), max_batch=b, w4=True)
        return s
    t, e, k = case["t"], case["e"], case["top_k"]
    s["logits"] = (torch.randn(t, e, device=DEV, generator=gen) * 1.7).to(DT[case["dtype"]])
    s["bias"] = torch.randn(e, device=DEV, generator=gen) if case["bias"] else None
    sel = s["logits"].float() + (s["bias"] if case["bias"] else 0.0)
    s["ids"] = sel.topk(k, dim=1).indices.to(torch.int32)
    s["mask"] = torch.rand(t, device=DEV, generator=gen) < case["live"] if case["live"] < 1.0 else None
    s["grad_loss"] = torch.rand(1, device=DEV, generator=gen) + 0.5
    s["loss"] = torch.empty(1, device=DEV)
    s["counts"] = torch.empty(e + 1, dtype=torch.int32, device=DEV)
    s["dlogits"] = torch.empty_like(s["logits"]) if case["grad"] else None
    return s


# ----------------------------------------------------------------------- run
COEF = 0.01


def run(s):
    if own:
        return {"linear": _linear_own, "block": _block_own, "balance": _balance_own}[s["case"]["op"]](s)
    return {"linear": _linear, "block": _block, "balance": _balance}[s["case"]["op"]](s)


def _linear_own(s):
    from moe_decode_block_b200 import w4
    w4.linear(s["x"], s["w"], s["out"], s["case"]["g"], zeros=s["case"]["zeros"], bias=s["bias"])
    return s["out"]


def _block_own(s):
    c = s["case"]
    s["block"].forward_w4(s["x"], s["router_w"], s["w13"], s["w2"], s["s13"], s["s2"], s["out"], s["ids"], s["wts"], c["g"], zeros=c["zeros"])
    return {"out": s["out"], "ids": s["ids"], "weights": s["wts"]}


def _balance_own(s):
    from moe_decode_block_b200 import balance
    balance.balance_loss(s["logits"], s["ids"], s["loss"], s["counts"], token_mask=s["mask"], router_bias=s["bias"], coef=COEF, dlogits=s["dlogits"],
                         grad_loss=s["grad_loss"] if s["case"]["grad"] else None)
    out = {"loss": s["loss"], "counts": s["counts"]}
    if s["case"]["grad"]:
        out["dlogits"] = s["dlogits"]
    return out


def _linear(s):
    c = s["case"]
    y = s["x"].float() @ _unpack(s["w"], c["n"], c["k"], c["g"], c["zeros"], s["x"].dtype).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def _mlp(x, w13, w2, c):
    """[..., h] of tokens x [..., tokens, h] and packed expert weights [..., panels, panel bytes]."""
    h = x @ _unpack(w13, 2 * c["i"], c["h"], c["g"], c["zeros"], torch.bfloat16).transpose(-1, -2)
    gate, up = h[..., : c["i"]], h[..., c["i"]:]
    return (gate / (1.0 + torch.exp(-gate)) * up) @ _unpack(w2, c["h"], c["i"], c["g"], c["zeros"], torch.bfloat16).transpose(-1, -2)


def _block(s):
    c = s["case"]
    x = s["x"].float()
    # logits in 64 bits: the selection compares them
    val, ids = (s["x"].double() @ s["router_w"].double()).sort(dim=1, descending=True, stable=True)
    val, ids = val[:, : c["top_k"]].float(), ids[:, : c["top_k"]]
    wts = torch.exp(val - val[:, :1])
    wts = wts / wts.sum(dim=1, keepdim=True)
    y = x
    if c["b"] * c["top_k"] <= c["e"]:  # fewer choices than experts: each token's own experts, one choice of every token at a time
        for j in range(c["top_k"]):
            y = y + wts[:, j: j + 1] * _mlp(x[:, None], s["w13"][ids[:, j]], s["w2"][ids[:, j]], c)[:, 0]
    else:  # every expert for all tokens, in pieces that fit in 32 bits
        gates = torch.zeros(c["b"], c["e"], device=x.device).scatter_(1, ids, wts)
        n = max(1, (1 << 28) // (c["h"] * c["i"]))
        for e in range(0, c["e"], n):
            y = y + (gates[:, e: e + n].t()[..., None] * _mlp(x, s["w13"][e: e + n], s["w2"][e: e + n], c)).sum(dim=0)
    if c["shared"]:
        y = y + _mlp(x, s["s13"], s["s2"], c)
    return {"out": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": wts}


def _probs(s):
    z = s["logits"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    p = torch.exp(z - z.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    return p if s["mask"] is None else p * s["mask"][:, None]


def _balance(s):
    c = s["case"]
    p = _probs(s)
    ids = s["ids"].long()
    live = torch.ones(c["t"], dtype=torch.int64, device=p.device) if s["mask"] is None else s["mask"].long()
    counts = torch.zeros(c["e"], dtype=torch.int64, device=p.device).index_add_(0, ids.reshape(-1), live[:, None].expand(-1, c["top_k"]).reshape(-1))
    n = live.sum()
    factor = torch.where(n > 0, COEF * c["e"] / (c["top_k"] * n.double().clamp(min=1) ** 2), torch.zeros_like(n, dtype=torch.float64))
    loss = (factor * (counts.double() * p.sum(dim=0, dtype=torch.float64)).sum()).float().view(1)
    out = {"loss": loss, "counts": torch.cat([counts, n.view(1)]).to(torch.int32)}
    if c["grad"]:
        cf = counts.float()
        d = p * (cf - (p * cf).sum(dim=1, keepdim=True)) * (factor.float() * s["grad_loss"])
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "linear":
        b, k, n = case["b"], case["k"], case["n"]
        entry = 4 if case["zeros"] else 2
        return {"bytes": n * k / 2 + n * (k // case["g"]) * entry + 2 * b * (k + n) + (2 * n if case["bias"] else 0), "flops": 2 * b * k * n}
    if case["op"] == "block":
        b, h, e, i, k = case["b"], case["h"], case["e"], case["i"], case["top_k"]
        entry = 4 if case["zeros"] else 2
        expert = 3 * h * i / 2 + 3 * h * i / case["g"] * entry
        active = e * (1.0 - (1.0 - k / e) ** b) + (1 if case["shared"] else 0)  # distinct experts that b tokens choose, on average
        return {"bytes": active * expert + 2 * h * e + 4 * b * h + 8 * b * k, "flops": 6 * h * i * b * (k + (1 if case["shared"] else 0)) + 2 * b * h * e}
    t, e, k = case["t"], case["e"], case["top_k"]
    el = 4 if case["dtype"] == "fp32" else 2
    passes = 2 if case["grad"] else 1  # the logits once and the gradient once: the counts that it needs come from the ids
    return {"bytes": passes * t * e * el + 4 * t * k + 4 * e, "flops": (10 if case["grad"] else 5) * t * e}


# --------------------------------------------------------------------- exact
def _weights64(w, n, k, g, zeros, dtype):
    """float64 [n, k] of one packed matrix, each code looked up by its output's and its input's place."""
    r, c = torch.arange(n, device=w.device)[:, None], torch.arange(k, device=w.device)[None, :]
    lane = (r % 8) * 4 + (c % 32) // 8
    word = (c % 64) // 32 * 2 + (c % 8) // 4
    bit = 4 * ((r % 16) // 8 + 2 * ((c % 4) // 2)) + 16 * (c % 2)
    byte = (c // 64) * 512 + lane * 16 + word * 4 + bit // 8
    code = (w[(r // 16).expand(n, k), byte].to(torch.int32) >> (bit % 8)) & 15
    ent = w[:, k // 64 * 512:].contiguous().view(dtype).double()
    width = 4 if zeros else 2
    at = ((torch.arange(k // g, device=w.device)[None, :] * 8 + r % 8) * width) + (r % 16) // 8
    scale = ent[r // 16, at]
    zero = ent[r // 16, at + 2] if zeros else torch.full_like(scale, 8.0)
    return (code.double() - zero.repeat_interleave(g, dim=1)) * scale.repeat_interleave(g, dim=1)


def _expert64(x, w13, w2, case):
    i, h, g, zs = case["i"], case["h"], case["g"], case["zeros"]
    a = _weights64(w13, 2 * i, h, g, zs, torch.bfloat16)
    gate, up = x @ a[:i].T, x @ a[i:].T
    return (gate * torch.sigmoid(gate) * up) @ _weights64(w2, h, i, g, zs, torch.bfloat16).T


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = s["x"].double() @ _weights64(s["w"], case["n"], case["k"], case["g"], case["zeros"], s["x"].dtype).T
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "block":
        x = s["x"].double()
        logits = x @ s["router_w"].double()
        ids = torch.argsort(-logits, dim=1, stable=True)[:, : case["top_k"]]
        wts = torch.softmax(torch.gather(logits, 1, ids), dim=1)
        y = x.clone()
        for e in torch.unique(ids).tolist():
            t, j = (ids == e).nonzero(as_tuple=True)
            y[t] += wts[t, j][:, None] * _expert64(x[t], s["w13"][e], s["w2"][e], case)
        if case["shared"]:
            y += _expert64(x, s["s13"], s["s2"], case)
        return {"out": y, "ids": None, "weights": wts}
    z = s["logits"].double() + (s["bias"].double() if s["bias"] is not None else 0.0)
    rows = torch.ones(case["t"], dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"]
    n = int(rows.sum())
    p = torch.softmax(z[rows], dim=1)
    c = torch.bincount(s["ids"][rows].reshape(-1).long(), minlength=case["e"]).double()
    f = COEF * case["e"] / (case["top_k"] * n * n) if n else 0.0
    out = {"loss": (f * (p.sum(dim=0) * c).sum()).view(1), "counts": None}
    if case["grad"]:
        d = torch.zeros_like(z)
        d[rows] = f * s["grad_loss"].double() * p * (c - (p @ c)[:, None])
        out["dlogits"] = d
    return out
