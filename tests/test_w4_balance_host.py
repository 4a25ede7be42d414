"""Refusals of the 4-bit products and of the balance loss on the host (no GPU
needed: arguments are checked before anything is enqueued)."""
import ctypes

import pytest
import torch

import moe_decode_block_b200 as mdb
from moe_decode_block_b200 import balance, synth, w4
from moe_decode_block_b200 import build as mbuild

BAD, SHAPE = mdb.MOE_ERR_INVALID_ARG, mdb.MOE_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    mbuild.build_library()
    return mdb.load_library()


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(4096 + 64)
    mem.keep = buf
    return (ctypes.addressof(buf) + 63) // 64 * 64


def test_packed_bytes(lib):
    # codes, and 16-bit scales (and zero points) of panels of 16 outputs
    assert lib.moe_w4_packed_bytes(16, 64, 64, 0) == 512 + 32
    assert lib.moe_w4_packed_bytes(16, 64, 64, 1) == 512 + 64
    assert lib.moe_w4_packed_bytes(17, 128, 32, 0) == 2 * (1024 + 4 * 32)
    assert lib.moe_w4_packed_bytes(4096, 7168, 128, 0) == 4096 * 7168 // 2 + 4096 * 56 * 2
    for n, k, g in ((0, 64, 64), (16, 0, 64), (16, 96, 32), (16, 64, 128), (16, 192, 128), (16, 64, 16), (16, 64, 48),
                    (16, 32768 + 64, 64), (524288 + 1, 64, 64), (-1, 64, 64), (16, -64, 64), (16, 64, 0), (16, 64, -64)):
        assert lib.moe_w4_packed_bytes(n, k, g, 0) == 0, (n, k, g)
    with pytest.raises(ValueError):
        w4.packed_bytes(16, 100, 64)


def test_linear_refusals(lib, mem):
    def call(x=mem, w=mem, bias=None, out=mem + 1024, b=2, k=64, n=16, g=64, z=0, xs=64, os=16, dt=0):
        return lib.moe_w4_linear(x, w, bias, out, b, k, n, g, z, xs, os, dt, None)

    for kw in (dict(k=65), dict(k=32), dict(n=0), dict(g=16), dict(g=128), dict(b=65), dict(b=-1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(x=mem + 2), dict(w=mem + 8), dict(out=mem + 1), dict(bias=mem + 1),
               dict(dt=2), dict(dt=-1), dict(xs=68), dict(xs=-64), dict(os=15)):
        assert call(**kw) == BAD, kw
    assert call(b=0, x=None, w=None, out=None) == mdb.MOE_OK  # nothing to do
    if not torch.cuda.is_available():
        assert call() == mdb.MOE_ERR_NO_DEVICE


def test_pack_refusals(lib, mem):
    def call(c=mem, s=mem, z=None, p=mem, n=16, k=64, g=64, dt=0):
        return lib.moe_w4_pack(c, s, z, p, n, k, g, dt, None)

    for kw in (dict(k=65), dict(n=0), dict(g=16), dict(g=128)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(c=None), dict(s=None), dict(p=None), dict(s=mem + 1), dict(p=mem + 8), dict(dt=2)):
        assert call(**kw) == BAD, kw
    if not torch.cuda.is_available():
        assert call() == mdb.MOE_ERR_NO_DEVICE


def test_block_handle_shapes(lib):
    def ws(**kw):
        s = synth.FULL
        d = dict(hidden=s.hidden, n_experts=s.n_experts, top_k=s.top_k, inter=s.inter, shared_inter=s.shared_inter, n_shared=1,
                 max_batch=64, router_bias=None, flags=mdb.MOE_FLAG_W4_WEIGHTS)
        d.update(kw)
        return lib.moe_decode_workspace_bytes(ctypes.byref(mdb.Shapes(**d)))

    plain = ws(flags=0)
    # a row for every (token, choice) and the shared expert; above 8 tokens lists of 1,088 and 1,024 units besides
    lists = (16 + 3 * (1088 + 1024) * 4 + 255) // 256 * 256
    assert ws() == plain + 64 * 9 * 7168 * 4 + lists
    assert ws(n_shared=0, shared_inter=0) == ws(n_shared=0, shared_inter=0, flags=0) + 64 * 8 * 7168 * 4 + lists
    assert ws(max_batch=16) == ws(max_batch=16, flags=0) + 16 * 9 * 7168 * 4 + lists
    assert ws(max_batch=8) == ws(max_batch=8, flags=0) + 8 * 9 * 7168 * 4
    assert ws(flags=mdb.MOE_FLAG_W4_WEIGHTS | mdb.MOE_FLAG_PARTIAL_SUM) == ws()
    for kw in (dict(hidden=7168 + 32), dict(inter=2048 + 32), dict(shared_inter=2048 + 32)):
        assert ws(**kw) == 0, kw
    for other in (mdb.MOE_FLAG_TWO_STREAM, mdb.MOE_FLAG_TCGEN05, mdb.MOE_FLAG_TEST_HOLD_PANEL, mdb.MOE_FLAG_FP8_WEIGHTS):
        assert ws(flags=mdb.MOE_FLAG_W4_WEIGHTS | other) == 0
    assert lib.moe_decode_forward_w4(None, *([None] * 9), 1, 64, 0, None) == BAD


def test_balance_refusals(lib, mem):
    assert lib.moe_balance_workspace_bytes(384) > 0
    for e in (0, 4, 12, 1032, -8):
        assert lib.moe_balance_workspace_bytes(e) == 0
    with pytest.raises(ValueError):
        balance.workspace_bytes(12)

    def call(z=mem, bias=None, ids=mem, mask=None, loss=mem, counts=mem, d=None, g=None, t=2, e=16, k=2, zs=16, ds=16, dt=2, ws=mem):
        return lib.moe_balance_loss(z, bias, ids, mask, loss, counts, d, g, t, e, k, zs, ds, 1.0, dt, ws, None)

    for kw in (dict(e=12), dict(e=0), dict(e=1032), dict(k=0), dict(k=17), dict(e=64, k=33), dict(t=-1), dict(t=(1 << 24) + 1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(z=None), dict(ids=None), dict(loss=None), dict(counts=None), dict(ws=None, t=513), dict(z=mem + 4), dict(z=mem + 4, dt=0),
               dict(ids=mem + 2), dict(loss=mem + 2), dict(counts=mem + 1), dict(d=mem + 8), dict(g=mem + 2), dict(bias=mem + 1),
               dict(ws=mem + 8), dict(zs=15), dict(zs=18), dict(d=mem, ds=15), dict(d=mem, ds=18), dict(dt=3), dict(dt=-1)):
        assert call(**kw) == BAD, kw
    if not torch.cuda.is_available():
        assert call() == mdb.MOE_ERR_NO_DEVICE


def test_bindings_refuse_tensors_that_do_not_fit(lib):
    x, out = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 16, dtype=torch.bfloat16)
    packed = torch.zeros(w4.packed_bytes(16, 64, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        w4.linear(x, packed, out, 64)  # not on a GPU
    with pytest.raises(ValueError):
        w4.linear(x, packed[:-1], out, 64)
    with pytest.raises(ValueError):
        w4.linear(x.float(), packed, out.float(), 64)
    with pytest.raises(ValueError):
        w4.linear(x, packed, out[:1], 64)
    with pytest.raises(ValueError):
        w4.linear(x.t().contiguous().t(), packed, out, 64)
    with pytest.raises(ValueError):
        w4.linear(x, packed, out, 64, bias=torch.zeros(15, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        w4.pack(torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.bfloat16))
    z, ids = torch.zeros(3, 16), torch.zeros(3, 2, dtype=torch.int32)
    loss, counts = torch.zeros(1), torch.zeros(17, dtype=torch.int32)
    with pytest.raises(ValueError):
        balance.balance_loss(z, ids, loss, counts)  # not on a GPU
    for kw in (dict(topk_ids=ids.long()), dict(topk_ids=ids[:2]), dict(loss=torch.zeros(2)), dict(counts=counts[:16]),
               dict(logits=z.double()), dict(logits=z.t().contiguous().t()), dict(token_mask=torch.zeros(3)),
               dict(token_mask=torch.zeros(2, dtype=torch.bool)), dict(router_bias=torch.zeros(15)), dict(dlogits=z.bfloat16()),
               dict(grad_loss=torch.zeros(2))):
        args = dict(logits=z, topk_ids=ids, loss=loss, counts=counts)
        args.update(kw)
        with pytest.raises(ValueError):
            balance.balance_loss(**args)
