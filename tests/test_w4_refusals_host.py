"""Calls that forward_w4 refuses before anything reaches the library (no GPU needed): tensors too small for the batch,
of another type, with gaps, or elsewhere."""
import pytest
import torch

import moe_decode_block_b200 as mdb
from moe_decode_block_b200 import MoEDecode, Shapes, w4


class _Reached(Exception):
    pass


class _Library:
    def moe_decode_forward_w4(self, *args):
        raise _Reached


def _handle(partial=False):
    """A handle on "GPU" -1, the index that CPU tensors report, with a library that only says that it was reached."""
    blk = MoEDecode.__new__(MoEDecode)
    blk._lib, blk._h, blk._device, blk._tables = _Library(), None, -1, {}
    blk.shapes = Shapes(128, 8, 2, 64, 64, 1, 16, None, mdb.MOE_FLAG_W4_WEIGHTS | (mdb.MOE_FLAG_PARTIAL_SUM if partial else 0))
    return blk


def _args(b=3):
    bf = torch.bfloat16
    pk = lambda n, k, lead=(): torch.zeros(*lead, w4.packed_bytes(n, k, 64), dtype=torch.uint8).view(*lead, -(-n // 16), -1)  # noqa: E731
    return dict(x=torch.zeros(b, 128, dtype=bf), router_w=torch.zeros(128, 8, dtype=bf), w13=pk(128, 128, (8,)), w2=pk(128, 64, (8,)),
                shared_w13=pk(128, 128), shared_w2=pk(128, 64), out=torch.zeros(b, 128, dtype=bf),
                topk_ids=torch.zeros(b, 2, dtype=torch.int32), topk_w=torch.zeros(b, 2), group=64, stream=1)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from moe_decode_block_b200 import build as mbuild
    mbuild.build_library()


def test_calls_that_fit_reach_the_library():
    for kw in ({}, dict(batch=2), dict(batch=0), dict(w13=list(_args()["w13"])), dict(x=torch.zeros(9, 128, dtype=torch.bfloat16), batch=3)):
        with pytest.raises(_Reached):
            _handle().forward_w4(**{**_args(), **kw})
    with pytest.raises(_Reached):
        _handle(partial=True).forward_w4(**{**_args(), "out": torch.zeros(3, 128)})


@pytest.mark.parametrize("name,make", [
    ("x", lambda t: t.float()), ("x", lambda t: t.half()), ("x", lambda t: t[:, :64]), ("x", lambda t: t.t().contiguous().t()),
    ("router_w", lambda t: t.float()), ("router_w", lambda t: t.t()), ("router_w", lambda t: t[:64]),
    ("out", lambda t: t.float()), ("out", lambda t: t[:2]), ("out", lambda t: torch.zeros(3, 256, dtype=t.dtype)[:, :128]),
    ("topk_ids", lambda t: t.long()), ("topk_ids", lambda t: t[:2]), ("topk_w", lambda t: t.double()), ("topk_w", lambda t: t[:, :1]),
    ("w13", lambda t: t[:7]), ("w2", lambda t: t[..., :-1]), ("w13", lambda t: list(t.flip(1)[:, 1:])), ("shared_w2", lambda t: t[:-1]),
])
def test_tensors_that_do_not_fit_are_refused(name, make):
    args = _args()
    args[name] = make(args[name])
    with pytest.raises(ValueError, match=name):
        _handle().forward_w4(**args)


def test_a_batch_larger_than_the_tensors_is_refused():
    with pytest.raises(ValueError, match="x"):
        _handle().forward_w4(**_args(), batch=4)
    with pytest.raises(ValueError, match="topk_ids"):
        _handle().forward_w4(**{**_args(8), "topk_ids": torch.zeros(3, 2, dtype=torch.int32)}, batch=8)
    with pytest.raises(ValueError, match="out"):  # a partial sum is fp32
        _handle(partial=True).forward_w4(**_args())


def test_tensors_elsewhere_are_refused():
    blk = _handle()
    blk._device = 0
    with pytest.raises(ValueError, match="GPU 0"):
        blk.forward_w4(**_args())


def test_wait_limit_and_hold_are_set_on_the_host():
    lib = mdb.load_library()
    for probes in (1, 512, 1 << 31, 0):
        assert lib.moe_w4_linear_set_wait_limit(probes) == mdb.MOE_OK
    assert lib.moe_w4_test_hold(-1) == mdb.MOE_ERR_INVALID_ARG
    assert lib.moe_w4_test_hold(3) == mdb.MOE_OK and lib.moe_w4_test_hold(0) == mdb.MOE_OK


def test_numbers_beyond_32_bits_do_not_come_around():
    class Keeps:
        def moe_decode_forward_w4(self, *args):
            self.batch, self.group = args[10], args[11]
            raise _Reached

    blk = _handle()
    blk._lib = Keeps()
    for kw in (dict(group=2 ** 32 + 64), dict(group=48), dict(batch=1 - 2 ** 32)):
        with pytest.raises(_Reached):
            blk.forward_w4(**{**_args(), **kw})
        assert blk._lib.group == (0 if "group" in kw else 64) and blk._lib.batch == (-1 if "batch" in kw else 3)
    with pytest.raises(ValueError):
        blk.forward_w4(**_args(), batch=2 ** 32 + 1)
    for n, k, g in ((2 ** 32 + 16, 64, 64), (16, 2 ** 32 + 64, 64), (16, 64, 2 ** 32 + 64), (16, 64, -2 ** 32 + 64)):
        with pytest.raises(ValueError):
            w4.packed_bytes(n, k, g)
