"""The router's balance loss on logits of every magnitude: rows at a mask's usual fill value, maxima far from zero.

Tolerances as in test_gpu_balance.py (no bias here, which at 1e10 could not be added in fp32): a row's logits are
within 16 of its maximum, or so far below that their probability is zero in fp32 and in 64 bits alike.  The maximum
comes off exactly (Sterbenz) or, below 2^20, with one rounding of m log2(e) that all of the row shares."""
import pytest
import torch

from test_gpu_balance import _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [48, 384, 1000])
@pytest.mark.parametrize("t", [50, 1200])
def test_rows_of_one_large_value_are_uniform(t, e, dtype):
    """Every expert of a live row at the same value: probabilities 1 / E, whatever the value."""
    logits, _, ids, _ = _inputs(t, e, 3, dtype, seed=t + e)
    fills = [s * v for v in (2.0 ** 19, 2.0 ** 20, 1e6, 1e9, 2.0 ** 31, 5e9, 1e10, 1e20, 1e30, 2.0 ** 100, 3e38) for s in (-1, 1)]
    for i, v in enumerate(fills):
        logits[2 * i + 1] = v
    loss, counts, d = _run(logits, ids)
    assert bool(loss.isfinite()) and bool(d.isfinite().all())
    _check(logits, ids, None, None, 0.5, None, loss, counts, d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t", [50, 1200])
def test_large_maxima_with_others_below(t, dtype):
    """A maximum of +1e10 (and other sizes) over ordinary logits, two experts sharing it; masked experts at -1e10."""
    logits, _, ids, _ = _inputs(t, 256, 4, dtype, seed=t)
    for i, v in enumerate((1e5, 2.0 ** 20, 1e7, 3e9, 1e10, 1e30, 3e38)):
        logits[3 * i, 7] = v
        logits[3 * i, 200] = v
    logits[2, 10:] = -1e10
    logits[5, :255] = -1e30
    loss, counts, d = _run(logits, ids)
    assert bool(loss.isfinite()) and bool(d.isfinite().all())
    _check(logits, ids, None, None, 0.5, None, loss, counts, d)


@pytest.mark.parametrize("t", [50, 1200])
def test_rows_around_large_values(t):
    """fp32 rows about v, on v's own grid and within 16 of the maximum, on both sides of 2^20."""
    logits, _, ids, _ = _inputs(t, 384, 8, torch.float32, seed=3 * t)
    for i, v in enumerate((1e3, -1e4, 5e5, -5e5, 2.0 ** 20 - 20, -(2.0 ** 20), 2.0 ** 20 + 20, 3e6, -1e7, 1e8, -1.2e8)):
        logits[4 * i] += v
    loss, counts, d = _run(logits, ids)
    _check(logits, ids, None, None, 0.5, None, loss, counts, d)


@pytest.mark.parametrize("t", [50, 1200])
def test_a_row_of_nan_alone_is_not_hidden(t):
    """NaN in every expert, or in one beside -inf: the loss and that row's gradient are NaN, the other rows' are not."""
    logits, _, ids, _ = _inputs(t, 48, 3, torch.float32, seed=21)
    for only in (False, True):
        z = logits.clone()
        z[7] = float("nan") if only else -float("inf")
        z[7, 30] = float("nan")
        loss, counts, d = _run(z, ids)
        assert bool(loss.isnan()) and bool(d[7].isnan().all())
        assert bool(d[:7].isfinite().all()) and bool(d[8:].isfinite().all())
