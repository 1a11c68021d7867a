"""Corners of the block's training operators on the GPU (needs a GPU): values that must not reach their
neighbours, against the fp64 definitions.  Tolerances as derived in ``test_gpu_train.py``, whose helpers are
used here.
"""
import numpy as np
import pytest
import torch

from test_gpu_train import C_ROW, HALF, TYPES, U, g, np64, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def close_where_finite(got, ref, major, c, what):
    """NaN in the same places, and ``close`` everywhere else."""
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(np64(got)), nan), f"{what}: NaN in other places than the definition has it"
    half, got = HALF[got.dtype], np.where(nan, 0.0, np64(got))
    ref = np.where(nan, 0.0, ref)
    bad = np.abs(got - ref) > half * np.abs(ref) + c * U * major
    assert not bad.any(), f"{what}: {bad.sum()} out of tolerance"


@pytest.mark.parametrize("dtype", TYPES)
def test_gates_keep_a_nan_in_its_channel(g, dtype):
    """NaN and infinities in single channels of the gates' pre-activations: the gradients of all other
    channels are those of the formula."""
    shape = (1, 40, 2, 64)
    x = [rand(i, *shape, dtype=dtype) for i in range(6)]
    for i in range(3, 6):
        for t, c in ((3, 0), (4, 1), (5, 62), (6, 63), (20, 2 * i)):
            x[i][0, t, i % 2, c] = float("nan")
        x[i][0, 7, 0, 10], x[i][0, 7, 0, 13] = float("inf"), float("-inf")
    d = [rand(10 + i, *shape, dtype=dtype) for i in range(6)]
    conv = [rand(20 + i, 128, 4) for i in range(3)]
    outs = g.block_prologue_bwd(*x, *conv, *d)
    for i in range(3, 6):
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-np64(x[i])))
        ref = (-1.0 if i == 3 else 1.0) * np64(d[i]) * p * (1.0 - p)
        # an infinity shuts its gate: p (1 - p) = 0
        close_where_finite(outs[i], ref, np.where(np.isnan(ref), 0.0, np.abs(ref)), C_ROW, ("xa", "xb", "xw")[i - 3])
