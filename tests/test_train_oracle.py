"""Pins of the training oracle (``oracle/block_train.py``; CPU only): its gradients against central
differences and autograd of independent forwards, its 8-bit form against exact properties."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block_train as bt

rng = np.random.default_rng(7)


def _differences(f, x, d, eps=1e-6):
    """d/dx of sum(d * f(x)) by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + eps
        hi = (d * f()).sum()
        x[i] = keep - eps
        lo = (d * f()).sum()
        x[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_layer_norm_is_torchs():
    h, w, b = rng.standard_normal((5, 12)), rng.standard_normal(12), rng.standard_normal(12)
    ref = torch.nn.functional.layer_norm(torch.tensor(h), (12,), torch.tensor(w), torch.tensor(b), 1e-5)
    np.testing.assert_allclose(bt.layer_norm(h, w, b)[0], ref.numpy(), rtol=1e-12, atol=1e-12)


def test_layer_norm_bwd_is_the_difference_quotient():
    h, w, b, dy = (rng.standard_normal(s) for s in ((4, 7), 7, 7, (4, 7)))
    _, mean, rstd = bt.layer_norm(h, w, b)
    dx, dw, db = bt.layer_norm_bwd(dy, h, mean, rstd, w)
    f = lambda: bt.layer_norm(h, w, b)[0]  # noqa: E731
    for got, x in ((dx, h), (dw, w), (db, b)):
        np.testing.assert_allclose(got, _differences(f, x, dy), rtol=1e-6, atol=1e-8)
    dh = rng.standard_normal((4, 7))
    np.testing.assert_allclose(bt.layer_norm_bwd(dy, h, mean, rstd, w, dh)[0], dx + dh, rtol=1e-14)


def test_epilogue_bwd_is_the_difference_quotient_of_the_forward_oracle():
    o, z, g, dy = (rng.standard_normal(s) for s in ((2, 3, 5), (2, 3, 5), 5, (2, 3, 5)))
    f = lambda: oracle.block_epilogue(o, z, g)  # noqa: E731
    for got, x in zip(bt.block_epilogue_bwd(o, z, g, dy), (o, z, g)):
        np.testing.assert_allclose(got, _differences(f, x, dy), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("K", [1, 3, 4])
@pytest.mark.parametrize("cu", [None, [0, 2, 2, 6]])
def test_prologue_bwd_is_the_difference_quotient_of_the_forward_oracle(K, cu):
    lead, H, dk, dv = ((2, 3) if cu is None else (6,)), 2, 2, 3
    dims = (dk, dk, dv, dk, dk, dv)
    x = [rng.standard_normal((*lead, H, d)) for d in dims]
    W = [rng.standard_normal((H * d, K)) for d in (dk, dk, dv)]
    d = [rng.standard_normal(t.shape) for t in x]
    got = bt.block_prologue_bwd(*x, *W, *d, cu_seqlens=cu)
    f = lambda i: (lambda: oracle.block_prologue(*x, *W, cu_seqlens=cu)[i])  # noqa: E731
    for i in range(6):
        np.testing.assert_allclose(got[i], _differences(f(i), x[i], d[i]), rtol=1e-5, atol=1e-7)
    for i in range(3):
        np.testing.assert_allclose(got[6 + i], _differences(f(i), W[i], d[i]), rtol=1e-5, atol=1e-7)


def test_a_planted_mistake_in_the_conv_gradient_is_caught():
    """A gradient that crosses a sequence start differs from the difference quotient."""
    x = [rng.standard_normal((6, 1, 2)) for _ in range(6)]
    W = [rng.standard_normal((2, 4)) for _ in range(3)]
    d = [rng.standard_normal((6, 1, 2)) for _ in range(6)]
    right = bt.block_prologue_bwd(*x, *W, *d, cu_seqlens=[0, 3, 6])
    wrong = bt.block_prologue_bwd(*x, *W, *d, cu_seqlens=[0, 6])
    for i in (0, 1, 2, 6, 7, 8):
        assert np.abs(right[i] - wrong[i]).max() > 1e-3


def test_rows_behind_the_last_sequence_have_no_gradient():
    x = [rng.standard_normal((6, 1, 2)) for _ in range(6)]
    W = [rng.standard_normal((2, 4)) for _ in range(3)]
    d = [rng.standard_normal((6, 1, 2)) for _ in range(6)]
    got = bt.block_prologue_bwd(*x, *W, *d, cu_seqlens=[0, 4])
    cut = bt.block_prologue_bwd(*[t[:4] for t in x], *W, *[t[:4] for t in d], cu_seqlens=[0, 4])
    for i in range(6):
        assert (got[i][4:] == 0).all() and np.array_equal(got[i][:4], cut[i])
    for i in range(6, 9):
        assert np.array_equal(got[i], cut[i])


def test_act8_error_and_scale_are_as_stated():
    x = rng.standard_normal((9, 71)) * 10.0 ** rng.integers(-6, 6, (9, 1))
    codes, scales = bt.act8(x)
    back = bt.act8_values(codes, scales)
    assert np.abs(codes).max() <= 127 and scales.shape == (9, 3)
    unit = np.repeat(2.0 ** (scales - 127.0), 32, -1)[:, :71]
    assert (np.abs(back - x) <= unit / 2).all()
    for g in range(3):  # the next smaller power of two would not hold the group
        top = np.abs(x[:, 32 * g:32 * g + 32]).max(-1)
        assert (top <= 127 * 2.0 ** (scales[:, g] - 127.0)).all()
        assert (top > 127 * 2.0 ** (scales[:, g] - 128.0)).all()


def test_act8_corners():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 2] = 127.0, 0.5, 1.5     # scale 1: ties go to the even code
    codes, scales = bt.act8(x)
    assert scales.tolist() == [[127, 1]] and codes[0, :3].tolist() == [127, 0, 2]
    x[0, 0] = 127.0000001                            # just over: twice the scale
    assert bt.act8(x)[1][0, 0] == 128
    codes, scales = bt.act8(np.array([[3.4028234663852886e38, -1e38]]))  # the largest fp32 stays finite
    assert (codes[0, 0], scales[0, 0]) == (127, 121 + 127)
    assert np.isnan(bt.act8_values(np.zeros((1, 3), int), np.array([[255]]))).all()
