"""Corners of the block's training operators on the GPU (needs a GPU): values that must not reach their
neighbours, against the fp64 definitions.  Tolerances as derived in ``test_gpu_train.py``, whose helpers are
used here.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import block_train as bt
from test_gpu_train import C_ROW, C_SUM, HALF, TYPES, U, conv_major, g, hold, np64, rand  # noqa: F401

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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("ckpt", [False, True])
def test_a_nan_reaches_as_far_as_the_taps(g, dtype, K, ckpt):
    """A NaN in an input moves the gradients of the K - 1 tokens before and after that its taps join, in
    its head alone; with fewer than four taps there is no fourth one that it could pass through."""
    B, T, H, dims = 2, 60, 3, (64, 64, 64, 64, 64, 64)
    x = [rand(i, B, T, H, d, dtype=dtype) for i, d in enumerate(dims)]
    d = [rand(10 + i, B, T, H, n, dtype=dtype) for i, n in enumerate(dims)]
    conv = [rand(20 + i, H * n, K) for i, n in enumerate(dims[:3])]
    for i in range(3):
        x[i][0, 20, 1, 5] = x[i][0, 31, 1, 40] = float("nan")  # first and last token of a run
        x[i][0, T - 1, 0, 7] = float("nan")                    # the next sequence starts afresh
        d[i][1, 9, 2, 63] = d[i][1, T - 1, 1, 0] = float("nan")
    held = [hold(g, t, ckpt) for t in x]
    outs = g.block_prologue_bwd(*[h for h, _ in held], *conv, *d)
    flat = lambda v: v.reshape(B * T, H, -1)  # noqa: E731
    x64, d64, c64 = [flat(v) for _, v in held], [flat(np64(t)) for t in d], [np64(c) for c in conv]
    cu = [0, T, 2 * T]
    refs = bt.block_prologue_bwd(*x64, *c64, *d64, cu_seqlens=cu)
    for i in range(3):
        # what is finite does not depend on the NaN, so the majorants need not either
        mx, mW = conv_major(np.nan_to_num(x64[i], nan=0.0), c64[i], np.nan_to_num(d64[i], nan=0.0), i < 2, cu)
        close_where_finite(flat(outs[i]), refs[i], mx, C_ROW, "xqxkxv"[2 * i:2 * i + 2])
        close_where_finite(outs[6 + i], refs[6 + i], mW, C_SUM, "conv")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_a_nan_reaches_as_far_as_the_taps_forward(g, dtype, K):
    """The forward of the same: tokens more than K - 1 behind a NaN are those of the formula.  Tolerances
    are the forward's own (``test_gpu_block.py``)."""
    B, T, H, d = 2, 60, 3, 64
    x = [rand(i, B, T, H, d, dtype=dtype) for i in range(6)]
    conv = [rand(20 + i, H * d, K) for i in range(3)]
    for t in x[:3]:
        t[0, 20, 1, 5] = t[0, 31, 1, 40] = t[0, T - 1, 0, 7] = float("nan")
    outs = g.block_prologue(*x, *conv)
    for got, ref in zip(outs, oracle.block_prologue(*[np64(t) for t in x], *[np64(c) for c in conv])):
        got, nan = np64(got), np.isnan(ref)
        assert np.array_equal(np.isnan(got), nan)
        err = np.abs(got - ref)[~nan]
        if dtype is torch.float32:
            assert err.max() <= 1e-4 * np.abs(ref[~nan]).max()
        else:
            assert (err <= 1e-2 + 2e-2 * np.abs(ref[~nan])).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dv", [64, 256])
@pytest.mark.parametrize("tokens", [40, 5000])
def test_epilogue_bwd_keeps_a_nan_in_its_row(g, dtype, dv, tokens):
    """Rows lie side by side in a warp; a NaN in o, gate or dy reaches what its row's sums join, its channel
    of the weight's gradient, and nothing else."""
    H = 3
    o, z, dy = (rand(i, tokens, H, dv, dtype=dtype) for i in (1, 2, 3))
    nw = rand(4, dv, scale=0.2, shift=1.0)
    z[5, 1, 9] = dy[7, 0, 30] = float("nan")
    outs = g.block_epilogue_bwd(o, z, nw, dy)
    with_o = o.clone()
    with_o[11, 2, dv - 1] = float("nan")  # the whole row, and so the whole weight's gradient
    outs_o = g.block_epilogue_bwd(with_o, z, nw, dy)
    for o_, got in ((o, outs), (with_o, outs_o)):
        o64, z64, dy64, nw64 = (np64(t) for t in (o_, z, dy, nw))
        refs = bt.block_epilogue_bwd(o64, z64, nw64, dy64)
        o64, z64, dy64 = (np.nan_to_num(t, nan=0.0) for t in (o64, z64, dy64))
        r = 1 / np.sqrt((o64 ** 2).mean(-1, keepdims=True) + bt.RMS_EPS)
        sg = 1 / (1 + np.exp(-z64))
        aoh, s = np.abs(o64) * r, np.abs(z64) * sg
        ae = np.abs(dy64 * nw64) * s
        close_where_finite(got[0], refs[0], r * (ae + aoh * (ae * aoh).mean(-1, keepdims=True)), C_ROW, "do")
        close_where_finite(got[1], refs[1], np.abs(dy64 * nw64) * aoh * (sg + s), C_ROW, "dgate")
        close_where_finite(got[2], refs[2], (np.abs(dy64) * aoh * s).sum((0, 1)), C_SUM, "dnorm_weight")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [64, 100, 513, 2048, 8191])
@pytest.mark.parametrize("tokens", [8, 700])
def test_layer_norm_bwd_keeps_a_nan_in_its_row(g, dtype, width, tokens):
    """A NaN in dy reaches its row's dx and its channel of the weight's and the bias's gradients."""
    h, dy, dh = (rand(i, tokens, width, dtype=dtype) for i in (1, 2, 3))
    w = rand(4, width, scale=0.3, shift=1.0)
    out = g.layer_norm_fwd(h, w)
    dy[3, 17] = dy[6, width - 1] = float("nan")
    got = g.layer_norm_bwd(dy, h, out.mean, out.rstd, w, dh=dh)
    h64, dy64, dh64, w64, mean, rstd = (np64(t) for t in (h, dy, dh, w, out.mean, out.rstd))
    refs = bt.layer_norm_bwd(dy64, h64, mean, rstd, w64, dh64)
    dy64 = np.nan_to_num(dy64, nan=0.0)
    axh, ae = np.abs(h64 - mean[:, None]) * rstd[:, None], np.abs(dy64 * w64)
    major = rstd[:, None] * (ae + ae.mean(-1, keepdims=True) + axh * (ae * axh).mean(-1, keepdims=True)) + np.abs(dh64)
    close_where_finite(got[0], refs[0], major, C_ROW, "dx")
    close_where_finite(got[1], refs[1], (np.abs(dy64) * axh).sum(0), C_SUM, "dweight")
    close_where_finite(got[2], refs[2], np.abs(dy64).sum(0), C_SUM, "dbias")
