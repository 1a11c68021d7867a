"""fp64 definitions of the block's training operators (numpy), written apart from the CUDA path.

Layer norm and its backward, the backward of the block prologue and epilogue, and activations held in
8 bits.  They are pinned in ``tests/test_train_oracle.py``.
"""
import numpy as np

L2_EPS, RMS_EPS = 1e-6, 1e-5
GROUP = 32


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def _dsilu(y):
    s = _sigmoid(y)
    return s * (1.0 + y * (1.0 - s))


def layer_norm(h, weight, bias=None, eps=1e-5):
    """``(y, mean, rstd)`` over the last dimension of ``h``."""
    h = np.asarray(h, dtype=np.float64)
    mean = h.mean(-1)
    rstd = 1.0 / np.sqrt(((h - mean[..., None]) ** 2).mean(-1) + eps)
    y = (h - mean[..., None]) * rstd[..., None] * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_bwd(dy, h, mean, rstd, weight, dh=None):
    """``(dx, dweight, dbias)`` with the statistics taken as given."""
    xh = (h - mean[..., None]) * rstd[..., None]
    e = dy * weight
    dx = rstd[..., None] * (e - e.mean(-1, keepdims=True) - xh * (e * xh).mean(-1, keepdims=True))
    lead = tuple(range(dy.ndim - 1))
    return (dx if dh is None else dx + dh), (dy * xh).sum(lead), dy.sum(lead)


def block_epilogue_bwd(o, z, g, dy):
    """``(do, dz, dg)`` of y = RMSNorm(o) * g * SiLU(z) over the last dimension."""
    r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + RMS_EPS)
    oh, s = o * r, z * _sigmoid(z)
    e = dy * g * s
    do = r * (e - oh * (e * oh).mean(-1, keepdims=True))
    return do, dy * g * oh * _dsilu(z), (dy * oh * s).sum(tuple(range(o.ndim - 1)))


def _conv_bwd(x, W, d, l2):
    """One sequence of one convolution path: x, d ``[T, H, dim]``; W ``[H, dim, K]``."""
    T, K = x.shape[0], W.shape[-1]
    y = np.zeros_like(x)
    for t in range(T):
        for j in range(min(K, t + 1)):
            y[t] += W[..., K - 1 - j] * x[t - j]
    s = y * _sigmoid(y)
    if l2:
        n = 1.0 / np.sqrt((s * s).sum(-1, keepdims=True) + L2_EPS)
        d = n * d - n ** 3 * s * (s * d).sum(-1, keepdims=True)
    dy = d * _dsilu(y)
    dx, dW = np.zeros_like(x), np.zeros_like(W)
    for t in range(T):
        for j in range(min(K, t + 1)):
            dx[t - j] += W[..., K - 1 - j] * dy[t]
            dW[..., K - 1 - j] += dy[t] * x[t - j]
    return dx, dW


def block_prologue_bwd(xq, xk, xv, xa, xb, xw, Wq, Wk, Wv, dq, dk, dv, da, db, dw, cu_seqlens=None):
    """``(dxq, dxk, dxv, dxa, dxb, dxw, dWq, dWk, dWv)``; layouts as the forward oracle's.  Rows behind
    the last sequence of a packed batch have zero gradients."""
    H = xq.shape[-2]
    shape = xq.shape[:-2]
    if cu_seqlens is None:
        cu = [i * shape[1] for i in range(shape[0] + 1)]
    else:
        cu = [int(c) for c in cu_seqlens]
    flat = lambda t: np.asarray(t, dtype=np.float64).reshape(-1, H, t.shape[-1])  # noqa: E731
    dxs, dWs = [], []
    for x, W, d, l2 in ((xq, Wq, dq, True), (xk, Wk, dk, True), (xv, Wv, dv, False)):
        xf, df = flat(x), flat(d)
        Wf = np.asarray(W, dtype=np.float64).reshape(H, x.shape[-1], -1)
        dx, dW = np.zeros_like(xf), np.zeros_like(Wf)
        for b, e in zip(cu[:-1], cu[1:]):
            if e > b:
                gx, gW = _conv_bwd(xf[b:e], Wf, df[b:e], l2)
                dx[b:e] = gx
                dW += gW
        dxs.append(dx.reshape(x.shape))
        dWs.append(dW.reshape(W.shape))
    for x, d, sign in ((xa, da, -1.0), (xb, db, 1.0), (xw, dw, 1.0)):
        p = _sigmoid(np.asarray(x, dtype=np.float64))
        g = (sign * d * p * (1.0 - p)).reshape(-1, H, x.shape[-1])
        if cu_seqlens is not None:
            g[cu[-1]:] = 0.0
        dxs.append(g.reshape(x.shape))
    return (*dxs, *dWs)


def act8(x):
    """``(codes int, scales int)`` of finite ``x`` (any width; the last group of a row may be short)."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    codes = np.zeros(x.shape, dtype=np.int64)
    scales = np.zeros(x.shape[:-1] + (-(-D // GROUP),), dtype=np.int64)
    for g in range(scales.shape[-1]):
        part = np.clip(x[..., g * GROUP:(g + 1) * GROUP], -127.0 * 2.0 ** 121, 127.0 * 2.0 ** 121)
        top = np.abs(part).max(-1)
        e = np.full(top.shape, -126)
        for k in range(-126, 128):  # the least e that holds the largest value
            e = np.where(127.0 * 2.0 ** (k - 1) < top, k, e) if k > -126 else e
        scales[..., g] = e + 127
        codes[..., g * GROUP:(g + 1) * GROUP] = np.rint(part * 2.0 ** (-e[..., None].astype(np.float64)))
    return codes, scales


def act8_values(codes, scales):
    """The values that codes and scales stand for (NaN where the scale is 255)."""
    scales = np.repeat(np.asarray(scales, dtype=np.int64), GROUP, -1)[..., : codes.shape[-1]]
    unit = np.where(scales == 255, np.nan, 2.0 ** (np.minimum(scales, 254) - 127.0))
    return np.asarray(codes, dtype=np.float64) * unit
