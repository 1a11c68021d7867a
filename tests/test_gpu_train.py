"""The block's training operators on the GPU against their fp64 definitions (needs a GPU).

Tolerances count roundings.  A result that is rounded to bf16 is off by at most 2^-8 |y| for that
(2^-24 |y| for fp32); the fp32 arithmetic before it by at most C * 2^-24 * M, where M is the formula
evaluated with absolute values (so that cancellation is paid for where it happens) and C counts the
roundings on the longest way from an input to the result:
  * C = 64 for what is formed inside a row: at most 16 values per lane are added, then 5 shuffle steps,
    then 16 warps, beside about a dozen products, and the approximate exponential, reciprocal and
    reciprocal root (2 ulp each, the exponential's argument |x| log2 e rounded once: |x| <= 8 here);
  * C = 160 for weight gradients: up to 30 rows or 130 tokens one after another in one register in
    these tests, then every eighth of at most 592 partial sums, then eight.
What is held in 8 bits, and a residual sum, have to be equal.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import gdn2_workloads as W
import oracle
from oracle import block_train as bt

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
C_ROW, C_SUM = 64, 160
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_131_b200 as gdn2
    gdn2.lib()
    return gdn2


def np64(t):
    return t.double().cpu().numpy()


def close(got, ref, major, c, what):
    half = HALF[got.dtype]
    got = np64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= half * np.abs(ref) + c * U * major)
    worst = np.max(np.abs(got - ref) / (half * np.abs(ref) + c * U * major + 1e-300))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance, worst {worst:.2f} of the bound"


def rand(seed, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale + shift).to(dtype).cuda()


def hold(g, x, ckpt):
    """``x`` as it is handed over, and the fp64 values it stands for."""
    if not ckpt:
        return x, np64(x)
    a = g.act_pack(x)
    return a, bt.act8_values(a.codes.cpu().numpy(), a.scales.cpu().numpy())


# ------------------------------------------------------------------------------ activations in 8 bits

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1,), (5, 1), (3, 31), (2, 3, 32), (7, 33), (4, 40), (5, 72), (9, 130), (3, 1001),
                                   (17, 2048), (2, 5, 3, 64), (300, 4104), (1, 128)])
def test_act8_codes_scales_and_values(g, dtype, shape):
    x = rand(3, *shape, dtype=dtype) * (10.0 ** rand(4, *shape[:-1], 1).round()).to(dtype)
    a = g.act_pack(x)
    codes, scales = bt.act8(np64(x))
    assert np.array_equal(a.codes.cpu().numpy(), codes) and np.array_equal(a.scales.cpu().numpy(), scales)
    back = bt.act8_values(codes, scales)
    for dt in TYPES:
        assert np.array_equal(np64(g.act_unpack(a, dtype=dt)), back)


def test_act8_many_tensors_of_different_widths_in_one_call(g):
    shapes = [(3, 64), (0, 64), (5, 33), (2, 40), (1, 1), (4, 2, 256), (1000, 31), (64, 8192)]
    xs = [rand(10 + i, *s, dtype=torch.bfloat16) for i, s in enumerate(shapes)]
    acts = g.act_pack(xs)
    for x, a, v in zip(xs, acts, g.act_unpack(acts)):
        one = g.act_pack(x)
        assert torch.equal(a.codes, one.codes) and torch.equal(a.scales, one.scales)
        assert np.array_equal(np64(v), bt.act8_values(a.codes.cpu().numpy(), a.scales.cpu().numpy()))


@pytest.mark.parametrize("width", [64, 40, 37])
def test_act8_extremes(g, width):
    """Zeros, the type's smallest and largest values, ties, infinities and NaN: only the group that holds
    an infinity or a NaN reads back as NaN."""
    x = torch.zeros(8, width)
    x[1, 0], x[1, 1] = 3.4028234663852886e38, -1e37
    x[2, 0], x[2, 1] = 1e-45, -2.0 ** -126
    x[3, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    x[4, 0] = 127.5
    x[5, 1], x[6, 2], x[7, width - 1] = float("inf"), float("nan"), float("-inf")
    a = g.act_pack(x.cuda())
    codes, scales = a.codes.cpu().numpy(), a.scales.cpu().numpy()
    finite = x.numpy()[:5].astype(np.float64)
    rc, rs = bt.act8(finite)
    assert np.array_equal(codes[:5], rc) and np.array_equal(scales[:5], rs)
    for row, col in ((5, 1), (6, 2), (7, width - 1)):
        assert scales[row, col // 32] == 255 and (np.delete(scales[row], col // 32) == 1).all()
        assert (codes[row] == 0).all()
    for dt in TYPES:
        v = np64(g.act_unpack(a, dtype=dt))
        assert np.array_equal(v, bt.act8_values(codes, scales), equal_nan=True)
        assert np.isnan(v[5, :32]).all() and not np.isnan(v[5, 32:]).any()


# ------------------------------------------------------------------------------------------ layer norm

WIDTHS = [1, 7, 32, 64, 100, 513, 1001, 1024, 2048, 2056, 5000, 8191, 8192]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("residual,bias", [(False, True), (True, False)])
def test_layer_norm_fwd(g, dtype, width, residual, bias):
    tokens = 37
    x = rand(1, tokens, width, dtype=dtype, shift=0.7)
    r = rand(2, tokens, width, dtype=dtype, scale=3.0) if residual else None
    w = rand(3, width, scale=0.2, shift=1.0)
    b = rand(4, width) if bias else None
    out = g.layer_norm_fwd(x, w, b, residual=r, checkpoint=True)
    h = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(out.h, h)
    h64, w64 = np64(h), np64(w)
    y, mean, rstd = bt.layer_norm(h64, w64, None if b is None else np64(b))
    am = np.abs(h64).mean(-1)
    close(out.mean, mean, am, C_ROW, "mean")
    # mean is off by C U am: that moves (h - mean)^2's average by 2 C U am |h - mean| at most
    spread = np.abs(h64 - mean[:, None]).mean(-1)
    close(out.rstd, rstd, rstd * (1 + rstd ** 2 * am * spread), C_ROW, "rstd")
    major = rstd[:, None] * np.abs(w64) * (am[:, None] + np.abs(h64 - mean[:, None]) * (1 + rstd ** 2 * am * spread)[:, None])
    close(out.y, y, major + (0 if b is None else np.abs(np64(b))), C_ROW, "y")
    rc, rs = bt.act8(h64)
    assert np.array_equal(out.checkpoint.codes.cpu().numpy(), rc)
    assert np.array_equal(out.checkpoint.scales.cpu().numpy(), rs)
    bare = g.layer_norm_fwd(x, w, b, residual=r, stats=False)
    assert torch.equal(bare.y, out.y) and bare.mean is None and bare.rstd is None and bare.checkpoint is None


@pytest.mark.parametrize("tokens", [0, 1, 2])
def test_layer_norm_few_rows_and_leading_shapes(g, tokens):
    x, w = rand(1, tokens, 3, 64), rand(2, 64)
    out = g.layer_norm_fwd(x, w)
    assert out.y.shape == x.shape and out.mean.shape == (tokens, 3)
    flat = g.layer_norm_fwd(x.reshape(-1, 64), w)
    assert torch.equal(out.y.reshape(-1, 64), flat.y)
    dx, dw, db = g.layer_norm_bwd(x, out.h, out.mean, out.rstd, w)
    assert dx.shape == x.shape and dw.shape == db.shape == (64,)
    if tokens == 0:
        assert (dw == 0).all() and (db == 0).all()


def test_layer_norm_constant_row_and_a_row_with_nan(g):
    x, w, b = rand(1, 5, 96), rand(2, 96), rand(3, 96)
    x[1] = 4.0
    x[3, 7] = float("nan")
    out = g.layer_norm_fwd(x, w, b, checkpoint=True)
    assert torch.equal(out.y[1], b)  # no deviation: the bias alone
    assert torch.isnan(out.y[3]).all()
    keep = [0, 1, 2, 4]
    clean = g.layer_norm_fwd(x[keep].contiguous(), w, b)
    assert torch.equal(out.y[keep], clean.y)
    assert out.checkpoint.scales[3].tolist()[0] == 255 and out.checkpoint.scales[3].tolist()[1] != 255


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("ckpt,along", [(False, True), (True, False), (True, True)])
def test_layer_norm_bwd(g, dtype, width, ckpt, along, tokens=149):
    h = rand(1, tokens, width, dtype=dtype, shift=0.5)
    dy = rand(2, tokens, width, dtype=dtype)
    dh = rand(3, tokens, width, dtype=dtype) if along else None
    w = rand(4, width, scale=0.3, shift=1.0)
    out = g.layer_norm_fwd(h, w)
    held, h64 = hold(g, h, ckpt)
    dx, dw, db = g.layer_norm_bwd(dy, held, out.mean, out.rstd, w, dh=dh)
    mean, rstd, w64, dy64 = np64(out.mean), np64(out.rstd), np64(w), np64(dy)
    rx, rw, rb = bt.layer_norm_bwd(dy64, h64, mean, rstd, w64, None if dh is None else np64(dh))
    axh = np.abs(h64 - mean[:, None]) * rstd[:, None]
    ae = np.abs(dy64 * w64)
    major = rstd[:, None] * (ae + ae.mean(-1, keepdims=True) + axh * (ae * axh).mean(-1, keepdims=True))
    close(dx, rx, major + (0 if dh is None else np.abs(np64(dh))), C_ROW, "dx")
    close(dw, rw, (np.abs(dy64) * axh).sum(0), C_SUM, "dweight")
    close(db, rb, np.abs(dy64).sum(0), C_SUM, "dbias")
    again = g.layer_norm_bwd(dy, held, out.mean, out.rstd, w, dh=dh)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))  # sums in a fixed order
    assert g.layer_norm_bwd(dy, held, out.mean, out.rstd, w, dh=dh, want_dbias=False)[2] is None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,tokens", [(w, t) for w in (1, 37, 1001, 2048, 8192) for t in (1, 7, 8, 9)]
                         + [(64, 17), (64, 127), (64, 128), (64, 129), (256, 31), (256, 32), (256, 33), (1024, 8)])
def test_layer_norm_bwd_of_few_rows(g, dtype, width, tokens):
    """Either side of the sizes that one cluster of blocks does in a single launch."""
    if width > 1:  # a row of one value has no variance
        test_layer_norm_bwd(g, dtype, width, tokens % 2 == 0, tokens % 3 != 0, tokens)
    else:
        dy, h, one = rand(1, tokens, 1, dtype=dtype), rand(2, tokens, 1, dtype=dtype), torch.ones(tokens, device="cuda")
        dw, db = g.layer_norm_bwd(dy, h, 0 * one, one, rand(3, 1))[1:]
        close(dw, (np64(dy) * np64(h)).sum(0), np.abs(np64(dy) * np64(h)).sum(0), C_SUM, "dweight")
        close(db, np64(dy).sum(0), np.abs(np64(dy)).sum(0), C_SUM, "dbias")


def off16(t):
    """A copy of ``t`` that starts on a 16-byte boundary and on no 32-byte one."""
    buf = torch.empty(t.numel() + 16 // t.element_size(), dtype=t.dtype, device=t.device)
    v = buf[16 // t.element_size():].view(t.shape)
    assert v.data_ptr() % 32 == 16
    return v.copy_(t)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [512, 2048, 8192])
@pytest.mark.parametrize("ckpt", [False, True])
def test_layer_norm_on_16_byte_boundaries(g, dtype, width, ckpt):
    """Rows that would move in 32-byte vectors, on pointers that forbid it."""
    tokens = 300
    h, dy, dh = (off16(rand(i, tokens, width, dtype=dtype)) for i in (1, 2, 3))
    w = off16(rand(4, width, scale=0.3, shift=1.0))
    out = g.layer_norm_fwd(h, w, off16(rand(5, width)), residual=dh)
    ref = g.layer_norm_fwd(h.clone(), w.clone(), rand(5, width), residual=dh.clone())
    assert torch.equal(out.y, ref.y) and torch.equal(out.h, ref.h) and torch.equal(out.rstd, ref.rstd)
    held, h64 = hold(g, h, ckpt)
    if ckpt:
        held = g.Act8(off16(held.codes), off16(held.scales))
    n = g.layer_norm_fwd(h, w)
    dx, dw, db = g.layer_norm_bwd(dy, held, n.mean, n.rstd, w, dh=dh)
    mean, rstd, w64, dy64 = np64(n.mean), np64(n.rstd), np64(w), np64(dy)
    rx, rw, rb = bt.layer_norm_bwd(dy64, h64, mean, rstd, w64, np64(dh))
    axh, ae = np.abs(h64 - mean[:, None]) * rstd[:, None], np.abs(dy64 * w64)
    major = rstd[:, None] * (ae + ae.mean(-1, keepdims=True) + axh * (ae * axh).mean(-1, keepdims=True))
    close(dx, rx, major + np.abs(np64(dh)), C_ROW, "dx")
    close(dw, rw, (np.abs(dy64) * axh).sum(0), C_SUM, "dweight")
    close(db, rb, np.abs(dy64).sum(0), C_SUM, "dbias")


def test_layer_norm_gradient_against_differences(g):
    """fp32: the gradient along a random direction, against central differences of the fp64 forward."""
    h, w, b, dy = rand(1, 23, 200), rand(2, 200), rand(3, 200), rand(4, 23, 200)
    out = g.layer_norm_fwd(h, w, b)
    grads = g.layer_norm_bwd(dy, out.h, out.mean, out.rstd, w)
    dirs = [rand(5, 23, 200), rand(6, 200), rand(7, 200)]
    args = [np64(t) for t in (h, w, b)]
    f = lambda s: (np64(dy) * bt.layer_norm(*[a + s * np64(d) for a, d in zip(args, dirs)])[0]).sum()  # noqa: E731
    want = (f(1e-5) - f(-1e-5)) / 2e-5
    got = sum((np64(p) * np64(d)).sum() for p, d in zip(grads, dirs))
    scale = sum((np.abs(np64(p)) * np.abs(np64(d))).sum() for p, d in zip(grads, dirs))
    assert abs(got - want) <= 1e-6 * scale


def test_layer_norm_in_place(g):
    """h over x or the residual, y over the other; dx over dy or dh."""
    L, tokens, width = g.lib(), 33, 1000
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    x, r, w = rand(1, tokens, width, dtype=torch.bfloat16), rand(2, tokens, width, dtype=torch.bfloat16), rand(3, width)
    out = g.layer_norm_fwd(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    assert L.gdn2_layer_norm_fwd(ptr(x2), ptr(r2), ptr(w), None, 1e-5, ptr(x2), ptr(r2), None, None, None, None, tokens,
                                 width, g.GDN2_BF16, s) == g.GDN2_OK
    assert torch.equal(x2, out.y) and torch.equal(r2, out.h)
    dy, dh = rand(4, tokens, width, dtype=torch.bfloat16), rand(5, tokens, width, dtype=torch.bfloat16)
    ref = g.layer_norm_bwd(dy, out.h, out.mean, out.rstd, w, dh=dh)
    for over in range(2):
        bufs, dw = [dy.clone(), dh.clone()], torch.empty(width, device="cuda")
        assert L.gdn2_layer_norm_bwd(ptr(bufs[0]), ptr(out.h), None, ptr(out.mean), ptr(out.rstd), ptr(w), ptr(bufs[1]),
                                     ptr(bufs[over]), ptr(dw), None, tokens, width, g.GDN2_BF16, s) == g.GDN2_OK
        assert torch.equal(bufs[over], ref[0]) and torch.equal(dw, ref[1])


# -------------------------------------------------------------------------------------- block epilogue

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dv", [64, 128, 256])
@pytest.mark.parametrize("tokens,H", [(1, 1), (77, 3), (1030, 2)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_epilogue_bwd(g, dtype, dv, tokens, H, ckpt):
    o, z, dy = (rand(i, tokens, H, dv, dtype=dtype, scale=s) for i, s in ((1, 0.5), (2, 1.0), (3, 1.0)))
    nw = rand(4, dv, scale=0.2, shift=1.0)
    (oh_, o64), (zh, z64) = hold(g, o, ckpt), hold(g, z, ckpt)
    do, dz, dg = g.block_epilogue_bwd(oh_, zh, nw, dy)
    dy64, nw64 = np64(dy), np64(nw)
    ro, rz, rg = bt.block_epilogue_bwd(o64, z64, nw64, dy64)
    r = 1 / np.sqrt((o64 ** 2).mean(-1, keepdims=True) + bt.RMS_EPS)
    aoh, s = np.abs(o64) * r, np.abs(z64) / (1 + np.exp(-z64))
    ae = np.abs(dy64 * nw64) * s
    close(do, ro, r * (ae + aoh * (ae * aoh).mean(-1, keepdims=True)), C_ROW, "do")
    sg = 1 / (1 + np.exp(-z64))
    close(dz, rz, np.abs(dy64 * nw64) * aoh * (sg + s), C_ROW, "dgate")
    close(dg, rg, (np.abs(dy64) * aoh * s).sum((0, 1)), C_SUM, "dnorm_weight")
    again = g.block_epilogue_bwd(oh_, zh, nw, dy)
    assert all(torch.equal(p, q) for p, q in zip((do, dz, dg), again))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dv,rows", [(64, (255, 513, 1024, 1025)), (128, (33, 256, 257, 512, 513)),
                                     (256, (9, 128, 129, 256, 257))])
def test_epilogue_bwd_of_few_rows(g, dtype, dv, rows):
    """Either side of the sizes that one cluster of blocks does in a single launch."""
    for n in rows:
        test_epilogue_bwd(g, dtype, dv, n, 1, n % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ckpt", [False, True])
def test_block_backwards_on_16_byte_boundaries(g, dtype, ckpt):
    """The same results on pointers that are 16-byte but not 32-byte aligned."""
    hand = (lambda t: g.Act8(*[off16(p) for p in g.act_pack(t)])) if ckpt else off16
    held = g.act_pack if ckpt else (lambda t: t)
    o, z, dy = (rand(i, 130, 3, 128, dtype=dtype) for i in (1, 2, 3))
    nw = rand(4, 128)
    for p, q in zip(g.block_epilogue_bwd(hand(o), hand(z), off16(nw), off16(dy)),
                    g.block_epilogue_bwd(held(o), held(z), nw, dy)):
        assert torch.equal(p, q)
    t = [rand(10 + i, 2, 60, 2, 64, dtype=dtype) for i in range(12)]
    conv = [rand(30 + i, 128, 4) for i in range(3)]
    for p, q in zip(g.block_prologue_bwd(*[hand(x) for x in t[:6]], *[off16(c) for c in conv], *[off16(d) for d in t[6:]]),
                    g.block_prologue_bwd(*[held(x) for x in t[:6]], *conv, *t[6:])):
        assert torch.equal(p, q)


def test_epilogue_bwd_without_tokens_zero_rows_and_far_gates(g):
    nw = rand(1, 64)
    e = torch.empty(0, 2, 64, device="cuda")
    do, dz, dg = g.block_epilogue_bwd(e, e, nw, e)
    assert do.shape == dz.shape == (0, 2, 64) and (dg == 0).all()
    o, z, dy = rand(2, 6, 1, 64), rand(3, 6, 1, 64), rand(4, 6, 1, 64)
    o[1] = 0.0                          # no norm to speak of: eps under the root
    z[2], z[3] = 200.0, -200.0          # gates fully open and shut
    do, dz, dg = g.block_epilogue_bwd(o, z, nw, dy)
    with np.errstate(over="ignore"):
        ro, rz, rg = bt.block_epilogue_bwd(*[np64(t) for t in (o, z, nw, dy)])
    assert torch.isfinite(do).all() and torch.isfinite(dz).all() and torch.isfinite(dg).all()
    # the longest row: |do| up to 1/sqrt(eps) * |dy nw s|; 64 roundings of the largest value bound all
    for got, ref in ((do, ro), (dz, rz), (dg, rg)):
        assert np.abs(np64(got) - ref).max() <= C_SUM * U * np.abs(ref).max() * 64
    assert (do[3].abs() <= 1e-30).all()


def test_epilogue_bwd_in_place(g):
    L, tokens, H, dv = g.lib(), 50, 2, 128
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    o, z, dy = (rand(i, tokens, H, dv, dtype=torch.bfloat16) for i in (1, 2, 3))
    nw, dg = rand(4, dv), torch.empty(dv, device="cuda")
    ref = g.block_epilogue_bwd(o, z, nw, dy)
    o2, z2 = o.clone(), z.clone()
    assert L.gdn2_block_epilogue_bwd(ptr(o2), ptr(z2), None, None, ptr(nw), ptr(dy), ptr(o2), ptr(z2), ptr(dg), tokens,
                                     H, dv, g.GDN2_BF16, s) == g.GDN2_OK
    assert torch.equal(o2, ref[0]) and torch.equal(z2, ref[1]) and torch.equal(dg, ref[2])


# -------------------------------------------------------------------------------------- block prologue

PRE = ("xq", "xk", "xv", "xa", "xb", "xw")
CONV = ("conv_q", "conv_k", "conv_v")


def lagged(x, j):
    """x_{t-j} of one sequence, zero before its start."""
    out = np.zeros_like(x)
    if j < x.shape[0]:
        out[j:] = x[:x.shape[0] - j]
    return out


def conv_major(x, Wt, d, l2, cu):
    """Majorants of dx and dW of one convolution path (flat rows): a rounding of y counts through
    SiLU' (at most 1.1) and SiLU'' (at most 0.5), and through the norm's sums with |s| <= conv |x|."""
    H, dim = x.shape[-2:]
    w = Wt.reshape(H, dim, -1)
    K = w.shape[-1]
    taps = [w[..., K - 1 - j] for j in range(K)]
    mx, mW = np.zeros_like(x), np.zeros_like(w)
    for b, e in zip(cu[:-1], cu[1:]):
        X, D = x[b:e], np.abs(d[b:e])
        ya = sum(np.abs(taps[j] * lagged(X, j)) for j in range(K))
        if l2:
            y = sum(taps[j] * lagged(X, j) for j in range(K))
            s = y / (1 + np.exp(-y))
            n = 1 / np.sqrt((s * s).sum(-1, keepdims=True) + bt.L2_EPS)
            grow = 1 + n ** 2 * (ya * ya).sum(-1, keepdims=True)
            D = (n * D + n ** 3 * ya * (ya * D).sum(-1, keepdims=True)) * grow
        dy = D * (1.1 + ya)
        for j in range(min(K, e - b)):
            mx[b:e - j] += (np.abs(taps[j]) * dy)[j:]
            mW[..., K - 1 - j] += (dy * np.abs(lagged(X, j))).sum(0)
    return mx, mW.reshape(-1, K)


def prologue_case(g, wl, K, seed, ckpt, lengths=None, pad=0):
    d = W.block_inputs(wl, device="cuda", seed=seed, conv_len=K, lengths=lengths)
    x = [d[n] for n in PRE]
    if pad:  # rows behind the last sequence
        x = [torch.cat([t, torch.full((pad, *t.shape[1:]), float("nan"), device="cuda", dtype=t.dtype)]) for t in x]
    dt = x[0].dtype
    grads = [rand(100 + i, *t.shape, dtype=dt) for i, t in enumerate(x)]
    held = [hold(g, t, ckpt) for t in x]
    conv = [d[n] for n in CONV]
    outs = g.block_prologue_bwd(*[h for h, _ in held], *conv, *grads, cu_seqlens=d["cu_seqlens"])
    torch.cuda.synchronize()
    H = x[0].shape[-2]
    tokens = x[0].shape[:-2].numel() - pad
    cu = [i * x[0].shape[1] for i in range(x[0].shape[0] + 1)] if d["cu_seqlens"] is None else d["cu_seqlens"].tolist()
    flat = lambda t: t.reshape(-1, H, t.shape[-1])[:tokens]  # noqa: E731
    x64, g64, c64 = [flat(v) for _, v in held], [flat(np64(t)) for t in grads], [np64(c) for c in conv]
    refs = bt.block_prologue_bwd(*x64, *c64, *g64, cu_seqlens=cu)
    for i in range(3):
        mx, mW = conv_major(x64[i], c64[i], g64[i], i < 2, cu)
        close(flat(outs[i]), refs[i], mx, C_ROW, PRE[i])
        close(outs[6 + i], refs[6 + i], mW, C_SUM, CONV[i])
    for i in range(3, 6):
        close(flat(outs[i]), refs[i], np.abs(refs[i]), C_ROW, PRE[i])
    again = g.block_prologue_bwd(*[h for h, _ in held], *conv, *grads, cu_seqlens=d["cu_seqlens"])
    for p, q in zip(outs, again):
        p, q = (flat(t) if t.dim() > 2 else t for t in (p, q))
        assert torch.equal(p, q)
    return d, held, grads, outs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("ckpt", [False, True])
def test_prologue_bwd_dense(g, dtype, K, ckpt):
    wl = W.Workload("train_dense", B=2, T=83, H=3, dk=128, dv=256, dtype=dtype)
    prologue_case(g, wl, K, 61, ckpt)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 256), (128, 64)])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("pad", [0, 9])
def test_prologue_bwd_packed(g, dk, dv, ckpt, pad):
    lengths = [1, 70, 0, 64, 1, 1, 0, 0, 131, 2, 3, 5]
    wl = W.Workload("train_packed", B=len(lengths), T=256, H=1, dk=dk, dv=dv, varlen=True)
    prologue_case(g, wl, 4, 62, ckpt, lengths=lengths, pad=pad)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
def test_prologue_bwd_short_sequences(g, T):
    wl = W.Workload("train_short", B=5, T=T, H=2, dk=64, dv=64, dtype="f32")
    prologue_case(g, wl, 4, 63, False)


def test_prologue_bwd_long_runs(g):
    """Enough tokens that every lane walks many batches, sequences ending inside runs and at their ends."""
    lengths = [4001, 96, 0, 2500, 1, 3000, 31]
    wl = W.Workload("train_runs", B=len(lengths), T=4096, H=8, dk=64, dv=64, varlen=True)
    prologue_case(g, wl, 4, 64, True, lengths=lengths)


def test_prologue_bwd_leaves_rows_behind_the_last_sequence(g):
    """Through the C ABI: guard bands around every output and the padded rows keep their content."""
    L, tokens, pad, H, dk, dv, K = g.lib(), 45, 6, 2, 64, 128, 4
    dims, dt, canary = (dk, dk, dv, dk, dk, dv), torch.bfloat16, -777.0
    x = [rand(i, tokens + pad, H, d, dtype=dt) for i, d in enumerate(dims)]
    gr = [rand(10 + i, tokens + pad, H, d, dtype=dt) for i, d in enumerate(dims)]
    conv = [rand(20 + i, H * d, K) for i, d in enumerate(dims[:3])]
    cu = torch.tensor([0, 20, tokens], dtype=torch.int32, device="cuda")
    band = 4096
    bufs = [torch.full((2 * band + t.numel(),), canary, device="cuda", dtype=t.dtype) for t in x]
    cbufs = [torch.full((2 * band + t.numel(),), canary, device="cuda") for t in conv]
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    outs = [b[band:band + t.numel()] for b, t in zip(bufs + cbufs, x + conv)]
    assert L.gdn2_block_prologue_bwd(*[ptr(t) for t in x], None, *[ptr(t) for t in conv], *[ptr(t) for t in gr],
                                     *[ptr(t) for t in outs], 2, tokens + pad, H, dk, dv, K, ptr(cu), g.GDN2_BF16,
                                     s) == g.GDN2_OK
    torch.cuda.synchronize()
    for b, t in zip(bufs + cbufs, outs):
        assert (b[:band] == canary).all() and (b[band + t.numel():] == canary).all()
    for t, d in zip(outs[:6], dims):
        rows = t.view(tokens + pad, H * d)
        assert (rows[tokens:] == canary).all() and not (rows[:tokens] == canary).any()


def test_prologue_bwd_without_tokens(g):
    x = [torch.empty(0, 2, 64, device="cuda") for _ in range(6)]
    conv = [rand(i, 128, 4) for i in range(3)]
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    outs = g.block_prologue_bwd(*x, *conv, *x, cu_seqlens=cu)
    assert all((t == 0).all() for t in outs[6:]) and all(t.shape == (0, 2, 64) for t in outs[:6])
    # tokens, but all of them behind the (empty) sequences
    x = [rand(i, 5, 2, 64) for i in range(6)]
    outs = g.block_prologue_bwd(*x, *conv, *x, cu_seqlens=cu)
    assert all((t == 0).all() for t in outs[6:])


# ----------------------------------------------------------------------------------- all of them together

def block_step(g, p, dtype, ckpt):
    """One training step of a block: norm, projections, mixer, gate, output projection, and back.
    Returns the loss's inputs' gradients; ``p`` holds the weights, the input and dL/dout."""
    B, T, H, d = p["shape"]
    D = H * d
    mm = lambda a, b: a.reshape(-1, a.shape[-1]) @ b  # noqa: E731
    heads = lambda t: t.reshape(B, T, H, d)  # noqa: E731
    n = g.layer_norm_fwd(p["x"], p["nw"], p["nb"], residual=p["r"], checkpoint=ckpt)
    pre = [heads(mm(n.y, w)).contiguous() for w in p["proj"]]   # xq xk xv xa xb xw z
    tok = g.block_prologue(*pre[:6], *p["conv"])
    o, _ = g.chunk_fwd(*tok)
    y = g.block_epilogue(o, pre[6], p["gw"])
    out = mm(y.reshape(B, T, D), p["wo"]).reshape(B, T, D) + n.h
    saved = dict(h=n.checkpoint, pre=g.act_pack(pre), o=g.act_pack(o)) if ckpt else dict(h=n.h, pre=pre, o=o)
    # backward
    dout = p["dout"]
    dyf = mm(dout, p["wo"].t())
    do, dz, dgw = g.block_epilogue_bwd(saved["o"], saved["pre"][6], p["gw"], heads(dyf).contiguous())
    if ckpt:  # q .. w formed again from the checkpoints
        tok = g.block_prologue(*g.act_unpack(saved["pre"][:6], dtype=dtype), *p["conv"])
    dtok = g.chunk_bwd(*tok, do, want_dS0=False)[:6]
    dpre = g.block_prologue_bwd(*saved["pre"][:6], *p["conv"], *dtok)
    dy = sum(mm(t.reshape(B, T, D), w.t()) for t, w in zip([*dpre[:6], dz], p["proj"])).reshape(B, T, D).contiguous()
    dx, dnw, dnb = g.layer_norm_bwd(dy, saved["h"], n.mean, n.rstd, p["nw"], dh=dout)
    return out, dict(x=dx, nw=dnw, nb=dnb, conv=dpre[6:], gw=dgw)


def block_params(dtype, seed=0, shape=(2, 70, 2, 64)):
    B, T, H, d = shape
    D = H * d
    p = dict(shape=shape, x=rand(seed, B, T, D, dtype=dtype), r=rand(seed + 1, B, T, D, dtype=dtype),
             nw=rand(seed + 2, D, scale=0.1, shift=1.0), nb=rand(seed + 3, D, scale=0.1),
             proj=[rand(seed + 4 + i, D, D, dtype=dtype, scale=D ** -0.5) for i in range(7)],
             conv=[rand(seed + 20 + i, D, 4, scale=0.5) for i in range(3)], gw=rand(seed + 30, d, scale=0.1, shift=1.0),
             wo=rand(seed + 31, D, D, dtype=dtype, scale=D ** -0.5), dout=rand(seed + 32, B, T, D, dtype=dtype))
    return p


def block_loss64(p, moved):
    """sum(dout * out) of the block in fp64 through the oracles, the named inputs replaced."""
    B, T, H, d = p["shape"]
    D = H * d
    q = {k: np64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    q.update({k: [np64(t) for t in p[k]] for k in ("proj", "conv")})
    q.update(moved)
    h = q["x"] + q["r"]
    y, _, _ = bt.layer_norm(h, q["nw"], q["nb"])
    pre = [(y.reshape(-1, D) @ w).reshape(B, T, H, d) for w in q["proj"]]
    tok = oracle.block_prologue(*pre[:6], *q["conv"])
    o, _ = oracle.recurrent(*tok)
    e = oracle.block_epilogue(o, pre[6], q["gw"])
    return (q["dout"] * ((e.reshape(-1, D) @ q["wo"]).reshape(B, T, D) + h)).sum()


def test_block_training_step_against_differences(g):
    """fp32: every gradient of the whole chain along a random direction, against central differences of
    the fp64 chain.  The chain's fp32 products and sums stay under 2^-24 times a few hundred; the
    differences' own error (step 1e-5, third derivatives of order 10) is under 1e-8."""
    p = block_params(torch.float32)
    torch.backends.cuda.matmul.allow_tf32 = False
    _, grads = block_step(g, p, torch.float32, False)
    for name, got in (("x", grads["x"]), ("nw", grads["nw"]), ("nb", grads["nb"]), ("gw", grads["gw"]),
                      ("conv", grads["conv"])):
        many = isinstance(got, tuple)
        gs = [np64(t) for t in (got if many else [got])]
        base = [np64(t) for t in (p[name] if many else [p[name]])]
        dirs = [np64(rand(77 + i, *t.shape)) for i, t in enumerate(gs)]
        moved = lambda s: {name: [b + s * v for b, v in zip(base, dirs)] if many else base[0] + s * dirs[0]}  # noqa: E731,B023
        want = (block_loss64(p, moved(1e-5)) - block_loss64(p, moved(-1e-5))) / 2e-5
        have = sum((a * v).sum() for a, v in zip(gs, dirs))
        size = np.sqrt(sum(((a * v) ** 2).sum() for a, v in zip(gs, dirs)))
        assert abs(have - want) <= 2e-4 * size, (name, have, want, size)


def test_block_training_step_from_checkpoints(g):
    """From 8-bit checkpoints the gradients differ from those of the saved activations by what the
    checkpoints' rounding moves them: under 1/126 of a group's largest value each, so their directions
    agree closely."""
    p = block_params(torch.bfloat16)
    out, full = block_step(g, p, torch.bfloat16, False)
    out8, held = block_step(g, p, torch.bfloat16, True)
    assert torch.equal(out, out8)  # the forward is the same
    for name in full:
        a, b = ([np64(t).ravel() for t in (v if isinstance(v, tuple) else [v])] for v in (full[name], held[name]))
        a, b = np.concatenate(a), np.concatenate(b)
        cos = (a * b).sum() / np.sqrt((a * a).sum() * (b * b).sum())
        assert cos > 0.99, (name, cos)


# --------------------------------------------------------------------- streams, graphs, sizes past 2^31

def _calls(g):
    """Each backward call on inputs of its own, as closures that return their outputs; the short ones
    (one launch of one cluster) beside the others."""
    bf = torch.bfloat16
    x, w = rand(1, 300, 1000, dtype=bf), rand(2, 1000)
    n = g.layer_norm_fwd(x, w)
    o, z, dy, nw = *(rand(3 + i, 90, 4, 128, dtype=bf) for i in range(3)), rand(7, 128)
    pre = [rand(10 + i, 2, 60, 2, 64, dtype=bf) for i in range(12)]
    conv = [rand(30 + i, 128, 4) for i in range(3)]
    acts = g.act_pack(pre[:6])
    def norm(**k):
        out = g.layer_norm_fwd(x, w, checkpoint=True, **k)
        return [out.y, out.mean, out.rstd, *out.checkpoint]  # (out.h is x itself)

    return [norm,
            lambda **k: list(g.layer_norm_bwd(x, n.h, n.mean, n.rstd, w, **k)),
            lambda **k: list(g.layer_norm_bwd(x[:7], n.h[:7], n.mean[:7], n.rstd[:7], w, **k)),
            lambda **k: list(g.block_epilogue_bwd(o[:11], z[:11], nw, dy[:11], **k)),
            lambda **k: list(g.block_epilogue_bwd(o, z, nw, dy, **k)),
            lambda **k: list(g.block_prologue_bwd(*pre[:6], *conv, *pre[6:], **k)),
            lambda **k: list(g.block_prologue_bwd(*acts, *conv, *pre[6:], **k)),
            lambda **k: g.act_unpack(g.act_pack(pre[:6], **k), **k)]


def test_calls_on_two_other_streams_at_once(g):
    calls = _calls(g)
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[c(stream=s) for c in calls for _ in range(5)] for s in streams]
    torch.cuda.synchronize()
    for per in outs:
        for i, got in enumerate(per):
            assert all(torch.equal(a, b) for a, b in zip(got, refs[i // 5]))


def test_calls_from_two_threads_at_once(g):
    calls = _calls(g)
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    outs = [[], []]

    def work(out):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out.append([c() for c in calls])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(out,)) for out in outs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for out in outs:
        assert len(out) == 20
        for turn in out:
            for got, ref in zip(turn, refs):
                assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_captured_calls_replay(g):
    """Two graphs with workspaces of their own, replayed in turn and at once on two streams."""
    calls = _calls(g)
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append([c() for c in calls])
        graphs.append(gr)
    for per in outs:
        for got in per:
            for t in got:
                t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for per in outs:
        for got, ref in zip(per, refs):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_offsets_past_32_bits(g):
    """More than 2^31 values: the last rows are those of a call on them alone."""
    bf, width, dv = torch.bfloat16, 8192, 256
    rows = 2 ** 31 // width + 40
    base = rand(1, 64, width, dtype=bf)
    x = base.repeat(rows // 64 + 1, 1)[:rows].contiguous()
    w = rand(2, width)
    tail = x[-40:].contiguous()
    big, small = g.layer_norm_fwd(x, w, checkpoint=True), g.layer_norm_fwd(tail, w, checkpoint=True)
    assert torch.equal(big.y[-40:], small.y) and torch.equal(big.checkpoint.codes[-40:], small.checkpoint.codes)
    assert torch.equal(big.checkpoint.scales[-40:], small.checkpoint.scales)
    dx = g.layer_norm_bwd(x, big.checkpoint, big.mean, big.rstd, w)[0]
    assert torch.equal(dx[-40:], g.layer_norm_bwd(tail, small.checkpoint, small.mean, small.rstd, w)[0])
    del dx
    a = g.act_pack(x)
    assert torch.equal(a.codes, big.checkpoint.codes) and torch.equal(g.act_unpack(a)[-40:], g.act_unpack(small.checkpoint))
    del a, big
    H = width // dv
    heads = lambda t: t.view(-1, H, dv)  # noqa: E731
    nw = rand(3, dv)
    do, dz, _ = g.block_epilogue_bwd(heads(x), heads(x), nw, heads(x))
    so, sz, _ = g.block_epilogue_bwd(heads(tail), heads(tail), nw, heads(tail))
    assert torch.equal(do[-40:], so) and torch.equal(dz[-40:], sz)
    del do, dz
    # one sequence that ends where the tail begins, so that the tail's convolution starts afresh
    cu = torch.tensor([0, rows - 40, rows], dtype=torch.int32, device="cuda")
    conv = [rand(5 + i, width, 4) for i in range(3)]
    k = 128
    xs = [x.view(rows, width // k, k)] * 6
    outs = g.block_prologue_bwd(*xs, *conv, *xs, cu_seqlens=cu)
    ts = [tail.view(40, width // k, k)] * 6
    ref = g.block_prologue_bwd(*ts, *conv, *ts, cu_seqlens=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    for p, q in zip(outs[:6], ref[:6]):
        assert torch.equal(p[-40:], q)


FIRST_CALL = """
import torch, gated_delta_rule_131_b200 as g
bf = torch.bfloat16
r = lambda *s: torch.randn(*s, device="cuda").to(bf)
x, w = r(40, 512), torch.ones(512, device="cuda")
mean, rstd = torch.zeros(40, device="cuda"), torch.ones(40, device="cuda")
o, nw = r(30, 2, 64), torch.ones(64, device="cuda")
t, conv = [r(1, 20, 2, 64) for _ in range(12)], [torch.randn(128, 4, device="cuda") for _ in range(3)]
def calls():
    a = g.act_pack(t[:6])
    n = g.layer_norm_fwd(x, w, residual=x, checkpoint=True)
    return [n.y, *g.layer_norm_bwd(x, x, mean, rstd, w), *g.block_epilogue_bwd(o, o, nw, o),
            *g.block_prologue_bwd(*a, *conv, *t[6:]), *g.act_unpack(a)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(out, calls()))
print("captured first")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """The pool, the kernels' limits and the kernels themselves are set up inside a stream capture."""
    import os
    import subprocess
    import sys
    root = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured first" in run.stdout, run.stderr[-2000:]


def test_what_the_binding_turns_down(g):
    """Layouts and devices that the library does not take, before anything is launched."""
    before = g.launch_count()
    x, w = rand(1, 8, 128, dtype=torch.bfloat16), rand(2, 128)
    n = rand(3, 8)
    bad = [lambda: g.layer_norm_fwd(x.t(), rand(4, 8)), lambda: g.layer_norm_fwd(x, w.cpu()),
           lambda: g.layer_norm_fwd(x, w, stream="not a stream"),
           lambda: g.layer_norm_bwd(x, x, n, n.cpu(), w), lambda: g.act_pack(x[:, ::2]), lambda: g.act_pack([x] * 9),
           lambda: g.act_pack(x.flatten()[1:129]),  # not on a 16-byte boundary
           lambda: g.layer_norm_fwd(rand(5, 2, 8200), rand(6, 8200)),
           lambda: g.block_epilogue_bwd(*[rand(i, 4, 2, 96) for i in (1, 2)], rand(3, 96), rand(4, 4, 2, 96)),
           lambda: g.block_prologue_bwd(*[rand(i, 1, 4, 2, 64) for i in range(6)], *[rand(i, 128, 5) for i in range(3)],
                                        *[rand(i, 1, 4, 2, 64) for i in range(6)])]
    for call in bad:
        with pytest.raises((ValueError, g.Gdn2Error, AttributeError)):
            call()
    assert g.launch_count() == before


def test_the_same_tensor_in_every_place(g):
    x, w = rand(1, 70, 128, dtype=torch.bfloat16), rand(2, 128)
    same, apart = g.layer_norm_fwd(x, w, w, residual=x), g.layer_norm_fwd(x, w, w.clone(), residual=x.clone())
    assert all(torch.equal(p, q) for p, q in zip(same[:4], apart[:4]))
    b = g.layer_norm_bwd(x, x, same.mean, same.rstd, w, dh=x)
    for p, q in zip(b, g.layer_norm_bwd(x.clone(), x, same.mean, same.rstd, w, dh=x.clone())):
        assert torch.equal(p, q)
    a = g.act_pack([x, x])
    assert torch.equal(a[0].codes, a[1].codes) and torch.equal(a[0].scales, a[1].scales)
    t, c = rand(3, 1, 33, 2, 64), rand(4, 128, 4)
    for p, q in zip(g.block_prologue_bwd(*[t] * 6, c, c, c, *[t] * 6),
                    g.block_prologue_bwd(*[t.clone() for _ in range(6)], c, c, c, *[t.clone() for _ in range(6)])):
        assert torch.equal(p, q)
