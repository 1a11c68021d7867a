"""The long forms of the block's training operators on the GPU (needs a GPU): runs of many tokens, blocks
that walk many rows and tiles, the widest rows.  Tolerances as derived in ``test_gpu_train.py``, whose
helpers are used here; where a sum has more terms than counted there, the count stands at the test.
"""
import numpy as np
import pytest
import torch

from oracle import block_train as bt
from test_gpu_train import TYPES, close, conv_major, g, lagged, np64, rand  # noqa: F401
from test_gpu_train import test_epilogue_bwd as check_epilogue_bwd
from test_gpu_train import test_layer_norm_bwd as check_layer_norm_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,width", [(torch.bfloat16, 2 ** 31 - 1), (torch.bfloat16, 2 ** 31 - 8),
                                         (torch.float32, 2 ** 31 - 4), (torch.float32, 2 ** 31 - 32)])
def test_act8_rows_of_nearly_31_bits(g, dtype, width):
    """The widest rows there are, of each kind (single values, vectors that end inside a group, whole
    groups): the same codes and values as of the row's groups one by one."""
    base = rand(1, 2 ** 20 + 7, dtype=dtype)
    x = base.repeat(width // base.numel() + 1)[:width]
    whole = width // 32 * 32
    a = g.act_pack(x)
    groups = g.act_pack(x[:whole].view(-1, 32))
    assert torch.equal(a.codes[:whole].view(-1, 32), groups.codes)
    assert torch.equal(a.scales[:whole // 32], groups.scales.view(-1))
    values = g.act_unpack(a, dtype=dtype)
    assert torch.equal(values[:whole].view(-1, 32), g.act_unpack(groups, dtype=dtype))
    if whole < width:
        last = g.act_pack(x[whole:].clone())
        assert torch.equal(a.codes[whole:], last.codes) and torch.equal(a.scales[whole // 32:], last.scales)
        assert torch.equal(values[whole:], g.act_unpack(last, dtype=dtype))


def conv_bwd64(x, Wt, d, l2, cu):
    """``(dx, dW)`` of one convolution path by whole sequences: x, d ``[tokens, H, dim]``, W ``[H, dim, K]``."""
    K = Wt.shape[-1]
    dx, dW = np.zeros_like(x), np.zeros_like(Wt)
    for b, e in zip(cu[:-1], cu[1:]):
        X, D = x[b:e], d[b:e]
        y = sum(Wt[..., K - 1 - j] * lagged(X, j) for j in range(K))
        sg = 1 / (1 + np.exp(-y))
        s = y * sg
        if l2:
            n = 1 / np.sqrt((s * s).sum(-1, keepdims=True) + bt.L2_EPS)
            D = n * D - n ** 3 * s * (s * D).sum(-1, keepdims=True)
        dy = D * sg * (1 + y * (1 - sg))
        for j in range(min(K, e - b)):
            dx[b:e - j] += (Wt[..., K - 1 - j] * dy)[j:]
            dW[..., K - 1 - j] += (dy * lagged(X, j)).sum(0)
    return dx, dW


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ckpt", [False, True])
def test_prologue_bwd_runs_of_several_hundred_tokens(g, dtype, ckpt):
    """Runs long enough that the taps' gradients move to their second level more than once (every 256
    tokens), and end between two moves; compared on three of the heads."""
    H, dk, dv, K, pad = 32, 128, 256, 4, 5
    lengths = [2500, 0, 1, 3999, 2, 2498]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    tokens = int(cu[-1])
    dims = (dk, dk, dv, dk, dk, dv)
    bytes_ = g.block_prologue_bwd_workspace_bytes(len(lengths), tokens + pad, H, dk, dv, K, packed=True, dtype=dtype)
    runs = bytes_ / (4 * H * (2 * dk + dv) * K)  # a row of partial sums each
    assert 2 * 256 < tokens / runs < 3 * 256 - 8, "the runs are not as long as this case wants them"
    gen = torch.Generator(device="cuda").manual_seed(71)
    draw = lambda d: torch.randn(tokens + pad, H, d, device="cuda", generator=gen).to(dtype)  # noqa: E731
    x, d = [draw(n) for n in dims], [draw(n) for n in dims]
    for t in x:
        t[tokens:] = float("nan")
    conv = [rand(80 + i, H * n, K, scale=0.5) for i, n in enumerate(dims[:3])]
    held = [g.act_pack(t) for t in x] if ckpt else x
    outs = g.block_prologue_bwd(*held, *conv, *d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    again = g.block_prologue_bwd(*held, *conv, *d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(outs[6:], again[6:]))
    values = g.act_unpack(held, dtype=torch.float32) if ckpt else x
    heads = [0, 13, 31]
    # a tap's gradient: a term's own roundings (64), 256 terms in a register, three of those, sixteen runs'
    # partial sums or so, and the adding up of those in two warps
    c_sum = 64 + 256 + 3 + 20 + 4
    for i in range(3):
        x64, d64 = (np64(t[:tokens, heads]) for t in (values[i], d[i]))
        w64 = np64(conv[i].view(H, -1, K)[heads])
        rx, rW = conv_bwd64(x64, w64, d64, i < 2, cu)
        mx, mW = conv_major(x64, w64.reshape(-1, K), d64, i < 2, cu)
        close(outs[i][:tokens, heads], rx, mx, 64, "dx")
        close(outs[6 + i].view(H, -1, K)[heads].reshape(-1, K), rW.reshape(-1, K), mW, c_sum, "dconv")


def test_the_definition_by_whole_sequences_is_the_oracle():
    gen = np.random.default_rng(5)
    x, d, w = gen.standard_normal((40, 2, 8)), gen.standard_normal((40, 2, 8)), gen.standard_normal((2, 8, 3))
    cu = [0, 7, 7, 8, 40]
    for l2 in (False, True):
        dx, dW = conv_bwd64(x, w, d, l2, cu)
        ref = [sum(bt._conv_bwd(x[b:e], w, d[b:e], l2)[1] for b, e in zip(cu[:-1], cu[1:]) if e > b),
               np.concatenate([bt._conv_bwd(x[b:e], w, d[b:e], l2)[0] for b, e in zip(cu[:-1], cu[1:]) if e > b])]
        assert np.allclose(dW, ref[0], rtol=1e-12, atol=1e-12) and np.allclose(dx, ref[1], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("dtype,width,tokens", [
    (torch.bfloat16, 2048, 1500),   # 4 rows a block at a time, three of each group one after another
    (torch.bfloat16, 512, 5000),    # 16 of one warp each
    (torch.bfloat16, 1000, 2000),   # rows that do not fill their threads
    (torch.bfloat16, 1001, 1237),   # single values
    (torch.float32, 1001, 1237),
    (torch.float32, 256, 9000),
    (torch.float32, 8192, 450),     # 16 fp32 values per thread, one row a block at a time
    (torch.float32, 5000, 450),
    (torch.float32, 8191, 450),
    (torch.bfloat16, 8191, 450),
])
@pytest.mark.parametrize("ckpt", [False, True])
def test_layer_norm_bwd_of_many_rows(g, dtype, width, tokens, ckpt):
    """Every group of a block walks several rows.  A weight's gradient adds under ten rows in a register,
    16 groups, 148 blocks' sums as 8 by 8 and 19 warps': with a term's own 64 roundings under the 160 that
    are allowed."""
    check_layer_norm_bwd(g, dtype, width, ckpt, True, tokens)


@pytest.mark.parametrize("dtype,dv,tokens,H", [(torch.bfloat16, 128, 15001, 2), (torch.float32, 128, 9001, 2),
                                               (torch.bfloat16, 256, 4999, 3), (torch.float32, 64, 20003, 2)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_epilogue_bwd_of_many_tiles(g, dtype, dv, tokens, H, ckpt):
    """Blocks that take a second and a third tile of 256 x 32 bytes, the last one not full.  The weight's
    gradient adds three rows in a register, 32 groups of a block, 296 blocks' sums as 8 by 8, twice, and 32
    warps': with a term's own 64 roundings under the 160 that are allowed."""
    tiles = tokens * H * dv / (4096 if dtype == torch.bfloat16 else 2048)
    assert tiles > 2 * 296
    check_epilogue_bwd(g, dtype, dv, tokens, H, ckpt)
