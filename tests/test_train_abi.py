"""Refusals and host arithmetic of the training operators (CPU only): every call here is turned down on
the host, or has nothing to do, before any launch or allocation."""
import ctypes
import os
import re

import pytest
import torch

import gated_delta_rule_131_b200 as gdn2
from gated_delta_rule_131_b200 import build as gbuild

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
FAKE, MIS4, MIS2 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10002)
OK, BAD, UNSUP = gdn2.GDN2_OK, gdn2.GDN2_ERR_INVALID_ARG, gdn2.GDN2_ERR_UNSUPPORTED
BF16 = gdn2.GDN2_BF16


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn2.lib()


@pytest.fixture(autouse=True)
def nothing_is_launched(L):
    before = L.gdn2_launch_count()
    yield
    assert L.gdn2_launch_count() == before


def test_limits_match_the_header():
    txt = open(os.path.join(ROOT, "include", "gdn2.h")).read()
    assert int(re.search(r"#define GDN2_ACT_MAX_TENSORS (\d+)", txt).group(1)) == gdn2.ACT_MAX_TENSORS
    assert int(re.search(r"#define GDN2_NORM_MAX_WIDTH (\d+)", txt).group(1)) == gdn2.NORM_MAX_WIDTH


# ---- layer norm.  forward pointers: x residual weight bias | y h mean rstd codes scales

def norm_fwd(L, change=None, eps=1e-5, tokens=4, width=64, dtype=BF16, base=FAKE):
    p = [base] * 10
    for i, v in (change or {}).items():
        p[i] = v
    return L.gdn2_layer_norm_fwd(*p[:4], eps, *p[4:], tokens, width, dtype, None)


def test_layer_norm_fwd_refusals(L):
    for i in (0, 2, 4):
        assert norm_fwd(L, {i: None}) == BAD, i
    for i in (0, 1, 2, 3, 4, 5, 8, 9):
        assert norm_fwd(L, {i: MIS4}) == BAD, i
    for i in (6, 7):
        assert norm_fwd(L, {i: MIS2}) == BAD, i
    for i in (1, 5, 6, 7, 8, 9):  # residual with h, mean with rstd, codes with scales
        assert norm_fwd(L, {i: None}) == BAD, i
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm_fwd(L, eps=eps) == BAD
    assert norm_fwd(L, tokens=-1) == BAD and norm_fwd(L, width=0) == BAD and norm_fwd(L, dtype=5) == BAD
    assert norm_fwd(L, tokens=1 << 60, width=8192) == BAD
    assert norm_fwd(L, width=8193) == UNSUP
    assert norm_fwd(L, {0: None, 4: None}, tokens=0) == OK


# ---- backward pointers: dy h scales mean rstd weight dh | dx dweight dbias

def norm_bwd(L, change=None, tokens=4, width=64, dtype=BF16):
    p = [FAKE] * 10
    for i, v in (change or {}).items():
        p[i] = v
    return L.gdn2_layer_norm_bwd(*p, tokens, width, dtype, None)


def test_layer_norm_bwd_refusals(L):
    for i in (0, 1, 3, 4, 5, 7, 8):
        assert norm_bwd(L, {i: None}) == BAD, i
    for i in (0, 1, 2, 5, 6, 7):
        assert norm_bwd(L, {i: MIS4}) == BAD, i
    for i in (3, 4, 8, 9):
        assert norm_bwd(L, {i: MIS2}) == BAD, i
    assert norm_bwd(L, tokens=-1) == BAD and norm_bwd(L, width=-1) == BAD and norm_bwd(L, dtype=-1) == BAD
    assert norm_bwd(L, width=8200) == UNSUP


# ---- epilogue backward pointers: o gate o_scales gate_scales norm_weight dy | do dgate dnorm_weight

def epi_bwd(L, change=None, tokens=4, H=2, dv=64, dtype=BF16):
    p = [FAKE] * 9
    for i, v in (change or {}).items():
        p[i] = v
    return L.gdn2_block_epilogue_bwd(*p, tokens, H, dv, dtype, None)


def test_epilogue_bwd_refusals(L):
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8):  # one of the two scales alone is refused too
        assert epi_bwd(L, {i: None}) == BAD, i
    for i in (0, 1, 2, 3, 5, 6, 7):
        assert epi_bwd(L, {i: MIS4}) == BAD, i
    for i in (4, 8):
        assert epi_bwd(L, {i: MIS2}) == BAD, i
    assert epi_bwd(L, tokens=-1) == BAD and epi_bwd(L, H=0) == BAD and epi_bwd(L, dtype=2) == BAD
    assert epi_bwd(L, tokens=1 << 60, H=16) == BAD
    assert epi_bwd(L, dv=96) == UNSUP


# ---- prologue backward pointers: x[6] scales conv[3] d[6] | dx[6] dconv[3]

def pro_bwd(L, change=None, scales=None, B=1, T=64, H=2, dk=64, dv=64, K=4, cu=None, dtype=BF16):
    p = [FAKE] * 25
    p[6] = None if scales is None else (ctypes.c_void_p * 6)(*scales)
    for i, v in (change or {}).items():
        p[i] = v
    return L.gdn2_block_prologue_bwd(*p, B, T, H, dk, dv, K, cu, dtype, None)


def test_prologue_bwd_refusals(L):
    for i in [k for k in range(25) if k != 6]:
        assert pro_bwd(L, {i: None}) == BAD, i
    for i in [*range(6), *range(10, 22)]:
        assert pro_bwd(L, {i: MIS4}) == BAD, i
    for i in [7, 8, 9, 22, 23, 24]:
        assert pro_bwd(L, {i: MIS2}) == BAD, i
    for i in range(6):
        one = [0x10000] * 6
        one[i] = None
        assert pro_bwd(L, scales=one) == BAD, i
        one[i] = 0x10008
        assert pro_bwd(L, scales=one) == BAD, i
    assert pro_bwd(L, cu=MIS2) == BAD
    assert pro_bwd(L, B=-1) == BAD and pro_bwd(L, T=-1) == BAD and pro_bwd(L, H=0) == BAD and pro_bwd(L, dtype=4) == BAD
    assert pro_bwd(L, H=65537) == BAD and pro_bwd(L, B=1 << 30, T=1 << 30, H=1 << 10) == BAD
    assert pro_bwd(L, K=0) == UNSUP and pro_bwd(L, K=5) == UNSUP
    assert pro_bwd(L, dk=256) == UNSUP and pro_bwd(L, dv=32) == UNSUP


# ---- activations in 8 bits

def act(fn, ptrs=(0x10000, 0x20000, 0x30000), rows=4, width=64, count=1, dtype=BF16, null=None):
    n = max(count, 1)
    arrays = [(ctypes.c_void_p * n)(*[p] * n) for p in ptrs]
    arrays += [(ctypes.c_longlong * n)(*[rows] * n), (ctypes.c_int * n)(*[width] * n)]
    if null is not None:
        arrays[null] = None
    return fn(*arrays, count, dtype, None)


@pytest.mark.parametrize("name", ["gdn2_act_pack", "gdn2_act_unpack"])
def test_act_refusals(L, name):
    fn = getattr(L, name)
    for i in range(5):
        assert act(fn, null=i) == BAD
    for i in range(3):
        p = [0x10000, 0x20000, 0x30000]
        p[i] = None
        assert act(fn, p) == BAD
        p[i] = 0x10008
        assert act(fn, p) == BAD
    assert act(fn, rows=-1) == BAD and act(fn, width=0) == BAD and act(fn, count=-1) == BAD and act(fn, dtype=3) == BAD
    assert act(fn, rows=1 << 60) == BAD
    assert act(fn, count=gdn2.ACT_MAX_TENSORS + 1) == UNSUP
    assert act(fn, count=0) == OK
    assert act(fn, (None, None, None), rows=0) == OK


def test_workspace_bytes(L):
    """One row of partial weight gradients for each block (148 SMs where there is no GPU); none where the
    few blocks of a short call are one cluster."""
    norm, epi = L.gdn2_layer_norm_bwd_workspace_bytes, L.gdn2_block_epilogue_bwd_workspace_bytes
    assert norm(8192, 2048, BF16) == 148 * 2 * 2048 * 4 == gdn2.layer_norm_bwd_workspace_bytes(8192, 2048)
    # a cluster is 8 blocks, of one row each or of sums of up to 1024 channels (width 256: four rows)
    assert norm(8, 2048, BF16) == 0 and norm(9, 2048, BF16) == 9 * 2 * 2048 * 4
    assert norm(32, 256, BF16) == 0 and norm(33, 256, BF16) == 33 * 2 * 256 * 4
    assert norm(0, 100, BF16) == norm(5, 8193, BF16) == norm(5, 64, 7) == 0
    assert epi(8192, 16, 128, BF16) == 296 * 128 * 4 == gdn2.block_epilogue_bwd_workspace_bytes(8192, 16, 128)
    # 256 threads x 16 channels: 32 rows of 128 a tile, two tiles for each of 8 blocks are the last cluster
    assert epi(512, 1, 128, BF16) == 0 and epi(513, 1, 128, BF16) == 17 * 128 * 4
    assert epi(256, 1, 128, gdn2.GDN2_F32) == 0 and epi(257, 1, 128, gdn2.GDN2_F32) == 17 * 128 * 4
    assert epi(5000, 1, 63, BF16) == epi(5000, 1, 64, 9) == 0
    n = L.gdn2_block_prologue_bwd_workspace_bytes(1, 2, 1, 64, 128, 3, 0, gdn2.GDN2_F32)
    assert n == (64 + 64 + 128) * 3 * 4  # one run
    assert L.gdn2_block_prologue_bwd_workspace_bytes(1, 2, 1, 64, 128, 5, 0, gdn2.GDN2_F32) == 0
    # bounded by the resident lanes however many tokens there are
    big = L.gdn2_block_prologue_bwd_workspace_bytes(64, 65536, 16, 128, 128, 4, 0, BF16)
    assert 0 < big < 64 << 20
    assert gdn2.block_prologue_bwd_workspace_bytes(1, 2, 1, 64, 128, 3, dtype=torch.float32) == n


def test_python_refusals():
    """Shapes and types are turned down before the library is called; so are CPU tensors."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    bad = [
        lambda: gdn2.layer_norm_fwd(z(4, 64), f(64)),                                    # a CPU tensor
        lambda: gdn2.layer_norm_fwd(z(4, 64), f(63)),
        lambda: gdn2.layer_norm_fwd(z(4, 64), z(64)),
        lambda: gdn2.layer_norm_fwd(z(4, 64), f(64), residual=f(4, 64)),
        lambda: gdn2.layer_norm_fwd(torch.zeros(4, 64, dtype=torch.float16), f(64)),
        lambda: gdn2.layer_norm_bwd(z(4, 64), z(4, 64), f(4), f(3), f(64)),
        lambda: gdn2.layer_norm_bwd(z(4, 64), f(4, 64), f(4), f(4), f(64)),
        lambda: gdn2.layer_norm_bwd(z(4, 64), gdn2.Act8(z(4, 64, dtype=torch.int8), z(4, 3, dtype=torch.uint8)), f(4),
                                    f(4), f(64)),
        lambda: gdn2.block_epilogue_bwd(z(4, 2, 64), gdn2.Act8(z(4, 2, 64, dtype=torch.int8),
                                                               z(4, 2, 2, dtype=torch.uint8)), f(64), z(4, 2, 64)),
        lambda: gdn2.block_epilogue_bwd(z(4, 2, 64), z(4, 2, 64), f(32), z(4, 2, 64)),
        lambda: gdn2.act_pack([z(4, 64), f(4, 64)]),
        lambda: gdn2.act_pack(z(4, 64)),
        lambda: gdn2.act_unpack(gdn2.Act8(z(4, 64, dtype=torch.int8), z(4, 2, dtype=torch.uint8)), dtype=torch.float16),
        lambda: gdn2.act_unpack(gdn2.Act8(z(4, 64), z(4, 2, dtype=torch.uint8))),
    ]
    x = [z(1, 8, 2, 64) for _ in range(6)]
    W = [f(128, 4) for _ in range(3)]
    bad += [
        lambda: gdn2.block_prologue_bwd(*x, *W, *x),
        lambda: gdn2.block_prologue_bwd(*x, f(128, 3), *W[1:], *x),
        lambda: gdn2.block_prologue_bwd(*x, *W, *x[:5], z(1, 8, 2, 128)),
        lambda: gdn2.block_prologue_bwd(*x, *W, *x, cu_seqlens=torch.zeros(2, dtype=torch.int32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    assert gdn2.act_pack([]) == [] and gdn2.act_unpack([]) == []
