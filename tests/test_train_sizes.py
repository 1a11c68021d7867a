"""Sizes and arguments that the binding of the training operators has to turn down itself (CPU only): tensors
on the ``meta`` device have a size and no memory.
"""
import pytest
import torch

import gated_delta_rule_131_b200 as gdn2

WIDE = 2 ** 32 + 64  # its low 32 bits are a width that the library takes
BF = torch.bfloat16


def meta(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def f32(*shape):
    return meta(*shape, dtype=torch.float32)


def act8(*shape):
    return gdn2.Act8(meta(*shape, dtype=torch.int8), meta(*shape[:-1], -(-shape[-1] // 32), dtype=torch.uint8))


def test_a_last_dimension_of_more_than_31_bits_is_not_cut():
    with pytest.raises(ValueError, match="last dimension of 1 to"):
        gdn2.act_pack(meta(WIDE))
    with pytest.raises(ValueError, match="last dimension of 1 to"):
        gdn2.act_pack([meta(4, 64), meta(2, WIDE)])
    with pytest.raises(ValueError, match="last dimension of 1 to"):
        gdn2.act_unpack(act8(1, WIDE))
    for width in (WIDE, 8193):
        with pytest.raises(gdn2.Gdn2Error) as e:
            gdn2.layer_norm_fwd(meta(1, width), f32(width))
        assert e.value.status == gdn2.GDN2_ERR_UNSUPPORTED
        with pytest.raises(gdn2.Gdn2Error) as e:
            gdn2.layer_norm_bwd(meta(1, width), meta(1, width), f32(1), f32(1), f32(width))
        assert e.value.status == gdn2.GDN2_ERR_UNSUPPORTED


@pytest.mark.parametrize("H,d", [(1, WIDE), (2 ** 32 + 1, 64)])
def test_heads_and_channels_of_more_than_31_bits_are_not_cut(H, d):
    with pytest.raises(gdn2.Gdn2Error) as e:
        gdn2.block_epilogue_bwd(meta(1, H, d), meta(1, H, d), f32(d), meta(1, H, d))
    assert e.value.status == gdn2.GDN2_ERR_UNSUPPORTED
    x = [meta(1, 1, H, d) for _ in range(6)]
    with pytest.raises(gdn2.Gdn2Error) as e:
        gdn2.block_prologue_bwd(*x, *[f32(H * d, 4) for _ in range(3)], *x)
    assert e.value.status == gdn2.GDN2_ERR_UNSUPPORTED


def test_workspace_queries_do_not_cut_sizes():
    assert gdn2.layer_norm_bwd_workspace_bytes(500, 64) > 0 == gdn2.layer_norm_bwd_workspace_bytes(500, WIDE)
    assert gdn2.layer_norm_bwd_workspace_bytes(500, 64 - 2 ** 32) == 0
    query = gdn2.block_epilogue_bwd_workspace_bytes
    assert query(5000, 2, 64) > 0 == query(5000, 2, WIDE) == query(5000, 2 ** 32 + 2, 64) == query(5000, 2, 64 - 2 ** 32)
    query, sizes = gdn2.block_prologue_bwd_workspace_bytes, [1, 500, 2, 64, 64, 4]
    assert query(*sizes) > 0
    for i in range(6):
        assert query(*sizes[:i], sizes[i] + 2 ** 32, *sizes[i + 1:]) == 0, i


def test_a_missing_tensor_is_named():
    """What a forward without statistics leaves out, for one: a ValueError, as for every other argument."""
    h, w, n = meta(4, 64), f32(64), f32(4)
    x, c, z = [meta(1, 8, 2, 64) for _ in range(6)], [f32(128, 4) for _ in range(3)], meta(4, 2, 64)
    without = lambda args, i: [None if k == i else a for k, a in enumerate(args)]  # noqa: E731
    calls = [lambda: gdn2.layer_norm_fwd(h, None)]
    calls += [lambda i=i: gdn2.layer_norm_bwd(h, *without([h, n, n, w], i)) for i in range(4)]
    calls += [lambda i=i: gdn2.block_epilogue_bwd(*without([z, z, w], i), z) for i in range(3)]
    calls += [lambda i=i: gdn2.block_prologue_bwd(*without([*x, *c], i), *x) for i in range(9)]
    calls += [lambda i=i: gdn2.block_prologue_bwd(*x, *c, *without(x, i)) for i in range(1, 6)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError) as e:
            call()
        assert "CUDA" not in str(e.value), i  # turned down for what is missing, not for where the others are
