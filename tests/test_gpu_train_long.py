"""The long forms of the block's training operators on the GPU (needs a GPU).  Tolerances as derived in
``test_gpu_train.py``, whose helpers are used here; where a sum has more terms than counted there, the
count stands at the test.
"""
import pytest
import torch

from test_gpu_train import g, rand  # noqa: F401

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
