"""CPU checks of the operators around the block: arguments at the edges of what their entries take, refused before anything is launched."""
import ctypes

import pytest

from edge_aware_graph_b200 import eaga
from test_operators_abi import L, adam, norm_dims, tensor  # noqa: F401  (L: the built library)


@pytest.mark.parametrize("cfg", [dict(eps=1e-50), dict(eps=1e39), dict(grad_scale=1e39), dict(grad_scale=-1e39), dict(lr=1e39)])
def test_adamw_scalars_are_checked_as_the_kernel_uses_them(L, cfg):  # noqa: F811
    """Finite in 64 bits, but 0 or infinite in the 32 that the step computes in."""
    assert adam(L, [tensor()], **cfg) == 1


def test_adamw_counts_beyond_an_int(L):  # noqa: F811
    """Not taken modulo 2^32, past the end of the table that was checked."""
    table = (eaga.AdamwTensor * 1)(tensor())
    for count in ((1 << 32) + 1, -(1 << 32) + 1, 1 << 31):
        with pytest.raises(ValueError, match="count"):
            eaga.adamw_unpack(table, count, 0)
        with pytest.raises(ValueError, match="count"):
            eaga.adamw_step(eaga.AdamwConfig(), table, count, None, None, 0)
    with pytest.raises(eaga.EagaError) as e:
        eaga.adamw_unpack(table, (1 << 20) + 1, 0)
    assert e.value.code == 2
    with pytest.raises(ValueError):
        eaga.adamw_unpack(table, 2, 0)


def test_structures_of_another_kind(L):  # noqa: F811
    """Long enough is not enough: each call takes its own structure."""
    import torch
    host = torch.zeros(64, 128, dtype=torch.bfloat16)
    wrong = norm_dims(), eaga.AdamwConfig(), bytearray(4096), (eaga.AdamwTensor * 9)(), None, 3
    for d in wrong:
        with pytest.raises(ValueError, match="LinearDims"):
            eaga.linear_forward(d, host, None, None, None, None, None, None)
        with pytest.raises(ValueError, match="LinearDims"):
            eaga.linear_backward(d, host, None, None, None, None, None, None, None)
        with pytest.raises(ValueError, match="AdamwTensor" if d is not wrong[3] else "state"):
            eaga.adamw_step(eaga.AdamwConfig(), d, 1, None)
    for d in (eaga.linear_dims(64, 128, 8), (eaga.ResidualNormDims * 2)()._type_, (ctypes.c_double * 64)()):
        with pytest.raises(ValueError, match="ResidualNormDims"):
            eaga.residual_norm_forward(d, None, host, None, None, None, None, None, None, None, None)
        with pytest.raises(ValueError, match="ResidualNormDims"):
            eaga.residual_norm_backward(d, *[None] * 17)
        with pytest.raises(ValueError, match="AdamwConfig"):
            eaga.adamw_step(d, (eaga.AdamwTensor * 1)(), 1, None)
    with pytest.raises(ValueError, match="u: a CUDA tensor"):
        eaga.residual_norm_forward(norm_dims(), None, host, None, None, None, None, None, None, None, None)


@pytest.mark.parametrize("w", [8, 64, 128, 333, 4096])
@pytest.mark.parametrize("group", [2 ** 63 - 1, 2 ** 63 - 40, 2 ** 40, 2 ** 31])
def test_norm_groups_beyond_the_limit(L, w, group):  # noqa: F811
    """Of a call without rows too, whose plan divides by the length of the groups' runs."""
    assert eaga.residual_norm_workspace_size(norm_dims(rows=0, w=w, rows_per_group=group)) == 0
    assert eaga.residual_norm_workspace_size(norm_dims(rows=0, w=w, rows_per_group=0x7fff0000)) >= 256


def test_adamw_step_count_and_rate_apart_from_the_tensors(L):  # noqa: F811
    """The step writes its count: not into a tensor's buffers, nor over the rate; and no buffer over the rate."""
    def call(tensors, state=0x10, lr=None):
        c = eaga.AdamwConfig(1e-3, 0.9, 0.999, 1e-8, 1.0, 1, 0, 8, 0)
        return L.eaga_adamw_step(ctypes.byref(c), (eaga.AdamwTensor * len(tensors))(*tensors), len(tensors), state, lr, None)

    two = [tensor(0), tensor(1)]
    for k in ("p", "master", "g", "m", "v", "m_scale", "v_scale"):
        assert call(two, state=getattr(two[1], k)) == 1, k
        assert call(two[::-1], state=getattr(two[1], k)) == 1, k
        if k != "g":
            assert call(two, lr=getattr(two[0], k)) == 1, k
    assert call(two, state=tensor().p + 192) == 1         # the last 8 of a weight's 200 bytes
    assert call(two, state=0x40, lr=0x48) == 1
    apart = call(two, lr=0x30)                            # what a call without overlaps answers without a GPU
    assert apart != 1 and call(two, lr=two[0].g + 16) == apart and call(two[::-1], state=tensor().p + 208) == apart
