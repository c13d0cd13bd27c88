"""CPU checks of the operators around the block: arguments at the edges of what their entries take, refused before anything is launched."""
import ctypes

import pytest

from edge_aware_graph_b200 import eaga
from test_operators_abi import L, adam, norm_dims, tensor  # noqa: F401  (L: the built library)


@pytest.mark.parametrize("cfg", [dict(eps=1e-50), dict(eps=1e39), dict(grad_scale=1e39), dict(grad_scale=-1e39), dict(lr=1e39)])
def test_adamw_scalars_are_checked_as_the_kernel_uses_them(L, cfg):  # noqa: F811
    """Finite in 64 bits, but 0 or infinite in the 32 that the step computes in."""
    assert adam(L, [tensor()], **cfg) == 1
