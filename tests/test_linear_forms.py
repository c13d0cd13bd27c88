"""The kernels that the linear operator chooses, and that its GPU tests reach every one of them (the choice is the host's, for 148 SMs)."""
import itertools

import pytest

import test_linear_forms_gpu
import test_linear_gpu
from edge_aware_graph_b200 import build as B
from edge_aware_graph_b200 import eaga

LARGE = [m.args[1] for m in test_linear_gpu.test_exact_products_of_large_tiles.pytestmark if m.args[0] == "rows,i,o"][0]


def names(*parts):
    return {" ".join(w for w in p if w) for p in itertools.product(*parts)}


ALL = {}
for dtype, most in (("bf16", 8), ("fp32", 16)):
    rows = names(["rows"], [str(r) for r in (1, 2, 4, 8, 16) if r <= most], ["", "wide"])
    for product in ("Y", "dX", "dW"):
        some = rows | names(["tc"], ["pair", "128", "64"], ["", "tma"], ["promoted"], ["", "split"])
        if dtype == "bf16" and product != "dW":
            some |= names(["tc"], ["128", "64"], ["", "tma"]) | {"tc 64 two tma"}
        if dtype == "fp32":
            some |= {"cores 32x32", "cores 32x32 split", "cores 64x64 split", "cores thin", "cores thin split"} if product == "dW" else \
                names(["cores"], ["warps 4", "warps 2", "128x16", "128x32", "64x64", "32x32"])
        ALL[dtype, product] = some


@pytest.mark.parametrize("dtype,product", list(ALL))
def test_every_form_is_tested(dtype, product):
    B.build()
    reached = {eaga.linear_form(eaga.linear_dims(r, i, o, act, dtype), product)
               for r, i, o in [*test_linear_gpu.SHAPES, *LARGE, *test_linear_forms_gpu.SHAPES] for act in ("none", "relu")}
    assert reached == ALL[dtype, product]


def test_form_arguments():
    d = eaga.linear_dims(8, 64, 64)
    with pytest.raises(ValueError):
        eaga.linear_form(d, "Z")
    with pytest.raises(eaga.EagaError) as e:
        eaga.linear_form(eaga.linear_dims(8, 0, 64), "Y")
    assert e.value.code == 1
    assert eaga.linear_form(eaga.linear_dims(0, 64, 64), "dW") == "none"
    import ctypes
    small = ctypes.create_string_buffer(4)
    assert eaga.lib().eaga_linear_form(ctypes.byref(d), 0, small, 4) == 4 and len(small.value) < 4
    assert eaga.lib().eaga_linear_form(ctypes.byref(d), 3, small, 4) == 1 and eaga.lib().eaga_linear_form(ctypes.byref(d), 0, None, 0) == 1
