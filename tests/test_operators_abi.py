"""CPU checks of the operators around the block: what the C entries refuse, before anything is launched."""
import ctypes

import pytest

from edge_aware_graph_b200 import build as B
from edge_aware_graph_b200 import eaga


@pytest.fixture(scope="module")
def L():
    B.build()
    return eaga.lib()


OK = 0x100000


def norm_call(L, d, **over):
    at = dict(x=1, u=2, M=3, gate=4, post_g=5, post_s=6, pre_g=7, pre_s=8, r=9, h=10)
    p = [over.get(k, OK + (i << 28)) for k, i in at.items()]
    return L.eaga_residual_norm_forward(ctypes.byref(d) if d else None, *p, None)


def norm_dims(**k):
    return eaga.residual_norm_dims(**{**dict(rows=64, w=128, pre="layer", post="layer", rows_per_group=8), **k})


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1, rows_per_group=8), 1), (dict(w=0), 1), (dict(rows_per_group=0), 1), (dict(rows_per_group=7), 1),
    (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(alpha=float("inf")), 1), (dict(dtype=5), 1),
    (dict(w=8193), 2), (dict(rows=1 << 31, rows_per_group=8), 2),
])
def test_norm_dims(L, change, code):
    d = norm_dims(**change)
    assert norm_call(L, d) == code
    assert eaga.residual_norm_workspace_size(d) == 0


def test_norm_pointers(L):
    d = norm_dims()
    assert eaga.residual_norm_workspace_size(d) >= 256
    assert norm_call(L, None) == 1
    for k in ("u", "h"):
        assert norm_call(L, d, **{k: None}) == 1
    for k in ("x", "u", "M", "gate", "post_g", "pre_s", "r", "h"):
        assert norm_call(L, d, **{k: OK + (20 << 28) + 4}) == 3
    assert norm_call(L, d, r=OK + (2 << 28) + 64) == 1                  # r inside u
    assert norm_call(L, norm_dims(post="none")) == 1                    # a gain without its norm
    assert norm_call(L, norm_dims(pre="none"), pre_g=None, pre_s=None) == 1    # h without a pre-norm
    assert norm_call(L, norm_dims(rows=0, rows_per_group=1), u=None, x=None, r=None) == 0
    with pytest.raises(ValueError):
        eaga.residual_norm_dims(4, 8, pre="batch")


def test_norm_backward_pointers(L):
    d = norm_dims()
    names = ("r u M gate post_g post_s pre_g dr dh dx du dgate dpost_g dpost_s dpre_g dpre_s").split()
    need = eaga.residual_norm_workspace_size(d)

    def call(ws=OK + (30 << 28), size=need, dims=d, **over):
        return L.eaga_residual_norm_backward(ctypes.byref(dims), *[over.get(k, OK + (i << 28)) for i, k in enumerate(names)],
                                             ws, size, None)

    assert call(size=need - 1) == 4
    for k in ("r", "dh", "u"):
        assert call(**{k: None}) == 1
    assert call(ws=None) == 1 and call(gate=None) == 1
    assert call(dx=OK + 8) == 3
    assert call(dx=OK + (7 << 28)) == 1                                 # dx over dr
    assert call(dpost_g=OK + (12 << 28), dpost_s=OK + (12 << 28)) == 1  # one output twice


def adam(L, tensors, state=OK + (50 << 28), count=None, **cfg):
    c = eaga.AdamwConfig(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, param_dtype=1, grad_dtype=0,
                                   state_bits=8, seed=0), **cfg})
    t = (eaga.AdamwTensor * max(1, len(tensors)))(*tensors)
    return L.eaga_adamw_step(ctypes.byref(c), t, len(tensors) if count is None else count, state, None, None)


def tensor(i=0, n=100, **over):
    base = {k: OK + ((j + 8 * i) << 24) for j, k in enumerate(("p", "master", "g", "m", "v", "m_scale", "v_scale"))}
    return eaga.AdamwTensor(**{**base, "n": n, "counter": 0, "weight_decay": 0.0, **over})


@pytest.mark.parametrize("cfg,code", [
    (dict(state_bits=16), 1), (dict(param_dtype=2), 1), (dict(grad_dtype=-1), 1), (dict(beta1=1.0), 1), (dict(beta2=-0.1), 1),
    (dict(eps=0.0), 1), (dict(lr=float("inf")), 1), (dict(lr=-1.0), 1), (dict(grad_scale=float("nan")), 1),
    (dict(param_dtype=0), 1),                                           # a master beside fp32 weights
])
def test_adamw_config(L, cfg, code):
    assert adam(L, [tensor()], **cfg) == code


def test_adamw_tensors(L):
    assert adam(L, [tensor()], state=None) == 1 and adam(L, [tensor()], state=OK + 8) == 3
    assert adam(L, [], count=-1) == 1
    for k in ("p", "g", "m", "v", "m_scale", "v_scale"):
        assert adam(L, [tensor(**{k: None})]) == 1, k
    assert adam(L, [tensor(n=-1)]) == 1 and adam(L, [tensor(n=1 << 41)]) == 2
    assert adam(L, [tensor(weight_decay=-1.0)]) == 1 and adam(L, [tensor(weight_decay=float("nan"))]) == 1
    assert adam(L, [tensor(p=OK + 2)]) == 3 and adam(L, [tensor(m_scale=OK + 2)]) == 3
    assert adam(L, [tensor(), tensor(1, master=None)]) == 1             # masters for some
    # buffers that overlap: within a tensor, between tensors in any order, a weight and another's gradient
    assert adam(L, [tensor(m=tensor().v)]) == 1
    assert adam(L, [tensor(0), tensor(0)]) == 1
    assert adam(L, [tensor(1), tensor(0), tensor(2, p=tensor(1).p + 16)]) == 1
    assert adam(L, [tensor(1), tensor(0, g=tensor(1).master + 16)]) == 1
    assert L.eaga_adamw_unpack((eaga.AdamwTensor * 1)(tensor(g=None, master=tensor().p)), 1, None) == 1
    assert L.eaga_adamw_unpack(None, 0, None) == 0


def test_adamw_needs_a_gpu():
    import torch
    from edge_aware_graph_b200.optim import AdamW
    with pytest.raises(ValueError):
        AdamW([torch.zeros(8)], [torch.zeros(8)])


def linear_call(L, d, **over):
    names = "X W b R Y Z".split()
    p = [over.get(k, OK + ((i + 1) << 28)) for i, k in enumerate(names)]
    return L.eaga_linear_forward(ctypes.byref(d) if d else None, *p, over.get("ws", OK + (30 << 28)),
                                 over.get("size", eaga.linear_workspace_size(d, False) if d else 0), None)


def linear_back(L, d, act_in=0, **over):
    at = {k: OK + ((i + 1) << 28) for i, k in enumerate("X W Z dY Zin dR dX dW db".split())}
    if not d.act:
        at["Z"] = None
    if not act_in:
        at["Zin"] = None
    at.update(over)
    return L.eaga_linear_backward(ctypes.byref(d), at["X"], at["W"], at["Z"], at["dY"], act_in, at["Zin"], at["dR"], at["dX"], at["dW"],
                                  at["db"], over.get("ws", OK + (30 << 28)),
                                  over.get("size", eaga.linear_workspace_size(d, True)), None)


@pytest.mark.parametrize("args,code", [
    ((-1, 8, 8), 1), ((4, 0, 8), 1), ((4, 8, 0), 1), ((4, 65537, 8), 2), ((4, 8, 65537), 2), ((1 << 31, 8, 8), 2), ((4, 8, 8, "none", 7), 1),
])
def test_linear_dims(L, args, code):
    d = eaga.linear_dims(*args)
    assert linear_call(L, d) == code and linear_back(L, d) == code
    assert eaga.linear_workspace_size(d, False) == 0 and eaga.linear_workspace_size(d, True) == 0


def test_linear_pointers(L):
    d = eaga.linear_dims(64, 40, 24, "silu", "bf16")
    assert linear_call(L, None) == 1
    for k in ("X", "W", "Y", "ws"):
        assert linear_call(L, d, **{k: None}) == 1, k
    for k in ("X", "W", "b", "R", "Y", "Z", "ws"):
        assert linear_call(L, d, **{k: OK + (20 << 28) + 8}) == 3, k
    assert linear_call(L, d, size=eaga.linear_workspace_size(d, False) - 1) == 4
    assert linear_call(L, d, Y=OK + (4 << 28)) == 1 and linear_call(L, d, Z=OK + (5 << 28)) == 1      # Y over R, Z over Y
    for k in ("X", "W", "Z", "dY", "ws"):
        assert linear_back(L, d, **{k: None}) == 1, k
    for k in ("X", "W", "Z", "dY", "dR", "dX", "dW", "db", "ws"):
        assert linear_back(L, d, **{k: OK + (20 << 28) + 8}) == 3, k
    assert linear_back(L, d, size=eaga.linear_workspace_size(d, True) - 1) == 4
    assert linear_back(L, d, dX=None, dW=None, db=None, dR=None) == 1
    assert linear_back(L, d, dW=None) == 1                              # db without dW
    assert linear_back(L, d, dX=None) == 1                              # dR without dX
    assert linear_back(L, d, act_in=9) == 1 and linear_back(L, d, act_in=2, Zin=None) == 1
    assert linear_back(L, d, Zin=OK + (21 << 28)) == 1                  # an input activation's z without the activation
    assert linear_back(L, eaga.linear_dims(64, 40, 24), Z=OK + (21 << 28)) == 1
    assert linear_back(L, d, dX=OK + (6 << 28)) == 1                    # dX over dR
    with pytest.raises(ValueError):
        eaga.linear_dims(4, 8, 8, "tanh")


def test_binding_refuses_host_tensors(L):
    import torch
    d, n = eaga.linear_dims(4, 8, 8), norm_dims()
    host = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        eaga.linear_forward(d, host, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        eaga.linear_forward(d, None, None, None, None, None, None, None)
    with pytest.raises((ValueError, TypeError)):
        eaga.linear_forward(None, host, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        eaga.residual_norm_forward(n, None, host, None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        eaga.linear_forward(ctypes.c_int(4), host, None, None, None, None, None, None)      # too small for the dims
