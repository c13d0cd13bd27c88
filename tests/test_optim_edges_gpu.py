"""AdamW over weights that a program also differentiates, and what its Python side refuses."""
import pytest
import torch

from edge_aware_graph_b200.optim import AdamW

pytestmark = pytest.mark.gpu


def make(bits=8, n=(300, 17), **kw):
    g = torch.Generator().manual_seed(1)
    p = [torch.randn(k, generator=g).to("cuda", torch.bfloat16) for k in n]
    d = [torch.randn(k, generator=g).cuda() for k in n]
    return p, d, AdamW(p, d, bits=bits, **kw)


def test_weights_of_a_program_that_differentiates():
    """Masters and states are plain tensors: no graph is kept through them, and none grows with the checkpoints."""
    p, d, plain = make()
    leaves = [torch.nn.Parameter(t.clone()) for t in p]
    opt = AdamW(leaves, d, bits=8)
    for t in opt.master + opt.m + opt.v:
        assert not t.requires_grad and t.grad_fn is None
    opt.step()
    plain.step()
    s = opt.state_dict()
    assert not any(t.requires_grad for k in ("master", "m", "v", "m_scale", "v_scale") for t in s[k])
    opt.load_state_dict(s)
    for a, b in zip(opt.params + opt.master + opt.m + opt.v, plain.params + plain.master + plain.m + plain.v):
        assert torch.equal(a.detach(), b)


def test_unpacking_on_another_device_is_refused(monkeypatch):
    p, d, opt = make()
    opt.step()
    m, v = opt.unpack()
    run = opt.unpacker(m, v)
    before = [t.clone() for t in m + v]
    opt.step()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        run()
    with pytest.raises(ValueError, match="current device"):
        opt.unpack(m, v)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, m + v))
    run()
    assert not torch.equal(before[0], m[0])


def test_states_of_other_tensors_leave_the_optimiser_as_it_was():
    """A checkpoint that does not fit is refused whole: no part of it is loaded before the misfit is found."""
    p, d, opt = make()
    opt.step()
    good = opt.state_dict()
    opt.step()
    now = opt.state_dict()
    for k in ("master", "m", "v", "m_scale", "v_scale"):
        bad = {**good, k: good[k][:-1] + [torch.zeros(5, dtype=good[k][-1].dtype, device="cuda")]}
        with pytest.raises(ValueError, match=k):
            opt.load_state_dict(bad)
        with pytest.raises(ValueError, match=k):
            opt.load_state_dict({**good, k: None})
        with pytest.raises(ValueError, match=k):          # codes read as numbers, or numbers as codes
            opt.load_state_dict({**good, k: [t.to(torch.int16) for t in good[k]]})
        after = opt.state_dict()
        assert after["step"] == now["step"]
        for name in ("master", "m", "v", "m_scale", "v_scale"):
            assert all(torch.equal(a, b) for a, b in zip(after[name], now[name])), (k, name)
    opt.load_state_dict(good)
    assert opt.steps == 1 and all(torch.equal(a, b) for a, b in zip(opt.m, good["m"]))
