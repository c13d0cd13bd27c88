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


@pytest.mark.parametrize("bits", [8, 32])
def test_offsets_beyond_2_31_elements(bits):
    """One tensor of 2^31 + 4099 elements: its far end takes the same step as a tensor of that end alone, its random bits among it."""
    n, far = (1 << 31) + 4099, (1 << 31) - 256
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    rng = torch.Generator(device="cuda").manual_seed(2)
    end = slice(far, n)
    p[end] = torch.randn(n - far, generator=rng, device="cuda").bfloat16()
    g[end] = torch.randn(n - far, generator=rng, device="cuda").bfloat16()
    kw = dict(bits=bits, master=False, weight_decay=0.0, lr=1e-2, seed=3)
    small_p, small_g = p[end].clone(), g[end].clone()
    big, small = AdamW([p], [g], counters=[5], **kw), AdamW([small_p], [small_g], counters=[5 + far], **kw)
    for _ in range(2):
        big.step()
        small.step()
    assert torch.equal(p[end], small_p) and torch.equal(big.m[0][end], small.m[0]) and torch.equal(big.v[0][end], small.v[0])
    if bits == 8:
        assert torch.equal(big.m_scale[0][far // 256:], small.m_scale[0]) and torch.equal(big.v_scale[0][far // 256:], small.v_scale[0])
    for t in (p[:far], big.m[0][:far], big.v[0][:far]):
        assert int(torch.count_nonzero(t)) == 0
