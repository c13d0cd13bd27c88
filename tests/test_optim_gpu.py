"""The AdamW step on the GPU against the same operations in numpy.

Every operation of the step is rounded to fp32 on its own, so numpy's float32
gives the same bits: weights, masters, states and 8-bit codes are compared for
equality.  The formula itself is checked in 64 bits: one fp32 rounding is off
by at most 2^-24 of its value, and m', v' and p' take at most 3, 4 and 8 of
them on terms no larger than the sum of the magnitudes added."""
import numpy as np
import pytest
import torch

from edge_aware_graph_b200 import eaga
from edge_aware_graph_b200 import inputs as I
from edge_aware_graph_b200.buffers import BlockBuffers, LayerBuffers
from edge_aware_graph_b200.optim import AdamW

pytestmark = pytest.mark.gpu
f4 = np.float32
U = 2.0 ** -24
TD = {"fp32": torch.float32, "bf16": torch.bfloat16}


def mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    lo = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x6C8E9CF5)) & lo
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x5B2D1A67)) & lo
    return x ^ (x >> np.uint64(16))


def blocks_of(a):
    pad = -len(a) % 256
    return np.concatenate([a, np.zeros(pad, a.dtype)]).reshape(-1, 256)


def encode(a, top, rnd, shift, most):
    """Codes of non-negative fp32 values over their block's scale, and the scales."""
    b = blocks_of(a)
    big = b.max(1, keepdims=True)
    scale = big / f4(top)
    with np.errstate(all="ignore"):
        y = np.where(big == 0, f4(0), b / scale) * f4(2.0 ** -112)
    y = np.ascontiguousarray(y.reshape(-1)[:len(a)])
    return np.minimum((y.view(np.uint32).astype(np.uint64) + rnd) >> np.uint64(shift), np.uint64(most)), scale.reshape(-1)


def decode(code, scale, shift):
    y = (code.astype(np.uint32) << np.uint32(shift)).view(f4) * f4(2.0 ** 112)
    return (blocks_of(y) * scale[:, None]).reshape(-1)[:len(code)]


def decode_m(code, scale):
    a = decode(code & 127, scale, 20)
    return np.where(code > 127, -a, a)


class Model:
    """One tensor's weight and states in numpy."""

    def __init__(self, p, bits, counter, wd):
        n = len(p)
        self.p, self.bits, self.counter, self.wd = p.copy(), bits, counter, f4(wd)
        self.m = np.zeros(n, f4 if bits == 32 else np.uint8)
        self.v = np.zeros(n, f4 if bits == 32 else np.uint8)
        self.ms = np.zeros(-(-n // 256), f4)
        self.vs = np.zeros(-(-n // 256), f4)

    def states(self):
        if self.bits == 32:
            return self.m, self.v
        r = decode(self.v, self.vs, 19)
        return decode_m(self.m, self.ms), r * r

    def step(self, g, t, lr, b1, b2, eps, scale=1.0, seed=0, round_p=None):
        m, v = self.states()
        g = g * f4(scale)
        m = m * f4(b1) + g * f4(1 - b1)
        v = v * f4(b2) + (g * g) * f4(1 - b2)
        r = np.sqrt(v)
        size, inv = f4(lr / (1 - b1 ** t)), f4(1 / np.sqrt(1 - b2 ** t))
        keep = f4(1.0 - lr * float(self.wd))
        self.p = self.p * keep - (m / (r * inv + f4(eps))) * size
        if round_p is not None:
            self.p = round_p(self.p)
        if self.bits == 32:
            self.m, self.v = m, v
            return
        key = mix(t * 0x9E3779B9 + seed)
        h = mix(np.arange(len(m), dtype=np.uint64) + np.uint64(self.counter) + key)
        a, self.ms = encode(np.abs(m), 1.875, h >> np.uint64(12), 20, 127)
        self.m = (a | (np.uint64(128) * (m < 0))).astype(np.uint8)
        h2 = (h * np.uint64(0x3C6EF35F)) & np.uint64(0xFFFFFFFF)
        b, self.vs = encode(r, 1.9375, h2 >> np.uint64(13), 19, 255)
        self.v = np.where(r > 0, np.maximum(b, 1), b).astype(np.uint8)


def to_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).float().numpy()


def make(sizes, pd, gd, bits, master, seed=0, **kw):
    rng = np.random.default_rng(seed)
    p = [rng.standard_normal(n).astype(f4) * f4(0.1) for n in sizes]
    dev = [torch.from_numpy(a).to("cuda", TD[pd]) for a in p]
    if pd == "bf16" and not master:
        p = [to_bf16(a) for a in p]
    g = [torch.zeros(n, dtype=TD[gd], device="cuda") for n in sizes]
    mast = [torch.from_numpy(a).cuda() for a in p] if master else (False if pd == "bf16" else None)
    opt = AdamW(dev, g, bits=bits, master=mast, seed=seed, **kw)
    decay = kw.get("weight_decay", 0.01)
    off = np.concatenate([[0], np.cumsum(sizes)])
    ref = [Model(a, bits, off[i], decay[i] if hasattr(decay, "__len__") else decay) for i, a in enumerate(p)]
    return dev, g, opt, ref, rng


def draw_grads(rng, g, step):
    out = []
    for i, t in enumerate(g):
        a = (rng.standard_normal(t.numel()) * 10.0 ** -(1 + (i + step) % 4)).astype(f4)
        if t.numel() > 3 and i % 3 == 1:
            a[:: 2] = 0                                 # elements that no gradient reached
        t.copy_(torch.from_numpy(a))
        out.append(t.float().cpu().numpy())
    return out


def same(opt, dev, ref, master):
    torch.cuda.synchronize()
    for i, r in enumerate(ref):
        p = dev[i].float().cpu().numpy()
        if master:
            assert np.array_equal(opt.master[i].cpu().numpy(), r.p), i
            assert np.array_equal(p, to_bf16(r.p)), i
        else:
            assert np.array_equal(p, r.p), i
        assert np.array_equal(opt.m[i].cpu().numpy(), r.m), i
        assert np.array_equal(opt.v[i].cpu().numpy(), r.v), i
        if r.bits == 8:
            assert np.array_equal(opt.m_scale[i].cpu().numpy(), r.ms), i
            assert np.array_equal(opt.v_scale[i].cpu().numpy(), r.vs), i


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,gd,master", [("fp32", "fp32", False), ("fp32", "bf16", False), ("bf16", "fp32", True),
                                          ("bf16", "bf16", True), ("bf16", "fp32", False), ("bf16", "bf16", False)])
def test_steps_equal_numpy(bits, pd, gd, master):
    """Odd lengths, ends inside a vector, a scale block and a tile, and one of several tiles."""
    sizes = [1, 5, 8, 255, 256, 257, 1000, 2047, 2049, 70001]
    decay = [0.0 if i % 2 else 0.1 for i in range(len(sizes))]
    dev, g, opt, ref, rng = make(sizes, pd, gd, bits, master, lr=3e-3, weight_decay=decay, seed=7)
    for t in range(1, 5):
        gr = draw_grads(rng, g, t)
        opt.step(grad_scale=0.5 if t == 3 else 1.0)
        for r, a in zip(ref, gr):
            r.step(a, t, 3e-3, 0.9, 0.999, 1e-8, 0.5 if t == 3 else 1.0, 7,
                   to_bf16 if pd == "bf16" and not master else None)
        same(opt, dev, ref, master)
    assert opt.steps == 4


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More tensors than one launch's table holds, empty ones among them: each takes the same step."""
    sizes = [(17 * i) % 301 for i in range(801)]
    dev, g, opt, ref, rng = make(sizes, "bf16", "fp32", bits, True, lr=1e-2)
    for t in (1, 2):
        gr = draw_grads(rng, g, t)
        opt.step()
        for r, a in zip(ref, gr):
            if len(a):
                r.step(a, t, 1e-2, 0.9, 0.999, 1e-8)
    same(opt, dev, ref, True)
    assert opt.steps == 2


def test_against_64_bits():
    n = 5000
    dev, g, opt, _, rng = make([n], "fp32", "fp32", 32, False, lr=1e-3, weight_decay=0.05)
    p, m, v = dev[0].double().cpu().numpy(), np.zeros(n), np.zeros(n)
    for t in range(1, 4):
        gr = draw_grads(rng, g, t)[0].astype(np.float64)
        opt.step()
        ep, em, ev = (x.cpu().numpy().astype(np.float64) for x in (dev[0], opt.m[0], opt.v[0]))
        m1, v1 = 0.9 * m + 0.1 * gr, 0.999 * v + 0.001 * gr ** 2
        up = 1e-3 / (1 - 0.9 ** t) * m1 / (np.sqrt(v1 / (1 - 0.999 ** t)) + 1e-8)
        p1 = (1 - 1e-3 * float(f4(0.05))) * p - up
        # the constants 0.1 and 0.001 are rounded to fp32 too: one more rounding of a term
        assert np.all(np.abs(em - m1) <= 4 * U * (np.abs(0.9 * m) + np.abs(0.1 * gr)))
        assert np.all(np.abs(ev - v1) <= 6 * U * v1 + 1e-44)
        small = np.abs(0.9 * m) + np.abs(0.1 * gr)      # m' may cancel: its own error enters the update
        eu = 12 * U * np.abs(up) + np.abs(up) * 4 * U * small / np.maximum(np.abs(m1), 1e-300)
        assert np.all(np.abs(ep - p1) <= 4 * U * np.abs(p) + eu)
        p, m, v = ep, em, ev                            # each step from the step before as it is held


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_count(bits):
    """A captured step counts its replays, reads its rate from the device, and equals as many steps one by one."""
    sizes = [300, 5000]
    dev, g, opt, ref, rng = make(sizes, "bf16", "fp32", bits, True, weight_decay=0.02, lr=1.0)
    lr = torch.tensor([1e-2], device="cuda")
    gr = draw_grads(rng, g, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        opt.step(lr=lr)
    assert opt.steps == 0
    rates = [1e-2, 5e-3, 2e-3]
    for t, x in enumerate(rates, 1):
        lr.fill_(x)
        graph.replay()
        for r, a in zip(ref, gr):
            r.step(a, t, float(f4(x)), 0.9, 0.999, 1e-8)
    same(opt, dev, ref, True)
    assert opt.steps == 3
    del graph


def test_other_stream():
    dev, g, opt, ref, rng = make([4096], "fp32", "fp32", 32, False)
    gr = draw_grads(rng, g, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    opt.step(stream=s)
    ref[0].step(gr[0], 1, 1e-3, 0.9, 0.999, 1e-8)
    same(opt, dev, ref, False)


def test_nothing_to_do_and_zero_gradients():
    dev, g, opt, ref, _ = make([512, 0, 3], "fp32", "fp32", 8, False, weight_decay=0.0)
    before = [d.clone() for d in dev]
    opt.step()                                          # m = v = 0: 0 / eps
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(dev, before))
    assert all(int(x.abs().sum()) == 0 for x in opt.m + opt.v)
    assert opt.steps == 1


def test_bad_gradient_shows():
    """A NaN reaches its own element at 32 bits, its block's states at 8, and no other block."""
    for bits in (32, 8):
        dev, g, opt, _, _ = make([1024], "fp32", "fp32", bits, False)
        g[0].fill_(0.5)
        g[0][300] = float("nan")
        opt.step()
        p = dev[0].cpu().numpy()
        assert np.isnan(p[300]) and np.isnan(p).sum() == 1
        m, v = opt.unpack() if bits == 8 else (opt.m, opt.v)
        bad = np.isnan(m[0].cpu().numpy())
        assert bad[300] and not bad[:256].any() and not bad[512:].any()


def test_unpack_and_state_dict():
    sizes = [700, 33]
    dev, g, opt, ref, rng = make(sizes, "bf16", "fp32", 8, True, seed=3)
    for t in (1, 2):
        gr = draw_grads(rng, g, t)
        opt.step()
        for r, a in zip(ref, gr):
            r.step(a, t, 1e-3, 0.9, 0.999, 1e-8, 1.0, 3)
    m, v = opt.unpack()
    for i, r in enumerate(ref):
        em, ev = r.states()
        assert np.array_equal(m[i].cpu().numpy(), em) and np.array_equal(v[i].cpu().numpy(), ev)
    saved = opt.state_dict()
    weights = [d.clone() for d in dev]
    gr = draw_grads(rng, g, 3)
    opt.step()
    after = [d.clone() for d in dev]
    for d, w in zip(dev, weights):
        d.copy_(w)
    again = AdamW(dev, g, bits=8, seed=3)
    again.load_state_dict(saved)
    again.step()
    torch.cuda.synchronize()
    assert again.steps == 3
    assert all(torch.equal(a, b) for a, b in zip(dev, after))
    assert all(torch.equal(a, b) for a, b in zip(again.m + again.v, opt.m + opt.v))


def test_8_bit_states_follow():
    """A slowly moving second moment is followed on average: a block whose
    gradients stop at half of its places.  After 300 steps the exact v there
    is 0.999^300 = 0.74 of what it was; rounding to nearest would leave the
    codes where they are next to places that hold their value.  The mean over
    1000 blocks' halves (128000 places) of a walk of 300 roundings, each at
    most 2^-4 of r and unbiased, is within 1 %."""
    n = 256 * 1000
    p, g = [torch.zeros(n, device="cuda")], [torch.ones(n, device="cuda")]
    one = torch.ones(n, device="cuda")
    opt = AdamW(p, g, bits=8, lr=0.0, weight_decay=0.0)
    for _ in range(20):
        opt.step()
    _, v0 = opt.unpack()
    # from here the even places see nothing, and the odd ones gradients that hold r where it is
    r0 = v0[0].sqrt()
    g[0].copy_(torch.where(torch.arange(n, device="cuda") % 2 == 1, r0, torch.zeros_like(one)))
    for _ in range(300):
        opt.step()
    _, v1 = opt.unpack()
    ratio = (v1[0].sqrt()[::2].double().mean() / r0[::2].double().mean()).item()
    assert abs(ratio - 0.999 ** 150) < 0.01 * 0.999 ** 150
    hold = (v1[0].sqrt()[1::2].double().mean() / r0[1::2].double().mean()).item()
    assert abs(hold - 1) < 0.01


def test_layer_and_block_optimizers():
    """A layer's and a block's own weights and flat gradients, one training step each."""
    p = I.preset("sbm", B=2)
    d, W = I.draw_inputs(p, with_grads=True), I.draw_weights(p)
    buf = LayerBuffers(p.B, p.n, p.dx, p.de, p.dy, p.H, p.dh, dtype=p.dtype)
    buf.load_inputs(d, W)
    buf.forward()
    buf.backward()
    opt = buf.optimizer(lr=1e-2, bits=32)
    before = {k: v.clone() for k, v in buf.W.items()}
    opt.step()
    torch.cuda.synchronize()
    for k, w in before.items():
        # the first step: m' / sqrt(v') is the gradient's sign (to eps), so a weight moves by lr where there is a gradient
        dw = buf.dW[k]
        want = (w.float() * (1 - (1e-2 * 0.01 if w.dim() > 1 else 0.0)) - 1e-2 * dw / (dw.abs() + 1e-8)).to(w.dtype)
        got, want = buf.W[k].float(), want.float()
        # under 16 fp32 roundings of the terms, which may cancel; then at most the neighbouring bf16 value, one step 2^-7
        tol = 16 * U * (w.float().abs() + 1e-2)
        assert torch.all((got - want).abs() <= 2.0 ** -7 * (want.abs() + tol) + tol)
    b = BlockBuffers(p.B, p.n, p.dx, p.de, p.dy, p.H, p.dh, dtype=p.dtype)
    b.load_inputs(d, W)
    b.load_block(I.draw_block_weights(p), I.draw_block_upstream(p))
    opt = b.optimizer(bits=8)
    b.block_forward()
    b.block_backward()
    w0 = b.Wb["x_W1"].clone()
    opt.step()
    assert opt.steps == 1 and len(opt.sizes) == 39
    assert not torch.equal(w0, b.Wb["x_W1"])
    assert eaga.get_device_status(b.bws_bwd) == 0
    with pytest.raises(ValueError):
        LayerBuffers(2, 16, 256, 64, 64, 8, 32, backward=False).optimizer()


def test_refusals():
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    for bad in (dict(bits=16), dict(weight_decay=[0.1, 0.2]), dict(m=[torch.zeros(63, device="cuda")]),
                dict(master=[p.clone()])):
        with pytest.raises(ValueError):
            AdamW([p], [g], **bad)
    for params, grads in (([p], [g, g]), ([p.half()], [g]), ([p], [g.cpu()]), ([p[::2]], [g[:32]]), ([], [])):
        with pytest.raises(ValueError):
            AdamW(params, grads)
    for kw, code in ((dict(weight_decay=-1.0), 1), (dict(betas=(1.0, 0.9)), 1), (dict(eps=0.0), 1),
                     (dict(lr=float("nan")), 1)):
        with pytest.raises(eaga.EagaError) as e:
            AdamW([p], [g], **kw).step()
        assert e.value.code == code
    for params, grads in (([p, p], [g, g.clone()]), ([p], [p]), ([p[:32], p[16:48]], [g[:32], g[32:].clone()])):
        with pytest.raises(eaga.EagaError) as e:     # the same memory written twice, or written and read
            AdamW(params, grads).step()
        assert e.value.code == 1
    with pytest.raises(eaga.EagaError) as e:
        AdamW([p[1:33]], [g[:32]]).step()
    assert e.value.code == 3
    shared = AdamW([p, p.clone()], [g, g], lr=0.0)     # a gradient may be read twice
    shared.step()
    with pytest.raises(ValueError):
        shared.unpack()
