"""A training step of a gated feed-forward sub-layer, as a program around the block strings the operators together:
norm, product with gelu, product, gated residual with the norm after and the next one before, a head's product; back through all
of them; one AdamW step over every parameter.  Against autograd in 64 bits.

Bounds (norm of the difference over norm of the gradient): in fp32 each of the eight operators adds at most K + 40 steps of
2^-23 of the magnitudes (K = 256, the longest reduction) and a norm passes errors on times at most about 4; in bf16 about ten tensors
are stored on the way, half a step of 2^-8 each, with the same 4."""
import pytest
import torch

from edge_aware_graph_b200 import eaga
from edge_aware_graph_b200.optim import AdamW

pytestmark = pytest.mark.gpu
TD = {"fp32": torch.float32, "bf16": torch.bfloat16}
BOUND = {"fp32": 8 * 4 * (256 + 40) * 2.0 ** -23, "bf16": 10 * 4 * 2.0 ** -8}
B, N, W, F, O = 6, 37, 136, 256, 48                       # graphs, rows of each, width, hidden width, outputs
EPS = 1e-5


class Step:
    def __init__(self, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        td = TD[dtype]
        new = lambda *s, d=1.0, m=0.0: (torch.randn(*s, generator=g) * d + m).to(td).cuda()
        rows = B * N
        self.x, self.gate, self.c = new(rows, W), new(B, W, d=0.3, m=1.0), new(rows, O)
        real = torch.randint(0, N + 1, (B, 1), generator=g)
        real[0] = 0                                       # a graph without a real row
        self.M = (torch.arange(N)[None] < real).to(torch.uint8).reshape(-1).cuda()
        self.P = dict(g0=new(W, d=0.1, m=1.0), s0=new(W, d=0.1), W1=new(W, F, d=W ** -0.5), b1=new(F, d=0.1), W2=new(F, W, d=F ** -0.5),
                      b2=new(W, d=0.1), pg=new(W, d=0.1, m=1.0), ps=new(W, d=0.1), g1=new(W, d=0.1, m=1.0), W3=new(W, O, d=W ** -0.5), b3=new(O, d=0.1))
        self.G = {k: torch.full(v.shape, float("nan"), device="cuda") for k, v in self.P.items()}
        e = lambda *s: torch.full(s, float("nan"), dtype=td, device="cuda")
        self.h0, self.Z1, self.a, self.u, self.r, self.h1, self.y = e(rows, W), e(rows, F), e(rows, F), e(rows, W), e(rows, W), e(rows, W), e(rows, O)
        self.dh1, self.dr, self.du, self.dgate, self.dZ1, self.dh0, self.dx = e(rows, W), e(rows, W), e(rows, W), e(B, W), e(rows, F), e(rows, W), e(rows, W)
        self.n0 = eaga.residual_norm_dims(rows, W, pre="layer", eps=EPS, dtype=dtype)
        self.n1 = eaga.residual_norm_dims(rows, W, pre="rms", post="layer", rows_per_group=N, eps=EPS, alpha=0.5, dtype=dtype)
        self.l1, self.l2, self.l3 = (eaga.linear_dims(rows, i, o, act, dtype) for i, o, act in ((W, F, "gelu"), (F, W, "none"), (W, O, "none")))
        self.l1b = eaga.linear_dims(rows, W, F, "none", dtype)      # its activation's gradient is taken in the second product's backward
        size = max([eaga.linear_workspace_size(d, b) for d in (self.l1, self.l1b, self.l2, self.l3) for b in (False, True)]
                   + [eaga.residual_norm_workspace_size(d) for d in (self.n0, self.n1)])
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.opt = AdamW(list(self.P.values()), list(self.G.values()), lr=1e-2, weight_decay=[0.01 if v.dim() > 1 else 0.0 for v in self.P.values()], bits=8)

    def forward(self):
        P = self.P
        eaga.residual_norm_forward(self.n0, None, self.x, None, None, None, None, P["g0"], P["s0"], None, self.h0)
        eaga.linear_forward(self.l1, self.h0, P["W1"], P["b1"], None, self.a, self.Z1, self.ws)
        eaga.linear_forward(self.l2, self.a, P["W2"], P["b2"], None, self.u, None, self.ws)
        eaga.residual_norm_forward(self.n1, self.x, self.u, self.M, self.gate, P["pg"], P["ps"], P["g1"], None, self.r, self.h1)
        eaga.linear_forward(self.l3, self.h1, P["W3"], P["b3"], None, self.y, None, self.ws)

    def backward(self):
        P, G = self.P, self.G
        eaga.linear_backward(self.l3, self.h1, P["W3"], None, self.c, self.dh1, G["W3"], G["b3"], self.ws)
        eaga.residual_norm_backward(self.n1, self.r, self.u, self.M, self.gate, P["pg"], P["ps"], P["g1"], None, self.dh1, self.dr, self.du, self.dgate,
                                    G["pg"], G["ps"], G["g1"], None, self.ws)
        eaga.linear_backward(self.l2, self.a, P["W2"], None, self.du, self.dZ1, G["W2"], G["b2"], self.ws, act_in="gelu", Zin=self.Z1)
        eaga.linear_backward(self.l1b, self.h0, P["W1"], None, self.dZ1, self.dh0, G["W1"], G["b1"], self.ws)
        eaga.residual_norm_backward(self.n0, self.x, None, None, None, None, None, P["g0"], self.dr, self.dh0, None, self.dx, None,
                                    None, None, G["g0"], G["s0"], self.ws)

    def step(self):
        self.forward()
        self.backward()
        self.opt.step()

    def reference(self):
        D = {k: v.double().requires_grad_() for k, v in self.P.items()}
        x, gate = self.x.double().requires_grad_(), self.gate.double().requires_grad_()

        def layer(z, gain, shift):
            z = z - z.mean(1, keepdim=True)
            return z / (z.pow(2).mean(1, keepdim=True) + EPS).sqrt() * gain + shift

        h0 = layer(x, D["g0"], D["s0"])
        z1 = h0 @ D["W1"] + D["b1"]
        u = (z1 * torch.special.ndtr(z1)) @ D["W2"] + D["b2"]
        r = 0.5 * x + gate.repeat_interleave(N, 0) * layer(u, D["pg"], D["ps"])
        keep = self.M[:, None].double()
        h1 = r / (r.pow(2).mean(1, keepdim=True) + EPS).sqrt() * D["g1"] * keep
        y = h1 @ D["W3"] + D["b3"]
        (y * self.c.double()).sum().backward()
        return dict(y=y, dx=x.grad, dgate=gate.grad, **{k: v.grad for k, v in D.items()})


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gradients_through_all(dtype):
    s = Step(dtype)
    s.forward()
    s.backward()
    ref = s.reference()
    got = dict(y=s.y, dx=s.dx, dgate=s.dgate, **s.G)
    for k, want in ref.items():
        err = float((got[k].double() - want.detach()).norm() / want.detach().norm())
        assert err <= BOUND[dtype], (k, err)
    assert (s.r[s.M == 0] == 0).all() and (s.h1[s.M == 0] == 0).all() and (s.dgate[0] == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_steps_replayed(dtype):
    """Three captured steps give, bit for bit, what three plain ones give: losses' inputs, gradients, weights, 8-bit states, the count."""
    a, b = Step(dtype), Step(dtype)
    for _ in range(3):
        a.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                         # nothing is left to look up while capturing
        Step(dtype, seed=1).step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert a.opt.steps == b.opt.steps == 3
    for k in a.P:
        assert torch.equal(a.P[k], b.P[k]) and torch.equal(a.G[k], b.G[k]), k
    assert torch.equal(a.y, b.y) and torch.equal(a.dx, b.dx)
    for x, y in zip(a.opt.m + a.opt.v, b.opt.m + b.opt.v):
        assert torch.equal(x, y)


def test_weights_move_against_their_gradients():
    s = Step("fp32")
    before = {k: v.clone() for k, v in s.P.items()}
    s.step()
    for k, v in s.P.items():
        g = s.G[k]
        moved = (v - before[k]) * g
        # the first step of AdamW is lr in the gradient's direction, decay aside (1e-4 of the weight)
        assert (moved[g.abs() > 1e-3 * g.abs().max()] < 0).float().mean() > 0.9, k
