"""The residual step with its norms on the GPU against the formulas in 64 bits.

Tolerances come from a forward error analysis that runs beside the reference:
each value carries a bound of its absolute error.  One fp32 rounding is off by
2^-24 of its value; a sum over a row takes at most 40 of them on the sum of
magnitudes (8 to 16 in a thread, 9 levels of threads, the division); stores
round to half a step of the storage dtype (2^-8 for bf16, 2^-24 for fp32)."""
import numpy as np
import pytest
import torch

from edge_aware_graph_b200 import eaga

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SUM = 40 * U
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TD = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS, ALPHA = 1e-5, -0.75


class V:
    """A value and a bound of its error."""

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, np.float64)
        self.e = np.broadcast_to(np.asarray(e, np.float64), self.v.shape)

    def __add__(self, o):
        v = self.v + o.v
        return V(v, self.e + o.e + U * np.abs(v))

    def __sub__(self, o):
        return self + V(-o.v, o.e)

    def __mul__(self, o):
        v = self.v * o.v
        return V(v, self.e * np.abs(o.v) + o.e * np.abs(self.v) + self.e * o.e + U * np.abs(v))

    def mean(self):
        return V(self.v.mean(-1, keepdims=True), self.e.mean(-1, keepdims=True) + SUM * np.abs(self.v).mean(-1, keepdims=True))


def rsqrt(var):
    """1 / sqrt(var + eps), with a few roundings of its own."""
    s = var.v + EPS
    r = 1 / np.sqrt(s)
    rel = var.e / s
    return V(r, r * (np.where(rel < 0.5, 0.75 * rel, 10 * rel) + 6 * U))


def centre(z, kind):
    return z - z.mean() if kind == "layer" else z


def norm(z, kind, g, s):
    if kind == "none":
        return z
    c = centre(z, kind)
    y = c * rsqrt((c * c).mean())
    y = y * V(g) if g is not None else y
    return y + V(s) if s is not None else y


def norm_back(d, z, kind, g):
    """(gradient at z, z normalised)."""
    c = centre(z, kind)
    rs = rsqrt((c * c).mean())
    e = d * V(g) if g is not None else d
    zh = c * rs
    t = e - c * ((e * c).mean() * (rs * rs))
    if kind == "layer":
        t = t - e.mean()
    return t * rs, zh


def rows_sum(x):
    """Over rows: the kernel's order is a tree of runs; any order is off by at most (rows + 8) roundings of the magnitudes."""
    return V(x.v.sum(0), x.e.sum(0) + (len(x.v) + 8) * U * np.abs(x.v).sum(0))


def close(got, ref, dtype, name):
    got = got.detach().double().cpu().numpy().reshape(ref.v.shape)
    assert np.isfinite(got).all(), name
    tol = ref.e + HALF[dtype] * (np.abs(ref.v) + ref.e) + 1e-37
    bad = np.abs(got - ref.v) > tol
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref.v) / tol):.3g} of the bound"


class Case:
    def __init__(self, rows, w, group, pre, post, dtype, gate=True, res=True, mask="none", affine=True, shift=0.0, seed=0):
        g = torch.Generator().manual_seed(seed)
        td = TD[dtype]
        self.k = dict(rows=rows, w=w, group=group, pre=pre, post=post, dtype=dtype, gate=gate, res=res)
        new = lambda *s, m=0.0, d=1.0: (torch.randn(*s, generator=g) * d + m).to(td)
        self.t = t = {}
        t["u"], t["r"] = new(rows, w, m=shift, d=1.5), new(rows, w, m=shift)
        t["dr"], t["dh"] = new(rows, w), new(rows, w) if pre != "none" else None
        t["x"] = new(rows, w) if res else None
        t["gate"] = new(rows // group, w, m=0.5, d=0.5) if gate else None
        for n, kind in (("post", post), ("pre", pre)):
            t[n + "_g"] = new(w, m=1.0, d=0.2) if affine and kind != "none" else None
            t[n + "_s"] = new(w, d=0.2) if affine and kind == "layer" else None
        M = None
        if mask == "random":
            M = (torch.rand(rows, generator=g) < 0.6).to(torch.uint8)
        elif mask == "groups":                            # whole groups without a real row
            M = (torch.arange(rows) // group % 2 == 1).to(torch.uint8)
        elif mask == "none of them":
            M = torch.zeros(rows, dtype=torch.uint8)
        t["M"] = M
        self.d = eaga.residual_norm_dims(rows, w, pre=pre, post=post, rows_per_group=group, eps=EPS, alpha=ALPHA, dtype=dtype)

    def gpu(self):
        """The tensors on the GPU; masked rows hold what must not be read."""
        out = {k: None if v is None else v.cuda() for k, v in self.t.items()}
        if out["M"] is not None:
            dead = out["M"] == 0
            for k in ("u", "r", "dr", "dh", "x"):
                if out[k] is not None:
                    out[k][dead] = float("nan") if k != "x" else float("inf")
        return out

    def np(self, k):
        v = self.t[k]
        return None if v is None else v.double().numpy()

    def keep(self):
        return np.ones((self.k["rows"], 1)) if self.t["M"] is None else self.np("M")[:, None]

    def gates(self):
        return None if self.t["gate"] is None else V(np.repeat(self.np("gate"), self.k["group"], 0))

    def forward_ref(self):
        p = norm(V(self.np("u")), self.k["post"], self.np("post_g"), self.np("post_s"))
        r = p if self.t["gate"] is None else p * self.gates()
        if self.t["x"] is not None:
            r = r + V(self.np("x")) * V(ALPHA)
        keep = V(self.keep())
        h = norm(r, self.k["pre"], self.np("pre_g"), self.np("pre_s"))
        return r * keep, h * keep

    def backward_ref(self):
        keep, out, k = V(self.keep()), {}, self.k
        g = V(self.np("dr")) * keep
        if k["pre"] != "none":
            dh = V(self.np("dh")) * keep
            d, zh = norm_back(dh, V(self.np("r")), k["pre"], self.np("pre_g"))
            g = g + d
            out["dpre_g"], out["dpre_s"] = rows_sum(dh * zh), rows_sum(dh)
        out["dx"] = g * V(ALPHA)
        dp = g if self.t["gate"] is None else g * self.gates()
        u = V(self.np("u"))
        if self.t["gate"] is not None:
            gp = g * norm(u, k["post"], self.np("post_g"), self.np("post_s")) * keep
            n = k["rows"] // k["group"]
            gp = V(gp.v.reshape(n, k["group"], k["w"]).swapaxes(0, 1), gp.e.reshape(n, k["group"], k["w"]).swapaxes(0, 1))
            out["dgate"] = rows_sum(gp)
        out["du"] = dp
        if k["post"] != "none":
            out["du"], uh = norm_back(dp, u, k["post"], self.np("post_g"))
            out["dpost_g"], out["dpost_s"] = rows_sum(dp * uh), rows_sum(dp)
        out["du"] = out["du"] * keep
        return out

    def run_forward(self, stream=None):
        t = self.gpu()
        r = torch.full((self.k["rows"], self.k["w"]), 7.0, dtype=TD[self.k["dtype"]], device="cuda")
        h = r.clone() if self.k["pre"] != "none" else None
        eaga.residual_norm_forward(self.d, t["x"], t["u"], t["M"], t["gate"], t["post_g"], t["post_s"], t["pre_g"],
                                   t["pre_s"], r, h, stream)
        torch.cuda.synchronize()
        return r, h

    def outputs(self):
        k, td = self.k, TD[self.k["dtype"]]
        new = lambda *s, dtype=td: torch.full(s, 7.0, dtype=dtype, device="cuda")
        f = torch.float32
        o = dict(dx=new(k["rows"], k["w"]), du=new(k["rows"], k["w"]))
        o["dgate"] = new(k["rows"] // k["group"], k["w"]) if k["gate"] else None
        for n in ("post", "pre"):
            for x in ("_g", "_s"):
                o["d" + n + x] = new(k["w"], dtype=f) if k[n] != "none" else None
        return o

    def call_backward(self, t, o, ws, stream=None):
        eaga.residual_norm_backward(self.d, t["r"], t["u"], t["M"], t["gate"], t["post_g"], t["post_s"], t["pre_g"],
                                    t["dr"], t["dh"], o["dx"], o["du"], o["dgate"], o["dpost_g"], o["dpost_s"],
                                    o["dpre_g"], o["dpre_s"], ws, stream)

    def workspace(self):
        return torch.full((eaga.residual_norm_workspace_size(self.d),), 255, dtype=torch.uint8, device="cuda")

    def run_backward(self):
        o = self.outputs()
        self.call_backward(self.gpu(), o, self.workspace())
        torch.cuda.synchronize()
        return o

    def check(self):
        r, h = self.run_forward()
        er, eh = self.forward_ref()
        close(r, er, self.k["dtype"], "r")
        if h is not None:
            close(h, eh, self.k["dtype"], "h")
        got = self.run_backward()
        for n, ref in self.backward_ref().items():
            close(got[n], ref, "fp32" if n.startswith(("dpre", "dpost")) else self.k["dtype"], n)


WIDTHS = [1, 2, 7, 8, 16, 63, 64, 100, 129, 256, 257, 264, 777, 1024, 2048, 2056, 4096, 4097, 5000, 8192]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("w", WIDTHS)
def test_widths(w, dtype):
    Case(21, w, 7, "layer", "layer", dtype, mask="random", seed=w).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pre,post", [("layer", "none"), ("none", "layer"), ("rms", "rms"), ("rms", "none"),
                                      ("none", "rms"), ("rms", "layer"), ("none", "none")])
@pytest.mark.parametrize("gate,res,affine", [(True, True, True), (False, True, False), (True, False, True),
                                             (False, False, True)])
def test_forms(pre, post, gate, res, affine, dtype):
    Case(50, 96, 10, pre, post, dtype, gate=gate, res=res, affine=affine, seed=3).check()


@pytest.mark.parametrize("rows,group", [(1, 1), (33, 1), (33, 33), (200, 8), (5000, 1250), (4001, 4001), (30000, 15000)])
@pytest.mark.parametrize("mask", ["none", "random", "groups", "none of them"])
def test_rows_and_masks(rows, group, mask):
    Case(rows, 64, group, "layer", "layer", "bf16", mask=mask, seed=rows).check()


@pytest.mark.parametrize("w", [256, 1024, 6000])
@pytest.mark.parametrize("mask", ["groups", "none of them"])
def test_wide_masks(w, mask):
    Case(600, w, 60, "rms", "layer", "bf16", mask=mask, seed=w).check()


def test_far_mean_and_constant_rows():
    """Rows far from zero lose nothing to cancellation, and rows without variance divide by sqrt(eps)."""
    Case(64, 128, 64, "layer", "layer", "fp32", gate=False, shift=1000.0, seed=1).check()
    c = Case(8, 64, 8, "layer", "layer", "bf16", gate=False, res=False, seed=2)
    c.t["u"][:] = 3.25
    c.t["r"][:] = -2.0
    c.check()


def test_norm_alone():
    """A pre-norm alone: its input as u, no residual output."""
    c = Case(40, 200, 40, "layer", "none", "bf16", gate=False, res=False, seed=5)
    t = c.gpu()
    h = torch.empty_like(t["u"])
    eaga.residual_norm_forward(c.d, None, t["u"], None, None, None, None, t["pre_g"], t["pre_s"], None, h)
    torch.cuda.synchronize()
    close(h, c.forward_ref()[1], "bf16", "h")
    # backward: u is r, only dh comes in, and du is the gradient at the input
    du, dg = torch.empty_like(h), torch.empty(200, device="cuda")
    eaga.residual_norm_backward(c.d, t["u"], t["u"], None, None, None, None, t["pre_g"], None, t["dh"], None, du, None,
                                None, None, dg, None, c.workspace())
    torch.cuda.synchronize()
    d, zh = norm_back(V(c.np("dh")), V(c.np("u")), "layer", c.np("pre_g"))
    close(du, d, "bf16", "du")
    close(dg, rows_sum(V(c.np("dh")) * zh), "fp32", "dpre_g")


@pytest.mark.parametrize("pre,post", [("layer", "layer"), ("rms", "rms")])
def test_against_differences(pre, post):
    """The gradients along a direction against central differences of the
    forward formula in 64 bits (step 1e-6: off by its square and by 1e-10 of
    rounding over it, under 1e-7 of the terms' sum; the kernel's own 32 bits
    are allowed 200 roundings of that sum)."""
    c = Case(12, 40, 4, pre, post, "fp32", seed=9)
    r, h = c.forward_ref()
    c.t["r"] = torch.from_numpy(r.v).float()             # the forward's own r
    got = c.run_backward()
    rng = np.random.default_rng(0)

    def loss():
        r, h = c.forward_ref()
        return (r.v * c.np("dr")).sum() + (h.v * c.np("dh")).sum()

    for n in ("x", "u", "gate", "post_g", "post_s", "pre_g", "pre_s"):
        if c.t[n] is None:
            continue
        base, dirn = c.t[n], torch.from_numpy(rng.standard_normal(tuple(c.t[n].shape)))
        vals = []
        for s in (1e-6, -1e-6):
            c.t[n] = base.double() + s * dirn
            vals.append(loss())
        c.t[n] = base
        terms = got["d" + n].double().cpu().numpy() * dirn.numpy()
        size = np.abs(terms).sum() + np.abs(r.v * c.np("dr")).sum()
        assert abs(terms.sum() - (vals[0] - vals[1]) / 2e-6) <= (1e-7 + 200 * U) * size, n


def test_reproducible_captured_and_on_a_stream():
    c = Case(3000, 64, 1000, "layer", "layer", "bf16", mask="random", seed=11)
    t, ws = c.gpu(), c.workspace()
    first = c.run_backward()
    o = c.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.call_backward(t, o, ws, s)
    for _ in range(2):
        for v in o.values():
            if v is not None:
                v.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for n, v in first.items():
            assert v is None or torch.equal(v, o[n]), n
    del graph
    r, h = c.run_forward(stream=torch.cuda.default_stream())
    r2, h2 = c.run_forward()
    assert torch.equal(r, r2) and torch.equal(h, h2)


def test_no_rows():
    c = Case(0, 64, 1, "layer", "layer", "bf16", gate=True)
    r, h = c.run_forward()
    o = c.run_backward()
    assert r.numel() == 0 and all(float(o[n].abs().sum()) == 0 for n in ("dpre_g", "dpre_s", "dpost_g", "dpost_s"))


def test_far_offsets():
    """More than 2^31 elements: the last rows are where they belong."""
    rows, w = (1 << 31) // 8192 + 3, 8192
    d = eaga.residual_norm_dims(rows, w, pre="rms", rows_per_group=1, eps=EPS, alpha=1.0)
    u = torch.zeros(rows, w, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    tail = torch.randn(5, w, generator=g).to(torch.bfloat16)
    u[-5:] = tail.cuda()
    h = torch.full_like(u, 7.0)
    eaga.residual_norm_forward(d, None, u, None, None, None, None, None, None, None, h)
    torch.cuda.synchronize()
    assert float(h[:-5].abs().max()) == 0.0
    close(h[-5:], norm(V(tail.double().numpy()), "rms", None, None), "bf16", "h")


def test_refusals():
    c = Case(10, 64, 5, "layer", "layer", "bf16")
    t, ws = c.gpu(), c.workspace()
    r, h = torch.empty_like(t["u"]), torch.empty_like(t["u"])
    call = lambda **k: eaga.residual_norm_forward(
        c.d, *[{**t, "r": r, "h": h, **k}[n] for n in ("x", "u", "M", "gate", "post_g", "post_s", "pre_g", "pre_s", "r", "h")])
    call()
    for bad in (dict(u=t["u"].float()), dict(u=t["u"][:9]), dict(gate=t["gate"][:1]), dict(r=r.t().contiguous().t()),
                dict(u=t["u"].cpu()), dict(u=None)):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(h=None), dict(h=r), dict(r=t["u"])):
        with pytest.raises(eaga.EagaError) as e:
            call(**bad)
        assert e.value.code == 1
    o = c.outputs()
    with pytest.raises(eaga.EagaError) as e:
        c.call_backward(t, o, ws[:-256])
    assert e.value.code == 4
    with pytest.raises(eaga.EagaError) as e:
        c.call_backward(t, {**o, "du": o["dx"]}, ws)
    assert e.value.code == 1
    torch.cuda.synchronize()
