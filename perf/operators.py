"""The operators around the graph-transformer block that a training or serving program calls beside it, as cases to measure:

  linear_forward    Y = act(X W + b) + R, and Z = X W + b where the backward needs it
  linear_backward   dZ = act'(Z) dY;  dX = act_in'(Zin) (dZ W^T) + dR;  dW = X^T dZ;  db = sum of dZ's rows
  norm_forward      p = post_norm(u);  r = alpha x + gate p;  h = pre_norm(r)      (rows that M masks: r = h = 0)
  norm_backward     the gradients of x, u, the gate and the norms' gains and shifts from dr and dh
  adamw             one AdamW step over all tensors of a model, with states in 32 or in 8 bits

`run` computes them from elementary torch operations in 32 bits where `own` is false, and calls the framework where it is true."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    L, B, N, G, A = "linear_forward", "linear_backward", "norm_forward", "norm_backward", "adamw"
    return [
        # serving one token or graph: the weights are read once for a single row
        dict(name="linear 1x4096x4096", op=L, rows=1, inp=4096, out=4096, act="none", bias=True, res=True, save=False, dtype="bf16"),
        # the first FFN product on the edges of the SBM batch (32 graphs of 192 nodes), bound by memory
        dict(name="linear edges 64x128", op=L, rows=32 * 192 * 192, inp=64, out=128, act="relu", bias=True, res=False, save=False, dtype="bf16"),
        # a wide FFN product of a training step, bound by the tensor cores
        dict(name="linear 8192x4096x4096", op=L, rows=8192, inp=4096, out=4096, act="gelu", bias=True, res=True, save=True, dtype="bf16"),
        # an output head in 32 bits: odd sizes, rows that are not aligned
        dict(name="linear fp32 1001x257x131", op=L, rows=1001, inp=257, out=131, act="silu", bias=True, res=False, save=True, dtype="fp32"),
        # the second FFN product on the nodes of the SBM batch, its gradient passed on through the relu before it
        dict(name="linear bwd nodes 512x256", op=B, rows=32 * 192, inp=512, out=256, act="none", act_in="relu", bias=True, res=False, dtype="bf16"),
        # the same product at the size of a wide model, with the residual's gradient added
        dict(name="linear bwd 8192x4096x4096", op=B, rows=8192, inp=4096, out=4096, act="none", act_in="none", bias=True, res=True, dtype="bf16"),
        # the global features of 32 graphs: the smallest call
        dict(name="norm y 32x64", op=N, rows=32, w=64, group=1, pre="layer", post="layer", gate=True, res=True, mask=False, dtype="bf16"),
        # a long prompt's rows at the width of a wide model
        dict(name="norm rms 8192x4096", op=N, rows=8192, w=4096, group=8192, pre="rms", post="rms", gate=False, res=True, mask=False, dtype="bf16"),
        # the edges of the SBM batch, gated per graph, padded rows masked
        dict(name="norm bwd edges x64", op=G, rows=32 * 192 * 192, w=64, group=192 * 192, pre="layer", post="layer", gate=True, res=True, mask=True, dtype="bf16"),
        # nodes in 32 bits at an odd width
        dict(name="norm bwd fp32 777x333", op=G, rows=777, w=333, group=37, pre="layer", post="none", gate=True, res=True, mask=False, dtype="fp32"),
        # one block of the SBM configuration: 39 small tensors, where latency counts
        dict(name="adamw 1 block", op=A, blocks=1, dx=256, de=64, dy=64, bits=32, dtype="bf16", grad="fp32", step=10),
        # a deep stack at the widest block, states in 8 bits
        dict(name="adamw 8 bit 24 blocks", op=A, blocks=24, dx=512, de=64, dy=64, bits=8, dtype="bf16", grad="fp32", step=1000),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A row length: mostly a multiple of 8, sometimes any number."""
    v = _spread(rng, lo, hi)
    return v if rng.random() < 0.3 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["linear_forward", "linear_forward", "linear_backward", "linear_backward", "norm_forward", "norm_backward", "adamw"])
    yes = lambda p=0.5: rng.random() < p  # noqa: E731
    if op.startswith("linear"):
        dtype = "bf16" if yes(0.8) else "fp32"
        inp, out = _width(rng, 8, 4096), _width(rng, 4, 4096)
        # at most the largest listed case's products, and a tenth of it in 32 bits
        top = min(1_200_000, (8192 * 4096 * 4096 // (1 if dtype == "bf16" else 10)) // (inp * out), 75_000_000 // max(inp, out))
        c = dict(op=op, rows=_spread(rng, 1, max(1, top)), inp=inp, out=out, act=rng.choice(["none", "relu", "gelu", "silu"]), bias=yes(0.8), res=yes(), dtype=dtype)
        if op == "linear_forward":
            return dict(c, save=yes())
        # most gradients have passed the activation already, in the product that made them
        return dict(c, act=c["act"] if yes(0.3) else "none", act_in=rng.choice(["none", "relu", "gelu", "silu"]))
    if op.startswith("norm"):
        w = _width(rng, 16, 8192)
        rows = _spread(rng, 1, 33_554_432 // w)
        group = _spread(rng, 1, rows)
        rows = rows // group * group
        kinds = rng.choice([("layer", "layer"), ("layer", "none"), ("none", "layer"), ("rms", "rms"), ("rms", "none"), ("rms", "layer")])
        return dict(op=op, rows=rows, w=w, group=group, pre=kinds[0], post=kinds[1], gate=yes(), res=yes(0.8), mask=yes(), dtype="bf16" if yes(0.8) else "fp32")
    dtype = rng.choice(["bf16", "fp32"])
    return dict(op=op, blocks=_spread(rng, 1, 16), dx=rng.choice([64, 120, 256, 512]), de=rng.choice([24, 64]), dy=_width(rng, 8, 128), bits=rng.choice([8, 32]), dtype=dtype,
                grad=rng.choice(["fp32", "fp32", "bf16"]), step=_spread(rng, 1, 100000) - 1)


# ---------------------------------------------------------------- inputs

def _sizes(case):
    """Element counts of the parameters of `blocks` graph-transformer blocks and the attention layers in them."""
    dx, de, dy, hd, f = case["dx"], case["de"], case["dy"], 256, 16
    one = [dx * hd, hd] * 3 + [de * f, dy * f, f, 8 * de, hd * dx, dx]
    for w in (dx, de, dy):
        one += [w, w, 2 * w * w, 2 * w, 2 * w * w, w, w, w]
    return (one + [dx * dy, de * dy, dy]) * case["blocks"]


def _offsets(sizes, to=256):
    """Where each tensor begins in a flat buffer, on whole blocks of `to` elements, and the buffer's length."""
    at, off = [], 0
    for n in sizes:
        at.append(off)
        off += -(-n // to) * to
    return at, off


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)

    s = dict(case=dict(case))
    op = case["op"]
    if op.startswith("linear"):
        n, k, o = case["rows"], case["inp"], case["out"]
        s["W"] = normal(k, o, scale=k ** -0.5)
        s["b"] = normal(o, scale=0.5) if case["bias"] else None
        if op == "linear_forward":
            s["X"], s["R"] = normal(n, k), normal(n, o) if case["res"] else None
        else:
            s["Zin"] = normal(n, k) if case["act_in"] != "none" else None
            s["X"] = normal(n, k) if s["Zin"] is None else _act(s["Zin"].float(), case["act_in"]).to(dt)
            s["Z"] = normal(n, o) if case["act"] != "none" else None
            s["dY"], s["dR"] = normal(n, o), normal(n, k) if case["res"] else None
    elif op.startswith("norm"):
        n, w = case["rows"], case["w"]
        s["u"] = normal(n, w, scale=1.5, shift=0.3)
        s["x"] = normal(n, w) if case["res"] else None
        s["gate"] = normal(n // case["group"], w, scale=0.5, shift=0.5) if case["gate"] else None
        for k in ("post", "pre"):
            s[k + "_g"] = normal(w, scale=0.2, shift=1.0) if case[k] != "none" else None
            s[k + "_s"] = normal(w, scale=0.2) if case[k] == "layer" else None
        s["M"] = None
        if case["mask"]:  # padded graphs: each group's first rows are real, as many as it has
            real = torch.rand(n // case["group"], 1, generator=g, device=DEV) * (case["group"] + 1)
            s["M"] = (torch.arange(case["group"], device=DEV)[None] < real).to(torch.uint8).reshape(-1).contiguous()
        if op == "norm_backward":
            s["r"], s["dr"], s["dh"] = normal(n, w, shift=0.2), normal(n, w), normal(n, w) if case["pre"] != "none" else None
    else:
        sizes = _sizes(case)
        at, n = _offsets(sizes)
        s["sizes"], s["at"] = sizes, at
        live = torch.zeros(n, device=DEV)
        s["decay"] = torch.zeros(n, device=DEV)  # matrices decay, biases and gains do not
        size = torch.zeros(n, device=DEV)  # each tensor's gradients have a size of their own
        for i, (a, m) in enumerate(zip(at, sizes)):
            live[a:a + m] = 1
            s["decay"][a:a + m] = 0.01 if m > 1024 else 0.0
            size[a:a + m] = 10.0 ** -(1 + i % 5)
        grad = torch.randn(n, generator=g, device=DEV) * size * live
        s["g"] = grad.to(DTYPES[case["grad"]])
        p = torch.randn(n, generator=g, device=DEV) * 0.05 * live
        s["p"] = p.to(dt)
        s["master"] = p if case["dtype"] == "bf16" else None
        m = torch.randn(n, generator=g, device=DEV) * size * 0.3 * live
        r = size * (0.5 + torch.rand(n, generator=g, device=DEV)) * live
        if case["step"] == 0:
            m, r = m * 0, r * 0
        if case["bits"] == 32:
            s["m"], s["v"] = m, r * r
        else:
            h = _mix(torch.arange(n, device=DEV) + int(seed) % 1000)
            s["m"], s["m_scale"] = _pack_m(m, h)
            s["v"], s["v_scale"] = _pack_r(r, h)
        s["t"] = torch.full((), case["step"], dtype=torch.int64, device=DEV)
        s["seed"] = 1234
    if own:
        _plan(s, op, case)
    return s


# ---------------------------------------------------------------- the plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * (0.5 + 0.5 * torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 + 0.5 * torch.erf(z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    e = 1 / (1 + torch.exp(-z))
    return e * (1 + z * (1 - e))


def _f(t):
    return None if t is None else t.float()


def _linear_forward(s, c, dt):
    z = _f(s["X"]) @ _f(s["W"])
    if s["b"] is not None:
        z = z + _f(s["b"])
    y = _act(z, c["act"])
    if s["R"] is not None:
        y = y + _f(s["R"])
    return dict(Y=y.to(dt), Z=z.to(dt)) if c["save"] else dict(Y=y.to(dt))


def _linear_backward(s, c, dt):
    dz = _f(s["dY"])
    if s["Z"] is not None:
        dz = dz * _slope(_f(s["Z"]), c["act"])
    dx = dz @ _f(s["W"]).t()
    if s["Zin"] is not None:
        dx = dx * _slope(_f(s["Zin"]), c["act_in"])
    if s["dR"] is not None:
        dx = dx + _f(s["dR"])
    r = dict(dX=dx.to(dt), dW=_f(s["X"]).t() @ dz)
    if s["b"] is not None:
        r["db"] = dz.sum(0)
    return r


EPS, ALPHA = 1e-5, 0.75


def _centre(x, kind):
    """x, less its mean where the norm takes it off, and one over its deviation."""
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    return x, 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)


def _normed(x, kind, gain, shift):
    if kind == "none":
        return x
    x, inv = _centre(x, kind)
    y = x * inv * _f(gain)
    return y if shift is None else y + _f(shift)


def _back(x, kind, gain, dy):
    """(gradient of x, normalised x) of a norm."""
    x, inv = _centre(x, kind)
    xh, d = x * inv, dy * _f(gain)
    dx = d - xh * (d * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - d.mean(1, keepdim=True)
    return dx * inv, xh


def _rows(s, c, dt=None):
    """The gate for each row, or None."""
    return None if s["gate"] is None else _f(s["gate"]).repeat_interleave(c["group"], 0)


def _norm_forward(s, c, dt):
    p = _normed(_f(s["u"]), c["post"], s["post_g"], s["post_s"])
    gate = _rows(s, c)
    r = p if gate is None else p * gate
    if s["x"] is not None:
        r = r + ALPHA * _f(s["x"])
    h = _normed(r, c["pre"], s["pre_g"], s["pre_s"]) if c["pre"] != "none" else None
    if s["M"] is not None:
        keep = s["M"][:, None] != 0
        r = torch.where(keep, r, torch.zeros_like(r))
        h = torch.where(keep, h, torch.zeros_like(h)) if h is not None else None
    return dict(r=r.to(dt), h=h.to(dt)) if h is not None else dict(r=r.to(dt))


def _norm_backward(s, c, dt):
    u, gr, out = _f(s["u"]), _f(s["dr"]), {}
    keep = s["M"][:, None] != 0 if s["M"] is not None else None
    zero = (lambda t: t) if keep is None else lambda t: torch.where(keep, t, torch.zeros_like(t))
    if c["pre"] != "none":
        dh = zero(_f(s["dh"]))
        d, rh = _back(_f(s["r"]), c["pre"], s["pre_g"], dh)
        gr = gr + d
        out["dpre_g"] = (dh * zero(rh)).sum(0)
        if s["pre_s"] is not None:
            out["dpre_s"] = dh.sum(0)
    gr = zero(gr)
    if s["x"] is not None:
        out["dx"] = (ALPHA * gr).to(dt)
    gate, dp = _rows(s, c), gr
    if gate is not None:
        p = zero(_normed(u, c["post"], s["post_g"], s["post_s"]))
        out["dgate"] = (gr * p).reshape(-1, c["group"], c["w"]).sum(1).to(dt)
        dp = gr * gate
    du = dp
    if c["post"] != "none":
        du, uh = _back(u, c["post"], s["post_g"], dp)
        out["dpost_g"] = (dp * zero(uh)).sum(0)
        if s["post_s"] is not None:
            out["dpost_s"] = dp.sum(0)
    out["du"] = zero(du).to(dt)
    return out


# States in 8 bits: blocks of 256 values share a scale, the largest value of a block becomes the largest code. A code of the first moment is
# a sign, 4 bits of exponent and 3 of fraction; the second moment is held as its square root r, 4 bits of exponent and 4 of fraction.
# Rounding is up or down at random (by a hash of seed, step and place), so that slow averages do not stand still; a positive r never becomes 0.

BLOCK, LO32 = 256, 0xFFFFFFFF
LR, BETA1, BETA2, ADAM_EPS = 1e-3, 0.9, 0.999, 1e-8


def _mix(x):
    """A 32-bit hash, in 64-bit whole numbers."""
    x = x & LO32
    x = ((x ^ (x >> 16)) * 0x6C8E9CF5) & LO32
    x = ((x ^ (x >> 15)) * 0x5B2D1A67) & LO32
    return x ^ (x >> 16)


def _scaled(a, top):
    """The non-negative values of each block over the block's scale, and the scales."""
    a = a.reshape(-1, BLOCK)
    big = a.amax(1, keepdim=True)
    scale = big / torch.full_like(big, top)
    x = torch.where(big == 0, torch.zeros_like(a), a / scale)
    return (x * 2.0 ** -112).reshape(-1), scale.reshape(-1)


def _pack_m(m, h):
    y, scale = _scaled(m.abs(), 1.875)
    code = ((y.view(torch.int32).to(torch.int64) + (h >> 12)) >> 20).clamp(max=127)
    return (code | ((m < 0).to(torch.int64) << 7)).to(torch.uint8), scale


def _pack_r(r, h):
    y, scale = _scaled(r, 1.9375)
    h = (h * 0x3C6EF35F) & LO32
    code = ((y.view(torch.int32).to(torch.int64) + (h >> 13)) >> 19).clamp(max=255)
    return torch.where(r > 0, code.clamp(min=1), code).to(torch.uint8), scale


def _unpack_m(code, scale):
    a = ((code.to(torch.int32) & 127) << 20).view(torch.float32) * 2.0 ** 112
    a = (a.reshape(-1, BLOCK) * scale[:, None]).reshape(-1)
    return torch.where(code > 127, -a, a)


def _unpack_r(code, scale):
    a = (code.to(torch.int32) << 19).view(torch.float32) * 2.0 ** 112
    return (a.reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _adamw(s, c, dt):
    s["t"] += 1
    t = s["t"].double()
    bc1, bc2 = 1 - torch.pow(BETA1, t), 1 - torch.pow(BETA2, t)
    size, inv = (LR / bc1).float(), (1 / torch.sqrt(bc2)).float()
    g, p = _f(s["g"]), s["master"] if s["master"] is not None else s["p"]
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m, v = _unpack_m(s["m"], s["m_scale"]), _unpack_r(s["v"], s["v_scale"])
        v = v * v
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    r = torch.sqrt(v)
    p = p * (1 - LR * s["decay"].double()).float() - (m / (r * inv + ADAM_EPS)) * size
    s["p"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        key = _mix(s["t"] * 0x9E3779B9 + s["seed"])
        h = _mix(torch.arange(m.numel(), device=m.device) + key)
        for k, (code, scale) in (("m", _pack_m(m, h)), ("v", _pack_r(r, h))):
            s[k].copy_(code)
            s[k + "_scale"].copy_(scale)
        m, v = _unpack_m(s["m"], s["m_scale"]), _unpack_r(s["v"], s["v_scale"])
        v = v * v
    out = dict(p=s["p"], m=m, v=v)
    if s["master"] is not None:
        out["master"] = s["master"]
    return out


PLAIN = dict(linear_forward=_linear_forward, linear_backward=_linear_backward, norm_forward=_norm_forward, norm_backward=_norm_backward, adamw=_adamw)


# ---------------------------------------------------------------- the framework's calls

def _plan(s, op, c):
    """What a program keeps between its calls: dims, output tensors, workspaces, the optimiser."""
    from edge_aware_graph_b200 import eaga
    from edge_aware_graph_b200.optim import AdamW
    dt = DTYPES[c["dtype"]]
    new = lambda like, dtype=dt: None if like is None else torch.empty(like.shape, dtype=dtype, device=DEV)  # noqa: E731
    f32 = torch.float32
    if op.startswith("linear"):
        back = op == "linear_backward"
        s["dims"] = eaga.linear_dims(c["rows"], c["inp"], c["out"], c["act"], c["dtype"])
        s["ws"] = torch.empty(eaga.linear_workspace_size(s["dims"], back), dtype=torch.uint8, device=DEV)
        if back:
            s["dX"], s["dW"], s["db"] = new(s["X"]), new(s["W"], f32), new(s["b"], f32)
        else:
            s["Y"] = torch.empty(c["rows"], c["out"], dtype=dt, device=DEV)
            s["Z"] = torch.empty_like(s["Y"]) if c["save"] else None
    elif op.startswith("norm"):
        s["dims"] = eaga.residual_norm_dims(c["rows"], c["w"], pre=c["pre"], post=c["post"], rows_per_group=c["group"], eps=EPS, alpha=ALPHA, dtype=c["dtype"])
        if op == "norm_forward":
            s["r"], s["h"] = new(s["u"]), new(s["u"]) if c["pre"] != "none" else None
        else:
            s["ws"] = torch.empty(eaga.residual_norm_workspace_size(s["dims"]), dtype=torch.uint8, device=DEV)
            s["dx"], s["du"], s["dgate"] = new(s["x"]), new(s["u"]), new(s["gate"])
            for k in ("post_g", "post_s", "pre_g", "pre_s"):
                s["d" + k] = new(s[k], f32)
    else:
        part = lambda flat: None if flat is None else [flat[a:a + n] for a, n in zip(s["at"], s["sizes"])]  # noqa: E731
        scales = (lambda flat: [flat[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(s["at"], s["sizes"])]) if c["bits"] == 8 else lambda flat: None
        s["opt"] = AdamW(part(s["p"]), part(s["g"]), lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=[0.01 if n > 1024 else 0.0 for n in s["sizes"]], bits=c["bits"],
                         master=part(s["master"]), m=part(s["m"]), v=part(s["v"]), m_scale=scales(s.get("m_scale")), v_scale=scales(s.get("v_scale")),
                         counters=s["at"], seed=s["seed"], step=c["step"])
        if c["bits"] == 8:
            s["m32"], s["v32"] = torch.zeros(s["p"].numel(), device=DEV), torch.zeros(s["p"].numel(), device=DEV)
            s["unpack"] = s["opt"].unpacker(part(s["m32"]), part(s["v32"]))


def _call(s, c):
    from edge_aware_graph_b200 import eaga
    op = c["op"]
    some = lambda *names: {k: s[k] for k in names if s.get(k) is not None}  # noqa: E731
    if op == "linear_forward":
        eaga.linear_forward(s["dims"], s["X"], s["W"], s["b"], s["R"], s["Y"], s["Z"], s["ws"])
        return some("Y", "Z")
    if op == "linear_backward":
        eaga.linear_backward(s["dims"], s["X"], s["W"], s["Z"], s["dY"], s["dX"], s["dW"], s["db"], s["ws"], act_in=c["act_in"], Zin=s["Zin"], dR=s["dR"])
        return some("dX", "dW", "db")
    if op == "norm_forward":
        eaga.residual_norm_forward(s["dims"], s["x"], s["u"], s["M"], s["gate"], s["post_g"], s["post_s"], s["pre_g"], s["pre_s"], s["r"], s["h"])
        return some("r", "h")
    if op == "norm_backward":
        eaga.residual_norm_backward(s["dims"], s["r"], s["u"], s["M"], s["gate"], s["post_g"], s["post_s"], s["pre_g"], s["dr"], s["dh"], s["dx"], s["du"], s["dgate"],
                                    s["dpost_g"], s["dpost_s"], s["dpre_g"], s["dpre_s"], s["ws"])
        return some("dx", "du", "dgate", "dpost_g", "dpost_s", "dpre_g", "dpre_s")
    s["opt"].step()
    out = some("p", "master", "m", "v")
    if c["bits"] == 8:  # the states as the values that they stand for
        s["unpack"]()
        out.update(m=s["m32"], v=s["v32"])
    return out


def run(state):
    c = state["case"]
    if own:
        return _call(state, c)
    return PLAIN[c["op"]](state, c, DTYPES[c["dtype"]])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"].startswith("linear"):
        n, k, o = c["rows"], c["inp"], c["out"]
        if c["op"] == "linear_forward":
            return dict(bytes=e * (n * k + k * o + n * o * (1 + c["res"] + c["save"]) + o * c["bias"]), flops=2 * n * k * o)
        moved = n * k * (2 + (c["act_in"] != "none") + c["res"]) + k * o + n * o * (1 + (c["act"] != "none"))
        return dict(bytes=e * moved + 4 * (k * o + o * c["bias"]), flops=4 * n * k * o)
    if c["op"].startswith("norm"):
        n, w = c["rows"], c["w"]
        live = n // 2 if c["mask"] else n  # masked rows are written, not read
        params = w * ((c["pre"] != "none") + (c["pre"] == "layer") + (c["post"] != "none") + (c["post"] == "layer")) * e
        gate = (n // c["group"]) * w * c["gate"] * e
        if c["op"] == "norm_forward":
            return dict(bytes=e * w * (live * (1 + c["res"]) + n * (1 + (c["pre"] != "none"))) + params + gate, flops=0)
        reads = 2 * (c["pre"] != "none") + 1 + (c["gate"] or c["post"] != "none")
        return dict(bytes=e * w * (live * reads + n * (1 + c["res"])) + params * (1 + 4 // e) + 2 * gate, flops=0)
    n, state = sum(_sizes(c)), 2 * (1 if c["bits"] == 8 else 4) + (8 / BLOCK if c["bits"] == 8 else 0)
    weights = 8 + 2 if c["dtype"] == "bf16" else 8  # in 16 bits the 32-bit master is read and written, the weight written
    return dict(bytes=int(n * ((4 if c["grad"] == "fp32" else 2) + weights + 2 * state + (8 + state if c["bits"] == 8 else 0))), flops=0)


# ---------------------------------------------------------------- the definitions in 64 bits

def _activation64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _norm64(x, kind, gain, shift):
    if kind == "none":
        return x
    mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    y = (x - mean) * torch.rsqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS) * gain
    return y if shift is None else y + shift


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    D = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if c["op"] == "linear_forward":
        z = torch.matmul(D["X"], D["W"])
        z = z if D["b"] is None else z + D["b"]
        y = _activation64(z, c["act"])
        y = y if D["R"] is None else y + D["R"]
        return dict(Y=y, Z=z) if c["save"] else dict(Y=y)
    if c["op"] == "linear_backward":
        dz = D["dY"]
        if c["act"] != "none":
            z = D["Z"].clone().requires_grad_()
            dz, = torch.autograd.grad(_activation64(z, c["act"]), z, dz)
        dx = torch.matmul(dz, D["W"].T)
        if c["act_in"] != "none":
            z = D["Zin"].clone().requires_grad_()
            dx, = torch.autograd.grad(_activation64(z, c["act_in"]), z, dx)
        out = dict(dX=dx if D["dR"] is None else dx + D["dR"], dW=torch.matmul(D["X"].T, dz))
        if c["bias"]:
            out["db"] = torch.sum(dz, dim=0)
        return out
    if c["op"].startswith("norm"):
        keep = None if D["M"] is None else D["M"].reshape(-1, 1).double()
        grads = {k: D[k].requires_grad_() for k in ("u", "x", "gate", "post_g", "post_s", "pre_g", "pre_s") if D.get(k) is not None}
        p = _norm64(D["u"], c["post"], D["post_g"], D["post_s"])
        if D["gate"] is not None:
            p = (p.reshape(-1, c["group"], c["w"]) * D["gate"][:, None]).reshape(c["rows"], c["w"])
        r = p if D["x"] is None else ALPHA * D["x"] + p
        if c["op"] == "norm_forward":
            out = dict(r=r) if c["pre"] == "none" else dict(r=r, h=_norm64(r, c["pre"], D["pre_g"], D["pre_s"]))
            return {k: (v if keep is None else v * keep).detach() for k, v in out.items()}
        # the backward takes the r that the forward stored: what reaches r from h is taken there, and goes on through the sum from there
        dr = D["dr"] if keep is None else D["dr"] * keep
        out = {}
        if c["pre"] != "none":
            at = D["r"].requires_grad_()
            names = [k for k in ("pre_g", "pre_s") if k in grads]
            got = torch.autograd.grad(_norm64(at, c["pre"], D["pre_g"], D["pre_s"]), [at] + [grads[k] for k in names], D["dh"] if keep is None else D["dh"] * keep)
            dr = dr + got[0]
            out.update(zip(["d" + k for k in names], got[1:]))
        names = [k for k in ("u", "x", "gate", "post_g", "post_s") if k in grads]
        out.update(zip(["d" + k for k in names], torch.autograd.grad(r, [grads[k] for k in names], dr)))
        return out
    t = c["step"] + 1
    m, v = D["m"], D["v"]
    if c["bits"] == 8:  # the states of this step are read as held; those of the next are rounded at random, and have no such value
        bits = lambda code: (code.long() << 52 - 4)  # noqa: E731
        a, r = (D["m"].long() & 127) << 49, bits(D["v"])
        wide = lambda b, k: (b.view(torch.float64) * 2.0 ** 1008).reshape(-1, BLOCK) * D[k][:, None]  # noqa: E731
        m = wide(a, "m_scale").reshape(-1) * torch.where(D["m"] > 127, -1.0, 1.0).double()
        v = wide(r, "v_scale").reshape(-1) ** 2
    p = D["p"] if D["master"] is None else D["master"]
    m = BETA1 * m + (1 - BETA1) * D["g"]
    v = BETA2 * v + (1 - BETA2) * D["g"] ** 2
    p = (1 - LR * D["decay"]) * p - LR / (1 - BETA1 ** t) * m / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    out = dict(p=p, m=None if c["bits"] == 8 else m, v=None if c["bits"] == 8 else v)
    if D["master"] is not None:
        out["master"] = p
    return out
