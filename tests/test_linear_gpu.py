"""The linear operator on the GPU against its formulas in 64 bits.

Two kinds of tests.  With whole numbers as inputs every sum is exact in fp32,
whatever its order, so products and column sums have to be equal bit for bit
to the exact result rounded once.  With real numbers the bound is that of K
additions in any order, each off by at most one step of fp32 (2^-23, an
addition may truncate) of the sum of magnitudes; an activation adds a few steps
of fp32 (erff and expf are within two), a store half a step of its type."""
import math

import pytest
import torch

from edge_aware_graph_b200 import eaga

pytestmark = pytest.mark.gpu
TD = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
U = 2.0 ** -24


def empty(*shape, dtype):
    """An output: what it held before must not show."""
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def forward(X, W, b=None, R=None, act="none", dtype="bf16", save=True, stream=None):
    rows, i, o = X.shape[0], X.shape[1], W.shape[1]
    d = eaga.linear_dims(rows, i, o, act, dtype)
    ws = torch.full((eaga.linear_workspace_size(d, False),), 255, dtype=torch.uint8, device="cuda")
    Y = empty(rows, o, dtype=TD[dtype])
    Z = empty(rows, o, dtype=TD[dtype]) if save else None
    eaga.linear_forward(d, X, W, b, R, Y, Z, ws, stream)
    assert eaga.get_device_status(ws, stream) == 0
    return Y, Z


def backward(X, W, dY, Z=None, act="none", act_in="none", Zin=None, dR=None, dtype="bf16", dx=True, dw=True, db=True):
    rows, i, o = dY.shape[0], W.shape[0], W.shape[1]
    d = eaga.linear_dims(rows, i, o, act, dtype)
    ws = torch.full((eaga.linear_workspace_size(d, True),), 255, dtype=torch.uint8, device="cuda")
    dX = empty(rows, i, dtype=TD[dtype]) if dx else None
    dW = empty(i, o, dtype=torch.float32) if dw else None
    dB = empty(o, dtype=torch.float32) if db and dw else None
    eaga.linear_backward(d, X, W, Z, dY, dX, dW, dB, ws, act_in=act_in, Zin=Zin, dR=dR)
    assert eaga.get_device_status(ws) == 0
    return dX, dW, dB


def whole(g, *shape, dtype, top=3):
    return torch.randint(-top, top + 1, shape, generator=g).to(TD[dtype])


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


SHAPES = [  # rows, in, out: tile edges, rows that are not 16 bytes, one of each, reductions over many rows
    (1, 1, 1), (1, 512, 40), (3, 7, 5), (8, 64, 64), (9, 64, 64), (16, 8, 4), (127, 65, 33), (128, 64, 128), (129, 128, 256),
    (130, 72, 264), (257, 200, 136), (5, 1040, 72), (2, 4099, 131), (700, 8, 520), (64, 640, 8), (3000, 24, 16), (20011, 64, 128),
    (33, 300, 2056), (1000, 257, 131), (11, 3800, 9), (516, 2776, 132), (40, 9, 3801), (260, 12, 2000), (9, 1, 1), (64, 65536, 3),
    (40_000, 300, 60), (1174, 680, 520), (5000, 1300, 120), (4, 300, 200), (6, 1000, 1001), (7, 520, 1032), (12, 70, 300), (16, 1030, 45),
    (17, 64, 96), (50_000, 8, 8), (40_001, 7, 13), (30_000, 32, 12), (20_000, 33, 20), (25_000, 64, 64),
    (6580, 2576, 17), (3001, 70, 32), (100, 513, 7), (4000, 8, 1030), (2003, 31, 600), (20_000, 80, 20), (30_001, 257, 9),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,i,o", SHAPES)
def test_exact_products(rows, i, o, dtype):
    g = torch.Generator().manual_seed(rows * 7 + i + o)
    X, W, b, R = whole(g, rows, i, dtype=dtype), whole(g, i, o, dtype=dtype), whole(g, o, dtype=dtype), whole(g, rows, o, dtype=dtype)
    dY, dR = whole(g, rows, o, dtype=dtype), whole(g, rows, i, dtype=dtype)
    z = X.double() @ W.double() + b.double()
    for bias, res in ((b, R), (None, None)):
        Y, Z = forward(*cuda(X, W, bias, res), dtype=dtype)
        ref = z if bias is not None else z - b.double()
        assert torch.equal(Z.cpu(), ref.to(TD[dtype]))
        assert torch.equal(Y.cpu(), (ref + (R.double() if res is not None else 0)).to(TD[dtype]))
    dx = dY.double() @ W.double().T
    dX, dW, dB = backward(*cuda(X, W, dY), dR=dR.cuda(), dtype=dtype)
    assert torch.equal(dX.cpu(), (dx + dR.double()).to(TD[dtype]))
    assert torch.equal(dW.cpu().double(), X.double().T @ dY.double())
    assert torch.equal(dB.cpu().double(), dY.double().sum(0))
    # relu on either side keeps whole numbers whole
    Zin = whole(g, rows, i, dtype=dtype)
    zo = whole(g, rows, o, dtype=dtype)
    dz = dY.double() * (zo.double() > 0)
    dX, dW, dB = backward(*cuda(X, W, dY), Z=zo.cuda(), act="relu", act_in="relu", Zin=Zin.cuda(), dtype=dtype)
    assert torch.equal(dX.cpu().double(), ((dz @ W.double().T) * (Zin.double() > 0)).to(TD[dtype]).double())
    assert torch.equal(dW.cpu().double(), X.double().T @ dz)
    assert torch.equal(dB.cpu().double(), dz.sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,i,o", [(4000, 200, 2056), (3900, 136, 2051), (4000, 2056, 200), (3900, 2051, 140), (520, 4000, 2056),
                                      (777, 2200, 4099), (10_000, 1000, 1032)])
def test_exact_products_of_large_tiles(rows, i, o, dtype):
    """Results of many tiles, whole and ragged, and reductions of many steps."""
    g = torch.Generator().manual_seed(rows + i)
    X, W, b, R = cuda(*(whole(g, *s, dtype=dtype) for s in ((rows, i), (i, o), (o,), (rows, o))))
    dY, dR, Zin, zo = cuda(*(whole(g, *s, dtype=dtype) for s in ((rows, o), (rows, i), (rows, i), (rows, o))))
    z = X.double() @ W.double() + b.double()
    for res in (R, None):
        for save in (True, False):
            Y, Z = forward(X, W, b, res, act="relu", save=save, dtype=dtype)
            if save:
                assert torch.equal(Z, z.to(TD[dtype]))
            assert torch.equal(Y, (z.clamp(min=0) + (R.double() if res is not None else 0)).to(TD[dtype]))
    dX, dW, dB = backward(X, W, dY, dtype=dtype)
    assert torch.equal(dX, (dY.double() @ W.double().T).to(TD[dtype]))
    assert torch.equal(dW.double(), X.double().T @ dY.double())
    assert torch.equal(dB.double(), dY.double().sum(0))
    dz = dY.double() * (zo.double() > 0)
    dx = (dz @ W.double().T) * (Zin.double() > 0)
    for res in (dR, None):
        dX, dW, dB = backward(X, W, dY, Z=zo, act="relu", act_in="relu", Zin=Zin, dR=res, dtype=dtype)
        assert torch.equal(dX.double(), (dx + (dR.double() if res is not None else 0)).to(TD[dtype]).double())
        assert torch.equal(dW.double(), X.double().T @ dz)
        assert torch.equal(dB.double(), dz.sum(0))
    dX, _, _ = backward(None, W, dY, dR=dR, dw=False, dtype=dtype)
    assert torch.equal(dX, (dY.double() @ W.double().T + dR.double()).to(TD[dtype]))


@pytest.mark.parametrize("xbits,wbits", [(23, 1), (1, 23), (12, 12), (16, 8), (8, 16)])
def test_all_bits_of_fp32_operands(xbits, wbits):
    """Whole numbers of up to 24 bits, one product a sum: exact only if no part of an operand that counts is left out."""
    g = torch.Generator().manual_seed(xbits)
    rows, i, o = 200, 72, 40

    def numbers(bits, *s):
        return (torch.randint(1 << (bits - 1), 1 << bits, s, generator=g) * (2 * torch.randint(0, 2, s, generator=g) - 1)).float()

    X = numbers(xbits, rows, 1) * torch.nn.functional.one_hot(torch.arange(rows) % i, i).float()
    W = numbers(wbits, i, o)
    Y, _ = forward(*cuda(X, W), dtype="fp32")
    assert torch.equal(Y.cpu().double(), X.double() @ W.double())
    dY = numbers(xbits, rows, 1) * torch.nn.functional.one_hot(torch.arange(rows) % o, o).float()
    dX, _, _ = backward(None, *cuda(W, dY), dtype="fp32", dw=False)
    assert torch.equal(dX.cpu().double(), dY.double() @ W.double().T)
    X1, dY1 = numbers(xbits, i, i) * torch.eye(i), numbers(wbits, i, o)
    _, dW, _ = backward(*cuda(X1, W, dY1), dtype="fp32", dx=False)
    assert torch.equal(dW.cpu().double(), X1.double().T @ dY1.double())


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(z) if act == "silu" else z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def close(got, ref, err, dtype, name):
    got = got.detach().double().cpu()
    tol = err + HALF[dtype] * (ref.abs() + err) + 1e-37
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), name
    assert (off <= tol).all(), f"{name}: worst {float((off / tol).max()):.3g} of the bound"


def product(a, b):
    """a @ b and the bound of its fp32 error."""
    return a @ b, (a.shape[1] + 8) * 2 * U * (a.abs() @ b.abs())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("rows,i,o", [(1, 96, 80), (7, 33, 100), (61, 48, 200), (150, 130, 72), (300, 31, 57)])
def test_activations(rows, i, o, act, dtype):
    g = torch.Generator().manual_seed(rows + i)
    new = lambda *s, d=1.0: (torch.randn(*s, generator=g) * d).to(TD[dtype])
    X, W, b, R = new(rows, i), new(i, o, d=3 * i ** -0.5), new(o), new(rows, o)
    z, ez = product(X.double(), W.double())
    z, ez = z + b.double(), ez + 2 * U * (z.abs() + b.double().abs())
    Y, Z = forward(*cuda(X, W, b, R), act=act, dtype=dtype)
    close(Z, z, ez, dtype, "Z")
    y = act64(z, act)
    ey = 1.13 * ez + 8 * U * (z.abs() + y.abs())
    y = y + R.double()
    close(Y, y, ey + U * y.abs(), dtype, "Y")
    # the backward reads the stored Z
    dY, Zin, dR = new(rows, o), new(rows, i, d=2.0), new(rows, i)
    Zs = Z.cpu().double()
    dz = dY.double() * slope64(Zs, act)
    edz = dY.double().abs() * (16 + 8 * Zs.abs()) * U if act in ("gelu", "silu") else torch.zeros_like(dz)
    args = dict(Z=Z, act=act) if act != "none" else {}
    dX, dW, dB = backward(*cuda(X, W, dY), act_in="gelu", Zin=Zin.cuda(), dR=dR.cuda(), dtype=dtype, **args)
    dx, edx = product(dz, W.double().T)
    # two bf16 parts of dz carry all but 2^-16 of it
    parts = edz + (2.0 ** -16 * dz.abs() if dtype == "bf16" and act != "none" else 0)
    edx = edx + parts @ W.double().abs().T
    s = slope64(Zin.double(), "gelu")
    edx = edx * s.abs() + dx.abs() * (16 + 8 * Zin.double().abs()) * U
    dx = dx * s + dR.double()
    close(dX, dx, edx + U * dx.abs(), dtype, "dX")
    # three parts carry 24 bits
    parts = edz + (2.0 ** -24 * dz.abs() if dtype == "bf16" and act != "none" else 0)
    dw, edw = product(X.double().T, dz)
    close(dW, dw, edw + X.double().abs().T @ parts, "fp32", "dW")
    close(dB, dz.sum(0), (rows + 8) * 2 * U * dz.abs().sum(0) + parts.sum(0), "fp32", "db")


def test_gradients_against_differences():
    """<dL/dtheta, v> against (L(theta + h v) - L(theta - h v)) / 2h of the formula in 64 bits, at fp32 inputs."""
    g = torch.Generator().manual_seed(3)
    rows, i, o = 40, 24, 20
    X0, W, b, c = (torch.randn(*s, generator=g).float() for s in ((rows, i), (i, o), (o,), (rows, o)))
    f = lambda x, w, bb: (c.double() * act64(act64(x, "silu") @ w + bb, "gelu")).sum()
    Xa = act64(X0.double(), "silu").float()
    _, Z = forward(*cuda(Xa, W, b), act="gelu", dtype="fp32")
    dX, dW, dB = backward(*cuda(Xa, W, c), Z=Z, act="gelu", act_in="silu", Zin=X0.cuda(), dtype="fp32")
    for k, (grad, at) in enumerate(((dX, X0), (dW, W), (dB, b))):
        v = torch.randn(*at.shape, generator=g).double()
        args = [X0.double(), W.double(), b.double()]
        up, down = list(args), list(args)
        h = 1e-4
        up[k], down[k] = args[k] + h * v, args[k] - h * v
        num = float(f(*up) - f(*down)) / (2 * h)
        got = float((grad.double().cpu() * v).sum())
        # the difference is off by h^2 times the third derivative along v; |v|, |c|, the slopes' bounds give less than 1e-3 of the sum of magnitudes
        assert abs(got - num) <= 1e-4 * float((grad.double().cpu() * v).abs().sum()), k


@pytest.mark.parametrize("rows", [4, 40])
def test_not_a_number_stays_in_its_row(rows):
    g = torch.Generator().manual_seed(1)
    X, W, dY = whole(g, rows, 72, dtype="bf16"), whole(g, 72, 40, dtype="bf16"), whole(g, rows, 40, dtype="bf16")
    Z = torch.randn(rows, 40, generator=g).to(torch.bfloat16)
    X[1, 3], X[2, 5] = float("nan"), float("inf")
    Y, _ = forward(*cuda(X, W))
    bad = ~torch.isfinite(Y.float().cpu()).all(1)
    assert bad.tolist() == [r in (1, 2) for r in range(rows)]
    dY[3, 2] = float("-inf")
    W[:, 2] = 1
    Z[3, 2] = 1.0
    dX, dW, dB = backward(*cuda(whole(g, rows, 72, dtype="bf16"), W, dY), Z=Z.cuda(), act="silu")
    dX = dX.float().cpu()
    assert (dX[3] == float("-inf")).all() and torch.isfinite(dX[:3]).all() and torch.isfinite(dX[4:]).all()
    assert dB[2].item() == float("-inf") and torch.isfinite(dB[3:]).all()


def test_parts_of_the_backward():
    g = torch.Generator().manual_seed(2)
    for rows in (3, 50):
        X, W, dY = cuda(whole(g, rows, 40, dtype="bf16"), whole(g, 40, 24, dtype="bf16"), whole(g, rows, 24, dtype="bf16"))
        full = backward(X, W, dY)
        dX, _, _ = backward(None, W, dY, dw=False)
        assert torch.equal(dX, full[0])
        _, dW, dB = backward(X, W, dY, dx=False)
        assert torch.equal(dW, full[1]) and torch.equal(dB, full[2])
        _, dW, _ = backward(X, W, dY, dx=False, db=False)
        assert torch.equal(dW, full[1])


def test_no_rows():
    W = torch.zeros(24, 16, dtype=torch.bfloat16, device="cuda")
    X, dY = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    Y, _ = forward(X, W)
    assert Y.shape == (0, 16)
    _, dW, dB = backward(X, W, dY)
    assert (dW == 0).all() and (dB == 0).all()


def test_rows_beyond_2_31_elements():
    """Offsets that pass 31 bits: 300,000 rows of 8192 outputs (2.4e9 values), checked at both ends."""
    rows, i, o = 300_000, 8, 8192
    g = torch.Generator().manual_seed(5)
    W = whole(g, i, o, dtype="bf16").cuda()
    X = torch.zeros(rows, i, dtype=torch.bfloat16, device="cuda")
    for r in (0, 131_072, rows - 1):
        X[r] = whole(g, i, dtype="bf16").cuda()
    Y, _ = forward(X, W, save=False)
    for r in (0, 1, 131_072, rows - 2, rows - 1):
        assert torch.equal(Y[r].double(), X[r].double() @ W.double()), r
    dX, dW, dB = backward(X, W, Y)
    live = (0, 131_072, rows - 1)
    assert torch.equal(dW.double(), sum(torch.outer(X[r].double(), Y[r].double()) for r in live))
    assert torch.equal(dX[rows - 1].double(), (Y[rows - 1].double() @ W.double().T).to(torch.bfloat16).double())
    assert torch.equal(dB.double(), sum(Y[r].double() for r in live))


def test_replayed_and_beside_another_stream():
    """A captured call reads its inputs anew; calls on two streams with workspaces of their own do not disturb each other."""
    g = torch.Generator().manual_seed(4)
    rows, i, o = 500, 136, 264
    d = eaga.linear_dims(rows, i, o, "relu", "bf16")
    X, W, b, dY = cuda(whole(g, rows, i, dtype="bf16"), whole(g, i, o, dtype="bf16"), whole(g, o, dtype="bf16"), whole(g, rows, o, dtype="bf16"))
    sides = []
    for _ in range(2):
        t = dict(Y=empty(rows, o, dtype=torch.bfloat16), Z=empty(rows, o, dtype=torch.bfloat16), dX=empty(rows, i, dtype=torch.bfloat16),
                 dW=empty(i, o, dtype=torch.float32), db=empty(o, dtype=torch.float32), X=X.clone(), s=torch.cuda.Stream())
        t["wf"] = torch.empty(eaga.linear_workspace_size(d, False), dtype=torch.uint8, device="cuda")
        t["wb"] = torch.empty(eaga.linear_workspace_size(d, True), dtype=torch.uint8, device="cuda")
        sides.append(t)

    def step(t, stream=None):
        eaga.linear_forward(d, t["X"], W, b, None, t["Y"], t["Z"], t["wf"], stream)
        eaga.linear_backward(d, t["X"], W, t["Z"], dY, t["dX"], t["dW"], t["db"], t["wb"], stream=stream)

    torch.cuda.synchronize()
    for _ in range(5):
        for t in sides:
            step(t, t["s"])
    torch.cuda.synchronize()
    keys = ("Y", "Z", "dX", "dW", "db")
    first = {k: sides[0][k].clone() for k in keys}
    for k in keys:
        assert torch.equal(sides[0][k], sides[1][k]), k
    graph = torch.cuda.CUDAGraph()
    t = sides[0]
    with torch.cuda.graph(graph):
        step(t)
    t["X"].copy_(-X)
    graph.replay()
    torch.cuda.synchronize()
    step({**sides[1], "X": -X})
    torch.cuda.synchronize()
    for k in keys:
        assert torch.equal(t[k], sides[1][k]), k
    t["X"].copy_(X)
    graph.replay()
    torch.cuda.synchronize()
    for k in keys:
        assert torch.equal(t[k], first[k]), k


def test_refusals():
    """What the binding and the entries refuse, before anything is launched; the outputs stay as they were."""
    rows, i, o = 20, 24, 16
    d = eaga.linear_dims(rows, i, o, "gelu", "bf16")
    new = lambda *s, dtype=torch.bfloat16: torch.ones(*s, dtype=dtype, device="cuda")
    X, W, b, R, Y, Z = new(rows, i), new(i, o), new(o), new(rows, o), new(rows, o), new(rows, o)
    ws = torch.empty(eaga.linear_workspace_size(d, True), dtype=torch.uint8, device="cuda")
    good = dict(X=X, W=W, b=b, R=R, Y=Y, Z=Z, ws=ws)

    def call(**over):
        a = {**good, **over}
        eaga.linear_forward(d, a["X"], a["W"], a["b"], a["R"], a["Y"], a["Z"], a["ws"])

    for k, bad in (("X", X.float()), ("W", W[:, :8]), ("W", W.T.contiguous().T), ("b", b[:8]), ("Y", Y.cpu()), ("Z", new(rows + 1, o)), ("X", None), ("Y", None),
                   ("ws", None), ("ws", new(64, dtype=torch.float32)), ("X", [1, 2])):
        with pytest.raises(ValueError):
            call(**{k: bad})
    for over, code in ((dict(Y=R), 1), (dict(Z=Y), 1), (dict(ws=ws[:64]), 4), (dict(X=new(rows * i + 8)[4:-4].view(rows, i)), 3)):
        with pytest.raises(eaga.EagaError) as e:
            call(**over)
        assert e.value.code == code
    dY, dX, dW, db = new(rows, o), new(rows, i), new(i, o, dtype=torch.float32), new(o, dtype=torch.float32)
    with pytest.raises(eaga.EagaError):                   # gelu's backward needs Z
        eaga.linear_backward(d, X, W, None, dY, dX, dW, db, ws)
    with pytest.raises(ValueError):                       # weight gradients are fp32
        eaga.linear_backward(d, X, W, Z, dY, dX, dW.bfloat16(), db, ws)
    with pytest.raises(ValueError):
        eaga.linear_backward(d, X, W, Z, dY, dX, dW, db, ws, act_in="tanh")
    torch.cuda.synchronize()
    assert (Y == 1).all() and (Z == 1).all() and (dX == 1).all() and (dW == 1).all()
