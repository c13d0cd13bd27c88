"""What the linear operator's results may be off by, and what infinities and NaN become, beyond the parity tests."""
import pytest
import torch

from edge_aware_graph_b200 import eaga
from test_linear_gpu import backward, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,k,n", [(512, 65536, 9472), (500, 65536, 9467), (128, 32768, 18944)])
def test_long_sums_in_bf16_do_not_drift(rows, k, n):
    """Sums of positive products, where every truncation goes the same way, on pairs of CTAs and on single ones, unsplit.

    A bf16 result is the fp32 sum rounded once: off by half its spacing and by the sum's own error.  The sum leaves the
    accumulator every 1024 steps: 64 additions of 16 products, each off by one step of fp32 (2^-23) at most, then k / 1024
    additions rounded to nearest (2^-24)."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    new = lambda *s: (torch.rand(*s, generator=g, device="cuda") + 0.5).bfloat16()
    e = (2 * 64 + k / 1024) * 2.0 ** -24

    def check(got, exact):
        step = torch.exp2(torch.floor(torch.log2(exact * (1 + e))) - 7)
        off = (got.double() - exact).abs()
        assert (off <= step / 2 + e * exact).all(), float(((off - step / 2) / exact).max() / e)

    X, W = new(rows, k), new(k, n)
    exact = X.double() @ W.double()
    check(forward(X, W, save=False)[0], exact)
    W = W.t().contiguous()                                # the input gradient reduces over W's columns
    check(backward(None, W, X, dw=False)[0], exact)


NAN_SHAPES = [("bf16", 4, 72, 40), ("bf16", 6, 72, 41), ("bf16", 40, 72, 40), ("bf16", 300, 72, 41), ("bf16", 6144, 512, 256), ("fp32", 4, 72, 40),
              ("fp32", 13, 70, 37), ("fp32", 300, 200, 136), ("fp32", 1001, 257, 131), ("fp32", 3001, 70, 32), ("fp32", 20_000, 33, 20),
              ("fp32", 40_001, 7, 13)]


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("dtype,rows,i,o", NAN_SHAPES)
def test_a_nan_is_seen_behind_every_activation(dtype, rows, i, o, act):
    """It reaches the values that its own enters, and no others."""
    td = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(rows + i)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(td)
    nan = lambda t: torch.isnan(t.float())
    X, W, b, R = new(rows, i), new(i, o), new(o), new(rows, o)
    X[1, 3] = float("nan")
    row = torch.zeros(rows, 1, dtype=torch.bool, device="cuda")
    row[1] = True
    Y, Z = forward(X, W, b, R, act=act, dtype=dtype)
    assert torch.equal(nan(Y), row.expand(rows, o)) and torch.equal(nan(Z), row.expand(rows, o))
    X[1, 3] = 0
    Z, dY, dR, Zin = new(rows, o), new(rows, o), new(rows, i), new(rows, i)
    Zin[3, 2] = float("nan")
    (dY if act == "none" else Z)[2, 5] = float("nan")
    dX, dW, dB = backward(X, W, dY, Z=Z if act != "none" else None, act=act, act_in=act, Zin=Zin if act != "none" else None, dR=dR, dtype=dtype)
    want = torch.zeros(rows, i, dtype=torch.bool, device="cuda")
    want[2] = True
    want[3, 2] = act != "none"
    col = torch.arange(o, device="cuda") == 5
    assert torch.equal(nan(dX), want) and torch.equal(nan(dW), col.expand(i, o)) and torch.equal(nan(dB), col)


GELU_SHAPES = [(4, 8, 512), (13, 70, 128), (300, 200, 136), (2001, 257, 131), (20_001, 64, 128), (3001, 70, 32), (3001, 32, 70), (20_000, 33, 20), (700, 900, 260)]


@pytest.mark.parametrize("rows,i,o", GELU_SHAPES)
def test_gelu_in_fp32_is_right_in_its_relative_error(rows, i, o):
    """Every z exactly (one product a sum, by 1 or -1), from -9 to 9, tails and the slope's zero among them.  With s = 2^-23:

    Phi(-x) = t Q(t) e^(-x^2/2): t is off by 1.5 s (its divisor's rounding, the reciprocal), twice that in the result (d ln Phi / d ln t
    is 2 at the most), Q by 2.75 s (its steps' roundings, its argument's, its fit), e by 2.5 s (the power of two's 2 s, its correction's rounding),
    two products by half a step each: 9.25 s.  y = z Phi(z) rounds twice more: 10.25 s |y|.
    slope = Phi + z phi, phi = e^(-z^2/2) / sqrt(2 pi): 2.5 s and three roundings: 9.25 s Phi + 4 s |z phi| and a step of the sum."""
    g = torch.Generator().manual_seed(rows + o)
    s = 2.0 ** -23
    z = (torch.rand(rows, generator=g) * 18 - 9).float()
    z[:3] = torch.tensor([-3.0, 0.0, -0.7517916])
    X = torch.zeros(rows, i)
    X[torch.arange(rows), torch.arange(rows) % i] = z
    sign = (1 - 2 * (torch.arange(o) % 2)).float()
    W = sign.expand(i, o).contiguous()
    Z64 = z.double()[:, None] * sign.double()
    phi = torch.special.erfc(-Z64 / 2 ** 0.5) / 2        # (ndtr is 1 + erf: nothing of a tail)
    y = Z64 * phi
    Y, Z = forward(X.cuda(), W.cuda(), act="gelu", dtype="fp32")
    assert torch.equal(Z.cpu().double(), Z64)
    off = (Y.cpu().double() - y).abs()
    assert (off <= 10.25 * s * y.abs()).all(), float((off / (s * y.abs()).clamp(min=1e-300)).max())
    # the slope of Z, read off a product by 1: dX has one dZ in each row
    pdf = torch.exp(-Z64 * Z64 / 2) / (2 * torch.pi) ** 0.5
    slope = phi + Z64 * pdf
    tol = s * (9.25 * phi + 4 * (Z64 * pdf).abs() + slope.abs())
    dY = torch.zeros(rows, o)
    c = torch.arange(rows) % o
    dY[torch.arange(rows), c] = 1
    dX, _, _ = backward(None, W.cuda(), dY.cuda(), Z=Z, act="gelu", dw=False, dtype="fp32")
    want = (slope[torch.arange(rows), c] * sign.double()[c])[:, None]
    off = (dX.cpu().double() - want).abs()
    assert (off <= tol[torch.arange(rows), c][:, None]).all(), float((off / tol[torch.arange(rows), c][:, None]).max())
    # and of Zin, in the epilogue
    Zin = Z64[:, :1].float().expand(rows, i).contiguous()
    dX, _, _ = backward(None, torch.ones(i, o, device="cuda"), dY.cuda(), act_in="gelu", Zin=Zin.cuda(), dw=False, dtype="fp32")
    off = (dX.cpu().double() - slope[:, :1]).abs()
    assert (off <= tol[:, :1]).all(), float((off / tol[:, :1]).max())


FP32_SHAPES = [(rows, i, o) for dtype, rows, i, o in NAN_SHAPES if dtype == "fp32"] + [(200, 2048, 264), (777, 2200, 1030)]


@pytest.mark.parametrize("rows,i,o", FP32_SHAPES)
def test_infinities_in_fp32_stay_in_their_rows(rows, i, o):
    """In every form: the sums that an infinity, or a product beyond the type, enters are infinite or NaN, the others the same bits as without it."""
    g = torch.Generator(device="cuda").manual_seed(rows + o)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X, W, b, dY, R = new(rows, i), new(i, o), new(o), new(rows, o), new(rows, o)
    W[W == 0] = 1
    W[3] = W[3].sign() * (2 + W[3].abs())
    Y0, Z0 = forward(X, W, b, R, dtype="fp32")
    d0 = backward(X, W, dY, dtype="fp32")
    for v in (float("inf"), float("-inf"), 3e38):
        Xv, dYv = X.clone(), dY.clone()
        Xv[1, 3] = v
        row = torch.arange(rows, device="cuda") == 1
        for got, clean in zip(forward(Xv, W, b, R, dtype="fp32"), (Y0, Z0)):
            assert torch.equal(got[~row], clean[~row]) and not torch.isfinite(got[row]).any()
        dYv[2, 5] = v
        if abs(v) != float("inf"):
            continue                                      # (its products with weights and inputs below 1 are finite)
        dX, dW, dB = backward(X, W, dYv, dtype="fp32")
        row, col = torch.arange(rows, device="cuda") == 2, torch.arange(o, device="cuda") == 5
        assert torch.equal(dX[~row], d0[0][~row]) and not torch.isfinite(dX[row]).any()
        assert torch.equal(dW[:, ~col], d0[1][:, ~col]) and not torch.isfinite(dW[:, col]).any()
        assert torch.equal(dB[~col], d0[2][~col]) and not torch.isfinite(dB[col]).any()


@pytest.mark.parametrize("rows,i,o", FP32_SHAPES)
def test_the_largest_and_smallest_numbers_in_fp32(rows, i, o):
    """The type's lowest and largest values, as masks hold them, and tiny ones: one product a sum, by a power of two, is exact
    (the third part of a value of 2^-100 still has 9 bits above 2^-133)."""
    top = torch.finfo(torch.float32).max
    values = torch.tensor([top, -top, top * (1 - 2.0 ** -10), 2.0 ** -100 * (1 + 2.0 ** -23), -(2.0 ** -90) * (2 - 2.0 ** -23), 1 + 2.0 ** -23, -0.0])
    z = values[torch.arange(rows) % len(values)]
    X = torch.zeros(rows, i)
    X[torch.arange(rows), torch.arange(rows) % i] = z
    W = torch.tensor([0.5, -1.0, 0.125])[torch.arange(o) % 3].expand(i, o).contiguous()
    Y, _ = forward(X.cuda(), W.cuda(), dtype="fp32")
    assert torch.equal(Y.cpu().double(), z.double()[:, None] * W[:1].double())


@pytest.mark.parametrize("rows,i,o", [(23_661, 2376, 8), (40_000, 1500, 10), (26_000, 2376, 5)])
def test_bias_gradients_in_fp32_are_summed_in_short_chains(rows, i, o):
    """Equal positive values, whose roundings to a sum beyond 1024 all go one way.  A sum takes 16 rows by themselves (16 additions), then at most 2048 / 16
    such sums of its part of the rows, then at most 128 parts in eights (16 + 8): each off by half a step (2^-24) of the whole."""
    parts = eaga.linear_form(eaga.linear_dims(rows, i, o, "none", "fp32"), "dW")
    assert parts == "cores 32x32 split" or parts == "cores 64x64 split"
    dY = torch.full((rows, o), 1 + 0.49 * 2.0 ** -13, device="cuda")
    X, W = torch.zeros(rows, i, device="cuda"), torch.zeros(i, o, device="cuda")
    _, _, dB = backward(X, W, dY, dtype="fp32")
    exact = rows * dY[0, 0].double()
    assert ((dB.double() - exact).abs() <= (16 + 2048 / 16 + 24) * 2.0 ** -24 * exact).all(), float((dB.double() / exact - 1).abs().max() * 2 ** 24)
