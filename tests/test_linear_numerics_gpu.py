"""What the linear operator's results may be off by, and what infinities and NaN become, beyond the parity tests."""
import pytest
import torch

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
