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
