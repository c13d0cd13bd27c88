"""Each kernel that the linear operator may choose, at a size that chooses it, on whole numbers: exact sums, so equal bit for bit.

`test_linear_forms.py` checks, without a GPU, that these shapes and those of `test_linear_gpu.py` reach every kernel there is."""
import pytest
import torch

from test_linear_gpu import TD, backward, forward

pytestmark = pytest.mark.gpu

SHAPES = [  # rows, in, out
    # two CTAs an SM: whole and ragged, one step and four
    (100_000, 64, 64), (80_001, 40, 56), (77_000, 256, 64), (77_003, 64, 256), (90_000, 64, 250),
    # pairs with bf16 outputs by TMA, whole and ragged, unsplit and split
    (4096, 2048, 4096), (4000, 2040, 4072), (652, 6624, 1704), (151, 7736, 5981), (137, 7086, 3560), (3703, 1826, 1285),
    # fp32 input gradients by warps, long and short reductions; tiles of 128 x 32; weight gradients of narrow operands
    (2847, 5, 289), (285, 2, 204), (5001, 13, 300), (1000, 32, 75), (200_000, 24, 32), (60_003, 30, 23), (58_208, 50, 40), (19, 1, 1),
    # single tiles of 128 and 64 columns, unsplit and split, rows that are not 16 bytes
    (23, 4983, 1059), (15_481, 114, 83), (18_908, 165, 35),
    # two and five rows
    (2, 1, 8), (5, 1, 8), (2, 100, 88), (5, 300, 264),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,i,o", SHAPES)
def test_every_form(rows, i, o, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + i)
    new = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(TD[dtype])
    X, W, b, R, dY, dR, Zin, zo = (new(*s) for s in ((rows, i), (i, o), (o,), (rows, o), (rows, o), (rows, i), (rows, i), (rows, o)))
    z = X.double() @ W.double() + b.double()
    for res in (R, None):
        for save in (True, False):
            Y, Z = forward(X, W, b, res, act="relu", save=save, dtype=dtype)
            assert not save or torch.equal(Z, z.to(TD[dtype]))
            assert torch.equal(Y, (z.clamp(min=0) + (R.double() if res is not None else 0)).to(TD[dtype]))
    Y, _ = forward(X, W, save=False, dtype=dtype)
    assert torch.equal(Y, (z - b.double()).to(TD[dtype]))
    dx, dw = dY.double() @ W.double().T, X.double().T @ dY.double()
    for zi, res in ((None, None), (Zin, None), (None, dR), (Zin, dR)):
        dX, dW, dB = backward(X, W, dY, act_in="relu" if zi is not None else "none", Zin=zi, dR=res, dtype=dtype)
        want = dx * (Zin.double() > 0) if zi is not None else dx
        assert torch.equal(dX.double(), (want + (dR.double() if res is not None else 0)).to(TD[dtype]).double())
        assert torch.equal(dW.double(), dw) and torch.equal(dB.double(), dY.double().sum(0))
    dz = dY.double() * (zo.double() > 0)
    dX, dW, dB = backward(X, W, dY, Z=zo, act="relu", act_in="relu", Zin=Zin, dR=dR, dtype=dtype)
    assert torch.equal(dX.double(), ((dz @ W.double().T) * (Zin.double() > 0) + dR.double()).to(TD[dtype]).double())
    assert torch.equal(dW.double(), X.double().T @ dz) and torch.equal(dB.double(), dz.sum(0))
    # one gradient without the other
    assert torch.equal(backward(None, W, dY, dR=dR, dw=False, dtype=dtype)[0].double(), (dx + dR.double()).to(TD[dtype]).double())
    assert torch.equal(backward(X, W, dY, dx=False, dtype=dtype)[1].double(), dw)
