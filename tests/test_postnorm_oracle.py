"""Pins of the post-norm block's float64 oracle: finite differences for every gradient, torch's own
layer_norm and linear on the CPU, and the checkpoint format by its definition."""
import numpy as np
import pytest
import torch

from oracle import postnorm as P

R = np.random.default_rng(5)


def diff(f, a, g, h=1e-6, n=40):
    """Largest error of the gradient g of sum(f * seed) against central differences at n places."""
    worst = 0.0
    for _ in range(n):
        i = tuple(R.integers(0, s) for s in a.shape)
        keep = a[i]
        a[i] = keep + h
        hi = f()
        a[i] = keep - h
        lo = f()
        a[i] = keep
        worst = max(worst, abs((hi - lo) / (2 * h) - g[i]))
    return worst


@pytest.mark.parametrize("width", [1, 7, 32, 65])
def test_layer_norm_against_torch_and_differences(width):
    z, dy = R.normal(size=(3, 4, width)) + 0.5, R.normal(size=(3, 4, width))
    gain, bias, eps = R.normal(size=width), R.normal(size=width), 1e-3
    f = P.layer_norm(z, gain, bias, eps)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(z), (width,), torch.from_numpy(gain), torch.from_numpy(bias), eps)
    assert np.abs(f["y"] - ref.numpy()).max() < 1e-12
    b = P.layer_norm_backward(z, dy, gain, f["mean"], f["rstd"])
    loss = lambda: (P.layer_norm(z, gain, bias, eps)["y"] * dy).sum()
    # eps 1e-3: the third derivative of the norm is below 1e6, so the differences are good to 1e-6
    assert diff(loss, z, b["dz"]) < 1e-6
    assert diff(loss, gain, b["dgain"]) < 1e-6
    assert diff(loss, bias, b["dbias"]) < 1e-6


def test_mix_rows_and_revert_are_inverse_and_match_the_definition():
    B, T, D, H = 2, 6, 12, 4
    x = np.arange(B * T * D, dtype=np.float64).reshape(B, T, D)
    r = P.mix_rows(x, H)
    for b, h, t, j in [(0, 0, 0, 0), (1, 3, 5, 2), (0, 2, 4, 1)]:
        assert r[b, h, t * 3 + j] == x[b, t, h * 3 + j]
    assert np.array_equal(P.revert_rows(r, T), x)


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_linear_against_torch_and_differences(name):
    x, w, bias = R.normal(size=(5, 3, 6)), R.normal(size=(3, 4, 6)), R.normal(size=(3, 4))
    dy, res = R.normal(size=(5, 3, 4)), R.normal(size=(5, 3, 4))
    y, z = P.linear(x, w, bias, name, res)
    tz = torch.einsum("bgk,gnk->bgn", torch.from_numpy(x), torch.from_numpy(w)) + torch.from_numpy(bias)
    f = {"none": lambda t: t, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[name]
    assert np.abs(y - (f(tz).numpy() + res)).max() < 1e-12
    g = P.linear_backward(x, dy, z, w, name)
    loss = lambda: (P.linear(x, w, bias, name, res)[0] * dy).sum()
    for a, k in ((x, "dx"), (w, "dw"), (bias, "db")):
        assert diff(loss, a, g[k]) < 1e-6


def test_checkpoint_by_its_definition():
    z = R.normal(size=(50, 70)) * np.exp2(R.integers(-20, 20, size=(50, 1)).astype(float))
    code, e, val = P.checkpoint8(z)
    assert e.shape == (50, 3) and np.abs(code).max() <= 127
    step = np.repeat(np.exp2(e.astype(float)), 32, axis=1)[:, :70]
    assert (np.abs(val - z) <= step / 2).all()
    for r in range(50):                                    # the exponent is the smallest that holds the block
        for k in range(3):
            top = np.abs(z[r, 32 * k:32 * k + 32]).max()
            assert top <= 127 * 2.0 ** e[r, k] and top > 127 * 2.0 ** (e[r, k] - 1)


def test_checkpoint_borders():
    z = np.zeros((1, 32))
    assert P.checkpoint8(z)[1][0, 0] == -126 and not P.checkpoint8(z)[2].any()
    z[0, 0] = 127.0
    z[0, 1:4] = 0.5, 1.5, -2.5                             # ties to even
    code, e, val = P.checkpoint8(z)
    assert e[0, 0] == 0 and list(code[0, :4]) == [127, 0, 2, -2]
    z[0, 0] = 127.5
    assert P.checkpoint8(z)[1][0, 0] == 1
    z[0, 0] = np.inf
    z[0, 4] = np.nan
    code, e, val = P.checkpoint8(z)
    assert e[0, 0] == 127 and not code.any() and np.isnan(val).all()
    tiny = np.full((1, 5), 2.0 ** -140)
    assert P.checkpoint8(tiny)[1][0, 0] == -126 and not P.checkpoint8(tiny)[0].any()
