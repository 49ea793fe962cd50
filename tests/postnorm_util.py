"""Inputs and error bounds of the post-norm block's GPU tests.

Every bound is worst-case arithmetic, derived here before any run, with u = 2^-24 (half a step of fp32)
and h = half a step of the storage type relative to the value (bf16 2^-8, fp32 2^-24):

* a sum of n fp32 terms taken by threads, shuffles and blocks passes each term through at most
  d <= 32 + 9 + 16 additions for a row (32 in a thread, 9 shuffle and warp steps, the rest spare), so it
  is off by at most 64 u sum|terms| here;
* row sums over R rows (dgain, dbias, db) pass each term through at most R + 64 additions;
* a tensor-core contraction of depth K: products of bf16 are exact in fp32, additions are taken in an
  unknown order and may truncate (2 u each): (K + 8) 2 u sum|products|;
* bf16 activations use the short forms whose documented relative error is 3.7e-4 (gelu's tail) plus 4 u
  and the two exponentials' 2^-22 each: 5e-4 of |z| Q(|z|) <= 0.17, and of the value itself for silu;
  gelu's slope is documented to an absolute 1.6e-5, plus the exponential's and the polynomial's rounding
  (seven terms of at most 1, 2 u each): 2e-5.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda:0"


def draw(rng, shape, dtype, std=1.0, mean=0.0):
    """(device tensor, its float64 values) of normal values rounded to the storage type."""
    t = torch.from_numpy((rng.normal(size=shape) * std + mean).astype(np.float32)).to(DT[dtype])
    return t.to(DEV), t.double().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, want, tol):
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), got.size, got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, want.shape)[bad][:4])


def norm_tols(z, f, gain, bias, dtype):
    """Bounds of (mean, rstd, n without the storage rounding, y)."""
    g = np.ones(z.shape[-1]) if gain is None else np.abs(gain)
    b = 0.0 if bias is None else np.abs(bias)
    az = np.abs(z).mean(-1)
    tm = 67 * U * az                                       # the sum, 1/W and the product with it, z's addition (1 u)
    # d = z - mu is off by tm + 2 u (|z| + |mu|); squares summed (64 u), halved by the root, 4 more steps
    spread = np.abs(z - f["mean"][..., None]).max(-1)
    td = tm + 2 * U * (np.abs(z).max(-1) + np.abs(f["mean"]))
    # relative: half the sum's error, d's error times rstd, and rsqrtf's documented 2 ulp (4 u)
    tr = f["rstd"] * (70 * U + f["rstd"] * td * 1.01)
    tn = (td * f["rstd"])[..., None] + np.abs(f["n"]) * ((tr / f["rstd"])[..., None] + 4 * U)
    ty = tn * g + 2 * U * (np.abs(f["n"]) * g + b)
    ty = ty + HALF[dtype] * (np.abs(f["y"]) + ty)
    return tm, tr, tn, ty


def norm_bwd_tols(z, f, bwd, dy, gain, tn, dtype):
    """Bounds of (dz, dgain, dbias) when mean and rstd are the library's own."""
    rows = int(np.prod(z.shape[:-1]))
    n, dn, rs = np.abs(bwd["n"]) + tn, np.abs(bwd["dn"]), f["rstd"][..., None] * (1 + 1e-4)
    m1 = dn.mean(-1, keepdims=True)
    m2 = (dn * n).mean(-1, keepdims=True)
    # the two means (66 u, dn rounded: 1 u, n's error), the combination (4 u each term), rstd's error
    e2 = 68 * U * m2 + (dn * tn).mean(-1, keepdims=True)
    td = rs * (5 * U * (dn + m1 + n * m2) + 67 * U * m1 + n * e2 + tn * m2)
    rel = (tn.max(-1, keepdims=True) / np.maximum(np.abs(bwd["n"]).max(-1, keepdims=True), 1e-3))
    td = td + np.abs(bwd["dz"]) * (rel + 70 * U)
    tdz = td + HALF[dtype] * (np.abs(bwd["dz"]) + td)
    lead = tuple(range(z.ndim - 1))
    tg = ((rows + 64) * U * np.abs(dy) * n + np.abs(dy) * tn).sum(lead)
    tb = (rows + 64) * U * np.abs(dy).sum(lead)
    return (tdz, td, tg + HALF[dtype] * (np.abs(bwd["dgain"]) + tg), tb + HALF[dtype] * (np.abs(bwd["dbias"]) + tb))


def act_err(z, name, dtype):
    """Error of the activation itself at an exact z."""
    from scipy.special import expit, ndtr
    if dtype == "f32":
        return 16 * U * (np.abs(z) + 1.0) * (name != "none")     # CUDA's erfcf, expf: a few u each
    a = np.abs(z)
    return {"gelu": 5e-4 * a * ndtr(-a), "silu": 1e-5 * a * expit(z)}.get(name, 0.0 * a) + 4 * U * a


def slope_err(z, name, dtype):
    a = np.abs(z)
    if dtype == "f32":
        return 16 * U * (1.0 + a) * (name not in ("none", "relu"))
    return {"gelu": 0.0 * a + 2e-5, "silu": 1e-5 * (1 + a)}.get(name, 0.0 * a)


def linear_tols(x, w, bias, z, y, name, residual, dtype):
    """Bounds of (z before any rounding, y)."""
    K = x.shape[-1]
    mag = np.einsum("bgk,gnk->bgn", np.abs(x), np.abs(w)) + (0.0 if bias is None else np.abs(bias))
    tz = ((K + 8) * 2 * U) * mag
    ty = 1.13 * tz + act_err(z, name, dtype) + 2 * U * (np.abs(y) + (0.0 if residual is None else np.abs(residual)))
    return tz, ty + HALF[dtype] * (np.abs(y) + ty)


def linear_bwd_tols(x, dy, z, w, name, g, dtype, dx_add=None):
    """Bounds of (dx, dw, db) for the z that the library was given."""
    B, N = x.shape[0], w.shape[1]
    tdz = np.abs(dy) * slope_err(z, name, dtype) + 4 * U * np.abs(g["dz"])
    tdr = tdz if name == "none" else tdz + HALF[dtype] * (np.abs(g["dz"]) + tdz)   # dz stored for the products
    adz = np.abs(g["dz"]) + tdr
    tx = np.einsum("bgn,gnk->bgk", tdr + (N + 8) * 2 * U * adz, np.abs(w))
    tw = np.einsum("bgn,bgk->gnk", tdr + (B + 8) * 2 * U * adz, np.abs(x))
    tb = (tdz + (B + 64) * U * adz).sum(0)
    ax = np.abs(g["dx"] + (0.0 if dx_add is None else dx_add))
    tx = tx + 2 * U * (ax + np.abs(g["dx"]))
    h = HALF[dtype]
    return tx + h * (ax + tx), tw + h * (np.abs(g["dw"]) + tw), tb + h * (np.abs(g["db"]) + tb)
