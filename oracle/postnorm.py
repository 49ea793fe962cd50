"""Float64 oracle of the post-norm per-token block: layer norm, per-token linear layers, their
gradients, and the values of an 8-bit activation checkpoint.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code with the library.

Source: [digest] 2.3.1 Eq. 5-8 (post-norm token mixing LN(TM(X) + X) and per-token FFN of the
predecessor block) and its per-token FFN with bias; the gradients are the chain rule:

    z = x + r,  mu = mean(z),  s = 1 / sqrt(mean((z - mu)^2) + eps),  n = (z - mu) s,  y = n g + b
    dn = dy g,  dz = s (dn - mean(dn) - n mean(dn n)),  dg = sum dy n,  db = sum dy

    z = x W^T + b,  y = act(z) + r;  dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum dz
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np
from scipy.special import erfc, expit


def checkpoint8(z: np.ndarray):
    """(codes, exponents, values) of rows [..., width]: blocks of 32 values share 2^e, e the smallest
    integer with max|z| <= 127 * 2^e, at least -126 and at most 121; codes held to +-127.  A block with a
    value that is not finite has e = 127, codes 0 and values NaN."""
    z = np.asarray(z, np.float64)
    width = z.shape[-1]
    nblk = -(-width // 32)
    b = np.zeros(z.shape[:-1] + (nblk * 32,))
    b[..., :width] = z
    b = b.reshape(z.shape[:-1] + (nblk, 32))
    fin = np.isfinite(b).all(-1)
    b = np.where(fin[..., None], b, 0.0)
    top = np.abs(b).max(-1)
    m, x = np.frexp(top)                                   # top = m 2^x, m in [1/2, 1)
    e = np.where(top > 0, x - 7 + (m > 127.0 / 128.0), -126)
    e = np.clip(e, -126, 121)
    code = np.clip(np.rint(np.ldexp(b, -e[..., None])), -127, 127)
    val = np.where(fin[..., None], np.ldexp(code, e[..., None]), np.nan)
    e = np.where(fin, e, 127)
    cut = lambda a: a.reshape(z.shape[:-1] + (nblk * 32,))[..., :width]
    return cut(code).astype(np.int64), e.astype(np.int64), cut(val)


def mix_rows(x: np.ndarray, H: int) -> np.ndarray:
    """Row h, column t * dh + j of sample b is x[b, t, h * dh + j]."""
    B, T, D = x.shape
    dh = D // H
    return np.stack([x[:, :, h * dh:(h + 1) * dh].reshape(B, T * dh) for h in range(H)], axis=1)


def revert_rows(r: np.ndarray, T: int) -> np.ndarray:
    B, H, W = r.shape
    dh = W // T
    out = np.empty((B, T, H * dh))
    for h in range(H):
        out[:, :, h * dh:(h + 1) * dh] = r[:, h].reshape(B, T, dh)
    return out


def layer_norm(z: np.ndarray, gain, bias, eps: float) -> Dict[str, np.ndarray]:
    mu = z.mean(-1)
    d = z - mu[..., None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    n = d * rstd[..., None]
    y = n * (1.0 if gain is None else gain) + (0.0 if bias is None else bias)
    return {"y": y, "mean": mu, "rstd": rstd, "n": n}


def layer_norm_backward(z: np.ndarray, dy: np.ndarray, gain, mean: np.ndarray, rstd: np.ndarray) -> Dict[str, np.ndarray]:
    """dz, dgain, dbias; mean and rstd are the forward's (z may be what a checkpoint kept)."""
    n = (z - mean[..., None]) * rstd[..., None]
    dn = dy * (1.0 if gain is None else gain)
    dz = rstd[..., None] * (dn - dn.mean(-1, keepdims=True) - n * (dn * n).mean(-1, keepdims=True))
    lead = tuple(range(z.ndim - 1))
    return {"dz": dz, "dgain": (dy * n).sum(lead), "dbias": dy.sum(lead), "n": n, "dn": dn}


def act(z: np.ndarray, name: str) -> np.ndarray:
    return {"none": lambda: z, "relu": lambda: np.maximum(z, 0.0), "gelu": lambda: 0.5 * z * erfc(-z / np.sqrt(2.0)),
            "silu": lambda: z * expit(z)}[name]()


def act_slope(z: np.ndarray, name: str) -> np.ndarray:
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if name == "silu":
        s = expit(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def linear(x: np.ndarray, w: np.ndarray, bias, name: str, residual: Optional[np.ndarray] = None):
    """x [B, banks, K], w [banks, N, K]: (y, z)."""
    z = np.einsum("bgk,gnk->bgn", x, w)
    if bias is not None:
        z = z + bias
    y = act(z, name)
    return (y if residual is None else y + residual), z


def linear_backward(x: np.ndarray, dy: np.ndarray, z: np.ndarray, w: np.ndarray, name: str) -> Dict[str, np.ndarray]:
    dz = dy * act_slope(z, name)
    return {"dx": np.einsum("bgn,gnk->bgk", dz, w), "dw": np.einsum("bgn,bgk->gnk", dz, x), "db": dz.sum(0), "dz": dz}
