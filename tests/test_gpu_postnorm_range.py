"""GPU tests of the per-token linear layer's activations and slopes over every finite pre-activation of bf16 (each of the 65280
values, in bf16 and as fp32), through identity weights, against the float64 oracle; and of rows whose mean is large
against their spread.

The bounds, derived before any run; h is half a step of the storage type relative to the value:

* bf16 silu, z < 0: e^-z, whose exponent of up to 127 in fp32 with two roundings is off by 2 * 127 * 2^-24 = 1.5e-5;
  the exponential, the reciprocal and five steps (2^-20): 2e-4 of the value, as far as the reciprocal is a normal fp32
  number (2^-126).  Below that it is taken as 0: silu is at most 90 * 2^-126 < 2^-119 there.
* bf16 gelu, z < 0: the documented 3.7e-4 of the tail up to 6, an exponent of up to 30 there in fp32 with six roundings
  (6 * 30 u ln 2 = 8e-6), the exponential and two steps: 4.5e-4.  Past 6 the tail is documented to fall short by up to all
  of it: an absolute 6e-9 at most.
* z >= 0: the value is z less a tail with the same bound, and 4 u of z.
* fp32: expf is good to a few u, its argument's rounding is multiplied by at most |z| <= 90 before the tail leaves
  the normal numbers: 4 * 90 * u < 3e-5; erfcf's argument is multiplied by a^2 <= 180, 2 u of it: the same.
* slopes: the documented absolute bound, and h of the value;
* gelu's slope from -1.5 down keeps its relative precision as far as its exponential is a normal fp32 number: the
  documented 1.5e-4 in bf16, an exponent of up to 126 with three roundings (3 * 126 u ln 2 = 1.6e-5), and the exponential,
  the reciprocal and five steps whose cancellation at most doubles them (16 u): 2e-4.  In fp32 the exponent's rounding
  is multiplied by at most a^2 / 2 <= 90, erfcf's by a^2 <= 180 of a term that is a third of the other at 1.5 and less
  beyond, and expf and erfcf are good to a few u: below 2 * 300 u < 1e-4.  Below the normal numbers the slope may be
  taken as 0: at most 6 * 2^-126 there.
"""
import numpy as np
import pytest
import torch

from oracle import postnorm as P
from postnorm_util import DEV, DT, HALF, U, check, f64
from token_sparse_moe_b200 import _abi as A
from token_sparse_moe_b200 import api

pytestmark = pytest.mark.gpu
GONE = 2.0 ** -119                        # what a tail below the normal fp32 numbers may have held


def every_value(order):
    """All finite bf16 values as [8160, 8]: by their bits, or shuffled so that neighbours differ wildly."""
    bits = np.arange(65536, dtype=np.uint32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    if order == "shuffled":
        bits = np.random.default_rng(5).permutation(bits)
    return (bits << 16).view(np.float32).reshape(-1, 8)


def eye(banks, dtype):
    return torch.eye(8, dtype=DT[dtype], device=DEV).expand(banks, 8, 8).contiguous()


def forward_bound(z, y, act, dtype):
    rel = {"f32": 3e-5, "bf16": {"gelu": np.where(np.abs(z) <= 6, 4.5e-4, 1.0), "silu": 2e-4}.get(act, 0.0)}[dtype]
    tail = y if act == "relu" else np.where(z < 0, y, y - z)          # of positive z: z less the tail
    t = 0.0 * z if act == "relu" else rel * np.abs(tail) + GONE + 4 * U * np.maximum(z, 0)
    return t + HALF[dtype] * (np.abs(y) + t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["many", "one"])
@pytest.mark.parametrize("order", ["by bits", "shuffled"])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_activation_of_every_finite_value(dtype, form, order, act):
    """`many`: 8160 samples of one bank; `one`: one sample of 8160 banks."""
    z = every_value(order)
    shape = (8160, 1, 8) if form == "many" else (1, 8160, 8)
    x = torch.from_numpy(z).reshape(shape).to(DT[dtype]).to(DEV)
    y = api.pertoken_linear(x, api.Linear(eye(shape[1], dtype), None, act))
    z = z.astype(np.float64).reshape(shape)
    want = P.act(z, act)
    check(act, y, want, forward_bound(z, want, act, dtype))


def every_slope(act, dtype, save, order):
    """(pre-activations that the backward works from, dz for dy = 1) of all finite values."""
    z = torch.from_numpy(every_value(order)).reshape(8160, 1, 8).to(DT[dtype]).to(DEV)
    saved = z if save == "full" else api.checkpoint8_pack(z)
    if save == "ckpt8":
        z = api.checkpoint8_unpack(saved)
    one = torch.ones_like(z)
    dx, g = api.pertoken_linear_backward(one, one, api.Linear(eye(1, dtype), torch.zeros(1, 8, dtype=DT[dtype], device=DEV), act),
                                         saved)
    assert torch.isfinite(g["dw"]).all() and torch.isfinite(g["db"]).all()
    return f64(z), dx                     # dx = dz through the identity


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("save,order", [("full", "by bits"), ("full", "shuffled"), ("ckpt8", "by bits")])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_slope_of_every_finite_value(dtype, save, order, act):
    """Slopes of bf16 to the documented absolute bound (gelu 2e-5, silu 1e-5 with its roundings; fp32 16 u of 1 + |z| up
    to 20, past which the slope is 0 or 1 to 1e-7)."""
    z, dz = every_slope(act, dtype, save, order)
    want = P.act_slope(z, act)
    t = 0.0 * z
    if act != "relu":
        t = t + (16 * U * (1 + np.minimum(np.abs(z), 20)) if dtype == "f32" else {"gelu": 2e-5, "silu": 1e-5}[act])
    check(act, dz, want, t + HALF[dtype] * (np.abs(want) + t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("save", ["full", "ckpt8"])
def test_slope_of_gelu_keeps_its_precision_in_the_tail(dtype, save):
    z, dz = every_slope("gelu", dtype, save, "by bits")
    want = P.act_slope(z, "gelu")
    t = np.where(z <= -1.5, {"bf16": 2e-4, "f32": 1e-4}[dtype], np.inf) * np.abs(want) + 2.0 ** -123
    check("gelu", dz, want, t + HALF[dtype] * (np.abs(want) + t))


@pytest.mark.parametrize("width", [45, 384, 1000, 3000])
def test_rows_of_a_large_mean_from_the_checkpoint(width):
    """Values of 100 and, one in 16, 101 (exact in the checkpoint): the mean is 400 standard deviations.  With one row dgain
    is dy n, n = (z - mean) rstd: a subtraction, two products and, in fp32, nothing else to round: 4 u of it."""
    rng = np.random.default_rng(width)
    zo = 100.0 + (rng.random((1, 1, width)) < 1 / 16)
    zo[0, 0, 0] = 101.0
    do = rng.normal(size=zo.shape).astype(np.float32).astype(np.float64)
    z, dy = (torch.from_numpy(v).float().to(DEV) for v in (zo, do))
    sh = api.shape(1, 1, width, 1, "f32", 1e-6)
    _, saved = api.layer_norm(z, None, A.TM_LAYOUT_ROWS, sh, checkpoint8=True)
    assert torch.equal(api.checkpoint8_unpack(saved.ckpt), z)
    _, _, grads = api.layer_norm_backward(dy, saved, A.TM_LAYOUT_ROWS, sh)
    want = P.layer_norm_backward(zo, do, None, f64(saved.mean), f64(saved.rstd))["dgain"]
    check("dgain", grads["dgain"], want, 4 * U * np.abs(want) + 1e-30)
