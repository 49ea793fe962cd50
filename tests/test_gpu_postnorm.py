"""GPU tests of the post-norm block's operators against the float64 oracle (bounds: postnorm_util)."""
import numpy as np
import pytest
import torch

from oracle import postnorm as P
from postnorm_util import DEV, DT, HALF, U, act_err, check, draw, f64, linear_bwd_tols, linear_tols, norm_bwd_tols, norm_tols
from token_sparse_moe_b200 import _abi as A
from token_sparse_moe_b200 import api

pytestmark = pytest.mark.gpu
EPS = 1e-6


# ------------------------------------------------------------------ 8-bit checkpoints
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 32), (3, 31), (7, 33), (5, 8), (65, 72), (1000, 100), (37, 512),
                                        (2, 4097), (513, 64), (3000, 36)])
def test_checkpoint_is_the_format_to_the_bit(dtype, rows, width):
    rng = np.random.default_rng(rows * 7 + width)
    scale = torch.from_numpy(np.exp2(rng.integers(-60, 60, size=(rows, 1))))
    x, _ = draw(rng, (rows, width), dtype)
    x = (x.double() * scale.to(DEV)).to(DT[dtype])
    code, e, val = P.checkpoint8(f64(x))
    ck = api.checkpoint8_pack(x)
    assert np.array_equal(f64(ck.codes), code) and np.array_equal(f64(ck.exps), e)
    back = api.checkpoint8_unpack(ck)
    assert back.dtype == x.dtype and np.array_equal(f64(back), val)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [64, 45])
def test_checkpoint_of_values_at_the_borders(dtype, width):
    """Infinities and NaN (alone in a block, with others, whole blocks of them: the block reads back as NaN),
    the type's largest and smallest values, zeros, ties, and maxima on both sides of 127 * 2^e."""
    fin = torch.finfo(DT[dtype])
    x = torch.zeros(12, width)
    x[0, 3] = float("inf")
    x[1, :5] = torch.tensor([float("nan"), 1.0, -2.5, 0.5, float("-inf")])
    x[2] = float("nan")
    x[3, 0], x[3, 1] = fin.max, -fin.max
    x[4, :3] = torch.tensor([fin.tiny, -fin.tiny, fin.tiny / 4])
    x[5, 0], x[5, 1], x[5, 2] = 127.0, 0.5, 1.5
    x[6, 0], x[6, 1] = 127.5, 1.0
    x[7, 0], x[7, 1] = 128.0, -1.0
    x[8, 33], x[8, 0] = 3.0, float("inf")
    x[9] = -float("inf")
    x[10, 1] = fin.smallest_normal
    x[11, 31], x[11, 32] = 1e30, 1e-30
    x = x.to(DT[dtype]).to(DEV)
    code, e, val = P.checkpoint8(f64(x))
    ck = api.checkpoint8_pack(x)
    assert np.array_equal(f64(ck.codes), code) and np.array_equal(f64(ck.exps), e)
    assert np.array_equal(f64(api.checkpoint8_unpack(ck)), val, equal_nan=True)


# ------------------------------------------------------------------ layer norm
ROWS = [(1, 1, 1), (1, 1, 8), (3, 5, 64), (7, 3, 40), (5, 2, 128), (9, 4, 256), (33, 3, 384), (6, 2, 512), (5, 3, 768),
        (4, 2, 1024), (3, 1, 2048), (2, 2, 4096), (1, 2, 8200), (2, 1, 16384), (4, 3, 17), (3, 2, 300), (2, 2, 999),
        (2, 1, 5001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,banks,W", ROWS)
@pytest.mark.parametrize("with_res,ckpt", [(True, False), (False, True), (True, True)])
def test_layer_norm_rows(dtype, B, banks, W, with_res, ckpt):
    rng = np.random.default_rng(B * 1000 + W)
    x, xo = draw(rng, (B, banks, W), dtype, mean=0.7)
    res, ro = draw(rng, (B, banks, W), dtype) if with_res else (None, 0.0)
    gain, go = draw(rng, (W,), dtype, std=0.2, mean=1.0)
    bias, bo = draw(rng, (W,), dtype, std=0.2)
    dy, do = draw(rng, (B, banks, W), dtype)
    # the norm acts on the fp32 sum (exact rounding of the two stored values' sum)
    z = (xo + ro).astype(np.float32).astype(np.float64)
    f = P.layer_norm(z, go, bo, EPS)
    sh = api.shape(B, banks, W, 1, DT[dtype], EPS)
    y, saved = api.layer_norm(x, res, A.TM_LAYOUT_ROWS, sh, gain, bias, checkpoint8=ckpt)
    if W == 1:       # one value: the mean is the value, rstd 1 / sqrt(eps), y the bias
        check("y", y, np.broadcast_to(bo, z.shape), HALF[dtype] * np.abs(bo) + 1e-30)
        return
    tm, tr, tn, ty = norm_tols(z, f, go, bo, dtype)
    check("mean", saved.mean, f["mean"], tm)
    check("rstd", saved.rstd, f["rstd"], tr)
    check("y", y, f["y"], ty)
    zb = z
    if ckpt:
        code, e, zb = P.checkpoint8(z)
        assert np.array_equal(f64(saved.ckpt.codes), code) and np.array_equal(f64(saved.ckpt.exps), e)
    b = P.layer_norm_backward(zb, do, go, f["mean"], f["rstd"])
    tn = tn + np.abs(zb - z) * 0       # the checkpoint's values are exact in the library too
    tdz, _, tg, tb = norm_bwd_tols(zb, f, b, do, go, tn + np.abs(b["n"]) * (tr / f["rstd"])[..., None], dtype)
    kw = {} if ckpt else dict(x=x, residual=res)
    dx, dres, grads = api.layer_norm_backward(dy, saved, A.TM_LAYOUT_ROWS, sh, gain, **kw)
    check("dx", dx, b["dz"], tdz)
    assert (dres is dx) == with_res and (dres is None) == (not with_res)
    check("dgain", grads["dgain"], b["dgain"], tg)
    check("dbias", grads["dbias"], b["dbias"], tb)


MIXED = [(1, 2, 16, 2), (5, 8, 64, 8), (3, 4, 96, 2), (2, 3, 64, 8), (7, 16, 256, 16), (3, 32, 512, 32), (2, 48, 768, 48),
         (300, 5, 80, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,H", MIXED)
@pytest.mark.parametrize("ckpt", [False, True])
def test_layer_norm_mixed(dtype, B, T, D, H, ckpt):
    """Rows read through Mix; with T = H also the token mixing LN(Mix(X) + X) and X's whole gradient."""
    rng = np.random.default_rng(B + T * D + H)
    W = T * D // H
    x, xo = draw(rng, (B, T, D), dtype, mean=-0.4)
    gain, go = draw(rng, (W,), dtype, std=0.2, mean=1.0)
    bias, bo = draw(rng, (W,), dtype, std=0.2)
    dy, do = draw(rng, (B, H, W), dtype)
    sh = api.shape(B, T, D, H, DT[dtype], EPS)
    for self_ in ([False, True] if T == H else [False]):
        res, ro = (x, xo) if self_ else draw(rng, (B, H, W), dtype)
        z = (P.mix_rows(xo, H) + ro).astype(np.float32).astype(np.float64)
        f = P.layer_norm(z, go, bo, EPS)
        tm, tr, tn, ty = norm_tols(z, f, go, bo, dtype)
        y, saved = api.layer_norm(x, res, A.TM_LAYOUT_MIXED, sh, gain, bias, checkpoint8=ckpt)
        check("y", y, f["y"], ty)
        check("mean", saved.mean, f["mean"], tm)
        zb = P.checkpoint8(z)[2] if ckpt else z
        b = P.layer_norm_backward(zb, do, go, f["mean"], f["rstd"])
        tdz, td, tg, tb = norm_bwd_tols(zb, f, b, do, go, tn + np.abs(b["n"]) * (tr / f["rstd"])[..., None], dtype)
        kw = {} if ckpt else dict(x=x, residual=res)
        dx, dres, grads = api.layer_norm_backward(dy, saved, A.TM_LAYOUT_MIXED, sh, gain, residual_is_x=self_, **kw)
        if self_:
            assert dres is None
            whole = b["dz"] + P.revert_rows(b["dz"], T)
            t = td + P.revert_rows(td, T) + U * np.abs(whole)
            check("dX", dx, whole, t + HALF[dtype] * (np.abs(whole) + t))
        else:
            check("dresidual", dres, b["dz"], tdz)
            check("dx", dx, P.revert_rows(b["dz"], T), P.revert_rows(tdz, T))
        check("dgain", grads["dgain"], b["dgain"], tg)
        check("dbias", grads["dbias"], b["dbias"], tb)


# ------------------------------------------------------------------ per-token linear layer
LINEAR = [(1, 1, 8, 8), (1, 3, 64, 128), (5, 2, 72, 40), (64, 2, 64, 64), (128, 1, 256, 256), (129, 2, 128, 264),
          (200, 3, 136, 328), (300, 2, 320, 96), (33, 1, 768, 1536), (1000, 1, 40, 72), (700, 2, 384, 520)]
LINEAR_F32 = [(1, 1, 1, 1), (3, 2, 5, 7), (65, 2, 33, 70), (64, 8, 64, 128), (17, 1, 81, 196)]


def linear_case(dtype, B, banks, K, N, act, bias_, res_, save):
    rng = np.random.default_rng(B * 31 + K * 7 + N)
    x, xo = draw(rng, (B, banks, K), dtype)
    w, wo = draw(rng, (banks, N, K), dtype, std=K ** -0.5)
    bias, bo = draw(rng, (banks, N), dtype, std=0.3) if bias_ else (None, None)
    res, ro = draw(rng, (B, banks, N), dtype) if res_ else (None, None)
    dy, do = draw(rng, (B, banks, N), dtype)
    add, ao = draw(rng, (B, banks, K), dtype) if res_ else (None, None)
    lin = api.Linear(w, bias, act)
    yo, zo = P.linear(xo, wo, bo, act, ro)
    tz, ty = linear_tols(xo, wo, bo, zo, yo, act, ro, dtype)
    y, kept = api.pertoken_linear(x, lin, residual=res, save=save)
    check("y", y, yo, ty)
    zb = zo
    if act != "none":
        if save == "full":
            check("z", kept, zo, tz + HALF[dtype] * (np.abs(zo) + tz))
            zb = f64(kept)
        else:
            zb = f64(api.checkpoint8_unpack(api.Checkpoint8(kept.codes, kept.exps, torch.float32)))
            # half a step of the block's scale, which holds max|z| with at least 64 codes
            step = np.exp2(np.repeat(f64(kept.exps), 32, axis=-1)[..., :N])
            check("ckpt z", torch.from_numpy(zb), zo, step / 2 + tz)
            top = np.abs(np.pad(zo, ((0, 0), (0, 0), (0, -N % 32)))).reshape(B, banks, -1, 32).max(-1)
            assert (np.exp2(f64(kept.exps)) * 63.4 <= top + 1e-3).all()
    else:
        assert kept is None
    g = P.linear_backward(xo, do, zb, wo, act)
    tx, tw, tb = linear_bwd_tols(xo, do, zb, wo, act, g, dtype, ao)
    dx, grads = api.pertoken_linear_backward(x, dy, lin, kept, dx_add=add)
    check("dx", dx, g["dx"] + (0.0 if ao is None else ao), tx)
    check("dw", grads["dw"], g["dw"], tw)
    if bias_:
        check("db", grads["db"], g["db"], tb)
    else:
        assert "db" not in grads


@pytest.mark.parametrize("act,bias_,res_,save", [("none", True, True, "full"), ("none", False, False, "full"),
                                                 ("relu", True, False, "full"), ("gelu", True, True, "ckpt8"),
                                                 ("gelu", False, False, "full"), ("silu", True, False, "ckpt8"),
                                                 ("silu", True, True, "full"), ("relu", False, True, "ckpt8")])
@pytest.mark.parametrize("B,banks,K,N", LINEAR)
def test_linear_bf16(B, banks, K, N, act, bias_, res_, save):
    linear_case("bf16", B, banks, K, N, act, bias_, res_, save)


@pytest.mark.parametrize("act,bias_,res_,save", [("none", True, True, "full"), ("relu", True, False, "full"),
                                                 ("gelu", True, True, "ckpt8"), ("silu", False, False, "full")])
@pytest.mark.parametrize("B,banks,K,N", LINEAR_F32)
def test_linear_f32(B, banks, K, N, act, bias_, res_, save):
    linear_case("f32", B, banks, K, N, act, bias_, res_, save)


def test_no_device_error_was_recorded():
    api.get_device_error()
