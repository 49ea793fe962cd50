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


# (33 tokens of 264: checkpoint rows that are no multiple of 16 bytes; one token, one head)
MIXED = [(1, 2, 16, 2), (4, 1, 16, 1), (2, 33, 264, 33), (9, 20, 480, 20), (2, 24, 768, 24), (5, 8, 64, 8), (3, 4, 96, 2), (2, 3, 64, 8), (7, 16, 256, 16), (3, 32, 512, 32), (2, 48, 768, 48),
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


# (enough samples that several share a slot of shared memory, the last slot not full; odd and single heads)
MANY = [(1185, 16, 512, 16), (1301, 16, 256, 16), (1789, 8, 128, 8), (2501, 13, 104, 13), (6001, 4, 32, 4),
        (1207, 2, 128, 2), (20011, 3, 48, 3), (40009, 1, 16, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,H", MANY)
@pytest.mark.parametrize("ckpt", [False, True])
def test_layer_norm_of_many_small_samples(dtype, B, T, D, H, ckpt):
    test_layer_norm_mixed(dtype, B, T, D, H, ckpt)


# ------------------------------------------------------------------ per-token linear layer
LINEAR = [(1, 1, 8, 8), (1, 3, 64, 128), (5, 2, 72, 40), (64, 2, 64, 64), (128, 1, 256, 256), (129, 2, 128, 264),
          (200, 3, 136, 328), (300, 2, 320, 96), (33, 1, 768, 1536), (1000, 1, 40, 72), (700, 2, 384, 520)]
# (enough rows, columns and banks for the tiles of two SMs, with edges in every direction: the forward, dX, dW
# whole and dW split, in turn)
LINEAR_LARGE = [(390, 30, 264, 200), (450, 24, 200, 392), (4000, 2, 264, 392)]
# (one sample: contractions of more than one trip, columns that end inside a block of 32)
LINEAR_ONE = [(1, 5, 1032, 40), (1, 2, 520, 264), (1, 40, 768, 136), (1, 1, 16, 8)]
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


@pytest.mark.parametrize("act,bias_,res_,save", [("none", True, True, "full"), ("none", False, False, "full"),
                                                 ("relu", True, False, "full"), ("gelu", True, True, "ckpt8"),
                                                 ("gelu", False, False, "full"), ("silu", True, True, "ckpt8"),
                                                 ("silu", False, True, "full"), ("relu", False, True, "ckpt8")])
@pytest.mark.parametrize("B,banks,K,N", LINEAR_ONE)
def test_linear_bf16_of_one_sample(B, banks, K, N, act, bias_, res_, save):
    linear_case("bf16", B, banks, K, N, act, bias_, res_, save)


@pytest.mark.parametrize("act,bias_,res_,save", [("none", True, True, "full"), ("relu", True, False, "ckpt8"),
                                                 ("gelu", True, True, "full"), ("silu", False, True, "ckpt8")])
@pytest.mark.parametrize("B,banks,K,N", LINEAR_LARGE)
def test_linear_bf16_on_pairs(B, banks, K, N, act, bias_, res_, save):
    linear_case("bf16", B, banks, K, N, act, bias_, res_, save)


@pytest.mark.parametrize("act,bias_,res_,save", [("none", True, True, "full"), ("relu", True, False, "full"),
                                                 ("gelu", True, True, "ckpt8"), ("silu", False, False, "full")])
@pytest.mark.parametrize("B,banks,K,N", LINEAR_F32)
def test_linear_f32(B, banks, K, N, act, bias_, res_, save):
    linear_case("f32", B, banks, K, N, act, bias_, res_, save)


# ------------------------------------------------------------------ calls that the cases above do not make
def guarded(shape_, dtype, device=DEV):
    """A tensor between two stretches of a byte pattern: (tensor, check that they are intact)."""
    n = int(np.prod(shape_)) * torch.empty(0, dtype=dtype).element_size()
    pad = 4096
    buf = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device=device)
    t = buf[pad:pad + n].view(dtype).view(shape_)
    return t, lambda: bool((buf[:pad] == 0x5A).all()) and bool((buf[pad + n:] == 0x5A).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_is_written_beside_the_outputs(dtype):
    rng = np.random.default_rng(3)
    B, banks, K, N, T = 131, 3, 72, 200, 24
    x, _ = draw(rng, (B, banks, K), dtype)
    w, _ = draw(rng, (banks, N, K), dtype)
    dy, _ = draw(rng, (B, banks, N), dtype)
    lin = api.Linear(w, None, "gelu")
    checks = []

    def out(shape_, dt=DT[dtype]):
        t, ok = guarded(shape_, dt)
        checks.append(ok)
        return t
    y, z, codes, exps = out((B, banks, N)), out((B, banks, N)), out((B, banks, N), torch.int8), out((B, banks, 7), torch.int8)
    sh, c = api.shape(B, banks, K, 1, DT[dtype]), lin.c(banks, K, DT[dtype], 0)
    for kept in ({"z": z}, {"save": A.tm_ckpt8(codes.data_ptr(), exps.data_ptr())}):
        assert api.lib().tm_pertoken_linear(x.data_ptr(), None, sh, c, y.data_ptr(), kept.get("z", z).data_ptr() if "z" in kept else None,
                                            kept.get("save"), None) == 0
    dx, dw = out((B, banks, K)), out((banks, N, K))
    n = api.lib().tm_pertoken_linear_backward_workspace_bytes(sh, c)
    ws = out((n,), torch.uint8)
    assert api.lib().tm_pertoken_linear_backward(x.data_ptr(), dy.data_ptr(), z.data_ptr(), None, None, sh, c, dx.data_ptr(),
                                                 A.tm_linear_grads(dw.data_ptr(), None), ws.data_ptr(), n, None) == 0
    # norms: rows, and samples of both sizes
    for layout, Bn, bk, W in ((A.TM_LAYOUT_ROWS, 131, 3, 72), (A.TM_LAYOUT_MIXED, 7, T, T * 8), (A.TM_LAYOUT_MIXED, 7, 6, 96)):
        xs, _ = draw(rng, (Bn, bk, W), dtype)
        ds, _ = draw(rng, (Bn, bk, W), dtype)
        mixed = layout == A.TM_LAYOUT_MIXED
        shn = api.shape(Bn, bk, W, bk if mixed else 1, DT[dtype], EPS)
        wn = A.tm_layer_norm_w(bk, W, None, None)
        yn, mean, rstd = out((Bn, bk, W)), out((Bn * bk,), torch.float32), out((Bn * bk,), torch.float32)
        ck = A.tm_ckpt8(out((Bn, bk, W), torch.int8).data_ptr(), out((Bn, bk, (W + 31) // 32), torch.int8).data_ptr())
        assert api.lib().tm_layer_norm(xs.data_ptr(), xs.data_ptr(), layout, shn, wn, yn.data_ptr(), mean.data_ptr(),
                                       rstd.data_ptr(), ck, None) == 0
        n = api.lib().tm_layer_norm_backward_workspace_bytes(shn, layout, wn)
        dxn, dg, db, ws = out((Bn, bk, W)), out((W,)), out((W,)), out((n,), torch.uint8)
        for saved in (None, ck):
            assert api.lib().tm_layer_norm_backward(xs.data_ptr(), xs.data_ptr(), saved, mean.data_ptr(), rstd.data_ptr(),
                                                    ds.data_ptr(), layout, shn, wn, 1 if mixed else 0, dxn.data_ptr(), None,
                                                    A.tm_layer_norm_grads(dg.data_ptr(), db.data_ptr()), ws.data_ptr(), n,
                                                    None) == 0
        for width in (W, 45):
            xp = xs.reshape(-1)[:Bn * bk * 45].reshape(-1, 45) if width == 45 else xs
            cp = A.tm_ckpt8(out(xp.shape, torch.int8).data_ptr(), out((xp.numel() // width, (width + 31) // 32), torch.int8).data_ptr())
            back = out(xp.shape)
            assert api.lib().tm_checkpoint8_pack(xp.data_ptr(), A.TM_BF16 if dtype == "bf16" else A.TM_F32, xp.numel() // width,
                                                 width, cp, None) == 0
            assert api.lib().tm_checkpoint8_unpack(cp, A.TM_BF16 if dtype == "bf16" else A.TM_F32, xp.numel() // width, width,
                                                   back.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert all(ok() for ok in checks)


def chain(x, lin1, lin2, g, dy, sh, kept):
    """Every operator once, as a post-norm block's training step runs them."""
    s, n1 = api.layer_norm(x, x, A.TM_LAYOUT_MIXED, sh, g[0], g[1], checkpoint8=kept == "ckpt8")
    h, z = api.pertoken_linear(s, lin1, save=kept)
    o = api.pertoken_linear(h, lin2, residual=s)
    y, n2 = api.layer_norm(o, None, A.TM_LAYOUT_ROWS, sh, g[2], g[3], checkpoint8=kept == "ckpt8")
    do, _, g2 = api.layer_norm_backward(dy, n2, A.TM_LAYOUT_ROWS, sh, g[2], x=o)
    dh, w2 = api.pertoken_linear_backward(h, do, lin2)
    ds, w1 = api.pertoken_linear_backward(s, dh, lin1, z, dx_add=do)
    dx, _, g1 = api.layer_norm_backward(ds, n1, A.TM_LAYOUT_MIXED, sh, g[0], x=x, residual=x, residual_is_x=True)
    return {"s": s, "h": h, "o": o, "y": y, "do": do, "dh": dh, "ds": ds, "dx": dx, "dw1": w1["dw"], "db1": w1["db"],
            "dw2": w2["dw"], "db2": w2["db"], "dg1": g1["dgain"], "dg2": g2["dgain"]}


def chain_inputs(B, T, D, F, seed=1):
    rng = np.random.default_rng(seed)
    x, xo = draw(rng, (B, T, D), "bf16")
    w1, w1o = draw(rng, (T, F, D), "bf16", std=D ** -0.5)
    w2, w2o = draw(rng, (T, D, F), "bf16", std=F ** -0.5)
    b1, b1o = draw(rng, (T, F), "bf16", std=0.1)
    b2, b2o = draw(rng, (T, D), "bf16", std=0.1)
    g = [draw(rng, (D,), "bf16", std=0.1, mean=m) for m in (1.0, 0.0, 1.0, 0.0)]
    dy, dyo = draw(rng, (B, T, D), "bf16")
    dev = (x, api.Linear(w1, b1, "gelu"), api.Linear(w2, b2), [v[0] for v in g], dy, api.shape(B, T, D, T, "bf16", EPS))
    return dev, (xo, w1o, b1o, w2o, b2o, [v[1] for v in g], dyo)


def bf16(a):
    return torch.from_numpy(a).to(torch.bfloat16).double().numpy()


def oracle_chain(xo, w1, b1, w2, b2, g, dy, kept, store):
    """The block in float64; `store` rounds what the library stores, and the kept tensors go through 8 bits."""
    T = xo.shape[1]
    z1 = P.mix_rows(xo, T) + xo
    f1 = P.layer_norm(z1, g[0], g[1], EPS)
    s = store(f1["y"])
    h, zp = P.linear(s, w1, b1, "gelu")
    h = store(h)
    o = store(P.linear(h, w2, b2, "none", s)[0])
    f2 = P.layer_norm(o, g[2], g[3], EPS)
    q = (lambda v: P.checkpoint8(v)[2]) if kept == "ckpt8" and store is bf16 else (lambda v: store(v))
    n2 = P.layer_norm_backward(q(o), dy, g[2], f2["mean"], f2["rstd"])
    do = store(n2["dz"])
    l2 = P.linear_backward(h, do, o, w2, "none")
    dh = store(l2["dx"])
    zk = q(zp)
    l1 = P.linear_backward(s, dh, zk, w1, "gelu")
    dz = store(l1["dz"])
    ds = store(np.einsum("bgn,gnk->bgk", dz, w1) + do)
    dw1 = np.einsum("bgn,bgk->gnk", dz, s)
    n1 = P.layer_norm_backward(q(z1) if kept == "ckpt8" else z1, ds, g[0], f1["mean"], f1["rstd"])
    dx = n1["dz"] + P.revert_rows(n1["dz"], T)
    return {"s": s, "h": h, "o": o, "y": f2["y"], "do": do, "dh": dh, "ds": ds, "dx": dx, "dw1": dw1, "db1": l1["db"],
            "dw2": l2["dw"], "db2": l2["db"], "dg1": n1["dgain"], "dg2": n2["dgain"]}


@pytest.mark.parametrize("kept", ["full", "ckpt8"])
def test_post_norm_block_training_step(kept):
    """S = LN(Mix(X) + X); Y = LN(gelu(S W1^T + b1) W2^T + b2 + S) and its whole backward pass, operator by
    operator.  Against the exact block in float64 the library's outputs may be as far off (in rms) as a
    float64 model that rounds what the library stores (and quantises what it keeps in 8 bits), plus half of
    that again: roundings of the same size at the same places fall differently, their rms does not."""
    dev, host = chain_inputs(70, 16, 256, 384)
    got = chain(*dev, kept)
    exact = oracle_chain(*host, kept, lambda v: v)
    model = oracle_chain(*host, kept, bf16)
    for k, o in exact.items():
        rms = np.sqrt(np.mean(o * o))
        off = np.sqrt(np.mean((f64(got[k]) - o) ** 2)) / rms
        by_model = np.sqrt(np.mean((bf16(model[k]) - o) ** 2)) / rms
        assert off <= 1.5 * by_model, (k, off, by_model)


def test_same_bits_twice_in_a_graph_and_on_two_streams():
    dev, _ = chain_inputs(150, 16, 256, 264)
    x = dev[0]
    first = {k: v.clone() for k, v in chain(*dev, "ckpt8").items()}
    again = chain(*dev, "ckpt8")
    assert all(torch.equal(first[k], again[k]) for k in first)
    # captured: the replay works on what the inputs hold then
    keep = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(*dev, "ckpt8")
    x.copy_(keep.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    flipped = {k: v.clone() for k, v in out.items()}
    ref = chain(*dev, "ckpt8")
    assert all(torch.equal(flipped[k], ref[k]) for k in ref)
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], first[k]) for k in first)
    # two streams at once, each with workspaces of its own
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([chain(*dev, "ckpt8") for _ in range(3)][-1])
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], first[k]) for o in outs for k in first)
    # the stream argument, while another stream is the current one
    y, saved = api.layer_norm(x, x, A.TM_LAYOUT_MIXED, dev[5], *dev[3][:2], checkpoint8=True, stream=streams[0])
    h, z = api.pertoken_linear(y, dev[1], save="full", stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, first["s"]) and torch.equal(h, first["h"])


def test_a_bad_value_stays_in_its_sample():
    """NaN and infinity in one sample reach that sample's outputs and the sums over samples, nothing else; a
    checkpoint does not hide them from the backward pass."""
    rng = np.random.default_rng(8)
    B, banks, K, N = 140, 2, 64, 136
    x, _ = draw(rng, (B, banks, K), "bf16")
    w, _ = draw(rng, (banks, N, K), "bf16")
    dy, _ = draw(rng, (B, banks, N), "bf16")
    sh = api.shape(B, banks, K, 1, "bf16", EPS)
    clean = api.pertoken_linear(x, api.Linear(w, None, "silu"))
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[77, 1, 5] = bad
        lin = api.Linear(w, None, "silu")
        y, ck = api.pertoken_linear(xb, lin, save="ckpt8")
        rows = ~torch.isfinite(y).all(-1)
        assert rows.nonzero().tolist() == [[77, 1]] and torch.equal(y[~rows], clean[~rows])
        back = api.checkpoint8_unpack(ck)
        assert (~torch.isfinite(back).all(-1)).nonzero().tolist() == [[77, 1]]
        dx, g = api.pertoken_linear_backward(xb, dy, lin, ck)
        assert (~torch.isfinite(dx).all(-1)).nonzero().tolist() == [[77, 1]]
        assert torch.isfinite(g["dw"][0]).all() and not torch.isfinite(g["dw"][1]).any()
        yn, saved = api.layer_norm(xb, None, A.TM_LAYOUT_ROWS, sh, checkpoint8=True)
        assert (~torch.isfinite(yn).all(-1)).nonzero().tolist() == [[77, 1]]
        dn, _, _ = api.layer_norm_backward(yn.nan_to_num(), saved, A.TM_LAYOUT_ROWS, sh)
        assert (~torch.isfinite(dn).all(-1)).nonzero().tolist() == [[77, 1]]


def test_gain_and_bias_may_be_absent_and_gradients_not_wanted():
    rng = np.random.default_rng(9)
    x, xo = draw(rng, (9, 2, 96), "bf16")
    dy, do = draw(rng, (9, 2, 96), "bf16")
    sh, w = api.shape(9, 2, 96, 1, "bf16", EPS), A.tm_layer_norm_w(2, 96, None, None)
    f = P.layer_norm(xo, None, None, EPS)
    y, saved = api.layer_norm(x, None, A.TM_LAYOUT_ROWS, sh)
    check("y", y, f["y"], norm_tols(xo, f, None, None, "bf16")[3])
    dx, _, grads = api.layer_norm_backward(dy, saved, A.TM_LAYOUT_ROWS, sh, x=x)
    dx2, y2 = torch.empty_like(x), torch.empty_like(x)
    assert api.lib().tm_layer_norm_backward(x.data_ptr(), None, None, saved.mean.data_ptr(), saved.rstd.data_ptr(), dy.data_ptr(),
                                            A.TM_LAYOUT_ROWS, sh, w, 0, dx2.data_ptr(), None, None, None, 0, None) == 0
    assert api.lib().tm_layer_norm(x.data_ptr(), None, A.TM_LAYOUT_ROWS, sh, w, y2.data_ptr(), None, None, None, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(y, y2)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows come out as they do alone."""
    B, banks, W, N = 290000, 48, 160, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(B, banks, W, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    assert x.numel() > 2 ** 31
    sh, tail_sh = api.shape(B, banks, W, 1, "bf16", EPS), api.shape(3, banks, W, 1, "bf16", EPS)
    tail = x[-3:].clone()
    ck = api.checkpoint8_pack(x)
    assert torch.equal(ck.codes[-3:], api.checkpoint8_pack(tail).codes)
    assert torch.equal(api.checkpoint8_unpack(ck)[-3:], api.checkpoint8_unpack(api.checkpoint8_pack(tail)))
    del ck
    y, saved = api.layer_norm(x, None, A.TM_LAYOUT_ROWS, sh)
    yt, st = api.layer_norm(tail, None, A.TM_LAYOUT_ROWS, tail_sh)
    assert torch.equal(y[-3:], yt) and torch.equal(saved.mean[-3:], st.mean)
    dx, _, _ = api.layer_norm_backward(x, saved, A.TM_LAYOUT_ROWS, sh, x=x, dx=y)
    dt, _, _ = api.layer_norm_backward(tail, st, A.TM_LAYOUT_ROWS, tail_sh, x=tail)
    assert torch.equal(dx[-3:], dt)
    del y, dx
    lin = api.Linear(torch.empty(banks, N, W, dtype=torch.bfloat16, device=DEV).normal_(generator=g).mul_(0.1), None, "relu")
    out, z = api.pertoken_linear(x, lin, save="full")
    ot = api.pertoken_linear(tail, lin)
    assert torch.equal(out[-3:], ot)
    dxl, _ = api.pertoken_linear_backward(x, out, lin, z)
    dlt, _ = api.pertoken_linear_backward(tail, ot, lin, z[-3:])
    assert torch.equal(dxl[-3:], dlt)


def test_no_device_error_was_recorded():
    api.get_device_error()
