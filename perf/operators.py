"""Operators of the post-norm per-token block, their plain forms and the cases they are timed on.

The operators:
  * layer normalisation of the rows of a token tensor, y = LN(x + residual), the rows read as they
    are ([B, banks, width]) or through the Mix permutation of a token tensor [B, T, D] (the token
    mixing step S = LN(Mix(X) + X) of the post-norm block), with its backward pass;
  * the per-token linear layer y[b, n] = act(x[b, n] W[n]^T + bias[n]) + residual[b, n] (one weight
    matrix per bank), with its backward pass;
  * activation checkpoints in 8 bits (int8 codes, one power-of-two scale per 32 values of a row):
    packing and unpacking, and the backward passes of the other two reading them.

A case's "op" names what one pass runs:
  ln            the forward pass                          -> y, mean, rstd
  ln_train      forward, then backward for a given dy     -> y, dx, dresidual, dgain, dbias
  linear        the forward pass                          -> y
  linear_train  forward, then backward for a given dy     -> y, dx, dw, db
  ckpt8         packing, then unpacking                   -> the unpacked rows
In the two training operators "save" says what the backward pass works from: "full" (the operator's
inputs, or the pre-activation in the storage type) or "ckpt8" (the 8-bit checkpoint).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the small fp32 stack (B=64, T=8, D=64): a row pass where only the latency counts
        {"name": "ln_rows_small_f32", "op": "ln", "layout": "rows", "B": 64, "banks": 8, "width": 64,
         "residual": True, "dtype": "f32"},
        # token mixing of the MoE stack's token tensor (T=32, D=512, 16-column head pieces)
        {"name": "ln_mixed_bf16", "op": "ln", "layout": "mixed", "B": 8192, "banks": 32, "width": 512,
         "residual": True, "dtype": "bf16"},
        # training step of the same on the largest token tensor (T=48, D=768)
        {"name": "ln_train_mixed_bf16", "op": "ln_train", "layout": "mixed", "B": 4096, "banks": 48, "width": 768,
         "residual": True, "save": "full", "dtype": "bf16"},
        # the norm after the per-token FFN (rows of the non-square stack), an odd batch, from the checkpoint
        {"name": "ln_train_rows_ckpt8", "op": "ln_train", "layout": "rows", "B": 4097, "banks": 16, "width": 384,
         "residual": True, "save": "ckpt8", "dtype": "bf16"},
        # scoring one sample with the large stack's widths: the weights are the work
        {"name": "linear_one_sample", "op": "linear", "B": 1, "banks": 48, "width": 768, "out": 1536, "act": "silu",
         "bias": True, "residual": False, "dtype": "bf16"},
        # up projection of the dense block's FFN
        {"name": "linear_up_gelu", "op": "linear", "B": 4096, "banks": 16, "width": 256, "out": 1024, "act": "gelu",
         "bias": True, "residual": False, "dtype": "bf16"},
        # its down projection with the residual
        {"name": "linear_down_residual", "op": "linear", "B": 4096, "banks": 16, "width": 1024, "out": 256,
         "act": "none", "bias": True, "residual": True, "dtype": "bf16"},
        # the largest: the large stack's banks and widths at half its batch
        {"name": "linear_large_gelu", "op": "linear", "B": 8192, "banks": 48, "width": 768, "out": 1536,
         "act": "gelu", "bias": True, "residual": False, "dtype": "bf16"},
        # training step of the non-square stack's mixing banks, the pre-activation kept in 8 bits
        {"name": "linear_train_ckpt8", "op": "linear_train", "B": 4096, "banks": 8, "width": 768, "out": 1536,
         "act": "gelu", "bias": True, "save": "ckpt8", "dtype": "bf16"},
        # a small ragged training batch: sizes that fill no tile
        {"name": "linear_train_ragged", "op": "linear_train", "B": 333, "banks": 16, "width": 384, "out": 264,
         "act": "relu", "bias": True, "save": "full", "dtype": "bf16"},
        # the inputs of one block of the MoE stack, as a training step keeps them
        {"name": "ckpt8_block_input", "op": "ckpt8", "rows": 8192 * 32, "width": 512, "dtype": "bf16"},
        # rows that end inside a block of 32, fp32
        {"name": "ckpt8_odd_f32", "op": "ckpt8", "rows": 4099, "width": 100, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln_train", "linear", "linear_train", "ckpt8"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "ckpt8":
        width = _log(rng, 8, 4096)
        return {"op": op, "rows": max(1, min(_log(rng, 1, 300000), 2 ** 27 // width)), "width": width, "dtype": dtype}
    if op in ("ln", "ln_train"):
        c = {"op": op, "layout": rng.choice(["rows", "mixed"]), "dtype": dtype}
        if c["layout"] == "mixed":
            banks = rng.randint(2, 48)                       # T = H = banks, head width 8, 16, 24 or 32
            c.update(banks=banks, width=banks * rng.choice([h for h in (8, 16, 24, 32) if banks * h <= 768]))
        else:
            c.update(banks=rng.randint(1, 48), width=8 * _log(rng, 1, 256))
        row = c["banks"] * c["width"]
        c.update(B=max(1, min(_log(rng, 1, 8192), 2 ** 27 // row)), residual=c["layout"] == "mixed" or rng.random() < 0.7)
        if op == "ln_train":
            c["save"] = rng.choice(["full", "ckpt8"])
        return c
    if dtype == "f32":                                       # the small fp32 stack's range
        B, banks, width, out = _log(rng, 1, 256), rng.randint(1, 16), _log(rng, 16, 256), _log(rng, 16, 256)
    else:
        banks, width, out = rng.randint(1, 48), 8 * _log(rng, 8, 128), 8 * _log(rng, 8, 256)
        B = max(1, min(_log(rng, 1, 8192), 2 ** 37 // (banks * width * out)))
    c = {"op": op, "B": B, "banks": banks, "width": width, "out": out,
         "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.8, "dtype": dtype}
    if op == "linear":
        c["residual"] = rng.random() < 0.4
    elif dtype == "f32":
        # a pre-activation next to a border (zero for relu, half a code for the checkpoint) falls to either
        # side with the order of its fp32 sum, and moves an fp32 gradient by more than its own precision
        c.update(save="full", act=rng.choice(["none", "gelu", "silu"]))
    else:
        c["save"] = rng.choice(["full", "ckpt8"])
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPE[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dt)

    s = {"case": case}
    if case["op"] == "ckpt8":
        s["x"] = normal(case["rows"], case["width"])
        return s
    B, banks, width = case["B"], case["banks"], case["width"]
    s["x"] = normal(B, banks, width)                         # mixed: T = banks tokens of D = width
    if case["op"] in ("ln", "ln_train"):
        if case["residual"]:
            s["residual"] = s["x"] if case["layout"] == "mixed" else normal(B, banks, width, mean=0.2)
        s["gain"] = normal(width, std=0.1, mean=1.0)
        s["bias"] = normal(width, std=0.1)
        if case["op"] == "ln_train":
            s["dy"] = normal(B, banks, width)
        return s
    out = case["out"]
    s["w"] = normal(banks, out, width, std=width ** -0.5)
    if case["bias"]:
        s["bias"] = normal(banks, out, std=0.1)
    if case.get("residual"):
        s["residual"] = normal(B, banks, out)
    if case["op"] == "linear_train":
        s["dy"] = normal(B, banks, out)
    return s


def run(state):
    op = state["case"]["op"]
    if op == "ckpt8":
        return _run_ckpt8(state)
    if op in ("ln", "ln_train"):
        return _run_ln(state)
    return _run_linear(state)


# ------------------------------------------------------------------ the framework's calls
def _own_ln(s):
    from token_sparse_moe_b200 import _abi as A, api
    c = s["case"]
    B, banks, width = s["x"].shape
    mixed = c["layout"] == "mixed"
    layout = A.TM_LAYOUT_MIXED if mixed else A.TM_LAYOUT_ROWS
    sh = api.shape(B, banks, width, banks if mixed else 1, s["x"].dtype, EPS)
    res = s.get("residual")
    y, saved = api.layer_norm(s["x"], res, layout, sh, s["gain"], s["bias"], checkpoint8=c.get("save") == "ckpt8")
    if c["op"] == "ln":
        return {"y": y, "mean": saved.mean, "rstd": saved.rstd}
    dx, dres, grads = api.layer_norm_backward(s["dy"], saved, layout, sh, s["gain"], x=s["x"], residual=res,
                                              residual_is_x=mixed)
    return {"y": y, "dx": dx, "dresidual": dres, "dgain": grads["dgain"], "dbias": grads["dbias"]}


def _own_linear(s):
    from token_sparse_moe_b200 import api
    c = s["case"]
    lin = api.Linear(s["w"], s.get("bias"), c["act"])
    if c["op"] == "linear":
        return api.pertoken_linear(s["x"], lin, residual=s.get("residual"))
    y, saved = api.pertoken_linear(s["x"], lin, save="ckpt8" if c["save"] == "ckpt8" else "full")
    dx, grads = api.pertoken_linear_backward(s["x"], s["dy"], lin, saved)
    return {"y": y, "dx": dx, "dw": grads["dw"], "db": grads.get("db")}


def _own_ckpt8(s):
    from token_sparse_moe_b200 import api
    return api.checkpoint8_unpack(api.checkpoint8_pack(s["x"]))


# ------------------------------------------------------------------ plain forms, 32 bits
def _mix(x, heads):
    B, T, D = x.shape
    return x.reshape(B, T, heads, D // heads).transpose(1, 2).reshape(B, heads, T * D // heads)


def _through_8_bits(z):
    """The values that the 8-bit checkpoint of z's rows stands for: 32 values of a row share the scale
    2^e, e the smallest integer for which no code passes 127 (and at least -126)."""
    width = z.shape[-1]
    blocks = torch.nn.functional.pad(z, (0, -width % 32)).unflatten(-1, (-1, 32))
    m, x = torch.frexp(blocks.abs().amax(-1, keepdim=True))
    e = (x - 7 + (m > 127 / 128)).clamp(min=-126)
    codes = torch.round(torch.ldexp(blocks, -e))
    return torch.ldexp(codes, e).flatten(-2)[..., :width]


def _run_ckpt8(s):
    if own:
        return _own_ckpt8(s)
    return _through_8_bits(s["x"].float()).to(s["x"].dtype)


def _run_ln(s):
    if own:
        return _own_ln(s)
    c, dt = s["case"], s["x"].dtype
    mixed = c["layout"] == "mixed"
    x = s["x"].float()
    z = _mix(x, x.shape[1]) if mixed else x
    if c["residual"]:
        z = z + s["residual"].float()
    gain = s["gain"].float()
    mean = z.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((z - mean).square().mean(-1, keepdim=True) + EPS)
    y = ((z - mean) * rstd * gain + s["bias"].float()).to(dt)
    if c["op"] == "ln":
        return {"y": y, "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}
    n = ((_through_8_bits(z) if c["save"] == "ckpt8" else z) - mean) * rstd
    dy = s["dy"].float()
    dn = dy * gain
    dz = rstd * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    dgain, dbias = (dy * n).sum((0, 1)), dy.sum((0, 1))
    if mixed:                                                # x is the residual too: both gradients in one
        dx, dres = dz + _mix(dz, dz.shape[1]), None          # (with T = H, Mix is its own inverse)
    else:
        dx, dres = dz, dz if c["residual"] else None
    return {"y": y, "dx": dx.to(dt), "dresidual": dres if dres is None else dres.to(dt), "dgain": dgain.to(dt),
            "dbias": dbias.to(dt)}


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _run_linear(s):
    if own:
        return _own_linear(s)
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float().transpose(0, 1), s["w"].float()    # bank first
    z = torch.matmul(x, w.transpose(1, 2)).transpose(0, 1)
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["op"] == "linear":
        return (y + s["residual"].float() if c["residual"] else y).to(dt)
    kept = _through_8_bits(z) if c["save"] == "ckpt8" else z
    dz = s["dy"].float() * _act_grad(kept, c["act"])
    db = dz.sum(0).to(dt) if c["bias"] else None
    dz = dz.transpose(0, 1)
    dx = torch.matmul(dz, w).transpose(0, 1)
    dw = torch.matmul(dz.transpose(1, 2), x)
    return {"y": y.to(dt), "dx": dx.to(dt), "dw": dw.to(dt), "db": db}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ckpt8":                                # the codes and scales are written and read once
        n, blocks = case["rows"] * case["width"], case["rows"] * -(-case["width"] // 32)
        return {"bytes": 2 * n * e + 2 * (n + blocks), "flops": 4 * n}
    rows, width = case["B"] * case["banks"], case["width"]
    n = rows * width
    if case["op"] in ("ln", "ln_train"):
        ins = 2 if case["residual"] and case["layout"] == "rows" else 1
        fwd = (ins + 1) * n * e + 2 * width * e + 8 * rows
        if case["op"] == "ln":
            return {"bytes": fwd, "flops": 9 * n}
        again = 2 * (n + n // 32) if case["save"] == "ckpt8" else ins * n * e
        # rows: the residual's gradient is dx itself, so it costs no second write
        return {"bytes": fwd + again + 2 * n * e + 3 * width * e + 8 * rows, "flops": 22 * n}
    out, banks = case["out"], case["banks"]
    m, wts = rows * out, banks * out * width
    bias = banks * out if case["bias"] else 0
    if case["op"] == "linear":
        return {"bytes": (n + wts + bias + m * (2 if case["residual"] else 1)) * e, "flops": 2 * m * width}
    kept = 0 if case["act"] == "none" else 2 * (m + m // 32 if case["save"] == "ckpt8" else m * e)
    return {"bytes": (n + wts + bias + m) * e + kept + (m + n + wts + n + wts + bias) * e, "flops": 6 * m * width}


# ------------------------------------------------------------------ the definitions, 64 bits
def _exact_8_bits(z):
    out = torch.zeros(z.shape[:-1] + (-(-z.shape[-1] // 32) * 32,), dtype=torch.float64, device=z.device)
    out[..., :z.shape[-1]] = z
    b = out.view(*out.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 127.0))
    e = torch.where(top > 127.0 * torch.exp2(e), e + 1, torch.where(top <= 127.0 * torch.exp2(e - 1), e - 1, e))
    scale = torch.exp2(torch.where(top > 0, e, -126.0).clamp(min=-126.0))
    return ((b / scale).round() * scale).reshape(out.shape)[..., :z.shape[-1]]


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if k != "case"}
    if case["op"] == "ckpt8":
        return _exact_8_bits(d["x"])
    if case["op"] in ("ln", "ln_train"):
        x, mixed = d["x"], case["layout"] == "mixed"
        B, banks, width = x.shape
        at = None
        if mixed:                                            # Mix as a gather: row h, column t*dh+j <- token t, column h*dh+j
            dh = width // banks
            h, c = np.meshgrid(np.arange(banks), np.arange(width), indexing="ij")
            at = torch.from_numpy(((c // dh) * width + h * dh + c % dh).reshape(-1)).to(x.device)
            z = x.reshape(B, -1)[:, at].reshape(B, banks, width)
        else:
            z = x
        z = z + d["residual"] if case["residual"] else z
        mu = z.sum(-1) / width
        r = (((z - mu[..., None]) ** 2).sum(-1) / width + EPS) ** -0.5
        y = d["gain"] * ((z - mu[..., None]) * r[..., None]) + d["bias"]
        if case["op"] == "ln":
            return {"y": y, "mean": mu, "rstd": r}
        if case["save"] == "ckpt8":
            z = _exact_8_bits(z)
        n = (z - mu[..., None]) * r[..., None]
        gy = d["dy"] * d["gain"]
        dz = (gy - (gy.sum(-1) / width)[..., None] - n * ((gy * n).sum(-1) / width)[..., None]) * r[..., None]
        grads = {"dgain": torch.einsum("bnw,bnw->w", d["dy"], n), "dbias": torch.einsum("bnw->w", d["dy"])}
        if mixed:
            dx = dz.reshape(B, -1).clone()
            dx.index_add_(1, at, dz.reshape(B, -1))          # the adjoint of the gather, and the residual's part
            return {"y": y, "dx": dx.reshape(B, banks, width), "dresidual": None, **grads}
        return {"y": y, "dx": dz, "dresidual": dz if case["residual"] else None, **grads}
    z = torch.einsum("bnk,nok->bno", d["x"], d["w"])
    z = z + d["bias"] if case["bias"] else z
    act, root2 = case["act"], math.sqrt(2.0)
    cdf = 0.5 * torch.special.erfc(-z / root2) if act == "gelu" else torch.sigmoid(z) if act == "silu" else (z > 0).double()
    y = z if act == "none" else z * cdf
    if case["op"] == "linear":
        return y + d["residual"] if case["residual"] else y
    if case["save"] == "ckpt8":
        z = _exact_8_bits(z)
    if act == "gelu":
        slope = 0.5 * torch.special.erfc(-z / root2) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif act == "silu":
        slope = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    else:
        slope = (z > 0).double() if act == "relu" else torch.ones_like(z)
    dz = d["dy"] * slope
    return {"y": y, "dx": torch.einsum("bno,nok->bnk", dz, d["w"]), "dw": torch.einsum("bno,bnk->nok", dz, d["x"]),
            "db": dz.sum(0) if case["bias"] else None}
