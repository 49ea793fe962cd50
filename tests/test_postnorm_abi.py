"""The post-norm block's calls on the CPU: struct layouts, workspace queries and every refusal of the host
checks, all before any launch."""
import ctypes
import os
import subprocess

import pytest
import torch

from token_sparse_moe_b200 import _abi as A
from token_sparse_moe_b200 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = A.load()
MB = 1 << 20


def P(i):
    """A made-up device address, 64 MB apart."""
    return (i + 1) * 64 * MB


def test_struct_layouts(tmp_path):
    src = tmp_path / "l.c"
    src.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "tm.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu\n", sizeof(tm_ckpt8), sizeof(tm_layer_norm_w), sizeof(tm_layer_norm_grads),
         sizeof(tm_linear_w), sizeof(tm_linear_grads));
  printf("%zu %zu %zu %zu %zu\n", offsetof(tm_ckpt8, exps), offsetof(tm_layer_norm_w, bias), offsetof(tm_linear_w, act),
         offsetof(tm_linear_w, bias), offsetof(tm_linear_grads, db));
  printf("%d %d %d %d\n", TM_ACT_NONE, TM_ACT_RELU, TM_ACT_GELU, TM_ACT_SILU);
  return 0;
}
''')
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    s = ctypes.sizeof
    assert got == [s(A.tm_ckpt8), s(A.tm_layer_norm_w), s(A.tm_layer_norm_grads), s(A.tm_linear_w), s(A.tm_linear_grads),
                   A.tm_ckpt8.exps.offset, A.tm_layer_norm_w.bias.offset, A.tm_linear_w.act.offset,
                   A.tm_linear_w.bias.offset, A.tm_linear_grads.db.offset,
                   A.TM_ACT_NONE, A.TM_ACT_RELU, A.TM_ACT_GELU, A.TM_ACT_SILU]


INV, UNS, WS = A.TM_ERR_INVALID_ARG, A.TM_ERR_UNSUPPORTED, A.TM_ERR_WORKSPACE


def test_checkpoint_refusals():
    ck = A.tm_ckpt8(P(1), P(2))
    call = lambda x=P(0), dt=A.TM_BF16, rows=8, width=64, c=ck: (
        L.tm_checkpoint8_pack(x, dt, rows, width, c, None), L.tm_checkpoint8_unpack(c, dt, rows, width, x, None))
    for kw, want in [(dict(x=None), INV), (dict(dt=7), INV), (dict(rows=0), INV), (dict(width=0), INV),
                     (dict(width=-3), INV), (dict(c=A.tm_ckpt8(None, P(2))), INV), (dict(c=A.tm_ckpt8(P(1), None)), INV),
                     (dict(c=None), INV), (dict(x=P(0) + 8), INV), (dict(c=A.tm_ckpt8(P(1) + 4, P(2))), INV),
                     (dict(c=A.tm_ckpt8(P(0), P(2))), INV),                       # codes over x
                     (dict(c=A.tm_ckpt8(P(0) + 1008, P(2))), INV),                # codes over x's last bytes
                     (dict(rows=1 << 41), UNS)]:
        assert call(**kw) == (want, want), kw
    # exponents inside the codes: both written by the packing
    assert L.tm_checkpoint8_pack(P(0), A.TM_BF16, 8, 64, A.tm_ckpt8(P(1), P(1) + 256), None) == INV


def ln(x=P(0), res=P(1), layout=A.TM_LAYOUT_ROWS, sh=None, w=None, y=P(4), mean=P(5), rstd=P(6), save=None):
    sh = sh or api.shape(4, 8, 64, 8, "bf16")
    w = w or A.tm_layer_norm_w(8, 64, P(2), P(3))
    return L.tm_layer_norm(x, res, layout, sh, w, y, mean, rstd, save, None)


def test_layer_norm_refusals():
    bad_w = lambda **k: A.tm_layer_norm_w(k.get("banks", 8), k.get("width", 64), k.get("gain", P(2)), k.get("bias", P(3)))
    for kw, want in [(dict(x=None), INV), (dict(y=None), INV), (dict(x=P(0) + 2), INV), (dict(y=P(0)), INV),
                     (dict(y=P(1)), INV), (dict(y=P(0) + 4080), INV), (dict(mean=P(5) + 2), INV), (dict(mean=P(4)), INV),
                     (dict(rstd=P(5)), INV), (dict(layout=5), INV), (dict(w=bad_w(banks=0)), INV),
                     (dict(w=bad_w(width=0)), INV), (dict(w=bad_w(gain=P(2) + 8)), INV), (dict(y=P(2)), INV),
                     (dict(w=bad_w(width=16385)), UNS), (dict(sh=api.shape(0, 8, 64, 8, "bf16")), INV),
                     (dict(sh=api.shape(1 << 26, 8, 64, 8, "bf16")), UNS),            # 2^29 rows
                     (dict(save=A.tm_ckpt8(P(7), None)), INV), (dict(save=A.tm_ckpt8(P(4), P(7))), INV),
                     (dict(layout=A.TM_LAYOUT_MIXED, w=bad_w(banks=4)), INV),
                     (dict(layout=A.TM_LAYOUT_MIXED, w=bad_w(width=32)), INV),
                     # head width 4: no 16-byte vectors
                     (dict(layout=A.TM_LAYOUT_MIXED, sh=api.shape(4, 8, 32, 8, "bf16"), w=bad_w(width=32)), UNS)]:
        assert ln(**kw) == want, kw


def ln_bwd(x=P(0), res=P(1), saved=None, mean=P(5), rstd=P(6), dy=P(7), layout=A.TM_LAYOUT_ROWS, sh=None, w=None, self_=0,
           dx=P(8), dres=None, grads=None, ws=P(11), wsb=1 << 30):
    sh = sh or api.shape(4, 8, 64, 8, "bf16")
    w = w or A.tm_layer_norm_w(8, 64, P(2), None)
    grads = grads or A.tm_layer_norm_grads(P(9), P(10))
    return L.tm_layer_norm_backward(x, res, saved, mean, rstd, dy, layout, sh, w, self_, dx, dres, grads, ws, wsb, None)


def test_layer_norm_backward_refusals():
    M = A.TM_LAYOUT_MIXED
    n = L.tm_layer_norm_backward_workspace_bytes(api.shape(4, 8, 64, 8, "bf16"), A.TM_LAYOUT_ROWS,
                                                 A.tm_layer_norm_w(8, 64, None, None))
    assert n == 32 * 2 * 64 * 4                                                   # at most one partial sum a row
    assert L.tm_layer_norm_backward_workspace_bytes(api.shape(4, 8, 64, 8, "bf16"), A.TM_LAYOUT_ROWS,
                                                    A.tm_layer_norm_w(8, 1 << 15, None, None)) == 0
    big = api.shape(4, 64, 1024, 64, "bf16")                                      # 64 * 1024 * 4 bytes a sample
    for kw, want in [(dict(x=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV), (dict(dy=None), INV),
                     (dict(dx=None), INV), (dict(dx=P(7)), INV), (dict(dx=P(0)), INV), (dict(wsb=n - 1), WS),
                     (dict(ws=None), WS), (dict(ws=P(11) + 8), INV), (dict(ws=P(8)), INV), (dict(dres=P(12)), INV),
                     (dict(self_=1), INV), (dict(layout=M, self_=1), INV),             # the residual is not x
                     (dict(layout=M, self_=1, res=P(0), dres=P(12)), INV),
                     (dict(layout=M, self_=1, res=P(0), sh=api.shape(4, 8, 64, 4, "bf16"),
                           w=A.tm_layer_norm_w(4, 128, None, None)), INV),             # T != H
                     (dict(layout=M, self_=1, res=P(0), sh=big, w=A.tm_layer_norm_w(64, 1024, None, None)), UNS),
                     (dict(grads=A.tm_layer_norm_grads(P(9), P(9))), INV),
                     (dict(saved=A.tm_ckpt8(P(12), None)), INV), (dict(saved=A.tm_ckpt8(P(8), P(12))), INV)]:
        assert ln_bwd(**kw) == want, kw


def lin(x=P(0), res=P(1), sh=None, w=None, y=P(4), z=None, save=None):
    sh = sh or api.shape(4, 1, 1, 1, "bf16")
    w = w or A.tm_linear_w(2, 64, 32, A.TM_ACT_GELU, P(2), P(3))
    return L.tm_pertoken_linear(x, res, sh, w, y, z, save, None)


def test_linear_refusals():
    W = lambda banks=2, width=64, out=32, act=A.TM_ACT_GELU, w=P(2), b=P(3): A.tm_linear_w(banks, width, out, act, w, b)
    f32 = api.shape(4, 1, 1, 1, "f32")
    for kw, want in [(dict(x=None), INV), (dict(y=None), INV), (dict(y=P(0)), INV), (dict(y=P(1)), INV), (dict(y=P(2)), INV),
                     (dict(x=P(0) + 2), INV), (dict(w=W(w=None)), INV), (dict(w=W(w=P(2) + 8)), INV), (dict(w=W(b=P(3) + 2)), INV),
                     (dict(w=W(banks=0)), INV), (dict(w=W(act=4)), INV), (dict(w=W(act=-1)), INV), (dict(w=W(width=60)), UNS),
                     (dict(w=W(out=28)), UNS), (dict(z=P(5), save=A.tm_ckpt8(P(6), P(7))), INV),
                     (dict(z=P(5), w=W(act=A.TM_ACT_NONE)), INV), (dict(save=A.tm_ckpt8(P(6), P(7)), w=W(act=A.TM_ACT_NONE)), INV),
                     (dict(z=P(4)), INV), (dict(save=A.tm_ckpt8(P(6), P(6))), INV), (dict(save=A.tm_ckpt8(None, P(6))), INV),
                     (dict(sh=api.shape(0, 1, 1, 1, "bf16")), INV), (dict(sh=api.shape(1 << 28, 1, 1, 1, "bf16")), UNS),
                     (dict(sh=f32, w=W(banks=70000)), UNS), (dict(w=W(banks=1 << 16, width=1 << 16)), UNS)]:
        assert lin(**kw) == want, kw


def test_linear_backward_refusals():
    sh = api.shape(4, 1, 1, 1, "bf16")
    w = A.tm_linear_w(2, 64, 32, A.TM_ACT_GELU, P(2), P(3))
    n = L.tm_pertoken_linear_backward_workspace_bytes(sh, w)
    assert n >= 4 * 2 * 32 * 2
    assert L.tm_pertoken_linear_backward_workspace_bytes(sh, A.tm_linear_w(2, 60, 32, 0, P(2), None)) == 0

    def call(x=P(0), dy=P(1), z=P(5), saved=None, add=None, w=w, dx=P(6), g=A.tm_linear_grads(P(7), P(8)), ws=P(9), wsb=1 << 30):
        return L.tm_pertoken_linear_backward(x, dy, z, saved, add, sh, w, dx, g, ws, wsb, None)
    for kw, want in [(dict(x=None), INV), (dict(dy=None), INV), (dict(z=None), INV), (dict(saved=A.tm_ckpt8(P(10), P(11))), INV),
                     (dict(z=None, saved=A.tm_ckpt8(P(10), None)), INV), (dict(add=P(12), dx=None), INV), (dict(dx=P(0)), INV),
                     (dict(dx=P(1)), INV), (dict(dx=P(2)), INV), (dict(add=P(6)), INV), (dict(wsb=n - 1), WS), (dict(ws=None), WS),
                     (dict(ws=P(1)), INV), (dict(g=A.tm_linear_grads(P(7), P(7))), INV), (dict(g=A.tm_linear_grads(P(2), None)), INV),
                     (dict(g=A.tm_linear_grads(P(7) + 4, None)), INV)]:
        assert call(**kw) == want, kw
    assert call(dx=None, g=A.tm_linear_grads(None, None)) == A.TM_OK              # nothing wanted: nothing launched


def test_binding_refuses_host_tensors_and_bad_arguments():
    x = torch.zeros(2, 3, 8)
    sh = api.shape(2, 3, 8, 1, torch.float32)
    with pytest.raises(ValueError, match="device"):
        api.layer_norm(x, None, A.TM_LAYOUT_ROWS, sh)
    with pytest.raises(ValueError, match="device"):
        api.checkpoint8_pack(x)
    with pytest.raises(ValueError, match="device"):
        api.checkpoint8_unpack(api.Checkpoint8(x.to(torch.int8), x.to(torch.int8), torch.float32))
    with pytest.raises(ValueError, match="activation"):
        api.Linear(x, None, "tanh")
    with pytest.raises(ValueError, match="banks, out, width"):
        api.Linear(x[0])
    with pytest.raises(ValueError, match="device"):
        api.pertoken_linear(x, api.Linear(x))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.checkpoint8_pack(x.half())
    with pytest.raises(ValueError, match="3-dimensional"):
        api.layer_norm(x[0], None, A.TM_LAYOUT_ROWS, sh)
