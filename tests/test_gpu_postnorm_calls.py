"""GPU tests of the post-norm block's binding: what a caller may hand in, and what is refused before a launch."""
import numpy as np
import pytest
import torch

from postnorm_util import DEV, draw
from token_sparse_moe_b200 import _abi as A
from token_sparse_moe_b200 import api

pytestmark = pytest.mark.gpu
EPS = 1e-6


def test_workspace_of_the_caller():
    """Of any dtype, dense and on the call's device; anything else is refused, whatever its size."""
    rng = np.random.default_rng(1)
    x, _ = draw(rng, (70, 3, 96), "bf16")
    dy, _ = draw(rng, (70, 3, 96), "bf16")
    w, _ = draw(rng, (3, 96, 96), "bf16")
    sh = api.shape(70, 3, 96, 1, "bf16", EPS)
    _, saved = api.layer_norm(x, None, A.TM_LAYOUT_ROWS, sh)
    lin = api.Linear(w, None, "silu")
    _, z = api.pertoken_linear(x, lin, save="full")
    norm = lambda ws: api.layer_norm_backward(dy, saved, A.TM_LAYOUT_ROWS, sh, x=x, workspace=ws)
    linear = lambda ws: api.pertoken_linear_backward(x, dy, lin, z, workspace=ws)
    for call in (norm, linear):
        ref = call(None)
        for ws in (torch.empty(1 << 22, dtype=torch.uint8, device=DEV), torch.empty(1 << 20, dtype=torch.float32, device=DEV),
                   torch.empty(16, dtype=torch.uint8, device=DEV)):
            got = call(ws)
            assert torch.equal(got[0], ref[0]) and all(torch.equal(got[-1][k], ref[-1][k]) for k in ref[-1])
        for ws in (torch.empty(1 << 22, dtype=torch.uint8), torch.empty(1 << 23, dtype=torch.uint8, device=DEV)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(ws)


@pytest.mark.parametrize("checkpoint8", [False, True])
def test_residual_is_x_needs_a_forward_whose_residual_was_x(checkpoint8):
    """Otherwise dz + Revert(dz) would be handed out where X's gradient is Revert(dz) alone."""
    rng = np.random.default_rng(2)
    B, T, D = 5, 8, 64
    x, _ = draw(rng, (B, T, D), "bf16")
    other, _ = draw(rng, (B, T, D), "bf16")
    dy, _ = draw(rng, (B, T, D), "bf16")
    sh, M = api.shape(B, T, D, T, "bf16", EPS), A.TM_LAYOUT_MIXED
    for res in (None, other):
        _, saved = api.layer_norm(x, res, M, sh, checkpoint8=checkpoint8)
        with pytest.raises((ValueError, A.TMError)):
            api.layer_norm_backward(dy, saved, M, sh, x=x, residual=res, residual_is_x=True)
    # X as both: the whole gradient is the sum of the two that come out one by one
    _, saved = api.layer_norm(x, x, M, sh, checkpoint8=checkpoint8)
    whole, none, _ = api.layer_norm_backward(dy, saved, M, sh, x=x, residual=x, residual_is_x=True)
    dx, dres, _ = api.layer_norm_backward(dy, saved, M, sh, x=x, residual=x)
    assert none is None
    two = dx.float() + dres.float()
    off = (whole.float() - two).abs()
    # the parts are rounded to bf16 each, their sum once more; in fp32 each is good to 100 u of rstd (dn + 1 + n^2) < 30
    assert (off <= 2.0 ** -8 * (dx.float().abs() + dres.float().abs() + whole.float().abs()) * 1.01 + 4e-4).all()


@pytest.mark.parametrize("width", [2 ** 31 - 5, 2 ** 31 - 8])
def test_checkpoint_of_the_widest_rows(width):
    """One row of nearly 2^31 values (value by value, and in vectors): codes, exponents and values, piece by piece."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(1, width, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    ck = api.checkpoint8_pack(x)
    back = api.checkpoint8_unpack(ck)
    step = 1 << 28
    for a in range(0, width, step):
        b = min(width, a + step)
        want = api.checkpoint8_pack(x[:, a:b].clone())       # (blocks of 32 are the same ones: step is a multiple)
        assert torch.equal(ck.codes[:, a:b], want.codes) and torch.equal(ck.exps[:, a // 32:(b + 31) // 32], want.exps)
        assert torch.equal(back[:, a:b], api.checkpoint8_unpack(want))


def test_a_refused_packing_leaves_the_checkpoint_as_it_was():
    kept = torch.ones(4, 64, dtype=torch.float32, device=DEV)
    ck = api.checkpoint8_pack(kept)
    for x in (torch.ones(5, 64, dtype=torch.bfloat16, device=DEV), torch.ones(64, 4, dtype=torch.bfloat16, device=DEV).t()):
        with pytest.raises(ValueError):
            api.checkpoint8_pack(x, out=ck)
        assert ck.dtype == torch.float32 and torch.equal(api.checkpoint8_unpack(ck), kept)
    other = api.checkpoint8_pack(torch.full((4, 64), 2.0, dtype=torch.bfloat16, device=DEV), out=ck)
    assert other is ck and ck.dtype == torch.bfloat16 and torch.equal(api.checkpoint8_unpack(ck).float(), 2 * kept)
