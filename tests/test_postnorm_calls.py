"""The post-norm block's binding on the CPU: arguments that are refused before anything is launched."""
import pytest
import torch

from token_sparse_moe_b200 import _abi as A
from token_sparse_moe_b200 import api


class _Elsewhere(torch.Tensor):
    """A dense tensor that says it is on GPU 1."""

    def get_device(self):
        return 1


def test_binding_refuses_a_workspace_that_the_kernels_cannot_use():
    for ws in (torch.empty(4096, dtype=torch.uint8), torch.empty(4096, dtype=torch.uint8).as_subclass(_Elsewhere)):
        with pytest.raises(ValueError, match="workspace"):
            api._scratch(1024, 0, ws)
    here = torch.empty(2048, dtype=torch.float32).as_subclass(_Elsewhere)
    with pytest.raises(ValueError, match="workspace"):
        api._scratch(1024, 1, here[::2])                       # the bytes between its elements are not its own
    ws, address, nbytes = api._scratch(8192, 1, here)
    assert ws is here and address == here.data_ptr() and nbytes == 8192


def test_the_widest_checkpoint_rows_have_their_size():
    """Of the last widths below 2^31 the blocks are counted right: exponents that would reach into the codes are seen."""
    lib, x, codes = A.load(), 1 << 40, 1 << 41
    for width in (2 ** 31 - 1, 2 ** 31 - 31, 2 ** 31 - 32):
        over = A.tm_ckpt8(codes, codes - 1024)
        assert lib.tm_checkpoint8_pack(x, A.TM_BF16, 1, width, over, None) == A.TM_ERR_INVALID_ARG
        assert lib.tm_checkpoint8_unpack(A.tm_ckpt8(codes, x - 1024), A.TM_BF16, 1, width, x, None) == A.TM_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_layers_of_nearly_2_31_columns_are_refused(dtype):
    """A tile's edge past 2^31 columns is no 32-bit integer."""
    lib, P = A.load(), lambda i: (i + 1) << 44
    sh = api.shape(2, 1, 1, 1, dtype)
    for banks, width, out in ((1, 2 ** 31 - 8, 8), (255, 8421504, 8), (1, 8, 2 ** 31 - 8), (255, 8, 8421504)):
        w = A.tm_linear_w(banks, width, out, A.TM_ACT_NONE, P(2), None)
        assert lib.tm_pertoken_linear(P(0), None, sh, w, P(4), None, None, None) == A.TM_ERR_UNSUPPORTED
        assert lib.tm_pertoken_linear_backward_workspace_bytes(sh, w) == 0
