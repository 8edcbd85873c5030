"""The operators around the layer on the host, at the edges of what their
entry points accept (these calls never reach HIP)."""
import ctypes

import pytest

import mixture_experts_layer_prefix_amd as M
from mixture_experts_layer_prefix_amd import _lib as L

A, B, C, D = ((i + 1) << 20 for i in range(4))  # aligned addresses that are never dereferenced
BF, F32 = L.MOE_BF16, L.MOE_F32


# ---- rows whose columns an int cannot count --------------------------------
@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("d", [(1 << 30) + 1, (1 << 31) - 8192, (1 << 31) - 1])
def test_wide_rows_are_refused(d, prec):
    lib, dims, n = L.lib(), M.Dims(1, d, 8, 1, 1).c(), ctypes.c_size_t(0)
    assert lib.moe_workspace_bytes(dims, prec, 5, ctypes.byref(n)) == L.MOE_EUNSUPPORTED
    assert lib.moe_sort_tokens(dims, prec, A, A, A, A, A, A, B, A, 1 << 40, None) == L.MOE_EUNSUPPORTED
    assert lib.moe_sort_tokens_backward(dims, prec, A, B, None, C, None) == L.MOE_EUNSUPPORTED
    assert lib.moe_unsort_tokens(dims, prec, A, B, B, None, C, None) == L.MOE_EUNSUPPORTED
    assert lib.moe_unsort_tokens_backward(dims, prec, A, B, B, B, C, D, None) == L.MOE_EUNSUPPORTED


def test_the_widest_row_has_a_workspace():
    n = ctypes.c_size_t(0)
    assert L.lib().moe_workspace_bytes(M.Dims(1, 1 << 30, 8, 1, 1).c(), BF, 5, ctypes.byref(n)) == L.MOE_OK


# ---- empty batches ---------------------------------------------------------
def test_empty_batches_need_no_addresses():
    """torch gives tensors without elements the null address."""
    lib, e = L.lib(), M.Dims(0, 100, 8, 2, 1).c()
    assert lib.moe_unsort_tokens_backward(e, BF, None, None, None, None, None, None, None) == L.MOE_OK
    assert lib.moe_unsort_tokens_backward(M.Dims(1, 100, 8, 2, 1).c(), BF, A, A, A, A, None, None, None) == L.MOE_EINVAL
    b = M.Block(0, 100).c()
    assert lib.moe_block_norm(b, BF, *[None] * 9, None) == L.MOE_OK
