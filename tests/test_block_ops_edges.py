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


# ---- tensors that overlap --------------------------------------------------
def outputs_are_distinct(out, counts, types, sources, norm=0):
    import numpy as np
    pack = lambda v, t: np.array(v, t).tobytes()  # noqa: E731
    return L.tensors().distinct(pack(out, np.uint64), pack(counts, np.int64), pack(types, np.int32),
                                pack(sources, np.uint64), norm)


def test_outputs_that_overlap_are_found():
    bf, f = 1, 0  # describe's types
    yes = outputs_are_distinct
    assert yes([100, 200], [50, 50], [bf, bf], [100, 200])          # in place, end to end
    assert not yes([100, 198], [50, 50], [bf, bf], [100, 198])      # one element shared
    assert not yes([100, 200], [26, 50], [f, bf], [100, 200])       # fp32 elements are four bytes
    assert not yes([100, 120], [50, 2], [bf, bf], [100, 120])       # one inside the other
    assert yes([100, 100, 120], [50, 0, 0], [bf] * 3, [100, 0, 0])  # empty tensors overlap nothing
    # into other tensors
    assert yes([1000, 1100], [50, 50], [bf, bf], [100, 200])
    assert yes([1000, 1100], [50, 50], [bf, bf], [100, 100])        # a gradient read twice
    assert yes([100, 1100], [50, 50], [bf, bf], [100, 200])         # one of them in place
    assert not yes([200, 100], [50, 50], [bf, bf], [100, 200])      # the gradients in another order
    assert not yes([102, 1100], [50, 50], [bf, bf], [100, 200])     # shifted by an element
    assert not yes([1000, 298], [50, 50], [bf, bf], [100, 200])     # its own gradient's last element
    assert not yes([1000, 198], [50, 2], [bf, bf], [100, 300])      # another's last element
    assert not yes([100, 140], [20, 20], [bf, bf], [100, 139])      # its own and another output
    assert yes([], [], [], [])
    # the norm
    assert not yes([100], [50], [bf], [100], 196)
    assert yes([100], [50], [bf], [100], 200) and yes([100], [50], [bf], [100], 96)
    with pytest.raises(TypeError):
        L.tensors().distinct(b"", b"", b"")
    with pytest.raises(TypeError):
        L.tensors().distinct(bytes(8), bytes(8), bytes(8), bytes(8), 0)  # types are four bytes each


def test_overlap_against_every_pair():
    import random
    rng = random.Random(3)
    found = 0
    for _ in range(3000):
        n = rng.randint(1, 4)
        counts, types = [rng.randint(0, 4) for _ in range(n)], [rng.randint(0, 1) for _ in range(n)]
        size = [c * (2 if t else 4) for c, t in zip(counts, types)]
        src = [rng.randrange(0, 200, 2) for _ in range(n)]
        out = [s if rng.random() < 0.3 else rng.randrange(0, 200, 2) for s in src]
        norm = rng.randrange(4, 200, 4)

        def meet(a, na, b, nb):
            return na > 0 and nb > 0 and a < b + nb and b < a + na
        good = not any(meet(out[i], size[i], norm, 4) for i in range(n))
        for i in range(n):
            for j in range(n):
                good &= i == j or not meet(out[i], size[i], out[j], size[j])
                good &= (i == j and out[i] == src[i]) or not meet(out[i], size[i], src[j], size[j])
        assert outputs_are_distinct(out, counts, types, src, norm) == good
        found += not good
    assert 300 < found < 2700


# ---- plans -----------------------------------------------------------------
def test_norm_plan_without_a_block_output():
    """The step before the first block keeps no second residual."""
    block = M.Block(4, 8, post_norm=True)
    plan = M.BlockNormPlan(block, device="cpu", output=False)
    assert plan.x_out is None and plan.a.shape == (4, 8)
    assert M.BlockNormPlan(block, device="cpu").x_out.shape == (4, 8)


# ---- sizes that the C structs cannot hold ----------------------------------
@pytest.mark.parametrize("make", [
    lambda: M.Dims(1, (1 << 32) + 64, 8, 1, 1), lambda: M.Dims(1, 64, (1 << 32) + 8, 1, 1),
    lambda: M.Dims(1, 64, 8, (1 << 32) + 1, 1), lambda: M.Dims((1 << 64) + 1, 64, 8, 1, 1),
    lambda: M.Dims(1, 1 << 31, 8, 1, 1), lambda: M.Block(1, (1 << 32) + 64), lambda: M.Block((1 << 64) + 1, 64),
    lambda: M.Block(1, 64, gate_every=1 << 64)])
def test_sizes_are_not_cut(make):
    """ctypes keeps the low bits: 2^32 + 64 channels would have run as 64."""
    with pytest.raises(ValueError):
        make().c()
    assert M.Dims(5, (1 << 31) - 1, 8, 1, 1).c().d == (1 << 31) - 1
