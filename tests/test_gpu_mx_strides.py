"""The operators in 8 and 4 bits refuse tensors that are not contiguous, of the
right type and shape otherwise."""
import pytest

import mixture_experts_layer_prefix_amd as M

torch = pytest.importorskip("torch")
from tests.test_gpu_mx_ops import BF, F32, U8, ids, randn, whole_problem  # noqa: E402

pytestmark = pytest.mark.gpu


def strided(t):
    """t's values in a tensor of its shape that is not contiguous."""
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=t.device)
    wide[..., ::2] = t
    out = wide[..., ::2]
    assert out.shape == t.shape and out.dtype == t.dtype and not out.is_contiguous()
    return out


def refused(f, *args, **kw):
    """f takes the tensors, and none of them strided."""
    f(*args, **kw)
    torch.cuda.synchronize()
    for i, t in enumerate(args):
        with pytest.raises(ValueError, match="contiguous"):
            f(*args[:i], strided(t), *args[i + 1:], **kw)


def test_quantize4():
    refused(M.quantize_mxfp4, randn(1, (128, 128)))
    with pytest.raises(ValueError, match="contiguous"):
        M.quantize_mxfp4(randn(1, (128, 128)).t())
    with pytest.raises(ValueError, match="contiguous"):
        M.quantize_mxfp4(randn(1, (1, 128)).expand(4, 128))
    codes, scale = M.quantize_mxfp4(randn(1, (128, 256)))
    refused(M.dequantize_mxfp4, codes, scale)
    with pytest.raises(ValueError, match="contiguous"):
        M.dequantize_mxfp4(codes.t(), scale)          # [128][128], as codes may be


def test_norm():
    b = M.Block(4, 96, post_norm=True)
    refused(lambda *a: M.block_norm_mxfp8(b, *a), randn(1, (4, 96)), randn(2, (4, 96)), randn(3, (96,), F32),
            randn(4, (96,), F32), randn(5, (b.gates, 96), F32))


def test_sort():
    dims = M.Dims(4, 64, 3, 2, 1)
    x, xs = torch.zeros(4, 64, dtype=U8, device="cuda"), torch.zeros(4, 2, dtype=U8, device="cuda")
    refused(lambda *a: M.sort_tokens_mxfp8(*a, dims), ids(1, 4, 2, 0, 3), x, xs)
    for name, t in (("x_perm", torch.zeros(8, 64, dtype=U8, device="cuda")),
                    ("x_perm_scale", torch.zeros(8, 2, dtype=U8, device="cuda"))):
        with pytest.raises(ValueError, match="contiguous"):
            M.SortMxfp8Plan(dims, **{name: strided(t)})


def test_experts():
    T, d, E, k, I = 3, 128, 2, 2, 128
    dims = M.Dims(T, d, E, k, I)
    x, xs, w = whole_problem(1, T, d, E, k, I)
    idx, tw, add = ids(1, T, k, 0, E), torch.rand(T, k, device="cuda"), randn(2, (T, d))
    refused(lambda *a: M.routed_ffn_mxfp4(*a[:4], w, dims, a[4]), x, xs, idx, tw, add)
    for n, t in vars(w).items():
        with pytest.raises(ValueError, match="contiguous"):
            M.routed_ffn_mxfp4(x, xs, idx, tw, M.WeightsMxfp4(**dict(vars(w), **{n: strided(t)})), dims)


def test_prepare():
    dims = M.Dims(1, 128, 2, 1, 128)
    w = {n: randn(i, (2, 128, 128), BF) for i, n in enumerate(("w_gate", "w_up", "w_down"))}
    M.prepare_mxfp4(M.Weights(None, **w), dims)
    for n in w:
        with pytest.raises(ValueError, match="contiguous"):
            M.prepare_mxfp4(M.Weights(None, **dict(w, **{n: w[n].transpose(1, 2)})), dims)
