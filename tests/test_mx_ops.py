"""The operators that serve the layer in 8 and 4 bits on the host: their
refusals (these calls never reach HIP) and the 64-bit references."""
import ctypes

import numpy as np
import pytest

import mixture_experts_layer_prefix_amd as M
from mixture_experts_layer_prefix_amd import _lib as L

torch = pytest.importorskip("torch")
from tests import mx_ref as R  # noqa: E402

FAKE = 1 << 20  # an aligned address that is never dereferenced
BF, MX = L.MOE_BF16, L.MOE_MXFP8


def norm_status(x=FAKE, y=FAKE, w_post=None, gate=None, w_pre=None, x_out=FAKE, a=FAKE, a_q=FAKE, a_scale=FAKE,
                r_post=None, r_pre=None, **kw):
    b = M.Block(**dict(dict(T=4, d=96), **kw)).c()
    return L.lib().moe_block_norm_mxfp8(b, x, y, w_post, gate, w_pre, x_out, a, a_q, a_scale, r_post, r_pre, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), L.MOE_EINVAL), (dict(d=0), L.MOE_EINVAL), (dict(d=100), L.MOE_EUNSUPPORTED),
    (dict(d=16416), L.MOE_EUNSUPPORTED), (dict(T=1 << 23), L.MOE_EUNSUPPORTED), (dict(eps=0.0), L.MOE_EINVAL),
    (dict(a_q=None), L.MOE_EINVAL), (dict(a_scale=None), L.MOE_EINVAL), (dict(a_q=FAKE + 8), L.MOE_EINVAL),
    (dict(a=FAKE + 1), L.MOE_EINVAL), (dict(x=None), L.MOE_EINVAL), (dict(x_out=None), L.MOE_EINVAL),
    (dict(y=None), L.MOE_EINVAL), (dict(y=None, x_out=None, gate=FAKE), L.MOE_EINVAL), (dict(w_post=FAKE), L.MOE_EINVAL),
    (dict(w_pre=FAKE + 2), L.MOE_EINVAL), (dict(gate=FAKE, gate_every=-1), L.MOE_EINVAL),
    (dict(T=0, x=None, y=None, x_out=None, a=None, a_q=None, a_scale=None), L.MOE_OK)])
def test_block_norm_mxfp8_refuses(bad, status):
    assert norm_status(**bad) == status


def sort_status(idx=FAKE, x=FAKE, xs=FAKE, counts=FAKE, xp=2 * FAKE, xps=2 * FAKE, ws=FAKE, ws_bytes=1 << 40, **kw):
    d = M.Dims(**dict(dict(T=16, d=96, E=8, k=2, I=1), **kw))
    return L.lib().moe_sort_tokens_mxfp8(d.c(), idx, x, xs, counts, FAKE, FAKE, FAKE, xp, xps, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), L.MOE_EINVAL), (dict(d=0), L.MOE_EINVAL), (dict(d=100), L.MOE_EUNSUPPORTED), (dict(E=0), L.MOE_EINVAL),
    (dict(E=1025), L.MOE_EINVAL), (dict(k=17), L.MOE_EINVAL), (dict(T=1 << 23), L.MOE_EUNSUPPORTED),
    (dict(idx=None), L.MOE_EINVAL), (dict(x=None), L.MOE_EINVAL), (dict(xs=None), L.MOE_EINVAL),
    (dict(xp=None), L.MOE_EINVAL), (dict(xps=None), L.MOE_EINVAL), (dict(xp=FAKE), L.MOE_EINVAL),
    (dict(xps=FAKE), L.MOE_EINVAL), (dict(x=FAKE + 8), L.MOE_EINVAL), (dict(xs=FAKE + 2), L.MOE_EINVAL),
    (dict(counts=None), L.MOE_EINVAL), (dict(ws=None), L.MOE_EWORKSPACE), (dict(ws_bytes=4), L.MOE_EWORKSPACE),
    (dict(ws=FAKE + 8), L.MOE_EINVAL)])
def test_sort_tokens_mxfp8_refuses(bad, status):
    assert sort_status(**bad) == status


def test_quantize_mxfp4_refuses():
    lib = L.lib()
    for f in (lib.moe_quantize_mxfp4, lambda a, r, c, b, s, q: lib.moe_dequantize_mxfp4(a, s, r, c, b, q)):
        assert f(FAKE, 4, 96, FAKE, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, -1, 128, FAKE, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, 4, -128, FAKE, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, 1 << 28, 128, FAKE, FAKE, None) == L.MOE_EUNSUPPORTED
        assert f(FAKE, 4, (1 << 24) + 128, FAKE, FAKE, None) == L.MOE_EUNSUPPORTED
        assert f(None, 4, 128, FAKE, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, 4, 128, None, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, 4, 128, FAKE, None, None) == L.MOE_EINVAL
        assert f(FAKE + 8, 4, 128, FAKE, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, 4, 128, FAKE + 8, FAKE, None) == L.MOE_EINVAL
        assert f(FAKE, 4, 128, FAKE, FAKE + 2, None) == L.MOE_EINVAL
        assert f(None, 0, 128, None, None, None) == L.MOE_OK and f(None, 4, 0, None, None, None) == L.MOE_OK


def ffn_status(x=FAKE, xs=FAKE, idx=FAKE, w=FAKE, add=None, y=FAKE, ws=FAKE, ws_bytes=1 << 50, weights=None, **kw):
    d = M.Dims(**dict(dict(T=3, d=256, E=8, k=2, I=128), **kw))
    wt = L.moe_weights_mxfp4(**dict({n: FAKE for n, _ in L.moe_weights_mxfp4._fields_}, **(weights or {})))
    return L.lib().moe_routed_ffn_mxfp4(d.c(), x, xs, idx, w, wt, add, y, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), L.MOE_EINVAL), (dict(d=0), L.MOE_EINVAL), (dict(I=0), L.MOE_EINVAL), (dict(E=0), L.MOE_EINVAL),
    (dict(E=1025), L.MOE_EINVAL), (dict(k=0), L.MOE_EINVAL), (dict(k=17), L.MOE_EINVAL),
    (dict(T=1 << 23), L.MOE_EUNSUPPORTED), (dict(d=192), L.MOE_EUNSUPPORTED), (dict(I=96), L.MOE_EUNSUPPORTED),
    (dict(d=1 << 16, I=1 << 16), L.MOE_EUNSUPPORTED), (dict(T=1 << 20, d=2048), L.MOE_EUNSUPPORTED),
    (dict(T=1 << 21, k=8), L.MOE_EUNSUPPORTED), (dict(E=1024, d=1 << 14, I=1 << 13), L.MOE_EUNSUPPORTED),
    (dict(x=None), L.MOE_EINVAL), (dict(x=FAKE + 8), L.MOE_EINVAL),
    (dict(xs=None), L.MOE_EINVAL), (dict(xs=FAKE + 2), L.MOE_EINVAL), (dict(idx=None), L.MOE_EINVAL),
    (dict(w=None), L.MOE_EINVAL), (dict(add=FAKE + 8), L.MOE_EINVAL), (dict(y=None), L.MOE_EINVAL),
    (dict(weights=dict(q_up=None)), L.MOE_EINVAL), (dict(weights=dict(q_down=FAKE + 8)), L.MOE_EINVAL),
    (dict(weights=dict(q_gate_scale=None)), L.MOE_EINVAL), (dict(weights=dict(q_gate_scale=FAKE + 1)), L.MOE_EINVAL),
    (dict(ws=None), L.MOE_EWORKSPACE), (dict(ws_bytes=64), L.MOE_EWORKSPACE), (dict(ws=FAKE + 8), L.MOE_EINVAL),
    (dict(T=0, x=None, y=None, ws=None, ws_bytes=0), L.MOE_OK)])
def test_routed_ffn_refuses(bad, status):
    assert ffn_status(**bad) == status


def test_routed_ffn_workspace():
    n = ctypes.c_size_t(0)
    f = L.lib().moe_workspace_bytes
    assert f(M.Dims(7, 256, 4, 8, 128).c(), MX, 6, ctypes.byref(n)) == L.MOE_OK and n.value >= 56 * (128 + 4 + 4 * 256)
    assert f(M.Dims(0, 256, 4, 8, 128).c(), MX, 6, ctypes.byref(n)) == L.MOE_OK
    assert f(M.Dims(7, 96, 4, 8, 128).c(), MX, 6, ctypes.byref(n)) == L.MOE_EUNSUPPORTED
    assert f(M.Dims(7, 256, 4, 8, 128).c(), MX, 6, None) == L.MOE_EINVAL


def test_wrappers_refuse():
    u8, bf = torch.uint8, torch.bfloat16
    d = M.Dims(4, 128, 2, 2, 128)
    x, xs = torch.zeros(4, 128, dtype=u8), torch.zeros(4, 4, dtype=u8)
    idx, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    q, qs = torch.zeros(2, 128, 64, dtype=u8), torch.zeros(1, 256, 4, dtype=u8)
    wt = M.WeightsMxfp4(q, qs, q, qs, q, qs)
    for call in (lambda: M.quantize_mxfp4(torch.zeros(4, 128, dtype=bf)), lambda: M.quantize_mxfp4(None),
                 lambda: M.dequantize_mxfp4(q[0], qs), lambda: M.sort_tokens_mxfp8(idx, x, xs, d),
                 lambda: M.routed_ffn_mxfp4(x, xs, idx, w, wt, d), lambda: M.prepare_mxfp4(M.Weights(None), d),
                 lambda: M.block_norm_mxfp8(M.Block(4, 128), torch.zeros(4, 128, dtype=bf)),
                 lambda: M.BlockNormMxfp8Plan(M.Block(4, 128, "f32"), "cpu"),
                 lambda: M.BlockNormMxfp8Plan(M.Block(4, 100), "cpu"),
                 lambda: M.SortMxfp8Plan(M.Dims(4, 100, 2, 2, 1), "cpu")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.MoeError):
        M.RoutedFfnPlan(M.Dims(4, 96, 2, 2, 128), "cpu")
    # a plan on the CPU refuses its tensors before anything is launched
    with pytest.raises(ValueError):
        M.RoutedFfnPlan(d, "cpu").run(x, xs, idx, w, wt)


# ---- the references --------------------------------------------------------
def test_reference_rounding_to_e2m1():
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert [int(R.e2m1_round(v)) for v in grid] == list(range(8))
    # half way: the even code; beyond the largest: the largest
    assert [int(R.e2m1_round(v)) for v in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0)] == [0, 2, 2, 4, 4, 6, 6, 7]
    v = np.random.default_rng(3).uniform(-6, 6, 4096)
    near = np.array([min(abs(abs(a) - g) for g in grid) for a in v])
    assert np.array_equal(np.abs(np.abs(v) - R.E2M1[R.e2m1_round(v)]), near)


def test_reference_quantizer():
    rng = np.random.default_rng(4)
    w = rng.standard_normal((5, 256)) * 2.0 ** rng.integers(-20, 20, (5, 1))
    w[2, :32] = 0
    w[3, 32:64] = 6.0 * 2.0 ** -3
    w[3, 64] = 6.0001
    codes, scale = R.quantize4(w)
    v = R.values4(codes, scale)
    assert codes.shape == (5, 128) and scale.shape == (2, 5, 4)
    assert scale[0, 2, 0] == 0 and not codes[2, :16].any() and scale[0, 3, 1] == 124 and scale[0, 3, 2] == 128
    # nothing is clipped, and no finer scale would do
    b, e = np.abs(w).reshape(5, 8, 32).max(-1), scale.transpose(1, 0, 2).reshape(5, 8).astype(int) - 127
    assert np.all(b <= 6 * 2.0 ** e) and np.all((b > 3 * 2.0 ** e) | (b == 0))
    # off by at most half of the widest step, 2, at the block's scale
    assert np.all(np.abs(v - w) <= np.repeat(2.0 ** e, 32, axis=1))


def test_reference_h_rounding_bound_covers_flips():
    rng = np.random.default_rng(5)
    h = rng.standard_normal((6, 64)) * np.exp(rng.standard_normal((6, 64)))
    h[0, :32] = 448.0 * 2.0 ** -9  # at the border of two scales
    eh = 1e-2 * np.abs(h)
    q, off = R.round_h(h, eh)
    for _ in range(50):
        q2, _ = R.round_h(h + eh * rng.uniform(-1, 1, h.shape), np.zeros_like(h))
        assert np.all(np.abs(q2 - q) <= off * (1 + 1e-12))


def test_reference_routed_ffn():
    """Against the layer oracle's experts, on values that 8 bits hold."""
    from oracle import moe_oracle as O
    rng = np.random.default_rng(6)
    E, d, I, T = 3, 128, 128, 4
    gate, up, down = (rng.standard_normal((E, *s)) * 0.1 for s in ((I, d), (I, d), (d, I)))
    x, idx, w = rng.standard_normal((T, d)), np.array([[0, 1], [2, 2], [-1, 3], [1, -5]]), rng.uniform(size=(T, 2))
    add = rng.standard_normal((T, d))
    y, bound = R.routed_ffn(x, idx, w, gate, up, down, add)
    for t in range(T):
        want = add[t].copy()
        for j in range(2):
            e = idx[t, j]
            if 0 <= e < E:
                _, _, _, h = O.swiglu_ffn(x[t:t + 1], gate[e], up[e], down[e])
                codes, scale = O.mx_quantize(h)
                want += w[t, j] * (down[e] @ R.values8(codes, scale)[0])
        assert np.allclose(y[t], want, rtol=1e-12, atol=1e-12)
    assert np.array_equal(y[2], add[2]) and np.all(bound > 0)
