"""The operators around the layer on the host: their refusals (these calls
never reach HIP) and the 64-bit references' gradients against differences."""
import ctypes

import pytest

import mixture_experts_layer_prefix_amd as M
from mixture_experts_layer_prefix_amd import _lib as L

torch = pytest.importorskip("torch")
from tests import block_ref as B  # noqa: E402

FAKE = 1 << 20  # an aligned address that is never dereferenced
BF, F32, MX = L.MOE_BF16, L.MOE_F32, L.MOE_MXFP8


# ---- refusals --------------------------------------------------------------
def sort_status(ws=FAKE, ws_bytes=1 << 40, prec=BF, x=FAKE, xp=2 * FAKE, idx=FAKE, **kw):
    d = dict(T=16, d=100, E=8, k=2, I=1)
    d.update(kw)
    return L.lib().moe_sort_tokens(M.Dims(**d).c(), prec, idx, x, FAKE, FAKE, FAKE, FAKE, xp, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), L.MOE_EINVAL), (dict(d=0), L.MOE_EINVAL), (dict(E=0), L.MOE_EINVAL), (dict(E=1025), L.MOE_EINVAL),
    (dict(k=0), L.MOE_EINVAL), (dict(k=17), L.MOE_EINVAL), (dict(T=1 << 23), L.MOE_EUNSUPPORTED),
    (dict(prec=MX), L.MOE_EUNSUPPORTED), (dict(prec=7), L.MOE_EINVAL), (dict(idx=None), L.MOE_EINVAL),
    (dict(idx=FAKE + 2), L.MOE_EINVAL), (dict(x=None), L.MOE_EINVAL), (dict(xp=FAKE), L.MOE_EINVAL),
    (dict(x=FAKE + 1), L.MOE_EINVAL), (dict(prec=F32, x=FAKE + 2), L.MOE_EINVAL), (dict(ws=None), L.MOE_EWORKSPACE),
    (dict(ws_bytes=4), L.MOE_EWORKSPACE), (dict(ws=FAKE + 8), L.MOE_EINVAL)])
def test_sort_refuses(bad, status):
    assert sort_status(**bad) == status


def test_sort_workspace():
    n = ctypes.c_size_t(0)
    lib = L.lib()
    # k above E and odd widths are fine here, unlike for the layer
    assert lib.moe_workspace_bytes(M.Dims(1000, 33, 4, 8, 0).c(), BF, 5, ctypes.byref(n)) == L.MOE_OK and n.value > 0
    assert lib.moe_workspace_bytes(M.Dims(1000, 33, 4, 8, 0).c(), BF, 1, ctypes.byref(n)) == L.MOE_EINVAL
    assert lib.moe_workspace_bytes(M.Dims(1000, 33, 4, 8, 0).c(), MX, 5, ctypes.byref(n)) == L.MOE_EUNSUPPORTED


def test_unsort_refuses():
    lib, d = L.lib(), M.Dims(16, 100, 8, 2, 1).c()
    a, b, c = FAKE, 2 * FAKE, 3 * FAKE
    assert lib.moe_unsort_tokens(d, MX, a, b, b, None, c, None) == L.MOE_EUNSUPPORTED
    assert lib.moe_unsort_tokens(d, BF, a, b, None, None, c, None) == L.MOE_EINVAL
    assert lib.moe_unsort_tokens(d, BF, a, None, b, None, c, None) == L.MOE_EINVAL
    assert lib.moe_unsort_tokens(d, BF, a, b, b, None, a, None) == L.MOE_EINVAL
    assert lib.moe_unsort_tokens(d, F32, a + 2, b, b, None, c, None) == L.MOE_EINVAL
    assert lib.moe_sort_tokens_backward(d, BF, None, b, None, c, None) == L.MOE_EINVAL
    assert lib.moe_sort_tokens_backward(d, BF, a, b, a + 1, c, None) == L.MOE_EINVAL
    f = lib.moe_unsort_tokens_backward
    assert f(d, BF, a, b, b, b, None, None, None) == L.MOE_EINVAL
    assert f(d, BF, a, b, b, None, c, None, None) == L.MOE_EINVAL  # do_perm needs the weights
    assert f(d, BF, a, None, b, b, None, c, None) == L.MOE_EINVAL  # dtopk_w needs o_perm
    assert f(d, BF, a, b, b, b, a, None, None) == L.MOE_EINVAL
    e = M.Dims(0, 100, 8, 2, 1).c()
    assert lib.moe_unsort_tokens(e, BF, None, None, None, None, None, None) == L.MOE_OK
    assert lib.moe_sort_tokens_backward(e, BF, None, None, None, None, None) == L.MOE_OK


def norm_status(prec=BF, x=FAKE, y=FAKE, w_post=None, gate=None, w_pre=None, x_out=FAKE, a=FAKE, r_post=None,
                r_pre=None, **kw):
    b = M.Block(**dict(dict(T=4, d=100), **kw)).c()
    if "every" in kw:
        b.gate_every = kw["every"]
    return L.lib().moe_block_norm(b, prec, x, y, w_post, gate, w_pre, x_out, a, r_post, r_pre, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), L.MOE_EINVAL), (dict(d=0), L.MOE_EINVAL), (dict(d=16385), L.MOE_EUNSUPPORTED),
    (dict(T=1 << 23), L.MOE_EUNSUPPORTED), (dict(prec=MX), L.MOE_EUNSUPPORTED), (dict(eps=0.0), L.MOE_EINVAL),
    (dict(eps=float("nan")), L.MOE_EINVAL), (dict(alpha=float("inf")), L.MOE_EINVAL),
    (dict(beta=float("nan")), L.MOE_EINVAL), (dict(x=None), L.MOE_EINVAL), (dict(x_out=None), L.MOE_EINVAL),
    (dict(x=FAKE + 1), L.MOE_EINVAL), (dict(res_f32=True, x=FAKE + 2), L.MOE_EINVAL),
    (dict(y=None), L.MOE_EINVAL), (dict(y=None, x_out=None, a=None), L.MOE_EINVAL),
    (dict(y=None, x_out=None, gate=FAKE), L.MOE_EINVAL), (dict(y=None, x_out=None, post_norm=True), L.MOE_EINVAL),
    (dict(w_post=FAKE), L.MOE_EINVAL), (dict(r_post=FAKE), L.MOE_EINVAL), (dict(a=None, w_pre=FAKE), L.MOE_EINVAL),
    (dict(a=None, r_pre=FAKE), L.MOE_EINVAL), (dict(w_pre=FAKE + 2), L.MOE_EINVAL),
    (dict(gate=FAKE, gate_every=-1), L.MOE_EINVAL), (dict(T=0), L.MOE_OK)])
def test_block_norm_refuses(bad, status):
    assert norm_status(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dx_out=None, da=None), L.MOE_EINVAL), (dict(dy=None), L.MOE_EINVAL), (dict(y=None), L.MOE_EINVAL),
    (dict(r_pre=None), L.MOE_EINVAL), (dict(x_out=None), L.MOE_EINVAL), (dict(da=None), L.MOE_EINVAL),
    (dict(post_norm=True), L.MOE_EINVAL), (dict(w_post=FAKE), L.MOE_EINVAL), (dict(dw_pre=FAKE), L.MOE_EINVAL),
    (dict(dgate=FAKE), L.MOE_EINVAL), (dict(dx=None), L.MOE_EINVAL), (dict(dx=FAKE + 1), L.MOE_EINVAL),
    (dict(ws=None), L.MOE_EWORKSPACE), (dict(ws_bytes=64), L.MOE_EWORKSPACE), (dict(ws=FAKE + 4), L.MOE_EINVAL),
    (dict(prec=MX), L.MOE_EUNSUPPORTED), (dict(y=None, dy=None, gate=FAKE), L.MOE_EINVAL)])
def test_block_norm_backward_refuses(bad, status):
    a = dict(prec=BF, dx_out=FAKE, da=FAKE, x_out=FAKE, y=FAKE, r_post=None, r_pre=FAKE, w_post=None, gate=None,
             w_pre=None, dx=FAKE, dy=FAKE, dw_post=None, dgate=None, dw_pre=None, ws=FAKE, ws_bytes=1 << 40)
    a.update({k: v for k, v in bad.items() if k != "post_norm"})
    b = M.Block(4, 100, post_norm=bad.get("post_norm", False)).c()
    prec = a.pop("prec")
    assert L.lib().moe_block_norm_backward(b, prec, *a.values(), None) == status


def host(ptrs, numel, types):
    n = len(numel)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types), n)


@pytest.mark.parametrize("ptrs,numel,types,status", [
    ([FAKE], [-1], [BF], L.MOE_EINVAL), ([None], [4], [BF], L.MOE_EINVAL), ([FAKE + 1], [4], [BF], L.MOE_EINVAL),
    ([FAKE + 2], [4], [F32], L.MOE_EINVAL), ([FAKE], [4], [MX], L.MOE_EUNSUPPORTED), ([FAKE], [4], [9], L.MOE_EINVAL)])
def test_clip_refuses_tensors(ptrs, numel, types, status):
    p, m, t, n = host(ptrs, numel, types)
    lib = L.lib()
    assert lib.moe_grad_norm(p, m, t, n, FAKE, FAKE, 1 << 40, None) == status
    assert lib.moe_clip_grads(p, p, m, t, n, 1.0, None, FAKE, FAKE, 1 << 40, None) == status


def test_clip_refuses():
    lib = L.lib()
    p, m, t, n = host([FAKE], [4], [BF])
    need = lib.moe_grad_norm_scratch_bytes(m, n)
    assert need > 0
    assert lib.moe_grad_norm(p, m, t, n, None, FAKE, need, None) == L.MOE_EINVAL
    assert lib.moe_grad_norm(p, m, t, n, FAKE, None, need, None) == L.MOE_EWORKSPACE
    assert lib.moe_grad_norm(p, m, t, n, FAKE, FAKE, need - 1, None) == L.MOE_EWORKSPACE
    assert lib.moe_grad_norm(None, m, t, n, FAKE, FAKE, need, None) == L.MOE_EINVAL
    assert lib.moe_grad_norm(p, m, t, -1, FAKE, FAKE, need, None) == L.MOE_EINVAL
    for bad in (float("nan"), float("inf"), -1.0):
        assert lib.moe_clip_grads(p, p, m, t, n, bad, None, FAKE, FAKE, need, None) == L.MOE_EINVAL
    assert lib.moe_clip_grads(p, None, m, t, n, 1.0, None, FAKE, FAKE, need, None) == L.MOE_EINVAL
    assert lib.moe_clip_grads(p, p, m, t, n, 1.0, None, None, FAKE, need, None) == L.MOE_EINVAL
    assert lib.moe_clip_grads(p, p, m, t, n, 1.0, FAKE + 2, FAKE, FAKE, need, None) == L.MOE_EINVAL


def test_wrappers_refuse_host_tensors():
    d = M.Dims(4, 8, 2, 2, 1)
    x = torch.zeros(4, 8)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.sort_tokens(idx, x, d, "f32")
    with pytest.raises(ValueError):
        M.unsort_tokens(torch.zeros(8, 8), idx, torch.zeros(4, 2), None, d, "f32")
    with pytest.raises(ValueError):
        M.unsort_tokens_backward(x, torch.zeros(8, 8), idx, torch.zeros(4, 2), d, "mxfp8")
    with pytest.raises(ValueError):
        M.block_norm(M.Block(4, 8, "f32"), x)
    with pytest.raises(ValueError):
        M.clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        M.grad_norm([])


# ---- the references' own gradients -----------------------------------------
@pytest.mark.parametrize("post,gate,output", [(True, True, True), (False, True, True), (True, False, True),
                                              (False, False, False)])
def test_reference_gradient_matches_differences(post, gate, output):
    g = torch.Generator().manual_seed(5)
    T, d, every, alpha, beta, eps = 5, 7, 2, 0.75, -0.5, 1e-3
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    p = dict(x=rn(T, d), y=rn(T, d) if output else None, w_post=rn(d) if post else None,
             gate=rn(3, d) if gate else None, w_pre=rn(d))
    dxo, da = rn(T, d), rn(T, d)

    def fwd(q):
        return B.norm_fwd_ref(q["x"], q["y"], q["w_post"], q["gate"], q["w_pre"], every, alpha, beta, eps, post)

    def loss(q):
        o = fwd(q)
        return ((o["x_out"] if output else q["x"]) * dxo).sum() + (o["a"] * da).sum()

    o = fwd(p)
    got = B.norm_bwd_ref(dxo, da, o["x_out"] if output else p["x"], p["y"], o.get("r_post"), o["r_pre"], p["w_post"],
                         p["gate"], p["w_pre"], every, alpha, beta, post)
    names = dict(x="dx", y="dy", w_post="dw_post", gate="dgate", w_pre="dw_pre")
    h = 1e-5
    for n, t in p.items():
        if t is None:
            assert names[n] not in got
            continue
        diff = torch.zeros_like(t)
        for i in range(t.numel()):
            q = dict(p)
            for s in (1, -1):
                q[n] = t.clone()
                q[n].view(-1)[i] += s * h
                diff.view(-1)[i] += s * loss(q) / (2 * h)
        # central differences: error of order h^2 = 1e-10 times third derivatives, plus 1e-16 / h
        assert torch.allclose(got[names[n]], diff, rtol=1e-6, atol=1e-7), n


def test_reference_sort_gradients_match_differences():
    g = torch.Generator().manual_seed(6)
    T, k, E, d = 6, 3, 4, 5
    idx = torch.randint(-1, E + 1, (T, k), generator=g)
    _, offsets, _, token_row = B.sort_ref(idx, E)
    o = torch.randn(T * k, d, generator=g, dtype=torch.float64)
    w = torch.randn(T, k, generator=g, dtype=torch.float64)
    dy = torch.randn(T, d, generator=g, dtype=torch.float64)
    do, dw, _ = B.unsort_bwd_ref(dy, o, token_row, w)
    h = 1e-4
    for i in range(w.numel()):  # the sum is linear in each argument: differences are exact up to 1e-12
        e = torch.zeros_like(w)
        e.view(-1)[i] = h
        diff = ((B.unsort_ref(o, token_row, w + e, None)[0] - B.unsort_ref(o, token_row, w - e, None)[0]) * dy).sum()
        assert abs(diff / (2 * h) - dw.view(-1)[i]) < 1e-9
    for row in range(int(offsets[-1])):
        e = torch.zeros_like(o)
        e[row, 1] = h
        diff = ((B.unsort_ref(o + e, token_row, w, None)[0] - B.unsort_ref(o - e, token_row, w, None)[0]) * dy).sum()
        assert abs(diff / (2 * h) - do[row][1]) < 1e-9


# ---- the wrappers' helper module --------------------------------------------
def test_tensor_helper_module():
    import numpy as np
    h = L.tensors()
    t = torch.zeros(2, 3)
    assert h.address(t, torch.float32, (2, 3), 0) == -1  # not on a GPU
    assert h.address(3, torch.float32, (2, 3), 0) == -1
    assert h.describe([]) == (b"", b"", b"", -1)
    assert h.describe([t]) == 0 and h.describe([None, t]) == 0
    with pytest.raises(TypeError):
        h.address(t, torch.float32, [2, 3], 0)
    with pytest.raises(TypeError):
        h.distinct(b"", "")
    pack = lambda v, n: (np.array(v, np.uint64).tobytes(), np.array(n, np.int64).tobytes())  # noqa: E731
    assert h.distinct(*pack([16, 32], [1, 1])) and h.distinct(*pack([16, 16], [1, 0]))
    assert not h.distinct(*pack([16, 32, 16], [1, 1, 2]))
