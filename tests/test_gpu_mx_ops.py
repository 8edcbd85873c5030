"""The operators that serve the layer in 8 and 4 bits on the GPU, each against
its definition in 64 bits."""
import numpy as np
import pytest

import mixture_experts_layer_prefix_amd as M
from oracle import moe_oracle as O

torch = pytest.importorskip("torch")
from tests import block_ref as B  # noqa: E402
from tests import mx_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


# ---- weights in 4 bits -----------------------------------------------------
def check4(w):
    codes, scale = M.quantize_mxfp4(w)
    want_codes, want_scale = R.quantize4(np64(w))
    assert np.array_equal(scale.cpu().numpy(), want_scale)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    back = M.dequantize_mxfp4(codes, scale)
    want = torch.from_numpy(R.values4(want_codes, want_scale)).to(BF)
    assert torch.equal(back.cpu(), want) and torch.equal(back.cpu().signbit(), want.signbit())


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (15, 640), (16, 512), (17, 1152), (100, 128), (33, 2048),
                                       (2, 7168)])
def test_quantize4_shapes(rows, cols):
    w = randn(rows, (rows, cols)) * torch.exp2(torch.randint(-30, 30, (rows, cols // 32, 1), generator=gen(2),
                                                             device="cuda")).expand(-1, -1, 32).reshape(rows, cols)
    check4(w.to(BF))


def test_quantize4_every_value():
    """Every finite bf16 below 2^125 in blocks whose largest magnitude is each
    of several, so that every rounding and every tie is met; zeros and
    subnormals among them."""
    v = torch.arange(65536, dtype=I32, device="cuda").to(torch.int16).view(BF)
    v = v[v.abs() < 2.0 ** 125]
    for top in (None, 1.0, 5.0, 6.0, 6.03125, 7.5, 2.0 ** -126, 2.0 ** -133, 2.0 ** 100):
        if top is None:
            n = v.numel() // 128 * 128
            check4(v[:n].view(-1, 128).contiguous())
        else:
            some = v[v.abs() <= top]
            n = (some.numel() + 30) // 31 * 31
            some = torch.cat([some, torch.zeros(n - some.numel(), dtype=BF, device="cuda")]).view(-1, 31)
            blocks = torch.cat([torch.full((some.shape[0], 1), top, dtype=BF, device="cuda"), some], 1)
            pad = -blocks.shape[0] % 4
            blocks = torch.cat([blocks, torch.zeros(pad, 32, dtype=BF, device="cuda")])
            check4(blocks.view(-1, 128).contiguous())


def test_dequantize4_every_scale():
    """Every byte of codes at every scale whose values bf16 holds; below its
    normal numbers the value is rounded once."""
    scale = torch.arange(253, dtype=U8, device="cuda").view(1, 253, 1).expand(1, 253, 4)
    codes = torch.arange(256, dtype=U8, device="cuda").view(1, 256).expand(253, 256).reshape(253, 4, 64)
    for i in range(4):
        c, s = codes[:, i].contiguous(), scale.contiguous()
        got = M.dequantize_mxfp4(c, s)
        want = torch.from_numpy(R.values4(c.cpu().numpy(), s.cpu().numpy())).to(BF)
        assert torch.equal(got.cpu(), want)


def test_quantize4_empty():
    codes, scale = M.quantize_mxfp4(torch.empty(0, 128, dtype=BF, device="cuda"))
    assert codes.shape == (0, 64) and M.dequantize_mxfp4(codes, scale).shape == (0, 128)


# ---- norms whose output is in 8 bits ---------------------------------------
@pytest.mark.parametrize("T,d,res_f32,post,gate_every,output", [
    (1, 32, False, False, None, True), (3, 64, True, True, 0, True), (5, 96, False, True, 2, True),
    (2, 2016, True, False, 0, True), (700, 256, False, True, 100, True), (9, 7168, False, True, 0, True),
    (4, 7168, True, True, 3, True), (3, 8192, False, False, None, False), (2, 12288, False, True, 0, True),
    (2, 16384, True, True, 1, True), (6, 4128, True, False, None, False)])
def test_block_norm_mxfp8(T, d, res_f32, post, gate_every, output):
    b = M.Block(T, d, "bf16", res_f32=res_f32, post_norm=post and output, alpha=0.75, beta=-0.5, eps=1e-5,
                gate_every=gate_every or 0)
    x = randn(1, (T, d), F32 if res_f32 else BF, 2.0)
    y = randn(2, (T, d)) if output else None
    w_pre = 1 + randn(3, (d,), F32, 0.3)
    w_post = 1 + randn(4, (d,), F32, 0.1) if b.post_norm else None
    gate = None if gate_every is None or not output else randn(5, (b.gates, d), F32)
    x[0, :32] = 0
    if output:
        y[0, :32] = 0  # a block of zeros
    x_out, a, plan = M.block_norm(b, x, y, w_pre, w_post, gate)
    got, q, s, mx = M.block_norm_mxfp8(b, x, y, w_pre, w_post, gate)
    assert torch.equal(got, x_out) and torch.equal(mx.a, a) and torch.equal(mx.r_pre, plan.r_pre)
    assert not b.post_norm or torch.equal(mx.r_post, plan.r_post)
    codes, scale = O.mx_quantize(np64(a))
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(q.cpu().numpy(), codes)
    want = M.quantize_mxfp8(a, 0) if d % 128 == 0 else (q, s)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and int(s[0, 0]) == 0
    _, q2, s2, alone = M.block_norm_mxfp8(b, x, y, w_pre, w_post, gate, keep_a=False)
    assert alone.a is None and torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(alone.r_pre, mx.r_pre)
    ref = B.norm_fwd_ref(x, y, w_post, gate, w_pre, b.every, 0.75, -0.5, 1e-5, b.post_norm)["a"]
    # half a step of bf16, half a step of E4M3, a subnormal's half step, and fp32's roundings
    top = ref.view(T, -1, 32).abs().amax(-1, keepdim=True).expand(-1, -1, 32).reshape(T, d)
    off = (torch.from_numpy(R.values8(q.cpu().numpy(), s.cpu().numpy())) - ref).abs()
    assert bool((off <= ref.abs() * (2.0 ** -8 + 2.0 ** -4 + 2.0 ** -8) + top * (2.0 ** -17 + 2.0 ** -16)).all())


def test_block_norm_mxfp8_backward_takes_its_statistics():
    T, d = 33, 256
    b = M.Block(T, d, "bf16", res_f32=True, post_norm=True)
    x, y, w, wp = randn(1, (T, d), F32), randn(2, (T, d)), 1 + randn(3, (d,), F32, 0.1), 1 + randn(4, (d,), F32, 0.1)
    dx_out, da = randn(5, (T, d), F32), randn(6, (T, d))
    x0, _, p0 = M.block_norm(b, x, y, w, wp)
    x1, _, _, p1 = M.block_norm_mxfp8(b, x, y, w, wp, keep_a=False)
    r0 = M.block_norm_backward(b, dx_out, da, x0, y, p0.r_pre, p0.r_post, w, wp)
    r1 = M.block_norm_backward(b, dx_out, da, x1, y, p1.r_pre, p1.r_post, w, wp)
    assert torch.equal(r0[0], r1[0]) and torch.equal(r0[1], r1[1])
    assert all(torch.equal(r0[2][n], r1[2][n]) for n in r0[2])


def test_block_norm_mxfp8_empty():
    x_out, q, s, _ = M.block_norm_mxfp8(M.Block(0, 64), torch.empty(0, 64, dtype=BF, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 2)


# ---- tokens in 8 bits sorted by expert -------------------------------------
def ids(seed, T, k, lo, hi):
    return torch.randint(lo, hi, (T, k), generator=gen(seed), device="cuda", dtype=I32)


@pytest.mark.parametrize("T,d,E,k,lo,hi", [
    (1, 32, 1, 1, 0, 1), (1, 128, 4, 8, -1, 5), (7, 96, 5, 3, -2, 7), (256, 1056, 64, 8, -8, 72),
    (257, 160, 16, 8, 0, 16), (2000, 256, 33, 6, -1, 34), (5000, 64, 256, 8, -32, 288), (9, 7168, 256, 8, 0, 256),
    (40, 64, 3, 16, 3, 9)])
def test_sort_tokens_mxfp8(T, d, E, k, lo, hi):
    idx = ids(T, T, k, lo, hi)
    x = torch.randint(0, 256, (T, d), generator=gen(1), device="cuda", dtype=U8)
    xs = torch.randint(0, 256, (T, d // 32), generator=gen(2), device="cuda", dtype=U8)
    xp = torch.full((T * k, d), 0x55, dtype=U8, device="cuda")
    xps = torch.full((T * k, d // 32), 0xAA, dtype=U8, device="cuda")
    rt = torch.full((T * k,), -7, dtype=I32, device="cuda")
    plan = M.SortMxfp8Plan(M.Dims(T, d, E, k, 1), x_perm=xp, x_perm_scale=xps, row_token=rt)
    for _ in range(2):
        counts, offsets, row_token, token_row, x_perm, x_perm_scale = plan.run(idx, x, xs)
    rc, ro, rr, rtr = B.sort_ref(idx.cpu(), E)
    n = int(ro[-1])
    assert torch.equal(counts.cpu(), rc) and torch.equal(offsets.cpu(), ro) and torch.equal(token_row.cpu(), rtr)
    assert torch.equal(row_token[:n].cpu(), rr) and bool((row_token[n:] == -7).all())
    src = rr.long().cuda()
    assert torch.equal(x_perm[:n], x[src]) and torch.equal(x_perm_scale[:n], xs[src])
    assert bool((x_perm[n:] == 0x55).all()) and bool((x_perm_scale[n:] == 0xAA).all())


def test_sort_tokens_mxfp8_empty():
    e = torch.empty
    out = M.sort_tokens_mxfp8(e(0, 2, dtype=I32, device="cuda"), e(0, 64, dtype=U8, device="cuda"),
                              e(0, 2, dtype=U8, device="cuda"), M.Dims(0, 64, 4, 2, 1))
    assert out[0].tolist() == [0] * 4 and out[1].tolist() == [0] * 5


# ---- the routed experts of a few tokens ------------------------------------
def whole_problem(seed, T, d, E, k, I):
    """Inputs whose gate and up products are whole multiples of 2^-4 below 2^10
    each, so that the matrix cores add them exactly: E4M3 values 0, +-1, +-2 and
    weights 0, +-0.5, +-1, +-1.5 at scales 2^-1 to 2^1, sparse enough for |G|
    below 16."""
    g = gen(seed)
    pick = lambda shape, values: torch.tensor(values, dtype=U8, device="cuda")[  # noqa: E731
        torch.randint(0, len(values), shape, generator=g, device="cuda")]
    x = pick((T, d), [0x00] * 4 + [0x38, 0xB8, 0x40, 0xC0])
    xs = pick((T, d // 32), [126, 127, 128])
    out = {}
    thin = max(1, d // 64)
    for name, rows, cols, zeros in (("gate", I, d, 2 * thin), ("up", I, d, 2 * thin), ("down", d, I, 2)):
        lo, hi = (pick((E, rows, cols // 2), [0] * zeros + [1, 2, 3, 9, 10, 11]) for _ in range(2))
        out["q_" + name] = lo | (hi << 4)
        out["q_%s_scale" % name] = pick((cols // 128, E * rows, 4), [126, 127, 128])
    return x, xs, M.WeightsMxfp4(**out)


def real_problem(seed, T, d, E, k, I):
    w = {n: randn(seed + i, (E, *s), BF, s[1] ** -0.5)
         for i, (n, s) in enumerate((("w_gate", (I, d)), ("w_up", (I, d)), ("w_down", (d, I))))}
    x, xs = M.quantize_mxfp8(randn(seed + 5, (T, d)), 0)
    return x, xs, M.prepare_mxfp4(M.Weights(None, **w), M.Dims(T, d, E, k, I))


def host_weights(w, E):
    out = []
    for n in ("gate", "up", "down"):
        q, s = getattr(w, "q_" + n), getattr(w, "q_%s_scale" % n)
        v = R.values4(q.reshape(-1, q.shape[-1]).cpu().numpy(), s.cpu().numpy())
        out.append(v.reshape(E, -1, v.shape[-1]))
    return out


def reference(x, xs, idx, tw, w, E, add=None, **kw):
    return R.routed_ffn(R.values8(x.cpu().numpy(), xs.cpu().numpy()), idx.cpu().numpy(), np64(tw), *host_weights(w, E),
                        None if add is None else np64(add), **kw)


def poisoned(dims):
    plan = M.RoutedFfnPlan(dims)
    plan.ws.fill_(0xFF)  # NaN as E4M3, E8M0 and fp32; -1 as an index
    plan.y.fill_(float("nan"))
    return plan


@pytest.mark.parametrize("T,d,E,k,I,lo,hi,add", [
    (1, 128, 1, 1, 128, 0, 1, False), (1, 128, 4, 3, 256, 0, 4, True), (2, 256, 3, 5, 128, -1, 4, True),
    (5, 384, 6, 4, 384, -2, 8, False), (16, 128, 2, 2, 128, 0, 2, True), (17, 256, 2, 1, 128, 0, 2, True),
    (33, 128, 1, 1, 256, 0, 1, False), (70, 128, 3, 2, 128, -1, 3, True), (130, 128, 2, 2, 128, 0, 2, True),
    (3, 1152, 5, 2, 128, 0, 5, False), (4, 128, 9, 16, 1152, -4, 12, True), (300, 128, 40, 8, 128, -5, 45, False)])
def test_routed_ffn_whole_numbers(T, d, E, k, I, lo, hi, add):
    """Element by element: gate and up are exact, so h moves by SwiGLU's own
    roundings alone."""
    x, xs, w = whole_problem(T + d, T, d, E, k, I)
    idx, tw = ids(T, T, k, lo, hi), torch.rand(T, k, generator=gen(3), device="cuda")
    tw[(idx < 0) | (idx >= E)] = float("nan")  # not read
    y_add = randn(4, (T, d)) if add else None
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w, y_add)
    want, bound = reference(x, xs, idx, tw, w, E, y_add, exact_gu=True)
    got = np64(y)
    assert np.all(np.abs(got - want) <= bound), np.abs(got - want).max()
    gone = ((idx < 0) | (idx >= E)).all(1)
    assert torch.equal(y[gone], y_add[gone] if add else torch.zeros_like(y[gone]))


@pytest.mark.parametrize("T,d,E,k,I", [(1, 2048, 8, 6, 768), (3, 1024, 4, 2, 512), (20, 512, 6, 3, 640)])
def test_routed_ffn_real_values(T, d, E, k, I):
    """Normally distributed tokens and weights, in the 2-norm.  G and U are off
    by at most 2^-11 of themselves in the mean (products cut at 2^-13 of their
    group's largest), h by about as much; a share of at most 2 * 2^-11 / 2^-4 of
    its elements rounds the other way, each by at most 2^-3 of itself: sqrt(2^-6)
    2^-3 = 2^-6.  With y's rounding, 2^-8, 2e-2."""
    x, xs, w = real_problem(T, T, d, E, k, I)
    idx, tw = ids(T, T, k, 0, E), torch.rand(T, k, generator=gen(3), device="cuda")
    add = randn(4, (T, d))
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w, add)
    want, _ = reference(x, xs, idx, tw, w, E, add, bound=False)
    assert np.linalg.norm(np64(y) - want) <= 2e-2 * np.linalg.norm(want)


@pytest.mark.parametrize("T,E,k", [(9, 5, 3), (40, 16, 4), (150, 3, 2), (700, 8, 4)])
def test_routed_ffn_token_alone_gives_the_same_bits(T, E, k):
    d, I = 512, 384
    x, xs, w = real_problem(7, T, d, E, k, I)
    idx, tw = ids(1, T, k, -1, E + 1), torch.rand(T, k, generator=gen(2), device="cuda")
    add = randn(3, (T, d))
    y = M.routed_ffn_mxfp4(x, xs, idx, tw, w, M.Dims(T, d, E, k, I), add)
    one = M.RoutedFfnPlan(M.Dims(1, d, E, k, I))
    for t in (0, 1, T // 2, T - 1):
        s = slice(t, t + 1)
        assert torch.equal(one.run(x[s], xs[s], idx[s], tw[s], w, add[s]), y[s]), t
    order = torch.randperm(T, generator=gen(4), device="cuda")
    part = order[:T // 2]
    z = M.routed_ffn_mxfp4(x[part], xs[part], idx[part], tw[part], w, M.Dims(T // 2, d, E, k, I), add[part])
    assert torch.equal(z, y[part])
    # in place: y_add is the output
    plan = M.RoutedFfnPlan(M.Dims(T, d, E, k, I))
    plan.y.copy_(add)
    assert torch.equal(plan.run(x, xs, idx, tw, w, plan.y), y)


def test_routed_ffn_same_id_twice_and_many_ids():
    d, I, E, T, k = 256, 128, 2, 5, 16
    x, xs, w = whole_problem(3, T, d, E, k, I)
    idx = ids(4, T, k, 0, E)
    tw = torch.rand(T, k, generator=gen(5), device="cuda")
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w)
    want, bound = reference(x, xs, idx, tw, w, E, exact_gu=True)
    assert np.all(np.abs(np64(y) - want) <= bound)


def test_routed_ffn_all_routes_absent_and_empty_batch():
    d, I, E, T, k = 128, 128, 4, 6, 2
    x, xs, w = whole_problem(3, T, d, E, k, I)
    x[:] = 0x7F  # NaN
    idx = torch.tensor([[-1, E], [-(1 << 31), (1 << 31) - 1]] * 3, dtype=I32, device="cuda")
    tw = torch.full((T, k), float("inf"), device="cuda")
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w)
    assert bool((y == 0).all())
    add = randn(1, (T, d))
    assert torch.equal(M.routed_ffn_mxfp4(x, xs, idx, tw, w, M.Dims(T, d, E, k, I), add), add)
    none = M.Dims(0, d, E, k, I)
    assert M.routed_ffn_mxfp4(x[:0], xs[:0], idx[:0], tw[:0], w, none).shape == (0, d)


def test_routed_ffn_nan_of_one_token_stays_with_it():
    d, I, E, T, k = 256, 128, 3, 20, 2
    x, xs, w = real_problem(5, T, d, E, k, I)
    idx, tw = ids(1, T, k, 0, E), torch.rand(T, k, generator=gen(2), device="cuda")
    dims = M.Dims(T, d, E, k, I)
    y = M.routed_ffn_mxfp4(x, xs, idx, tw, w, dims)
    x2 = x.clone()
    x2[7] = 0x7F
    y2 = M.routed_ffn_mxfp4(x2, xs, idx, tw, w, dims)
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(y2[keep], y[keep])


def test_routed_ffn_on_another_stream_and_captured():
    T, d, E, k, I = 6, 512, 8, 3, 256
    x, xs, w = real_problem(9, T, d, E, k, I)
    idx, tw = ids(1, T, k, -1, E), torch.rand(T, k, generator=gen(2), device="cuda")
    dims = M.Dims(T, d, E, k, I)
    y = M.routed_ffn_mxfp4(x, xs, idx, tw, w, dims).clone()
    plan, s = M.RoutedFfnPlan(dims), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = plan.run(x, xs, idx, tw, w)
    s.synchronize()
    assert torch.equal(got, y)
    # captured with its inputs in fixed buffers; every replay on new contents
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.run(x, xs, idx, tw, w)
    for i in range(4):
        x.copy_(M.quantize_mxfp8(randn(20 + i, (T, d)), 0)[0])
        idx.copy_(ids(30 + i, T, k, -1, E))
        graph.replay()
        torch.cuda.synchronize()
        kept = plan.y.clone()
        eager = M.routed_ffn_mxfp4(x, xs, idx, tw, w, dims)
        assert torch.equal(kept, eager), i


def test_wrappers_refuse_other_tensors():
    T, d, E, k, I = 2, 128, 2, 1, 128
    x, xs, w = whole_problem(1, T, d, E, k, I)
    idx, tw = ids(1, T, k, 0, E), torch.rand(T, k, device="cuda")
    plan = M.RoutedFfnPlan(M.Dims(T, d, E, k, I))
    for bad in ((x[:1], xs, idx, tw, w), (x.float(), xs, idx, tw, w), (x, xs[:, :2], idx, tw, w),
                (x, xs, idx.long(), tw, w), (x, xs, idx, tw.half(), w), (x.cpu(), xs, idx, tw, w),
                (x, xs, idx, tw, M.WeightsMxfp4(**dict(vars(w), q_up=w.q_up[:1]))),
                (x, xs, idx, tw, M.WeightsMxfp4(**dict(vars(w), q_down_scale=None)))):
        with pytest.raises(ValueError):
            plan.run(*bad)
    with pytest.raises(ValueError):
        plan.run(x, xs, idx, tw, w, y_add=torch.zeros(T, d, device="cuda"))
    with pytest.raises(ValueError):
        M.quantize_mxfp4(randn(1, (4, 100)))
    with pytest.raises(ValueError):
        M.quantize_mxfp4(randn(1, (128, 128)).t()[:, ::1].float())
    with pytest.raises(ValueError):
        M.dequantize_mxfp4(w.q_gate[0], w.q_gate_scale)
