"""Variants, limits and long tensors of the operators that serve the layer in
8 and 4 bits."""
import numpy as np
import pytest

import mixture_experts_layer_prefix_amd as M
from mixture_experts_layer_prefix_amd import _lib as L

torch = pytest.importorskip("torch")
from tests import block_ref as B  # noqa: E402
from tests.test_gpu_mx_ops import (BF, F32, I32, U8, gen, ids, np64, poisoned, randn, real_problem, reference,  # noqa: E402
                                   whole_problem)

pytestmark = pytest.mark.gpu


def used_experts(w, idx, E, dims):
    """The weights of the experts that idx names, and idx in their numbers."""
    names = sorted({int(e) for e in idx.reshape(-1).tolist() if 0 <= e < E})
    at = torch.tensor(names, device="cuda")
    part = {}
    for n, t in vars(w).items():
        part[n] = (t.view(t.shape[0], E, -1, 4)[:, at].reshape(t.shape[0], -1, 4) if n.endswith("scale")
                   else t[at]).contiguous()
    return M.WeightsMxfp4(**part), torch.tensor([[names.index(e) for e in row] for row in idx.tolist()], dtype=I32), names


# tokens in tiles of 32 with 128 weight rows a workgroup, whole and shared by
# several workgroups; odd numbers of slabs; sixteen routes of one token
@pytest.mark.parametrize("T,d,E,k,I,lo,hi", [
    (70, 384, 64, 4, 640, 0, 64), (300, 256, 4, 2, 2048, -1, 5), (140, 128, 70, 8, 512, -9, 78),
    (1, 256, 20, 16, 384, 0, 20), (1, 128, 3, 16, 128, -2, 5), (3, 1152, 24, 8, 896, 0, 24), (16, 128, 1, 1, 128, 0, 1),
    (17, 128, 2, 1, 128, 0, 1), (4, 256, 5, 4, 128, 0, 5)])
def test_routed_ffn_variants_whole_numbers(T, d, E, k, I, lo, hi):
    x, xs, w = whole_problem(T + I, T, d, E, k, I)
    idx, tw = ids(T + 1, T, k, lo, hi), torch.rand(T, k, generator=gen(3), device="cuda")
    add = randn(4, (T, d))
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w, add)
    want, bound = reference(x, xs, idx, tw, w, E, add, exact_gu=True)
    off = np.abs(np64(y) - want)
    assert np.all(off <= bound), (off / bound).max()


def test_routed_ffn_many_experts_by_expert():
    """As many routes as experts, whose shared experts outweigh a schedule.
    Bits of a token alone, and a token's numbers."""
    T, d, E, k, I = 64, 1024, 512, 8, 1024
    x, xs, w = real_problem(11, T, d, E, k, I)
    idx, tw = ids(5, T, k, 0, E), torch.rand(T, k, generator=gen(2), device="cuda")
    idx[3] = idx[2]
    idx[7, 2:5] = -1
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w)
    one = M.RoutedFfnPlan(M.Dims(1, d, E, k, I))
    for t in (0, 2, 3, 7, 63):
        s = slice(t, t + 1)
        assert torch.equal(one.run(x[s], xs[s], idx[s], tw[s], w), y[s]), t
    few, mine, names = used_experts(w, idx[:1], E, None)
    want, _ = reference(x[:1], xs[:1], mine, tw[:1], few, len(names), bound=False)
    assert np.linalg.norm(np64(y[:1]) - want) <= 2e-2 * np.linalg.norm(want)  # as in test_routed_ffn_real_values


def test_routed_ffn_experts_beyond_4_gb():
    """Codes of the last experts begin past 2^32 bytes."""
    T, d, E, k, I = 3, 7168, 620, 2, 2048
    assert (E - 2) * I * d // 2 > 1 << 32
    few_x, few_s, few = whole_problem(2, T, d, 2, k, I)
    big = {}
    for n, t in vars(few).items():
        if n.endswith("scale"):
            v = torch.full((t.shape[0], E * (t.shape[1] // 2), 4), 127, dtype=U8, device="cuda")
            v[:, -t.shape[1]:] = t
        else:
            v = torch.zeros(E, *t.shape[1:], dtype=U8, device="cuda")
            v[-2:] = t
        big[n] = v
    idx = torch.tensor([[0, 1], [1, 0], [1, -1]], dtype=I32, device="cuda")
    tw = torch.rand(T, k, generator=gen(3), device="cuda")
    want = M.routed_ffn_mxfp4(few_x, few_s, idx, tw, few, M.Dims(T, d, 2, k, I))
    far = torch.where(idx >= 0, idx + E - 2, idx)
    for t in (T, 1):
        got = M.routed_ffn_mxfp4(few_x[:t], few_s[:t], far[:t], tw[:t], M.WeightsMxfp4(**big), M.Dims(t, d, E, k, I))
        assert torch.equal(got, want[:t])


@pytest.mark.parametrize("T,d,E,k,I", [(600, 256, 8, 1, 128), (700, 128, 900, 1, 256), (1500, 128, 40, 1, 128)])
def test_routed_ffn_every_token_at_one_expert(T, d, E, k, I):
    """More tokens at one expert than its share of the workgroups takes at a
    time, with a schedule and without."""
    x, xs, w = whole_problem(T, T, d, E, k, I)
    idx = torch.full((T, k), E // 2, dtype=I32, device="cuda")
    tw = torch.rand(T, k, generator=gen(3), device="cuda")
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w)
    few, mine, names = used_experts(w, idx, E, None)
    want, bound = reference(x, xs, mine, tw, few, len(names), exact_gu=True)
    off = np.abs(np64(y) - want)
    assert np.all(off <= bound), (off / bound).max()


def test_routed_ffn_128_routes_by_expert():
    """Without a schedule, found by whole workgroups, down by expert."""
    T, d, E, k, I = 16, 1280, 130, 8, 1280
    x, xs, w = real_problem(17, T, d, E, k, I)
    idx, tw = ids(5, T, k, 0, E), torch.rand(T, k, generator=gen(2), device="cuda")
    idx[3] = idx[2]
    idx[7, 2:5] = -1
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w)
    one = M.RoutedFfnPlan(M.Dims(1, d, E, k, I))
    for t in range(T):
        s = slice(t, t + 1)
        assert torch.equal(one.run(x[s], xs[s], idx[s], tw[s], w), y[s]), t


def test_routed_ffn_nearly_every_token_at_one_expert():
    T, d, E, k, I = 512, 1024, 512, 1, 1024
    x, xs, w = real_problem(13, T, d, E, k, I)
    idx = torch.full((T, k), 77, dtype=I32, device="cuda")
    idx[100:110] = 3
    tw = torch.rand(T, k, generator=gen(2), device="cuda")
    y = poisoned(M.Dims(T, d, E, k, I)).run(x, xs, idx, tw, w)
    one = M.RoutedFfnPlan(M.Dims(1, d, E, k, I))
    for t in (0, 15, 16, 99, 105, 300, 511):
        s = slice(t, t + 1)
        assert torch.equal(one.run(x[s], xs[s], idx[s], tw[s], w), y[s]), t


def test_plans_write_the_tensors_that_they_hold():
    """A plan's output may be replaced by another tensor of its shape between
    two calls."""
    T, d, E, k, I = 6, 256, 4, 2, 128
    x, xs, w = real_problem(3, T, d, E, k, I)
    idx, tw = ids(1, T, k, -1, E), torch.rand(T, k, generator=gen(2), device="cuda")
    res, out = randn(1, (T, d)), randn(2, (T, d))
    plans = [M.BlockNormMxfp8Plan(M.Block(T, d)), M.SortMxfp8Plan(M.Dims(T, d, E, k, 1)),
             M.RoutedFfnPlan(M.Dims(T, d, E, k, I))]
    calls = [lambda p: p.run(res, out), lambda p: p.run(idx, x, xs), lambda p: (p.run(x, xs, idx, tw, w),)]
    for plan, run in zip(plans, calls):
        if hasattr(plan, "x_perm"):
            for t in (plan.row_token, plan.x_perm, plan.x_perm_scale):
                t.zero_()
        first = [t.clone() for t in run(plan)]
        for name, t in list(vars(plan).items()):
            if torch.is_tensor(t) and name != "ws":
                setattr(plan, name, torch.zeros_like(t))
        assert all(torch.equal(a, b) for a, b in zip(run(plan), first)), type(plan).__name__


def test_two_plans_at_once():
    T, d, E, k, I = 40, 512, 8, 3, 256
    x, xs, w = real_problem(9, T, d, E, k, I)
    dims = M.Dims(T, d, E, k, I)
    tw = torch.rand(T, k, generator=gen(2), device="cuda")
    many = [ids(i, T, k, -1, E) for i in range(6)]
    want = [M.routed_ffn_mxfp4(x, xs, i, tw, w, dims) for i in many]
    plans, streams = [M.RoutedFfnPlan(dims) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for n, i in enumerate(many):
        with torch.cuda.stream(streams[n % 2]):
            got.append(plans[n % 2].run(x, xs, i, tw, w).clone())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_routed_ffn_inputs_are_left_alone():
    T, d, E, k, I = 5, 256, 4, 2, 128
    x, xs, w = real_problem(3, T, d, E, k, I)
    idx, tw, add = ids(1, T, k, -1, E), torch.rand(T, k, device="cuda"), randn(2, (T, d))
    keep = [t.clone() for t in (x, xs, idx, tw, add, *vars(w).values())]
    M.routed_ffn_mxfp4(x, xs, idx, tw, w, M.Dims(T, d, E, k, I), add)
    assert all(torch.equal(a, b) for a, b in zip(keep, (x, xs, idx, tw, add, *vars(w).values())))


def test_addresses_that_are_not_aligned_are_refused():
    T, d, E, k, I = 2, 128, 2, 1, 128
    x, xs, w = whole_problem(1, T, d, E, k, I)
    idx, tw = ids(1, T, k, 0, E), torch.rand(T, k, device="cuda")
    odd = torch.zeros(T * d + 8, dtype=U8, device="cuda")[8:].view(T, d)
    with pytest.raises(L.MoeError):
        M.routed_ffn_mxfp4(odd, xs, idx, tw, w, M.Dims(T, d, E, k, I))
    with pytest.raises(L.MoeError):
        M.sort_tokens_mxfp8(idx, odd, xs, M.Dims(T, d, E, k, 1))
    with pytest.raises(L.MoeError):
        M.quantize_mxfp4(torch.zeros(T * d + 4, dtype=BF, device="cuda")[4:].view(T, d))
    with pytest.raises(L.MoeError):
        M.dequantize_mxfp4(torch.zeros(T * 64 + 4, dtype=U8, device="cuda")[4:].view(T, 64),
                           torch.zeros(1, T, 4, dtype=U8, device="cuda"))


def test_norm_takes_rows_at_odd_addresses():
    """Only the codes need 16 bytes: x and y may begin at any element."""
    T, d = 3, 96
    x, y = (torch.cat([torch.zeros(1, dtype=BF, device="cuda"), randn(i, (T * d,))])[1:].view(T, d) for i in (1, 2))
    b = M.Block(T, d)
    _, q, s, plan = M.block_norm_mxfp8(b, x, y)
    _, q2, s2, _ = M.block_norm_mxfp8(b, x.clone(), y.clone())
    assert torch.equal(q, q2) and torch.equal(s, s2)


# ---- long tensors ----------------------------------------------------------
def test_norm_rows_beyond_2_31_elements():
    T, d = 262200, 8192
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    tail = randn(1, (40, d))
    x[-40:] = tail
    _, q, s, _ = M.block_norm_mxfp8(M.Block(T, d), x, keep_a=False)
    _, q2, s2, _ = M.block_norm_mxfp8(M.Block(40, d), tail, keep_a=False)
    assert torch.equal(q[-40:], q2) and torch.equal(s[-40:], s2) and not bool(q[:100].any())


@pytest.mark.parametrize("T,d", [(40000, 7168), (1800, 7168)])
def test_sort_of_streamed_rows(T, d):
    """Rows that are written with the streaming hint; in the larger case past
    2^31 bytes."""
    E, k = 64, 8
    idx = ids(T, T, k, -1, E)
    x = torch.randint(0, 256, (T, d), generator=gen(1), device="cuda", dtype=U8)
    xs = torch.randint(0, 256, (T, d // 32), generator=gen(2), device="cuda", dtype=U8)
    counts, offsets, row_token, token_row, x_perm, x_perm_scale = M.sort_tokens_mxfp8(idx, x, xs, M.Dims(T, d, E, k, 1))
    n = int(offsets[-1])
    c2, o2, r2, t2, _ = M.sort_tokens(idx, None, M.Dims(T, d, E, k, 1), "bf16", gather=False)
    assert torch.equal(counts, c2) and torch.equal(token_row, t2) and torch.equal(row_token[:n], r2[:n])
    for a in range(0, n, 65536):
        s = slice(a, min(a + 65536, n))
        src = row_token[s].long()
        assert torch.equal(x_perm[s], x[src]) and torch.equal(x_perm_scale[s], xs[src])


def test_quantize4_beyond_2_31_elements():
    rows, cols = 300000, 7168
    w = torch.zeros(rows, cols, dtype=BF, device="cuda")
    tail = randn(1, (33, cols))
    w[-33:] = tail
    codes, scale = M.quantize_mxfp4(w)
    c2, s2 = M.quantize_mxfp4(tail)
    assert torch.equal(codes[-33:], c2) and torch.equal(scale[:, -33:], s2) and not bool(codes[:64].any())
    back = M.dequantize_mxfp4(codes, scale)
    assert torch.equal(back[-33:], M.dequantize_mxfp4(c2, s2)) and not bool(back[:64].any())


def test_norm_and_sort_captured_and_replayed():
    """Norm, sort and the rounding of weights in a graph, on new contents
    beside eager work."""
    T, d, E, k = 50, 256, 8, 3
    b, D = M.Block(T, d, res_f32=True, post_norm=True), M.Dims(T, d, E, k, 1)
    x, y, idx, w = randn(1, (T, d), F32), randn(2, (T, d)), ids(3, T, k, -1, E), randn(4, (64, d))
    norm, sort = M.BlockNormMxfp8Plan(b), M.SortMxfp8Plan(D)
    sort.x_perm.zero_(), sort.x_perm_scale.zero_()

    def step():
        x1, q, s = norm.run(x, y)
        return [x1, q, s, norm.a, *sort.run(idx, q, s), *M.quantize_mxfp4(w)]

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(randn(10 + i, (T, d), F32))
        idx.copy_(ids(20 + i, T, k, -1, E))
        w.copy_(randn(30 + i, (64, d)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        x1, q, s, plan = M.block_norm_mxfp8(b, x, y)
        eager = [x1, q, s, plan.a, *M.sort_tokens_mxfp8(idx, q, s, D), *M.quantize_mxfp4(w)]
        n = int(eager[5][-1])
        for j, (a, e) in enumerate(zip(got, eager)):
            a, e = (a[:n], e[:n]) if j in (6, 8, 9) else (a, e)
            assert torch.equal(a, e), (i, j)
