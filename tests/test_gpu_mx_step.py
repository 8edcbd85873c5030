"""The operators that serve the layer in 8 and 4 bits together, as a program
runs them: a block's norm gives codes, which the routed experts take in 4 bits
for a few tokens, or sorted through the grouped products in MXFP8 for many;
the next norm takes the sum."""
import numpy as np
import pytest

import mixture_experts_layer_prefix_amd as M

torch = pytest.importorskip("torch")
from tests.test_gpu_mx_ops import BF, F32, np64, randn, reference  # noqa: E402
from tests import block_ref as B  # noqa: E402

pytestmark = pytest.mark.gpu
E, k, d, I, Is = 8, 3, 512, 256, 256
EPS = 1e-6


def layer():
    w = {n: randn(10 + i, s, BF, s[-1] ** -0.5) for i, (n, s) in enumerate((
        ("w_router", (E, d)), ("w_gate", (E, I, d)), ("w_up", (E, I, d)), ("w_down", (E, d, I)),
        ("ws_gate", (1, Is, d)), ("ws_up", (1, Is, d)), ("ws_down", (1, d, Is))))}
    return M.Weights(**w)


def dims(T, E=E):
    return M.Dims(T, d, E, k, I, 1, Is)


def block_step(x, weights, w4, w_in, w_next, T):
    """Residual x [T][d] fp32 through norm, router, shared and routed experts
    and the next norm: (x', a' codes, scales, routing, y)."""
    D = dims(T)
    first, step = M.Block(T, d, "bf16", res_f32=True, eps=EPS), M.Block(T, d, "bf16", res_f32=True, beta=0.5, eps=EPS)
    _, q, s, plan = M.block_norm_mxfp8(first, x, w_pre=w_in)
    _, idx, tw = M.route(plan.a, weights.w_router, D, "bf16")
    shared = M.shared_ffn(plan.a, weights, D, "bf16")
    y = M.routed_ffn_mxfp4(q, s, idx, tw, w4, D, y_add=shared)
    x1, q1, s1, next_plan = M.block_norm_mxfp8(step, x, y, w_pre=w_next)
    return x1, q1, s1, next_plan.a, (plan.a, q, s, idx, tw, shared, y)


def test_decoded_tokens_through_the_block():
    T = 6
    weights = layer()
    w4 = M.prepare_mxfp4(weights, dims(T))
    x, w_in, w_next = randn(1, (T, d), F32), 1 + randn(2, (d,), F32, 0.1), 1 + randn(3, (d,), F32, 0.1)
    x1, q1, s1, a1, (a, q, s, idx, tw, shared, y) = block_step(x, weights, w4, w_in, w_next, T)
    want, _ = reference(q, s, idx, tw, w4, E, shared, bound=False)
    assert np.linalg.norm(np64(y) - want) <= 2e-2 * np.linalg.norm(want)
    ref = B.norm_fwd_ref(x, torch.from_numpy(want), None, None, w_next, T, 1, 0.5, EPS, False)
    # half of y's error arrives in x' (beta), beside which x is as large
    for got, exact in ((x1, ref["x_out"]), (a1, ref["a"])):
        off = np.linalg.norm(np64(got) - exact.numpy())
        assert off <= 2e-2 * np.linalg.norm(exact.numpy())
    # each token alone gives the same bits
    for t in range(T):
        one = block_step(x[t:t + 1], weights, w4, w_in, w_next, 1)
        assert torch.equal(one[0], x1[t:t + 1]) and torch.equal(one[1], q1[t:t + 1]) and torch.equal(one[2], s1[t:t + 1])


def test_many_tokens_through_the_grouped_products_agree():
    """The same weights and codes through sort, expert_ffn in MXFP8 and unsort:
    E2M1 values are E4M3 values, so the weights are the same numbers.  The
    grouped form rounds o to bf16 (2^-8); both round h to 8 bits, a share of
    2^-6 of whose elements may go either way in each (2^-6 in the norm each)."""
    T = 200
    weights = layer()
    D = dims(T)
    w4 = M.prepare_mxfp4(weights, D)
    a = randn(1, (T, d))
    _, q, s, plan = M.block_norm_mxfp8(M.Block(T, d), a)
    _, idx, tw = M.route(plan.a, weights.w_router, D, "bf16")
    idx[::7, 1] = -1  # dropped routes
    y = M.routed_ffn_mxfp4(q, s, idx, tw, w4, D)
    back = {}
    for n in ("gate", "up", "down"):
        codes = getattr(w4, "q_" + n)
        back["w_" + n] = M.dequantize_mxfp4(codes.view(-1, codes.shape[-1]), getattr(w4, "q_%s_scale" % n)).view(
            E, codes.shape[1], -1)
    w8 = M.prepare_mxfp8(M.Weights(weights.w_router, **back), D)
    _, offsets, _, token_row, x_perm, x_perm_scale = M.sort_tokens_mxfp8(idx, q, s, D)
    o = M.expert_ffn(x_perm, x_perm_scale, offsets, w8, D, "mxfp8")
    z = M.unsort_tokens(o, token_row, tw, None, D, "bf16")
    y, z = np64(y), np64(z)
    assert np.linalg.norm(y - z) <= (2 * 2.0 ** -6 + 2 * 2.0 ** -8) * np.linalg.norm(z)


def test_experts_split_over_two_ranks_in_4_bits():
    """Each rank holds half of the experts and adds its share to the other's."""
    T, half = 9, E // 2
    weights = layer()
    w4 = M.prepare_mxfp4(weights, dims(T))
    _, q, s, plan = M.block_norm_mxfp8(M.Block(T, d), randn(1, (T, d)))
    _, idx, tw = M.route(plan.a, weights.w_router, dims(T), "bf16")
    whole = M.routed_ffn_mxfp4(q, s, idx, tw, w4, dims(T))
    total = None
    for e0 in (0, half):
        part = {}
        for n, t in vars(w4).items():
            part[n] = (t.view(t.shape[0], E, -1, 4)[:, e0:e0 + half].reshape(t.shape[0], -1, 4) if n.endswith("scale")
                       else t[e0:e0 + half]).contiguous()
        total = M.routed_ffn_mxfp4(q, s, idx - e0, tw, M.WeightsMxfp4(**part), dims(T, half), y_add=total)
    # the sum of the shares is rounded once more, after the first rank
    a, b = np64(total), np64(whole)
    assert np.all(np.abs(a - b) <= 2.0 ** -7 * (np.abs(a) + np.abs(b)) + 2.0 ** -8 * np.abs(b).max())


def test_decode_step_captured_and_replayed():
    """A step of two tokens in a graph, replayed on new residuals beside eager
    work."""
    T = 2
    weights = layer()
    w4 = M.prepare_mxfp4(weights, dims(T))
    w_in, w_next = 1 + randn(2, (d,), F32, 0.1), 1 + randn(3, (d,), F32, 0.1)
    x = randn(1, (T, d), F32)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block_step(x, weights, w4, w_in, w_next, T)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block_step(x, weights, w4, w_in, w_next, T)
    for i in range(4):
        x.copy_(randn(40 + i, (T, d), F32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out[:4]]
        eager = block_step(x, weights, w4, w_in, w_next, T)
        assert all(torch.equal(a, b) for a, b in zip(got, eager[:4])), i
