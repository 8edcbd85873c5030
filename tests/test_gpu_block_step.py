"""The operators around the layer together with it, as a program runs them:
a residual block trained for one step (norm, layer, norm with gate and
residual, their gradients, clipping), one token decoded through the same
block, and the layer's experts split over two ranks by the sort with absent
routes."""
import numpy as np
import pytest

import gen
import mixture_experts_layer_prefix_amd as M
from oracle import moe_oracle as O
from tests.moe_parity import TOL, device_problem, rel_err, to_np

torch = pytest.importorskip("torch")
from tests import block_ref as B  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 1e-6


def randn(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def block_parts(D):
    p, t, md, w = device_problem(D)
    d, bf, f32 = D.d, torch.bfloat16, torch.float32
    own = dict(x=randn(1, (D.T, d), f32), w_in=1 + randn(2, (d,), f32, 0.1), w_post=1 + randn(3, (d,), f32, 0.1),
               gate=randn(4, ((D.T + 99) // 100, d), f32), w_next=1 + randn(5, (d,), f32, 0.1),
               dx_out=randn(6, (D.T, d), f32), da=randn(7, (D.T, d), bf))
    first = M.Block(D.T, d, "bf16", res_f32=True, eps=EPS)
    step = M.Block(D.T, d, "bf16", res_f32=True, post_norm=True, alpha=0.75, beta=0.5, eps=EPS, gate_every=100)
    return p, t, md, w, own, first, step


def oracle_args(p):
    h = {n: p.host(n) for n in ("w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")}
    return (h["w_router"], p.logit_bias(), h["w_gate"], h["w_up"], h["w_down"], h["ws_gate"], h["ws_up"], h["ws_down"],
            p.dims.k)


def test_training_step_of_a_block():
    D = gen.Dims("block_step", 300, 256, 16, 4, 192, 1, 128, "bf16", 1.2)
    p, t, md, w, o, first, step = block_parts(D)
    # forward
    x, a, plan0 = M.block_norm(first, o["x"], w_pre=o["w_in"])
    y, routing = M.layer_forward(a, w, md, "bf16", bias=t["bias"], keep_gu=True)
    x1, a1, plan1 = M.block_norm(step, x, y, o["w_next"], o["w_post"], o["gate"])
    # backward of <x1, dx_out> + <a1, da>
    dx, dy, g1 = M.block_norm_backward(step, o["dx_out"], o["da"], x1, y, plan1.r_pre, plan1.r_post, o["w_next"],
                                       o["w_post"], o["gate"])
    da, grads = M.layer_backward(dy, a, M.prepare_backward(w), routing, md, "bf16")
    dx, none, g0 = M.block_norm_backward(first, dx, da, x, None, plan0.r_pre, None, o["w_in"])
    assert none is None
    every = list(grads.values()) + list(g0.values()) + list(g1.values())
    norm = M.grad_norm(every)
    keep = [v.clone() for v in every]
    M.clip_grads(every, 1.0)
    # the oracle: the layer on the same normalized tokens, everything else in 64 bits
    ah = B.f64(a).numpy()
    ref = B.norm_fwd_ref(o["x"], None, None, None, o["w_in"], 100, 1, 1, EPS, False)
    assert rel_err(to_np(a), ref["a"].numpy()) <= 2.0 ** -8
    fw = O.layer_forward(ah, *oracle_args(p))
    assert np.array_equal(routing["topk_idx"].cpu().numpy(), fw["topk_idx"])
    yr = torch.from_numpy(fw["y"])
    n1 = B.norm_fwd_ref(o["x"], yr, o["w_post"], o["gate"], o["w_next"], 100, 0.75, 0.5, EPS, True)
    tol = TOL["bf16"]
    assert rel_err(to_np(x1), n1["x_out"].numpy()) <= tol and rel_err(to_np(a1), n1["a"].numpy()) <= tol
    b1 = B.norm_bwd_ref(o["dx_out"], o["da"], n1["x_out"], yr, n1["r_post"], n1["r_pre"], o["w_post"], o["gate"],
                        o["w_next"], 100, 0.75, 0.5, True)
    bl = O.layer_backward(ah, *oracle_args(p), b1["dy"].numpy())
    b0 = B.norm_bwd_ref(b1["dx"], torch.from_numpy(bl["dx"]), o["x"], None, None, ref["r_pre"], None, None, o["w_in"],
                        100, 1, 1, False)
    for n, got, want in [("dx", dx, b0["dx"]), ("dw_in", g0["dw_pre"], b0["dw_pre"]),
                         ("dw_next", g1["dw_pre"], b1["dw_pre"]), ("dw_post", g1["dw_post"], b1["dw_post"]),
                         ("dgate", g1["dgate"], b1["dgate"])]:
        got = keep[[v is got for v in every].index(True)] if n != "dx" else got
        assert rel_err(to_np(got), want.numpy()) <= tol, n
    # the clipped gradients: the norm of what was there, each scaled by it
    ss = sum(B.f64(v).pow(2).sum() for v in keep)
    assert abs(float(norm) - float(ss.sqrt())) <= float(ss.sqrt()) * 2.0 ** -23 and float(norm) > 1.0
    for v, k in zip(every, keep):
        want = B.f64(k) / (float(norm) + 1e-6)
        B.check("clipped", v, want, want.abs(), 3)


def test_one_token_through_the_block():
    """A decoded token gives what it gives inside a batch."""
    D = gen.Dims("block_token", 64, 256, 16, 4, 192, 1, 128, "bf16", 0.0)
    _, t, md, w, o, first, step = block_parts(D)
    x, a, _ = M.block_norm(first, o["x"], w_pre=o["w_in"])
    y, _ = M.layer_forward(a, w, md, "bf16", bias=t["bias"])
    x1, a1, _ = M.block_norm(step, x, y, o["w_next"], o["w_post"], o["gate"])
    one_d = M.Dims(1, D.d, D.E, D.k, D.I, D.S, D.Is)
    for i in (0, 17, 63):
        s = slice(i, i + 1)
        b0 = M.Block(1, D.d, "bf16", res_f32=True, eps=EPS)
        b1 = M.Block(1, D.d, "bf16", res_f32=True, post_norm=True, alpha=0.75, beta=0.5, eps=EPS)
        xs, ai, _ = M.block_norm(b0, o["x"][s], w_pre=o["w_in"])
        assert torch.equal(ai, a[s])
        yi, _ = M.layer_forward(ai, w, one_d, "bf16", bias=t["bias"])
        xi, ni, _ = M.block_norm(b1, xs, yi, o["w_next"], o["w_post"], o["gate"][:1])
        assert torch.equal(yi, y[s]) and torch.equal(xi, x1[s]) and torch.equal(ni, a1[s])


def test_experts_split_over_two_ranks():
    """Each rank holds half of the experts: routes of the other half are
    absent from its sort.  The ranks' weighted sums add up to the layer's
    output, and their gradients to the layer's."""
    D = gen.Dims("block_ranks", 500, 256, 16, 4, 192, 0, 0, "bf16", 1.2)
    p, t, md, w = device_problem(D)
    x, half = t["x"], D.E // 2
    y, routing = M.layer_forward(x, w, md, "bf16", bias=t["bias"])
    h = {n: p.host(n) for n in ("w_router", "w_gate", "w_up", "w_down")}
    ref = O.layer_backward(p.host("x"), h["w_router"], p.logit_bias(), h["w_gate"], h["w_up"], h["w_down"], None, None,
                           None, D.k, p.host("dy"), with_router=False)
    dy = p.device("dy")
    total, dx, dw = None, None, torch.zeros(D.T, D.k, device="cuda")
    for rank in range(2):
        e0 = rank * half
        local = M.Dims(D.T, D.d, half, D.k, D.I)
        mine = M.Weights(w_router=t["w_router"], **{n: t[n][e0:e0 + half].contiguous()
                                                    for n in ("w_gate", "w_up", "w_down")})
        idx = routing["topk_idx"] - e0
        counts, offsets, _, token_row, x_perm = M.sort_tokens(idx, x, local, "bf16")
        o_perm = M.expert_ffn(x_perm, None, offsets, mine, local, "bf16")
        # the second rank adds the first one's share
        total = M.unsort_tokens(o_perm, token_row, routing["topk_w"], total, local, "bf16", y=total)
        do, part = M.unsort_tokens_backward(dy, o_perm, token_row, routing["topk_w"], local, "bf16")
        dw += part  # zero where the other rank has the route
        # the experts' input gradient in 64 bits, row by row
        da = torch.zeros_like(do)
        off = offsets.tolist()
        for e in range(half):
            r = slice(off[e], off[e + 1])
            if r.stop > r.start:
                a = B.f64(x_perm[r]).requires_grad_()
                g, u = (a @ torch.from_numpy(h[n][e0 + e]).T for n in ("w_gate", "w_up"))
                out = (torch.nn.functional.silu(g) * u) @ torch.from_numpy(h["w_down"][e0 + e]).T
                out.backward(B.f64(do[r]))
                da[r] = a.grad.to(da)
        dx = M.sort_tokens_backward(da, token_row, dx, local, "bf16", dx=dx)
        assert int(counts.sum()) == off[-1] < D.T * D.k
    tol = TOL["bf16"]
    assert rel_err(to_np(total), to_np(y)) <= tol
    assert rel_err(to_np(dw), ref["dtopk_w"]) <= tol
    assert rel_err(to_np(dx), ref["dx"]) <= tol
