"""The operators around the layer on the GPU where a workgroup takes many
rows, groups span several teams of rows, rows are streamed, or a list of
tensors leaves more partial sums than one launch adds up."""
import pytest

import mixture_experts_layer_prefix_amd as M

torch = pytest.importorskip("torch")
from tests import block_ref as B  # noqa: E402
from tests.test_gpu_block_ops import PRECS, TYPES, gen, norm_inputs, randn, unsort_inputs  # noqa: E402

pytestmark = pytest.mark.gpu

ROW = 2 * B.ROW_SUM + 16  # two row sums and a dozen products, as for a few rows


# ---- block norm: several rows a team ---------------------------------------
def check_both_directions(block, p, every, seed, col):
    """Forward and backward against the 64-bit references; col: roundings of a
    sum over tokens."""
    T, d, alpha, beta, post = block.T, block.d, block.alpha, block.beta, block.post_norm
    args = (p["x"], p["y"], p["w_post"], p["gate"], p["w_pre"], block.every, alpha, beta, block.eps, post)
    ref, mag = B.norm_fwd_ref(*args), B.norm_fwd_ref(*args, magnitude=True)
    x_out, a, plan = M.block_norm(block, p["x"], p["y"], p["w_pre"], p["w_post"], p["gate"])
    stat = B.ROW_SUM // 2 + 5  # half the row sum's error, eps, mean, root, quotient
    B.check("x_out", x_out, ref["x_out"], mag["x_out"], stat + 5)
    B.check("a", a, ref["a"], mag["a"], 2 * stat + 8)
    g = gen(seed)
    dxo, da = randn(g, (T, d), block.res, 0.3), randn(g, (T, d), block.act, 0.2)
    args = (dxo, da, x_out, p["y"], plan.r_post, plan.r_pre, p["w_post"], p["gate"], p["w_pre"], block.every, alpha,
            beta, post)
    ref, mag = B.norm_bwd_ref(*args), B.norm_bwd_ref(*args, magnitude=True)
    dx, dy, grads = M.block_norm_backward(block, dxo, da, x_out, p["y"], plan.r_pre, plan.r_post, p["w_pre"],
                                          p["w_post"], p["gate"])
    B.check("dx", dx, ref["dx"], mag["dx"], ROW)
    B.check("dy", dy, ref["dy"], mag["dy"], ROW)
    assert set(grads) == {n for n in ("dw_pre", "dw_post", "dgate") if n in ref}
    for n, t in grads.items():
        B.check(n, t, ref[n], mag[n], col)


# Teams take four or five consecutive rows (one team a workgroup, or five), so
# gate groups lie inside a team, begin or end in one, and span many; with 2 and
# 3 tokens a group there are more groups than teams.  8,200 channels keep the
# column sums in LDS (bf16), the others in registers.
LONG = [(1100, 8200, e) for e in (2, 3, 5, 7, 24, 1000, -1)] + [(1100, 4104, e) for e in (2, 3, 24, -1)] + \
    [(4000, 1032, e) for e in (2, 3, 9, 100)] + [(1100, 8195, 3), (4000, 1031, 3)]


@pytest.mark.parametrize("prec,res_f32", PRECS)
@pytest.mark.parametrize("T,d,every", LONG)
def test_norm_of_several_rows_a_team(T, d, every, prec, res_f32):
    block, p = norm_inputs(T, d, every, True, 0.75, 0.5, prec, res_f32, T + d + every, odd=d % 2 == 1)
    # a sum over tokens: at most 5 of a team and as many gate groups, 5 teams of
    # a workgroup, 40 for a way's share of 1,280 teams, 32 ways
    check_both_directions(block, p, every, every + 2, ROW + 90)


# More than 256 MB of rows, which the backward streams.
@pytest.mark.parametrize("prec,res_f32,T,d,every,post", [
    ("bf16", False, 3200, 7168, 100, True), ("bf16", False, 3200, 7168, 5, True), ("bf16", False, 2800, 8192, 9, False),
    ("bf16", False, 1500, 16384, 4, True), ("bf16", True, 2100, 7168, 100, True), ("bf16", True, 2100, 7168, 4, True),
    ("bf16", True, 1000, 16384, 3, True), ("f32", False, 1600, 7168, 5, True), ("f32", False, 700, 16384, 100, True),
    ("f32", False, 1600, 7168, -1, True), ("bf16", True, 2100, 7168, -1, False)])
def test_norm_of_streamed_rows(prec, res_f32, T, d, every, post):
    block, p = norm_inputs(T, d, every, post, 0.75, 0.5, prec, res_f32, T + d + every)
    size = {torch.bfloat16: 2, torch.float32: 4}
    assert T * d * 3 * (size[block.act] + size[block.res]) > 256 << 20
    # 13 rows of a team and as many gate groups, 8 for a way's share of 256 teams, 32 ways
    check_both_directions(block, p, every, every + 3, ROW + 70)


@pytest.mark.parametrize("res_f32", [False, True])
@pytest.mark.parametrize("n,copies,d,group", [(1000, 310, 7168, 62), (1000, 310, 7168, 310), (2049, 2047, 64, 89),
                                              (2049, 2047, 64, 2047)])
def test_weight_gradients_of_many_tokens(n, copies, d, group, res_f32):
    """A batch repeated `copies` times has that many times its weight
    gradients: 310,000 rows of 7,168 channels (1,211 a team), and the most
    tokens a call takes, 4,194,303 (1,024 a team).  `group` copies share a
    gate row."""
    g = gen(n + group)
    groups = copies // group
    small = M.Block(n, d, res_f32=res_f32, post_norm=True, alpha=0.5, beta=0.75)
    big = M.Block(n * copies, d, res_f32=res_f32, post_norm=True, alpha=0.5, beta=0.75, gate_every=n * group)
    assert big.gates == groups
    x, dxo = randn(g, (n, d), small.res), randn(g, (n, d), small.res, 0.3)
    y, da = randn(g, (n, d), small.act), randn(g, (n, d), small.act, 0.2)
    w_pre, w_post, gate = randn(g, (d,)), randn(g, (d,)), randn(g, (groups, d))
    x1, _, plan = M.block_norm(small, x, y, w_pre, w_post, gate[:1])
    many = lambda t: t.repeat(copies, *[1] * (t.dim() - 1))  # noqa: E731
    _, _, grads = M.block_norm_backward(big, many(dxo), many(da), many(x1), many(y), many(plan.r_pre),
                                        many(plan.r_post), w_pre, w_post, gate)
    ref, mag = dict(dw_post=0.0, dgate=[]), dict(dw_post=0.0, dgate=[])
    for i in range(groups):
        for out, m in ((ref, False), (mag, True)):
            one = B.norm_bwd_ref(dxo, da, x1, y, plan.r_post, plan.r_pre, w_post, gate[i:i + 1], w_pre, n, 0.5, 0.75,
                                 True, magnitude=m)
            out["dw_pre"] = one["dw_pre"] * copies
            out["dw_post"] = out["dw_post"] + one["dw_post"] * group
            out["dgate"].append(one["dgate"] * group)
    # up to 1,211 rows of a team, 16 teams of a workgroup, 128 for a way's share
    # of 4,096 teams, 32 ways, and the gate groups of a team
    for name, t in grads.items():
        r, m = (torch.cat(v) if isinstance(v, list) else v for v in (ref[name], mag[name]))
        B.check(name, t, r, m, ROW + 1211 + 16 + 128 + 32 + 23)


# ---- unsort: rows beyond the caches ----------------------------------------
@pytest.mark.parametrize("prec,T", [("bf16", 1800), ("f32", 900)])
@pytest.mark.parametrize("d", [7168, 7001])
def test_unsort_of_streamed_rows(prec, T, d):
    k = 16
    dims, rows, token_row, w, add, n = unsort_inputs(T, d, k, "some", prec, T + d)
    assert T * k * d * rows.element_size() > 384 << 20 and n < T * k
    tr = token_row.cpu()
    ref, mag = B.unsort_ref(rows, tr, w.cpu(), add)
    B.check("y", M.unsort_tokens(rows, token_row, w, add, dims, prec), ref, mag, k + 1)  # k fma and the addend
    ref, mag = B.unsort_ref(rows, tr, None, None)
    B.check("dx", M.sort_tokens_backward(rows, token_row, None, dims, prec), ref, mag, k + 1)


# ---- clip: more partial sums than one launch's workgroups -------------------
def test_clip_of_many_partial_sums():
    """500 tensors of 50,001 to 99,999 elements: three norm tables, two of them
    of more chunks than workgroups, and four scaling launches."""
    g = gen(11)
    grads = [randn(g, (50001 + (i * 6151) % 49999,), TYPES["f32" if i % 3 == 1 else "bf16"], 10.0 ** (i % 5 - 2),
                   odd=i % 2 == 1) for i in range(500)]
    chunks = [-(-t.numel() // 16384) for t in grads]
    assert sum(min(sum(chunks[i:i + 240]), 1024) for i in range(0, 500, 240)) > 2048
    ref = torch.stack([B.f64(t).pow(2).sum() for t in grads]).sum().sqrt()
    norm = M.grad_norm(grads)
    assert abs(norm.double().cpu() - ref) <= ref * (B.U + 2.0 ** -27)  # 64-bit sums (2^26 terms), one rounding
    max_norm = 0.37 * float(norm)
    f = max_norm / (float(norm) + 1e-6)
    out, joined = M.clip_grads(grads, max_norm, out=[torch.empty_like(t) for t in grads])
    given, same = M.clip_grads(grads, max_norm, norm=norm, out=[torch.empty_like(t) for t in grads])
    assert torch.equal(joined, norm) and same is norm
    for o, v, t in zip(out, given, grads):
        B.check("clipped", o, B.f64(t) * f, (B.f64(t) * f).abs(), 3)  # max_norm to fp32, sum, quotient
        assert torch.equal(o, v)
    again, joined = M.clip_grads(grads, max_norm)  # in place
    assert again is grads and torch.equal(joined, norm) and all(torch.equal(a, b) for a, b in zip(grads, out))
