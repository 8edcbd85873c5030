"""The operators around the layer on the GPU at the edges of what their entry
points accept: empty batches."""
import pytest

import mixture_experts_layer_prefix_amd as M

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


# ---- empty batches ---------------------------------------------------------
@pytest.mark.parametrize("prec,res_f32", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("every", [0, 3])
def test_empty_batch_has_zero_weight_gradients(prec, res_f32, every):
    """Exact zeros whatever the weights hold: no gate row belongs to a batch
    without tokens (gate_every 3: the gate has none; 0: its one row is not
    read)."""
    b = M.Block(0, 24, prec, res_f32=res_f32, post_norm=True, gate_every=every)
    x, y = torch.empty(0, 24, dtype=b.res, device="cuda"), torch.empty(0, 24, dtype=b.act, device="cuda")
    r, w = torch.empty(0, device="cuda"), torch.full((24,), float("nan"), device="cuda")
    gate = torch.full((b.gates, 24), float("nan"), device="cuda")
    assert gate.shape[0] == (0 if every else 1)
    dx, dy, grads = M.block_norm_backward(b, x, y, x, y, r, r, w, w, gate)
    assert dx.shape == dy.shape == (0, 24) and set(grads) == {"dw_pre", "dw_post", "dgate"}
    for name, t in grads.items():
        assert bool((t == 0).all()), name


@pytest.mark.parametrize("need_do,need_dw", [(True, True), (True, False), (False, True)])
def test_empty_batch_of_the_weighted_sums_gradient(need_do, need_dw):
    dims = M.Dims(0, 24, 6, 2, 1)
    x, w = torch.empty(0, 24, device="cuda"), torch.empty(0, 2, device="cuda")
    do, dw = M.unsort_tokens_backward(x, x, torch.empty(0, 2, dtype=torch.int32, device="cuda"), w, dims, "f32",
                                      need_do=need_do, need_dw=need_dw)
    assert (do.shape == (0, 24)) if need_do else do is None
    assert (dw.shape == (0, 2)) if need_dw else dw is None


# ---- tensors that overlap (refused before anything is launched) -------------
def test_clip_refuses_tensors_that_overlap():
    t = torch.ones(100, device="cuda")
    keep, norm = t.clone(), torch.ones(1, device="cuda")
    a, b = t[:50], t[50:]
    for grads, kw in [([t, t[10:20]], {}), ([t[:60], t[40:]], {}), ([a, b], dict(out=[b, a])),
                      ([a, b], dict(out=[t[1:51], torch.empty(50, device="cuda")])), ([a, b], dict(out=[a, t[25:75]])),
                      ([norm, a], dict(norm=norm))]:
        with pytest.raises(ValueError):
            M.clip_grads(grads, 1.0, **kw)
    assert torch.equal(t, keep)
    # views side by side, and one gradient into two outputs
    M.clip_grads([a, b], 5.0)
    assert bool((t - 0.5).abs().max() < 1e-6)
    out, n = M.clip_grads([a, a], 1e9, out=[torch.empty(50, device="cuda") for _ in range(2)])
    assert abs(float(n) - 5.0) < 1e-5 and all(torch.equal(o, a) for o in out)


# ---- plans -----------------------------------------------------------------
def test_norm_without_a_block_output_keeps_no_residual():
    x, y = torch.ones(3, 64, device="cuda"), torch.ones(3, 64, device="cuda")
    block = M.Block(3, 64, "f32")
    same, a, plan = M.block_norm(block, x)
    assert same is x and plan.x_out is None
    x_out, b, whole = M.block_norm(block, x, torch.zeros_like(y))
    assert whole.x_out is x_out and torch.equal(x_out, x) and torch.equal(a, b)
    with pytest.raises(M._lib.MoeError):  # a block output has nowhere to go
        plan.run(x, y)
    again, b = plan.run(x)
    assert again is x and b is plan.a and torch.equal(a, b)
