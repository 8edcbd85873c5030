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
