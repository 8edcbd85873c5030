"""Paths of the routed experts in 4 bits that calls take for other reasons than
their size alone: which kernels serve a call, the rounds that an expert's tokens
need, the schedule that sorts them.  A token alone takes the direct path with the
down projection by token; every other must give the same bits."""
import numpy as np
import pytest

import mixture_experts_layer_prefix_amd as M

torch = pytest.importorskip("torch")
from tests.test_gpu_mx_ops import I32, gen, ids, np64, poisoned, randn, real_problem, reference, whole_problem  # noqa: E402

pytestmark = pytest.mark.gpu


def same_alone(y, x, xs, idx, tw, w, dims, tokens, add=None):
    one = M.RoutedFfnPlan(M.Dims(1, dims.d, dims.E, dims.k, dims.I))
    for t in tokens:
        s = slice(t, t + 1)
        got = one.run(x[s], xs[s], idx[s], tw[s], w, None if add is None else add[s])
        assert torch.equal(got, y[s]), t


@pytest.mark.parametrize("T,d,E,k,I", [(8, 256, 64, 1, 384), (2, 128, 2, 1, 128), (16, 384, 16, 1, 1152), (13, 512, 40, 1, 256)])
def test_few_routes_of_one_each(T, d, E, k, I):
    """As many experts as routes or more, one route a token: without a schedule,
    the down projection by expert."""
    dims = M.Dims(T, d, E, k, I)
    x, xs, w = real_problem(T, T, d, E, k, I)
    tw, add = torch.rand(T, k, generator=gen(2), device="cuda"), randn(3, (T, d))
    for case in range(4):
        idx = ids(case, T, k, 0, E)
        if case == 1:
            idx[:] = E - 1                            # all at one expert
        if case == 2:
            idx[::2] = -1                             # absent
        if case == 3:
            idx[T // 2:] = idx[:T - T // 2].clone()           # repeated
        y = poisoned(dims).run(x, xs, idx, tw, w, add)
        same_alone(y, x, xs, idx, tw, w, dims, range(T), add)
    x, xs, w = whole_problem(T, T, d, E, k, I)
    idx = ids(7, T, k, -1, E + 1)
    y = poisoned(dims).run(x, xs, idx, tw, w, add)
    want, bound = reference(x, xs, idx, tw, w, E, add, exact_gu=True)
    assert np.all(np.abs(np64(y) - want) <= bound)


def test_few_routes_of_large_experts():
    """Sixteen routes of sixteen experts whose weights are worth reading once:
    the down projection by expert with two routes a token."""
    T, d, E, k, I = 8, 4096, 16, 2, 3200
    dims = M.Dims(T, d, E, k, I)
    x, xs, w = real_problem(5, T, d, E, k, I)
    tw = torch.rand(T, k, generator=gen(2), device="cuda")
    for hi in (E, 3):
        idx = ids(hi, T, k, -1, hi)
        same_alone(poisoned(dims).run(x, xs, idx, tw, w), x, xs, idx, tw, w, dims, range(T))


# tiles of 48, 32 and 32 tokens with 128, 128 and 64 weight rows
@pytest.mark.parametrize("T,d,E,k,I", [(300, 256, 4, 2, 2048), (160, 384, 64, 4, 640), (200, 256, 3, 2, 256)])
@pytest.mark.parametrize("skew", ["most at one", "all at one", "spread"])
def test_an_experts_tokens_in_several_rounds(T, d, E, k, I, skew):
    """After a schedule: more tokens at one expert than its workgroups take at a
    time, so that they go on to further ones over the LDS that held the sums."""
    dims = M.Dims(T, d, E, k, I)
    x, xs, w = real_problem(T, T, d, E, k, I)
    idx = ids(1, T, k, -1, E)
    if skew != "spread":
        idx[:] = 1
    if skew == "most at one":
        idx[::7] = ids(2, (T + 6) // 7, k, -1, E)
        idx[3, 0] = idx[5, 1] = -1
    tw, add = torch.rand(T, k, generator=gen(2), device="cuda"), randn(3, (T, d))
    y = poisoned(dims).run(x, xs, idx, tw, w, add)
    same_alone(y, x, xs, idx, tw, w, dims, list(range(0, T, 9)) + [1, 2, 3, 5, T - 1], add)


@pytest.mark.parametrize("T,E,k,lo,hi", [(4200, 64, 8, -6, 70), (34000, 3, 1, 0, 3)])
def test_more_routes_than_one_launch_sorts(T, E, k, lo, hi):
    """The schedule of more than 32,768 routes, which counts, scans and ranks
    them in the call's workspace."""
    d = I = 128
    dims = M.Dims(T, d, E, k, I)
    x, xs, w = whole_problem(T, T, d, E, k, I)
    idx, tw = ids(1, T, k, lo, hi), torch.rand(T, k, generator=gen(2), device="cuda")
    y = poisoned(dims).run(x, xs, idx, tw, w)
    some = torch.cat([torch.randperm(T, generator=gen(4), device="cuda")[:200], torch.tensor([0, T - 1], device="cuda")])
    want, bound = reference(x[some], xs[some], idx[some], tw[some], w, E, exact_gu=True)
    assert np.all(np.abs(np64(y[some]) - want) <= bound)
    same_alone(y, x, xs, idx, tw, w, dims, some[:20].tolist() + [0, T - 1])
    gone = ((idx < 0) | (idx >= E)).all(1)
    assert bool((y[gone] == 0).all())


def test_ids_of_every_kind_in_every_path():
    """The ends of the 32-bit range beside present ids, at counts of routes on
    both sides of every limit."""
    d, I, E, k = 256, 128, 12, 2
    far = torch.tensor([-(1 << 31), -1, E, (1 << 31) - 1], dtype=I32, device="cuda")
    for T in (1, 8, 9, 31, 32, 33, 64, 100, 511, 512, 513):
        dims = M.Dims(T, d, E, k, I)
        x, xs, w = real_problem(3, T, d, E, k, I)
        idx = ids(T, T, k, 0, E)
        idx[::3, 1] = far[torch.arange(len(idx[::3]), device="cuda") % 4]
        idx[::5, 0] = far[torch.arange(len(idx[::5]), device="cuda") % 4]
        tw = torch.rand(T, k, generator=gen(2), device="cuda")
        tw[(idx < 0) | (idx >= E)] = float("nan")
        y = poisoned(dims).run(x, xs, idx, tw, w)
        assert bool(torch.isfinite(y).all())
        same_alone(y, x, xs, idx, tw, w, dims, sorted({0, T // 2, T - 1}))
