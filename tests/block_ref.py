"""The operators around the layer in 64 bits on the CPU, from their
definitions, and bounds of the kernels' fp32 rounding.

Bounds.  u = 2^-24 is half a step of fp32.  Every kernel value is a chain of
fp32 operations, each off by at most u relative to its result; a value's error
is at most (roundings on the longest path) * u * M, where M is the same
expression with every term taken in magnitude (differences become sums).  A
row sum of d <= 16384 elements passes at most 16 fma in a thread, 6 steps over
the wave and 16 over the waves: 38 roundings.  An output is then rounded once
more, by at most half a step of its type relative to the value."""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ROW_SUM = 38


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


# ---- sort and unsort -------------------------------------------------------
def sort_ref(idx, E):
    """(counts, offsets, row_token of the present rows, token_row) as lists."""
    T, k = idx.shape
    lists = [[] for _ in range(E)]
    for r, e in enumerate(idx.reshape(-1).tolist()):
        if 0 <= e < E:
            lists[e].append(r)
    counts = [len(v) for v in lists]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    routes = [r for v in lists for r in v]
    token_row = [-1] * (T * k)
    for row, r in enumerate(routes):
        token_row[r] = row
    i32 = torch.int32
    return (torch.tensor(counts, dtype=i32), torch.tensor(offsets, dtype=i32),
            torch.tensor([r // k for r in routes], dtype=i32), torch.tensor(token_row, dtype=i32).reshape(T, k))


def unsort_ref(rows, token_row, w, add):
    """(value, magnitude): the weighted sum of the present routes' rows."""
    rows, add = f64(rows), f64(add)
    T, k = token_row.shape
    d = rows.shape[1]
    y = torch.zeros(T, d, dtype=torch.float64) if add is None else add.clone()
    m = y.abs()
    for t in range(T):
        for j in range(k):
            row = int(token_row[t, j])
            if row >= 0:
                v = (1.0 if w is None else float(w[t, j])) * rows[row]
                y[t] += v
                m[t] += v.abs()
    return y, m


def unsort_bwd_ref(dy, o_perm, token_row, w):
    """(do_perm rows {row: value}, dtopk_w, its magnitude)."""
    dy, o = f64(dy), f64(o_perm)
    T, k = token_row.shape
    dw, m, do = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64), {}
    for t in range(T):
        for j in range(k):
            row = int(token_row[t, j])
            if row >= 0:
                do[row] = float(w[t, j]) * dy[t]
                dw[t, j] = (dy[t] * o[row]).sum()
                m[t, j] = (dy[t] * o[row]).abs().sum()
    return do, dw, m


# ---- block norm ------------------------------------------------------------
def gate_rows(gate, T, every):
    return 1.0 if gate is None else f64(gate)[torch.arange(T) // every]


def norm_fwd_ref(x, y, w_post, gate, w_pre, every, alpha, beta, eps, post_norm, pre_norm=True, magnitude=False):
    """dict(x_out, a, r_post, r_pre); magnitude: the same with |x|, |y|, ... in
    x' (the row statistics stay those of the values)."""
    x, y = f64(x), f64(y)
    one = torch.ones(x.shape[1], dtype=torch.float64)
    w_post, w_pre = one if w_post is None else f64(w_post), one if w_pre is None else f64(w_pre)
    out = {}
    z = zm = x
    if y is not None:
        n = y
        if post_norm:
            out["r_post"] = (y.pow(2).mean(1) + eps).rsqrt()
            n = y * out["r_post"][:, None] * w_post
        n = beta * n * gate_rows(gate, x.shape[0], every)
        z, zm = alpha * x + n, (alpha * x).abs() + n.abs()
        out["x_out"] = zm if magnitude else z
    else:
        zm = x.abs()
    if pre_norm:
        out["r_pre"] = (z.pow(2).mean(1) + eps).rsqrt()
        if magnitude:
            # x' is off by up to (..) u zm, and r(x') with it
            spread = (z.abs() * zm).mean(1) / (z.pow(2).mean(1) + eps)
            out["a"] = (zm + z.abs() * spread[:, None]) * out["r_pre"][:, None] * w_pre.abs()
            out["r_pre"] = out["r_pre"] * (1 + spread)
        else:
            out["a"] = z * out["r_pre"][:, None] * w_pre
    return out


def norm_bwd_ref(dx_out, da, x_out, y, r_post, r_pre, w_post, gate, w_pre, every, alpha, beta, post_norm,
                 magnitude=False):
    """dict(dx, dy, dw_pre, dw_post, dgate) of the formulas for the inputs as
    given; magnitude: every term taken in magnitude."""
    mag = (lambda t: t.abs()) if magnitude else (lambda t: t)
    sub = (lambda a, b: a + b) if magnitude else (lambda a, b: a - b)
    some = da if dx_out is None else dx_out
    T, d = some.shape
    zero, one = torch.zeros(T, d, dtype=torch.float64), torch.ones(d, dtype=torch.float64)
    dx_out = zero if dx_out is None else mag(f64(dx_out))
    wq, wp = one if w_pre is None else mag(f64(w_pre)), one if w_post is None else mag(f64(w_post))
    out = {}
    dz = dx_out
    if da is not None:
        r = f64(r_pre)[:, None]
        xh, da = mag(f64(x_out)) * r, mag(f64(da))
        u = da * wq
        dz = dx_out + r * sub(u, xh * (u * xh).mean(1, keepdim=True))
        out["dw_pre"] = (da * xh).sum(0)
    if y is None:
        out["dx"] = dz
        return out
    out["dx"] = abs(alpha) * dz if magnitude else alpha * dz
    e = abs(beta) * dz if magnitude else beta * dz
    g = gate_rows(gate, T, every)
    g = mag(g) if gate is not None else g
    y = mag(f64(y))
    yh = y * f64(r_post)[:, None] if post_norm else y
    if gate is not None:
        groups = (T + every - 1) // every
        out["dgate"] = torch.zeros(groups, d, dtype=torch.float64).index_add_(0, torch.arange(T) // every, e * yh * wp)
    dn = e * g
    if post_norm:
        out["dw_post"] = (dn * yh).sum(0)
        v = dn * wp
        dn = f64(r_post)[:, None] * sub(v, yh * (v * yh).mean(1, keepdim=True))
    out["dy"] = dn
    return out


def check(name, got, ref, mag, roundings):
    """|got - ref| <= roundings * u * magnitude + half a step of got's type."""
    got64 = f64(got)
    bound = roundings * U * mag + HALF_STEP[got.dtype] * (ref.abs() + roundings * U * mag) + 1e-38
    bad = (got64 - ref).abs() > bound
    bad |= got64.isnan()
    if bool(bad.any()):
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError("%s: %d of %d off, first at %d: got %r, expected %r, bound %.3e" % (
            name, int(bad.sum()), bad.numel(), i, got64.reshape(-1)[i].item(), ref.reshape(-1)[i].item(),
            bound.reshape(-1)[i].item()))
