"""Speed cases of the operators around an MoE layer: tokens sorted by expert
and back (with gradients), the norms before and after a residual block (with
gradients), and the global gradient norm with clipping.

`listed()` names the cases, `draw(rng)` makes more of the same ranges,
`prepare` makes a case's inputs on the GPU, `run` is one pass through the
operator (plain torch in 32 bits, or the library's kernels where `own` is
true), `work` counts what a pass cannot do without and `exact` gives its
outputs from the definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _norm(name, T, d, prec="bf16", res_f32=False, post=True, gate="one", alpha=1.0, beta=1.0):
    return dict(name=name, op="norm", T=T, d=d, prec=prec, res_f32=res_f32, post=post, gate=gate, alpha=alpha,
                beta=beta)


def _routes(name, op, T, d, E, k, prec="bf16", absent="none"):
    return dict(name=name, op=op, T=T, d=d, E=E, k=k, prec=prec, absent=absent)


def listed():
    return [
        # One decoded token between two layers: residual add and the next block's norm.
        _norm("norm_token", 1, 7168, post=False, gate="none"),
        # A training batch: norms on both sides of the block, a learned gate per channel,
        # scaled residual, bf16 throughout.
        _norm("norm_batch", 8192, 7168, alpha=0.75, beta=0.5),
        # The backward of that batch at twice the tokens.
        dict(_norm("norm_grad", 16384, 7168, alpha=0.75, beta=0.5), op="norm_bwd"),
        # Ragged sizes: an odd width, sequences of 100 tokens each with a gate of its own, the
        # residual stream in fp32.
        dict(_norm("norm_grad_odd", 1531, 2047, res_f32=True, gate="seq100"), op="norm_bwd"),
        # Sixteen decoded tokens sent to their experts.
        _routes("sort_decode", "sort", 16, 7168, 256, 8),
        # A padded training batch: an eighth of its tokens hold no routes.
        _routes("sort_batch", "sort", 8192, 7168, 256, 8, absent="padding"),
        # One rank's share of the experts: 32 of 256, so most routes are another rank's.
        _routes("unsort_share", "unsort", 16384, 6144, 32, 8, absent="share8"),
        # The gradient of the weighted sum, every route present.
        _routes("unsort_grad", "unsort_bwd", 8192, 4096, 128, 8),
        # Odd width in fp32, a few routes dropped: the gradient of the sort.
        _routes("sort_grad_odd", "sort_bwd", 777, 1001, 64, 6, prec="f32", absent="dropped"),
        # A small layer's eight gradients.
        dict(name="clip_small", op="clip", sizes="8x64x256,8x64x256,8x256x64,64x256,64x256,256x64,256x8:f32,256:f32",
             copies=1),
        # The gradients of a layer of 64 experts (weights bf16, the router's fp32).
        dict(name="clip_layer", op="clip",
             sizes="64x768x2048,64x768x2048,64x2048x768,768x2048,768x2048,2048x768,64x2048:f32", copies=1),
        # Many tensors of odd sizes, as of a model of many small parts.
        dict(name="clip_many", op="clip", sizes="97x1031,2047,1:f32,33x64x65,4099:f32,777x1001", copies=100),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case; one that would move more bytes than the largest listed
    case is halved (tokens, or copies of the tensors) until it does not."""
    case = _draw(rng)
    most = max(work(c)["bytes"] for c in listed())
    while work(case)["bytes"] > most:
        key = "copies" if case["op"] == "clip" else "T"
        case[key] = case[key] // 2
    return case


def _draw(rng):
    op = rng.choice(["norm", "norm_bwd", "sort", "sort_bwd", "unsort", "unsort_bwd", "clip"])
    if op in ("norm", "norm_bwd"):
        T, d = _log_int(rng, 1, 16384), _log_int(rng, 64, 7168)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        prec = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, T=T, d=d, prec=prec, res_f32=rng.random() < 0.4, post=rng.random() < 0.6,
                    gate=rng.choice(["none", "one", "seq%d" % _log_int(rng, 1, 4096)]),
                    alpha=rng.choice([1.0, 0.5, 0.875]), beta=rng.choice([1.0, 0.25, 1.5]))
    if op == "clip":
        n = rng.randint(1, 12)
        return dict(op=op, sizes=",".join("%d%s" % (_log_int(rng, 1, 2000000), rng.choice(["", "", ":f32"]))
                                          for _ in range(n)),
                    copies=_log_int(rng, 1, 24))
    E = _log_int(rng, 1, 512)
    k = rng.randint(1, min(E, 12))
    T, d = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096)
    if rng.random() < 0.6:
        d = max(64, d // 64 * 64)
    return dict(op=op, T=T, d=d, E=E, k=k, prec=rng.choice(["bf16", "bf16", "f32"]),
                absent=rng.choice(["none", "padding", "dropped", "share%d" % rng.choice([2, 4, 8])]))


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _gate_every(case):
    """Tokens that share one row of the gate."""
    return int(case["gate"][3:]) if case["gate"].startswith("seq") else case["T"]


def _parse_sizes(case):
    """(shape, type) of every gradient tensor of a clip case."""
    one = []
    for s in case["sizes"].split(","):
        dims, _, t = s.partition(":")
        one.append((tuple(int(v) for v in dims.split("x")), t or "bf16"))
    return one * case["copies"]


def _make_routes(case, g):
    """Expert ids [T][k] (distinct, ascending) and router weights: skewed
    loads; ids outside [0, E) stand for routes that are not here."""
    T, E, k, absent = case["T"], case["E"], case["k"], case["absent"]
    total = E * int(absent[5:]) if absent.startswith("share") else E
    skew = torch.log(torch.arange(1, total + 1, device="cuda", dtype=torch.float32)) * -0.6
    skew = skew[torch.randperm(total, generator=g, device="cuda")]
    score = torch.rand(T, total, generator=g, device="cuda").clamp_(min=1e-9).log_().neg_().log_().neg_() + skew
    top, idx = torch.topk(score, k, dim=1)
    idx, order = torch.sort(idx, dim=1)
    w = torch.softmax(torch.gather(top, 1, order), dim=1)
    if absent.startswith("share"):
        idx = idx - (total - E) // 2  # the local experts are the middle ones
    elif absent == "padding":
        idx = torch.where((torch.rand(T, 1, generator=g, device="cuda") < 0.125), -1, idx)
    elif absent == "dropped":
        idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, idx)
    return idx.to(torch.int32).contiguous(), w.contiguous()


def _sorted_rows(idx, E):
    """token_row [T][k] (-1: absent) of the expert-major, token-ascending layout."""
    flat = idx.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    order = torch.sort(torch.where(valid, flat, E), stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    return torch.where(valid, rows, -1).to(torch.int32).reshape(idx.shape)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case=case)
    if op == "clip":
        st["grads"] = [_randn(g, s, _TYPES[t], 10.0 ** (-3 + i % 4)) for i, (s, t) in enumerate(_parse_sizes(case))]
        # the clipped gradients go into one flat bucket per type, tensor after tensor
        st["flat"], st["out"] = {}, [None] * len(st["grads"])
        for name, dtype in _TYPES.items():
            mine = [i for i, t in enumerate(st["grads"]) if t.dtype == dtype]
            if mine:
                flat = st["flat"][name] = torch.empty(sum(st["grads"][i].numel() for i in mine), dtype=dtype,
                                                      device="cuda")
                for i, part in zip(mine, flat.split([st["grads"][i].numel() for i in mine])):
                    st["out"][i] = part.view(st["grads"][i].shape)
        return st
    T, d, act = case["T"], case["d"], _TYPES[case["prec"]]
    if op in ("norm", "norm_bwd"):
        res = torch.float32 if case["res_f32"] else act
        every = _gate_every(case)
        st["w_pre"] = 1.0 + _randn(g, (d,), torch.float32, 0.1)
        st["w_post"] = 1.0 + _randn(g, (d,), torch.float32, 0.1) if case["post"] else None
        st["gate"] = None if case["gate"] == "none" else _randn(g, ((T + every - 1) // every, d), torch.float32, 0.7)
        st["y"] = _randn(g, (T, d), act)
        st["x"] = _randn(g, (T, d), res, 2.0)
        if op == "norm_bwd":
            st["da"] = _randn(g, (T, d), act, 0.02)
            st["dx_out"] = _randn(g, (T, d), res, 0.02)
            st["r_pre"] = torch.rsqrt(st["x"].float().square().mean(1) + 1e-6)
            st["r_post"] = torch.rsqrt(st["y"].float().square().mean(1) + 1e-6) if case["post"] else None
        if own:
            import mixture_experts_layer_prefix_amd as M
            block = M.Block(T, d, case["prec"], res_f32=case["res_f32"], post_norm=case["post"],
                            alpha=case["alpha"], beta=case["beta"], eps=1e-6, gate_every=every)
            if op == "norm":
                st["plan"] = M.BlockNormPlan(block)
            else:
                st["plan"] = M.BlockNormBackwardPlan(block, gate=st["gate"] is not None)
        return st
    idx, w = _make_routes(case, g)
    st["idx"], st["w"] = idx, w
    R = T * case["k"]
    if op == "sort":
        st["x"] = _randn(g, (T, d), act)
        st["x_perm"] = torch.zeros(R, d, dtype=act, device="cuda")
        st["row_token"] = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    else:
        st["token_row"] = _sorted_rows(idx, case["E"])
        st["rows"] = _randn(g, (R, d), act)  # o_perm or dx_perm
        st["tok"] = _randn(g, (T, d), act)   # y_add, dx_add or dy
        if op == "unsort_bwd":
            st["do_perm"] = torch.zeros(R, d, dtype=act, device="cuda")
    if own:
        import mixture_experts_layer_prefix_amd as M
        st["dims"] = M.Dims(T, d, case["E"], case["k"], 1)
        if op == "sort":
            st["plan"] = M.SortPlan(st["dims"], case["prec"], x_perm=st["x_perm"], row_token=st["row_token"])
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import mixture_experts_layer_prefix_amd as M
    case = st["case"]
    op, prec = case["op"], case.get("prec")
    if op == "norm":
        plan = st["plan"]
        plan.run(st["x"], st["y"], w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"])
        return dict(x_out=plan.x_out, a=plan.a, r_pre=plan.r_pre, **({"r_post": plan.r_post} if case["post"] else {}))
    if op == "norm_bwd":
        plan = st["plan"]
        dx, dy, grads = plan.run(st["dx_out"], st["da"], st["x"], st["y"], st["r_pre"], st["r_post"],
                                 w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"])
        return dict(grads, dx=dx, dy=dy)
    if op == "sort":
        counts, offsets, row_token, token_row, x_perm = st["plan"].run(st["idx"], st["x"])
        return dict(counts=counts, offsets=offsets, row_token=row_token, token_row=token_row, x_perm=x_perm)
    if op == "sort_bwd":
        return dict(dx=M.sort_tokens_backward(st["rows"], st["token_row"], st["tok"], st["dims"], prec))
    if op == "unsort":
        return dict(y=M.unsort_tokens(st["rows"], st["token_row"], st["w"], st["tok"], st["dims"], prec))
    if op == "unsort_bwd":
        do_perm, dw = M.unsort_tokens_backward(st["tok"], st["rows"], st["token_row"], st["w"], st["dims"], prec,
                                               do_perm=st["do_perm"])
        return dict(do_perm=do_perm, dtopk_w=dw)
    _, norm = M.clip_grads(st["grads"], 1.0, out=st["out"])
    return dict(st["flat"], norm=norm)


def _gate_rows(st):
    """The gate as it multiplies the tokens: [1][d], or [T][d] for several sequences."""
    gate = st["gate"]
    if gate is None or gate.shape[0] == 1:
        return gate
    return gate.repeat_interleave(_gate_every(st["case"]), dim=0)[:st["case"]["T"]]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        x, n = st["x"].float(), st["y"].float()
        out = {}
        if case["post"]:
            r = torch.rsqrt((n * n).mean(1, keepdim=True) + 1e-6)
            n = n * r * st["w_post"]
            out["r_post"] = r[:, 0]
        if st["gate"] is not None:
            n = n * _gate_rows(st)
        z = case["alpha"] * x + case["beta"] * n
        r = torch.rsqrt((z * z).mean(1, keepdim=True) + 1e-6)
        out.update(x_out=z.to(st["x"].dtype), a=(z * r * st["w_pre"]).to(st["y"].dtype), r_pre=r[:, 0])
        return out
    if op == "norm_bwd":
        y, da = st["y"].float(), st["da"].float()
        rp = st["r_pre"][:, None]
        xh, u = st["x"].float() * rp, da * st["w_pre"]
        dz = st["dx_out"].float() + rp * (u - xh * (u * xh).mean(1, keepdim=True))
        out = dict(dw_pre=(da * xh).sum(0), dx=(case["alpha"] * dz).to(st["x"].dtype))
        e = case["beta"] * dz
        yh = y * st["r_post"][:, None] if case["post"] else y
        dn = e
        if st["gate"] is not None:
            n = yh * st["w_post"] if case["post"] else y
            en, every = e * n, _gate_every(case)
            if st["gate"].shape[0] == 1:
                out["dgate"] = en.sum(0, keepdim=True)
            else:
                whole = torch.zeros(st["gate"].shape[0] * every, en.shape[1], device=en.device)
                whole[:case["T"]] = en
                out["dgate"] = whole.view(-1, every, en.shape[1]).sum(1)
            dn = e * _gate_rows(st)
        if case["post"]:
            out["dw_post"] = (dn * yh).sum(0)
            v = dn * st["w_post"]
            dn = st["r_post"][:, None] * (v - yh * (v * yh).mean(1, keepdim=True))
        out["dy"] = dn.to(st["y"].dtype)
        return out
    if op == "clip":
        total = sum(g.float().square().sum(dtype=torch.float64) for g in st["grads"])
        norm = total.sqrt().float()
        c = (1.0 / (norm + 1e-6)).clamp(max=1.0)
        for o, g in zip(st["out"], st["grads"]):
            o.copy_(g.float() * c)
        return dict(st["flat"], norm=norm.reshape(1))
    T, E, k = case["T"], case["E"], case["k"]
    if op == "sort":
        flat = st["idx"].reshape(-1).long()
        key = torch.where((flat >= 0) & (flat < E), flat, E)
        skey, order = torch.sort(key, stable=True)
        here = skey < E
        counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))[:E]
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
        offsets[1:] = counts.cumsum(0)
        tok = order // k
        st["row_token"].copy_(torch.where(here, tok.to(torch.int32), st["row_token"]))
        token_row = torch.empty_like(key)
        token_row[order] = torch.where(here, torch.arange(T * k, device=flat.device), -1)
        st["x_perm"].copy_(torch.where(here[:, None], st["x"][tok], st["x_perm"]))
        return dict(counts=counts.to(torch.int32), offsets=offsets, row_token=st["row_token"],
                    token_row=token_row.to(torch.int32).reshape(T, k), x_perm=st["x_perm"])
    row, tok = st["token_row"].long(), st["tok"]
    here = row >= 0
    safe = row.clamp(min=0)
    if op in ("sort_bwd", "unsort"):
        acc = torch.zeros(T, case["d"], device=tok.device)
        for j in range(k):
            w = here[:, j].float() if op == "sort_bwd" else torch.where(here[:, j], st["w"][:, j], 0.0)
            acc = acc + w[:, None] * st["rows"][safe[:, j]].float()
        return {"dx" if op == "sort_bwd" else "y": (acc + tok.float()).to(tok.dtype)}
    dy = tok.float()
    dw = torch.stack([(dy * st["rows"][safe[:, j]].float()).sum(1) for j in range(k)], 1)
    R = T * k
    route = torch.full((R + 1,), R, dtype=torch.int64, device=tok.device)
    route[torch.where(here, row, R).reshape(-1)] = torch.arange(R, device=tok.device)
    route[R] = R
    route = route[:R]
    used, src = route < R, route.clamp(max=R - 1)
    do = st["w"].reshape(-1)[src][:, None] * dy[src // k]
    st["do_perm"].copy_(torch.where(used[:, None], do.to(tok.dtype), st["do_perm"]))
    return dict(do_perm=st["do_perm"], dtopk_w=torch.where(here, dw, 0.0))


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def _valid_routes(case):
    """Expected number of routes that are here."""
    n, a = case["T"] * case["k"], case["absent"]
    if a == "padding":
        return n * 7 / 8
    if a == "dropped":
        return n * 9 / 10
    return n / int(a[5:]) if a.startswith("share") else n


def work(case):
    op = case["op"]
    if op == "clip":
        n = [(math.prod(s), _TYPES[t].itemsize) for s, t in _parse_sizes(case)]
        return dict(bytes=sum(2 * c * b for c, b in n) + 4, flops=sum(3 * c for c, _ in n))
    T, d, b = case["T"], case["d"], _TYPES[case["prec"]].itemsize
    if op in ("norm", "norm_bwd"):
        rb = 4 if case["res_f32"] else b
        rows = 0 if case["gate"] == "none" else -(-T // _gate_every(case))
        vec = (1 + case["post"] + rows) * d * 4 * (1 if op == "norm" else 2) + (1 + case["post"]) * T * 4
        n = 2 if op == "norm" else 3
        return dict(bytes=n * T * d * (b + rb) + vec, flops=(10 if op == "norm" else 22) * T * d)
    V, ids = _valid_routes(case), 4 * T * case["k"]
    if op == "sort":
        return dict(bytes=(T + V) * d * b + 2 * ids + 4 * V + 8 * case["E"] + 4, flops=0)
    if op == "unsort_bwd":
        return dict(bytes=(T + 2 * V) * d * b + 3 * ids, flops=3 * V * d)
    return dict(bytes=(V + 2 * T) * d * b + ids * (2 if op == "unsort" else 1), flops=2 * V * d)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "clip":
        ss = torch.zeros((), dtype=f64, device="cuda")
        for g in st["grads"]:
            flat = g.reshape(-1).to(f64)
            ss += torch.dot(flat, flat)
        norm = math.sqrt(ss.item())
        c = min(1.0, 1.0 / (norm + 1e-6))
        out = {name: torch.cat([g.reshape(-1).to(f64) * c for g in st["grads"] if g.dtype == _TYPES[name]])
               for name in st["flat"]}
        return dict(out, norm=torch.full((1,), norm, dtype=f64, device="cuda"))
    T, d = case["T"], case["d"]
    if op in ("norm", "norm_bwd"):
        return _exact_norm(case, st) if op == "norm" else _exact_norm_bwd(case, st)
    E, k = case["E"], case["k"]
    if op == "sort":
        ids = st["idx"].reshape(-1).cpu().tolist()
        lists = [[] for _ in range(E)]
        for r, e in enumerate(ids):
            if 0 <= e < E:
                lists[e].append(r)
        counts = [len(v) for v in lists]
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        routes = [r for v in lists for r in v]
        token_row = [-1] * len(ids)
        for row, r in enumerate(routes):
            token_row[r] = row
        i32 = dict(dtype=torch.int32, device="cuda")
        x_perm, row_token = st["x_perm"].to(f64), st["row_token"].clone()
        if routes:
            src = torch.tensor(routes, dtype=torch.int64, device="cuda") // k
            x_perm[:len(routes)] = st["x"].to(f64)[src]
            row_token[:len(routes)] = src.to(torch.int32)
        return dict(counts=torch.tensor(counts, **i32), offsets=torch.tensor(offsets, **i32), row_token=row_token,
                    token_row=torch.tensor(token_row, **i32).reshape(T, k), x_perm=x_perm)
    # the routes that are here, one list of (route, row) pairs
    row = st["token_row"].reshape(-1).long()
    route = torch.nonzero(row >= 0).reshape(-1)
    row, tok = row[route], route // k
    if op in ("sort_bwd", "unsort"):
        y = st["tok"].to(f64)
        for c in range(0, d, 1024):  # column slices bound the memory
            v = st["rows"][:, c:c + 1024].to(f64)[row]
            if op == "unsort":
                v = v * st["w"].reshape(-1)[route].to(f64)[:, None]
            y[:, c:c + 1024].index_add_(0, tok, v)
        return {"dx" if op == "sort_bwd" else "y": y}
    dy = st["tok"].to(f64)
    dw = torch.zeros(T * k, dtype=f64, device="cuda")
    do = st["do_perm"].to(f64)
    w = st["w"].reshape(-1).to(f64)
    for c in range(0, route.numel(), 8192):
        r, p, t = route[c:c + 8192], row[c:c + 8192], tok[c:c + 8192]
        dw[r] = (dy[t] * st["rows"][p].to(f64)).sum(1)
        do[p] = w[r][:, None] * dy[t]
    return dict(do_perm=do, dtopk_w=dw.reshape(T, k))


def _groups(case, dev="cuda"):
    """Gate row of every token."""
    return torch.div(torch.arange(case["T"], device=dev), _gate_every(case), rounding_mode="floor")


def _exact_norm(case, st):
    f64, d = torch.float64, case["d"]
    out = {}
    y = st["y"].to(f64)
    scale = torch.full((case["T"], 1), case["beta"], dtype=f64, device="cuda")
    if case["post"]:
        rms = (y.pow(2).sum(1) / d + 1e-6).sqrt()
        out["r_post"] = 1.0 / rms
        scale = scale / rms[:, None]
        y *= st["w_post"].to(f64)
    if st["gate"] is not None:
        y *= st["gate"].to(f64)[_groups(case)]
    y *= scale
    y.add_(st["x"].to(f64), alpha=case["alpha"])
    rms = (y.pow(2).sum(1) / d + 1e-6).sqrt()
    out["r_pre"] = 1.0 / rms
    out["a"] = y / rms[:, None] * st["w_pre"].to(f64)
    out["x_out"] = y
    return out


def _exact_norm_bwd(case, st):
    """Jacobian by rows: d(v r)/dv applied to a gradient q is r q - v r^3 <q, v> / d."""
    f64, T, d = torch.float64, case["T"], case["d"]
    out = dict(dw_pre=torch.zeros(d, dtype=f64, device="cuda"))
    if case["post"]:
        out["dw_post"] = torch.zeros(d, dtype=f64, device="cuda")
    if st["gate"] is not None:
        out["dgate"] = torch.zeros(st["gate"].shape, dtype=f64, device="cuda")
    out["dx"] = torch.empty(T, d, dtype=f64, device="cuda")
    out["dy"] = torch.empty(T, d, dtype=f64, device="cuda")
    group = _groups(case)
    one = torch.ones(d, dtype=f64, device="cuda")
    for a in range(0, T, 2048):
        s = slice(a, min(a + 2048, T))
        z, y, da = st["x"][s].to(f64), st["y"][s].to(f64), st["da"][s].to(f64)
        r2 = st["r_pre"][s].to(f64)[:, None]
        out["dw_pre"] += (da * z * r2).sum(0)
        q = da * st["w_pre"].to(f64)
        dz = st["dx_out"][s].to(f64) + r2 * q - z * r2 ** 3 * ((q * z).sum(1, keepdim=True) / d)
        out["dx"][s] = case["alpha"] * dz
        r1 = st["r_post"][s].to(f64)[:, None] if case["post"] else 1.0
        w1 = st["w_post"].to(f64) if case["post"] else one
        gate = st["gate"].to(f64)[group[s]] if st["gate"] is not None else 1.0
        if st["gate"] is not None:
            out["dgate"].index_add_(0, group[s], case["beta"] * dz * y * r1 * w1)
        if case["post"]:
            out["dw_post"] += (case["beta"] * dz * gate * y * r1).sum(0)
        q = case["beta"] * gate * w1 * dz
        if case["post"]:
            q = r1 * q - y * r1 ** 3 * ((q * y).sum(1, keepdim=True) / d)
        out["dy"][s] = q
    return out
