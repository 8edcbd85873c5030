"""Speed cases of the operators that serve an MoE layer in 8 and 4 bits: block
norms that give E4M3 codes and scales, the sort of such rows by expert, expert
weights rounded to E2M1 codes with a scale per 32, and the routed experts of a
few tokens on those weights.

`listed()` names the cases, `draw(rng)` makes more of the same ranges,
`prepare` makes a case's inputs on the GPU, `run` is one pass through the
operator (plain torch in 32 bits, or the library's kernels where `own` is
true), `work` counts what a pass cannot do without and `exact` gives its
outputs from the definition in 64 bits.
"""
import math

import torch

own = False

_F8, _E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _norm(name, T, d, res_f32=False, post=True, gate="one", keep_a=True, alpha=1.0, beta=1.0):
    return dict(name=name, op="norm", T=T, d=d, res_f32=res_f32, post=post, gate=gate, keep_a=keep_a, alpha=alpha,
                beta=beta)


def _sort(name, T, d, E, k, absent="none"):
    return dict(name=name, op="sort", T=T, d=d, E=E, k=k, absent=absent)


def _ffn(name, T, d, E, k, I, absent="none", add=True):
    return dict(name=name, op="ffn", T=T, d=d, E=E, k=k, I=I, absent=absent, add=add)


def listed():
    return [
        # One decoded token between two layers: residual add, the next block's norm, its codes.
        _norm("norm_token", 1, 7168, post=False, gate="none"),
        # A prompt's tokens: norms on both sides of the block, a learned gate per channel, bf16 throughout.
        _norm("norm_batch", 8192, 7168, alpha=0.75, beta=0.5),
        # Ragged sizes: 63 scale blocks a row, sequences of 100 tokens each with a gate of its own, the residual
        # stream in fp32, codes alone.
        _norm("norm_odd", 1531, 2016, res_f32=True, gate="seq100", keep_a=False),
        # Sixteen decoded tokens sent to their experts.
        _sort("sort_decode", 16, 7168, 256, 8),
        # A padded prompt batch: an eighth of its tokens hold no routes.
        _sort("sort_batch", 8192, 7168, 256, 8, absent="padding"),
        # One matrix of a small layer's shared expert to 4 bits and back.
        dict(name="round4_small", op="round4", rows=768, d=2048),
        # The gate projections of 32 experts to 4 bits and back.
        dict(name="round4_experts", op="round4", rows=32 * 2048, d=7168),
        # One decoded token through 8 of 256 experts.
        _ffn("ffn_token", 1, 7168, 256, 8, 2048),
        # Sixteen decoded tokens, about 100 experts between them.
        _ffn("ffn_decode", 16, 7168, 256, 8, 2048),
        # 256 tokens on one of eight ranks: 32 of 256 experts, most routes are another rank's.
        _ffn("ffn_share", 256, 7168, 32, 8, 2048, absent="share8", add=False),
        # Five tokens (one and its drafts) of a small layer.
        _ffn("ffn_small", 5, 2048, 64, 6, 768),
        # An odd batch that reaches every expert of a middle-sized layer, some routes dropped.
        _ffn("ffn_batch", 333, 4096, 128, 8, 1536, absent="dropped"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case; one that would move more bytes or compute more than the
    largest listed case is halved until it does not."""
    case = _draw(rng)
    most = {n: max(work(c)[n] for c in listed()) for n in ("bytes", "flops")}
    while any(work(case)[n] > most[n] for n in most):
        key = "rows" if case["op"] == "round4" else "T" if case["op"] != "ffn" or case["T"] > 1 else "I"
        case[key] = max(128, case[key] // 256 * 128) if key == "I" else case[key] // 2
    return case


def _draw(rng):
    op = rng.choice(["norm", "sort", "round4", "ffn", "ffn"])
    wide = lambda step, most: max(step, _log_int(rng, step, most) // step * step)  # noqa: E731
    if op == "norm":
        return dict(op=op, T=_log_int(rng, 1, 16384), d=wide(32, 7168), res_f32=rng.random() < 0.4,
                    post=rng.random() < 0.6, gate=rng.choice(["none", "one", "seq%d" % _log_int(rng, 1, 4096)]),
                    keep_a=rng.random() < 0.6, alpha=rng.choice([1.0, 0.5, 0.875]), beta=rng.choice([1.0, 0.25, 1.5]))
    if op == "round4":
        return dict(op=op, rows=_log_int(rng, 1, 65536), d=wide(128, 7168))
    E = _log_int(rng, 1, 256)
    k = rng.randint(1, min(E, 8))
    absent = rng.choice(["none", "padding", "dropped", "share%d" % rng.choice([2, 4, 8])])
    if op == "sort":
        return dict(op=op, T=_log_int(rng, 1, 8192), d=wide(32, 7168), E=E, k=k, absent=absent)
    return dict(op=op, T=_log_int(rng, 1, 512), d=wide(128, 7168), E=E, k=k, I=wide(128, 2048), absent=absent,
                add=rng.random() < 0.7)


# --------------------------------------------------------------------------
# Blocks of 32 with a power-of-two scale, in 32 bits
# --------------------------------------------------------------------------
def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], from its bits: a power function
    is not exact for every one of them."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).view(torch.float32)


def _block_exp(v, top_exp, top_mant):
    """Exponents [..., n/32] of the finest scales at which no block's largest
    value passes the element type's largest, 2 top_mant 2^top_exp."""
    m, e = torch.frexp(v.unflatten(-1, (-1, 32)).abs().amax(-1))
    e = e - 1 - top_exp + (m > top_mant).to(e.dtype)
    return torch.where(m > 0, e.clamp(-127, 127), -127)


def _quantize8(v):
    """E4M3 codes [..., n] and E8M0 scales [..., n/32] of fp32 values."""
    e = _block_exp(v, 8, 0.875)
    codes = (v.unflatten(-1, (-1, 32)) * _pow2(-e)[..., None]).to(_F8)
    return codes.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


def _values8(codes, scale):
    v = codes.view(_F8).float().unflatten(-1, (-1, 32))
    return (v * _pow2(scale.to(torch.int32) - 127)[..., None]).flatten(-2)


def _quantize4(w):
    """E2M1 codes [rows][n/2] (the even element in the low half) and E8M0
    scales [n/128][rows][4] of fp32 values [rows][n]."""
    e = _block_exp(w, 2, 0.75)
    s = (w.unflatten(-1, (-1, 32)) * _pow2(-e)[..., None]).flatten(-2)
    a = s.abs()
    # half way between two values the one with the even code is taken
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
         + (torch.signbit(s).to(torch.uint8) << 3))
    return c[:, 0::2] | (c[:, 1::2] << 4), (e + 127).to(torch.uint8).unflatten(-1, (-1, 4)).transpose(0, 1).contiguous()


def _pairs(device="cuda"):
    """The two values of every byte of codes, [256][2]."""
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    v += [-x for x in v]
    return torch.tensor([[v[b & 15], v[b >> 4]] for b in range(256)], device=device)


def _values4(codes, scale, pairs):
    """fp32 values [..., n] of codes [..., n/2] and scales [..., n/32]."""
    v = pairs[codes.to(torch.int32)].flatten(-2).unflatten(-1, (-1, 32))
    return (v * _pow2(scale.to(torch.int32) - 127)[..., None]).flatten(-2)


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


def _make_routes(case, g):
    """Expert ids [T][k] (distinct, ascending) and router weights; ids outside
    [0, E) stand for routes that are not here."""
    T, E, k, absent = case["T"], case["E"], case["k"], case["absent"]
    total = E * int(absent[5:]) if absent.startswith("share") else E
    top, idx = torch.topk(torch.rand(T, total, generator=g, device="cuda"), k, dim=1)
    idx, order = torch.sort(idx, dim=1)
    w = torch.softmax(4.0 * torch.gather(top, 1, order), dim=1)
    if absent.startswith("share"):
        idx = idx - (total - E) // 2  # the local experts are the middle ones
    elif absent == "padding":
        idx = torch.where((torch.rand(T, 1, generator=g, device="cuda") < 0.125), -1, idx)
    elif absent == "dropped":
        idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, idx)
    return idx.to(torch.int32).contiguous(), w.contiguous()


def _make_weights(g, E, rows, cols):
    """Codes [E][rows][cols/2] and scales [cols/128][E rows][4] of normally
    distributed bf16 weights."""
    codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(cols // 128, E, rows, 4, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (rows * cols))
    for e in range(0, E, step):
        n = min(step, E - e)
        c, s = _quantize4(_randn(g, (n * rows, cols), torch.bfloat16, cols ** -0.5).float())
        codes[e:e + n] = c.view(n, rows, cols // 2)
        scale[:, e:e + n] = s.view(-1, n, rows, 4)
    return codes, scale.view(-1, E * rows, 4)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case=case)
    bf, d = torch.bfloat16, case["d"]
    if op == "round4":
        st["w"] = _randn(g, (case["rows"], d), bf, d ** -0.5)
        st["pairs"] = _pairs()
        return st
    T = case["T"]
    if op == "norm":
        every, post = _gate_every(case), case["post"]
        st["w_pre"] = 1.0 + _randn(g, (d,), torch.float32, 0.1)
        st["w_post"] = 1.0 + _randn(g, (d,), torch.float32, 0.1) if post else None
        st["gate"] = None if case["gate"] == "none" else _randn(g, ((T + every - 1) // every, d), torch.float32, 0.7)
        st["y"] = _randn(g, (T, d), bf)
        st["x"] = _randn(g, (T, d), torch.float32 if case["res_f32"] else bf, 2.0)
        if own:
            import mixture_experts_layer_prefix_amd as M
            st["plan"] = M.BlockNormMxfp8Plan(
                M.Block(T, d, "bf16", res_f32=case["res_f32"], post_norm=post, alpha=case["alpha"], beta=case["beta"],
                        eps=1e-6, gate_every=every), keep_a=case["keep_a"])
        return st
    st["idx"], st["w"] = _make_routes(case, g)
    st["x"], st["x_scale"] = _quantize8(_randn(g, (T, d), bf).float())
    E, k = case["E"], case["k"]
    if op == "sort":
        st["x_perm"] = torch.zeros(T * k, d, dtype=torch.uint8, device="cuda")
        st["x_perm_scale"] = torch.full((T * k, d // 32), 127, dtype=torch.uint8, device="cuda")
        st["row_token"] = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        if own:
            import mixture_experts_layer_prefix_amd as M
            st["plan"] = M.SortMxfp8Plan(M.Dims(T, d, E, k, 1), x_perm=st["x_perm"], x_perm_scale=st["x_perm_scale"],
                                         row_token=st["row_token"])
        return st
    I = case["I"]
    for name, rows, cols in (("gate", I, d), ("up", I, d), ("down", d, I)):
        st["q_" + name], st["q_%s_scale" % name] = _make_weights(g, E, rows, cols)
    st["y_add"] = _randn(g, (T, d), bf, 0.5) if case["add"] else None
    st["pairs"] = _pairs()
    if own:
        import mixture_experts_layer_prefix_amd as M
        st["weights"] = M.WeightsMxfp4(**{n: st[n] for n in st if n.startswith("q_")})
        st["plan"] = M.RoutedFfnPlan(M.Dims(T, d, E, k, I))
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import mixture_experts_layer_prefix_amd as M
    case = st["case"]
    op = case["op"]
    if op == "round4":
        return dict(w=M.dequantize_mxfp4(*M.quantize_mxfp4(st["w"])))
    plan = st["plan"]
    if op == "norm":
        x_out, a_q, a_scale = plan.run(st["x"], st["y"], w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"])
        out = dict(x_out=x_out, a_q=a_q.view(_F8), a_scale=a_scale.view(_E8), r_pre=plan.r_pre)
        if case["keep_a"]:
            out["a"] = plan.a
        if case["post"]:
            out["r_post"] = plan.r_post
        return out
    if op == "sort":
        counts, offsets, row_token, token_row, x_perm, x_perm_scale = plan.run(st["idx"], st["x"], st["x_scale"])
        return dict(counts=counts, offsets=offsets, row_token=row_token, token_row=token_row, x_perm=x_perm.view(_F8),
                    x_perm_scale=x_perm_scale.view(_E8))
    return dict(y=plan.run(st["x"], st["x_scale"], st["idx"], st["w"], st["weights"], y_add=st["y_add"]))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "round4":
        codes, scale = _quantize4(st["w"].float())
        return dict(w=_values4(codes, scale.transpose(0, 1).flatten(-2), st["pairs"]).to(torch.bfloat16))
    if op == "norm":
        return _plain_norm(st)
    if op == "sort":
        return _plain_sort(st)
    return _plain_ffn(st)


def _plain_norm(st):
    case = st["case"]
    x, n = st["x"].float(), st["y"].float()
    out = {}
    if case["post"]:
        r = torch.rsqrt((n * n).mean(1, keepdim=True) + 1e-6)
        n = n * r * st["w_post"]
        out["r_post"] = r[:, 0]
    gate = st["gate"]
    if gate is not None:
        n = n * (gate if gate.shape[0] == 1 else gate.repeat_interleave(_gate_every(case), dim=0)[:case["T"]])
    z = case["alpha"] * x + case["beta"] * n
    r = torch.rsqrt((z * z).mean(1, keepdim=True) + 1e-6)
    a = (z * r * st["w_pre"]).to(torch.bfloat16)
    codes, scale = _quantize8(a.float())  # of the rounded a, which the router and the shared expert take
    out.update(x_out=z.to(st["x"].dtype), a_q=codes.view(_F8), a_scale=scale.view(_E8), r_pre=r[:, 0])
    if case["keep_a"]:
        out["a"] = a
    return out


def _plain_sort(st):
    T, E, k = (st["case"][n] for n in ("T", "E", "k"))
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
    st["x_perm_scale"].copy_(torch.where(here[:, None], st["x_scale"][tok], st["x_perm_scale"]))
    return dict(counts=counts.to(torch.int32), offsets=offsets, row_token=st["row_token"],
                token_row=token_row.to(torch.int32).reshape(T, k), x_perm=st["x_perm"].view(_F8),
                x_perm_scale=st["x_perm_scale"].view(_E8))


def _expert_values(st, name, rows, chosen=None):
    """fp32 weights [experts][rows][cols] of all experts, or of the chosen ones."""
    codes, scale = st["q_" + name], st["q_%s_scale" % name]
    scale = scale.unflatten(1, (-1, rows)).permute(1, 2, 0, 3)
    if chosen is not None:
        codes, scale = codes[chosen], scale[chosen]
    return _values4(codes, scale.flatten(-2), st["pairs"])


def _plain_ffn(st):
    """Few routes: every route's expert is unpacked by itself.  Many: all
    experts are, and each of the three products is one over all of them."""
    T, d, E, k, I = (st["case"][n] for n in ("T", "d", "E", "k", "I"))
    x, idx = _values8(st["x"], st["x_scale"]), st["idx"].long()
    here = (idx >= 0) & (idx < E)
    idx = torch.where(here, idx, 0)
    w = torch.where(here, st["w"], 0.0)
    few = T * k <= E
    if few:
        chosen = idx.reshape(-1)
        xr = x.repeat_interleave(k, dim=0)[..., None]
        gate, up = (torch.matmul(_expert_values(st, n, I, chosen), xr)[..., 0].view(T, k, I) for n in ("gate", "up"))
    else:
        at = idx[..., None].expand(T, k, I)
        gate, up = (torch.matmul(x, _expert_values(st, n, I).view(E * I, d).t()).view(T, E, I).gather(1, at)
                    for n in ("gate", "up"))
    h = _values8(*_quantize8(gate / (1.0 + torch.exp(-gate)) * up))
    if few:
        o = torch.matmul(_expert_values(st, "down", d, chosen), h.view(T * k, I, 1)).view(T, k, d)
        y = (w[..., None] * o).sum(1)
    else:
        hw = torch.zeros(T, E, I, device=x.device).scatter_add_(1, at, w[..., None] * h)
        down = _expert_values(st, "down", d).transpose(1, 2)
        y = torch.matmul(hw.view(T, E * I), down.reshape(E * I, d))
    if st["y_add"] is not None:
        y = y + st["y_add"].float()
    return dict(y=y.to(torch.bfloat16))


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def _present(case):
    """Expected routes that are here, and experts that they reach."""
    T, E, k, a = case["T"], case["E"], case["k"], case["absent"]
    keep = 7 / 8 if a == "padding" else 9 / 10 if a == "dropped" else 1.0
    ranks = int(a[5:]) if a.startswith("share") else 1
    return T * k * keep / ranks, E * (1.0 - (1.0 - keep * k / (E * ranks)) ** T)


def work(case):
    op, d = case["op"], case["d"]
    if op == "round4":
        n = case["rows"] * d
        return dict(bytes=2 * (2 + 17 / 32) * n, flops=0)
    T = case["T"]
    if op == "norm":
        rows = 0 if case["gate"] == "none" else -(-T // _gate_every(case))
        vec = (1 + case["post"] + rows) * d * 4 + (1 + case["post"]) * T * 4
        per = 2 * (4 if case["res_f32"] else 2) + 2 + 2 * case["keep_a"] + 33 / 32
        return dict(bytes=per * T * d + vec, flops=12 * T * d)
    routes, experts = _present(case)
    ids = 4 * T * case["k"]
    if op == "sort":
        return dict(bytes=(T + routes) * d * 33 / 32 + 2 * ids + 4 * routes + 8 * case["E"] + 4, flops=0)
    weights = 3 * case["I"] * d
    return dict(bytes=experts * weights * 17 / 32 + T * d * (33 / 32 + 2 + 2 * case["add"]) + 2 * ids,
                flops=2 * routes * weights)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
_f64 = torch.float64


def _power(e):
    """2^e in fp64 for whole e, from its bits."""
    return (e.to(torch.int64) + 1023 << 52).view(_f64)


def _exact_round(v, mant, low, top):
    """Blocks of 32 of fp64 values rounded to elements of `mant` mantissa bits,
    smallest normal exponent `low` and largest value `top`: (elements, block
    exponents)."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -200) / top))
    e = torch.where(amax > top * _power(e), e + 1, e)  # where the logarithm was off by one step
    e = torch.where(amax <= top * _power(e - 1), e - 1, e)
    e = e.clamp(-127, 127)
    s = b / _power(e)
    binade = torch.floor(torch.log2(s.abs().clamp(min=2.0 ** low)))
    binade = torch.where(_power(binade + 1) <= s.abs(), binade + 1, binade)
    binade = torch.where(_power(binade) > s.abs().clamp(min=2.0 ** low), binade - 1, binade)
    step = _power(binade - mant)
    return (torch.round(s / step) * step).reshape(v.shape), e[..., 0]


def _exact_values(elements, e):
    return (elements.reshape(*e.shape, 32) * _power(e)[..., None]).reshape(elements.shape)


def _decode(bits, exp_bits, mant, bias):
    """fp64 values of sign, exponent and mantissa fields."""
    b = bits.to(torch.int64)
    m = (b & ((1 << mant) - 1)).to(_f64) / (1 << mant)
    f = (b >> mant) & ((1 << exp_bits) - 1)
    v = torch.where(f == 0, m * 2.0 ** (1 - bias), (1.0 + m) * _power(f - bias))
    return torch.where((b >> (mant + exp_bits)) & 1 == 1, -v, v)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "round4":
        w = st["w"]
        out = torch.empty(w.shape, dtype=_f64, device=w.device)
        for a in range(0, w.shape[0], 8192):
            out[a:a + 8192] = _exact_values(*_exact_round(w[a:a + 8192].to(_f64), 1, 0, 6.0))
        return dict(w=out)
    if op == "norm":
        return _exact_norm(case, st)
    if op == "sort":
        return _exact_sort(case, st)
    return _exact_ffn(case, st)


def _exact_norm(case, st):
    T, d = case["T"], case["d"]
    out = {}
    y = st["y"].to(_f64)
    scale = torch.full((T, 1), case["beta"], dtype=_f64, device="cuda")
    if case["post"]:
        rms = (y.pow(2).sum(1) / d + 1e-6).sqrt()
        out["r_post"] = 1.0 / rms
        scale = scale / rms[:, None]
        y *= st["w_post"].to(_f64)
    if st["gate"] is not None:
        y *= st["gate"].to(_f64)[torch.div(torch.arange(T, device="cuda"), _gate_every(case), rounding_mode="floor")]
    y *= scale
    y.add_(st["x"].to(_f64), alpha=case["alpha"])
    rms = (y.pow(2).sum(1) / d + 1e-6).sqrt()
    a = y / rms[:, None] * st["w_pre"].to(_f64)
    out.update(x_out=y, r_pre=1.0 / rms)
    if case["keep_a"]:
        out["a"] = a
    out["a_q"], e = _exact_round(a.to(torch.bfloat16).to(_f64), 3, -6, 448.0)
    out["a_scale"] = _power(e)
    return out


def _exact_sort(case, st):
    T, d, E, k = (case[n] for n in ("T", "d", "E", "k"))
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
    x_perm, row_token = torch.zeros(T * k, d, dtype=_f64, device="cuda"), torch.full((T * k,), -1, **i32)
    scale = torch.ones(T * k, d // 32, dtype=_f64, device="cuda")
    if routes:
        src = torch.tensor(routes, dtype=torch.int64, device="cuda") // k
        n = len(routes)
        x_perm[:n] = _decode(st["x"], 4, 3, 7)[src]
        scale[:n] = _power(st["x_scale"].to(torch.int64) - 127)[src]
        row_token[:n] = src.to(torch.int32)
    return dict(counts=torch.tensor(counts, **i32), offsets=torch.tensor(offsets, **i32), row_token=row_token,
                token_row=torch.tensor(token_row, **i32).reshape(T, k), x_perm=x_perm, x_perm_scale=scale)


def _exact_ffn(case, st):
    """Expert by expert, over the routes that chose it."""
    T, d, E, k, I = (case[n] for n in ("T", "d", "E", "k", "I"))
    x = _exact_values(_decode(st["x"], 4, 3, 7), st["x_scale"].to(_f64) - 127.0)
    y = torch.zeros(T, d, dtype=_f64, device="cuda") if st["y_add"] is None else st["y_add"].to(_f64)

    def weights(name, e, rows):
        codes = st["q_" + name][e]
        v = torch.stack([_decode(codes & 15, 2, 1, 1), _decode(codes >> 4, 2, 1, 1)], -1).reshape(rows, -1)
        s = st["q_%s_scale" % name][:, e * rows:(e + 1) * rows].to(_f64) - 127.0
        return _exact_values(v, s.permute(1, 0, 2).reshape(rows, -1))

    ids = st["idx"].cpu().tolist()
    for e in range(E):
        at = [(t, j) for t in range(T) for j in range(k) if ids[t][j] == e]
        if not at:
            continue
        tok, slot = (torch.tensor(v, device="cuda") for v in zip(*at))
        g, u = (x[tok] @ weights(n, e, I).t() for n in ("gate", "up"))
        h = _exact_values(*_exact_round(g * torch.sigmoid(g) * u, 3, -6, 448.0))
        y.index_add_(0, tok, st["w"].to(_f64)[tok, slot][:, None] * (h @ weights("down", e, d).t()))
    return dict(y=y)
