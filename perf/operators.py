"""The operators of grouped routing and of 8-bit routed experts, as they are measured.

Five operators around the routed experts of the layer:

route           scores of the experts from router logits (sigmoid, or softmax over all experts), a selection
                bias, groups of experts of which the best are kept, top-k, weights renormalised and scaled
route_backward  the gradient of the logits from the gradient of those weights
quantize        e4m3 values with one power-of-two scale (E8M0) for each 128 columns of a row, the rows taken
                through an index; or for each 128 x 128 block of stacked weight matrices
expert_gemm     the product of quantised rows with the quantised weights of the expert that each row belongs to
expert_ffn      the routed experts as a whole: rows of z quantised, gate and up products, SiTU, the hidden
                units quantised, output product

Where ``own`` is false ``run`` computes them in elementary torch operations, in 32 bits.

Formats.  A block's scale is 2^e with the smallest e >= -126 for which its largest magnitude is at most 448
scales; it is kept as the byte e + 127.  Rows [n, c]: scales [ceil(c / 512), n, 4], block b of row r at
[b // 4, r, b % 4].  Matrices [m, r, c]: scales [m, ceil(r / 128), 4 ceil(c / 512)].  Bytes past the last
block are 127.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
DEV = "cuda"
BETA1, BETA2 = 4.0, 25.0
CLAMP = 1e-9  # the least sum that weights are divided by


# ------------------------------------------------------------------ cases
def _route(name, op, n, experts, k, score, groups=1, kept=1, group_score="top2", renorm=True, scale=1.0):
    return {"name": name, "op": op, "n": n, "experts": experts, "k": k, "score": score, "groups": groups,
            "kept": kept, "group_score": group_score, "renorm": renorm, "scale": scale}


def listed():
    return [
        # one decode step of 64 sequences at the K3 width: latency
        _route("route_decode", "route", 64, 896, 16, "sigmoid", 14, 7, "top2", True, 2.5),
        # a training batch of the mid layer: softmax scores, weights as they are
        _route("route_softmax", "route", 16384, 64, 8, "softmax", 1, 1, "max", False, 1.0),
        # a prompt batch at the K3 width, the experts in groups
        _route("route_groups", "route", 8192, 896, 16, "sigmoid", 14, 7, "top2", True, 2.5),
        # the 0.5b layer's training step
        _route("route_backward_small", "route_backward", 4096, 16, 2, "sigmoid"),
        # dense gradients of softmax scores over many experts
        _route("route_backward_softmax", "route_backward", 8192, 896, 16, "softmax", 1, 1, "max", False, 2.5),
        # the mid layer's latent rows in expert order
        {"name": "quantize_rows", "op": "quantize", "what": "rows", "src": 16384, "rows": 131072, "cols": 1024,
         "dtype": "bf16"},
        # fp32 master weights of the 0.5b layer's experts, after an update
        {"name": "quantize_weights", "op": "quantize", "what": "weights", "mats": 16, "rows": 768, "cols": 384,
         "dtype": "f32"},
        # one dense projection: a single expert that has every row, ragged sizes
        {"name": "gemm_dense", "op": "expert_gemm", "n": 1000, "experts": 1, "k": 1, "n_in": 784, "n_out": 392,
         "dtype": "bf16", "skew": 0.0},
        # the mid layer's output projections
        {"name": "gemm_mid", "op": "expert_gemm", "n": 16384, "experts": 64, "k": 8, "n_in": 1024, "n_out": 1024,
         "dtype": "bf16", "skew": 0.0},
        # one decode step of 64 sequences at the K3 width: the weights of some 600 experts are read for a row or two each
        {"name": "ffn_decode", "op": "expert_ffn", "n": 64, "experts": 896, "k": 16, "latent": 3584, "ff": 512,
         "dtype": "bf16", "skew": 0.0},
        # the mid layer: compute
        {"name": "ffn_mid", "op": "expert_ffn", "n": 16384, "experts": 64, "k": 8, "latent": 1024, "ff": 1024,
         "dtype": "bf16", "skew": 0.0},
        # a prompt batch at the K3 width: about 146 rows for each expert
        {"name": "ffn_prompt", "op": "expert_ffn", "n": 8192, "experts": 896, "k": 16, "latent": 3584, "ff": 512,
         "dtype": "bf16", "skew": 0.3},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "quantize", "expert_gemm", "expert_ffn"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 3, 4, 7, 8, 14, 16])
        experts = groups * _log_int(rng, max(2, 8 // groups), 1024 // groups)
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(32, kept * (experts // groups)))
        # one renormalised weight is constant: it has no gradient
        renorm = rng.random() < 0.7 and not (op == "route_backward" and k == 1)
        case = _route("", op, _log_int(rng, 1, 16384), experts, k, rng.choice(["sigmoid", "softmax"]), groups, kept,
                      rng.choice(["top2", "max"]), renorm, rng.choice([1.0, 2.5]))
        del case["name"]
        return case
    if op == "quantize":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.5:
            src = _log_int(rng, 1, 16384)
            return {"op": op, "what": "rows", "src": src, "rows": src * rng.randint(1, 8),
                    "cols": 16 * _log_int(rng, 1, 64), "dtype": dtype}
        return {"op": op, "what": "weights", "mats": _log_int(rng, 1, 64), "rows": 8 * _log_int(rng, 1, 128),
                "cols": 16 * _log_int(rng, 1, 64), "dtype": dtype}
    experts = _log_int(rng, 1, 128)
    case = {"op": op, "n": _log_int(rng, 1, 8192), "experts": experts, "k": rng.randint(1, min(8, experts)),
            "dtype": "bf16", "skew": rng.choice([0.0, 0.5, 2.0])}
    if op == "expert_gemm":
        case.update(n_in=16 * _log_int(rng, 1, 128), n_out=8 * _log_int(rng, 1, 256))
    else:
        case.update(latent=16 * _log_int(rng, 2, 96), ff=16 * _log_int(rng, 2, 64))
    return case


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _keys64(case, logits, bias):
    """Selection keys in 64 bits."""
    x = logits.double()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    return s + bias.double()


def _near_tie(case, logits, bias):
    """Rows whose choice of groups, choice of experts or order hangs on a difference that 32 bits do not hold."""
    key = _keys64(case, logits, bias)
    n, experts = key.shape
    groups, kept, k = case["groups"], case["kept"], case["k"]
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    if kept < groups:
        by = key.view(n, groups, -1).sort(2, descending=True).values
        gs = by[..., :2].sum(2) if case["group_score"] == "top2" else by[..., 0]
        order = gs.sort(1, descending=True)
        bad |= order.values[:, kept - 1] - order.values[:, kept] < 1e-5 * order.values[:, kept - 1].abs() + 1e-7
        keep = torch.zeros(n, groups, dtype=torch.bool, device=DEV).scatter_(1, order.indices[:, :kept], True)
        key = key.masked_fill(~keep.repeat_interleave(experts // groups, 1), -math.inf)
    top = key.topk(min(k + 1, experts), 1).values
    gap = top[:, :-1] - top[:, 1:]
    return bad | (gap < 1e-5 * top[:, :-1].abs() + 1e-7).any(1)


def _route_inputs(case, seed):
    """Logits of a router over inputs of unit variance, a balance bias, no near ties (rows are drawn again)."""
    g = _gen(seed)
    n, experts = case["n"], case["experts"]
    bias = 0.05 * _randn(g, experts)
    if case["score"] == "softmax":
        bias /= experts
    logits = 1.2 * _randn(g, n, experts)
    for _ in range(8):
        at = _near_tie(case, logits, bias).nonzero().flatten()
        if not at.numel():
            break
        logits[at] = 1.2 * _randn(g, at.numel(), experts)
    else:  # what is left takes the values of a row without one: evenly spread logits, far apart
        spread = torch.linspace(-2.0, 2.0, experts, device=DEV)
        logits[_near_tie(case, logits, bias)] = spread
    return logits, bias


def _blocks(c):
    return (c + 127) // 128


def _words(c):
    return (c + 511) // 512


def _random_f8(g, mats, rows, cols):
    """Stacked matrices as a quantiser leaves them: normal values whose block maximum lies in the top binade."""
    q = torch.empty(mats, rows, cols, dtype=F8, device=DEV)
    step = max(1, (1 << 27) // max(1, rows * cols))
    for m in range(0, mats, step):
        x = _randn(g, min(step, mats - m), rows, cols)
        q[m:m + step] = x.mul_(80.0).clamp_(-448.0, 448.0).to(F8)
    scales = torch.full((mats, _blocks(rows), 4 * _words(cols)), 127, dtype=torch.uint8, device=DEV)
    scales[..., :_blocks(cols)] = torch.randint(113, 116, (mats, _blocks(rows), _blocks(cols)), generator=g,
                                                device=DEV).to(torch.uint8)
    return q, scales


def _dispatch(case, g):
    """Expert order of random routings: the token of each sorted pair and the experts' bounds."""
    n, experts, k = case["n"], case["experts"], case["k"]
    ids = (torch.rand(n, experts, generator=g, device=DEV) + case["skew"] * _randn(g, experts)).topk(k, 1).indices
    order = ids.flatten().sort(stable=True).indices
    counts = torch.bincount(ids.flatten(), minlength=experts)
    bounds = [0] + counts.cumsum(0).tolist()
    offsets = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    return (order // k).int().contiguous(), offsets, bounds


def _dims(case, latent, ff):
    import sigmoid_top_routing_latentmoe_b200 as lm
    return lm.make_dims(case["n"], 128, latent, case["experts"], case["k"], 0, ff, 0, BETA1, BETA2,
                        dtype=_dtype(case))


def prepare(case, seed):
    op = case["op"]
    st = {"case": case}
    if op in ("route", "route_backward"):
        st["logits"], st["bias"] = _route_inputs(case, seed)
        if op == "route_backward":
            st["ids"] = _select(case, _scores(case, st["logits"]) + st["bias"]).int()
            st["dw"] = _randn(_gen(seed + 1), case["n"], case["k"])
        if own:
            import sigmoid_top_routing_latentmoe_b200 as lm
            st["dims"] = lm.make_dims(case["n"], 128, 128, case["experts"], case["k"], 0, 128, 0,
                                      dtype=torch.float32)
            st["rule"] = lm.make_route_rule(
                score=lm.SCORE_SIGMOID if case["score"] == "sigmoid" else lm.SCORE_SOFTMAX,
                n_groups=case["groups"], topk_groups=case["kept"],
                group_score=lm.GROUP_TOP2 if case["group_score"] == "top2" else lm.GROUP_MAX,
                renormalise=case["renorm"], scale=case["scale"])
            if op == "route":
                st["out"] = (torch.empty(case["n"], case["k"], dtype=torch.int32, device=DEV),
                             torch.empty(case["n"], case["k"], device=DEV))
            else:
                st["out"] = torch.empty(case["n"], case["experts"], device=DEV)
        return st
    g = _gen(seed)
    if op == "quantize":
        if case["what"] == "rows":
            n, cols = case["rows"], case["cols"]
            # the latent rows differ in size from token to token
            st["x"] = (0.55 * _randn(g, case["src"], cols) * torch.exp(_randn(g, case["src"], 1))).to(_dtype(case))
            st["index"] = torch.randint(0, case["src"], (n,), generator=g, device=DEV).int()
            shape = (_words(cols), n, 4)
            qshape = (n, cols)
        else:
            m, n, cols = case["mats"], case["rows"], case["cols"]
            st["x"] = (0.02 * _randn(g, m, n, cols)).to(_dtype(case))
            shape = (m, _blocks(n), 4 * _words(cols))
            qshape = (m, n, cols)
        if own:
            st["out"] = (torch.empty(qshape, dtype=F8, device=DEV), torch.empty(shape, dtype=torch.uint8, device=DEV))
        return st
    st["perm"], st["offsets"], st["bounds"] = _dispatch(case, g)
    pairs, experts = case["n"] * case["k"], case["experts"]
    if op == "expert_gemm":
        n_in, n_out = case["n_in"], case["n_out"]
        st["a"] = _random_f8(g, 1, pairs, n_in)[0][0]
        scales = torch.full((pairs, 4 * _words(n_in)), 127, dtype=torch.uint8, device=DEV)
        scales[:, :_blocks(n_in)] = torch.randint(116, 121, (pairs, _blocks(n_in)), generator=g, device=DEV).to(torch.uint8)
        st["a_scales"] = scales.view(pairs, -1, 4).transpose(0, 1).contiguous()
        st["w"], st["w_scales"] = _random_f8(g, experts, n_out, n_in)
        latent, ff, out = n_in, n_out, n_out
    else:
        latent, ff, out = case["latent"], case["ff"], case["latent"]
        st["z"] = (0.55 * _randn(g, case["n"], latent)).to(_dtype(case))
        for name, rows, cols in (("w_g", ff, latent), ("w_u", ff, latent), ("w_o", latent, ff)):
            st[name], st[name + "_scales"] = _random_f8(g, experts, rows, cols)
    if own:
        import sigmoid_top_routing_latentmoe_b200 as lm
        st["dims"] = _dims(case, latent, ff)
        st["ws"] = lm.alloc_workspace(st["dims"])
        st["out"] = torch.empty(pairs, out, dtype=_dtype(case), device=DEV)
    return st


# ------------------------------------------------------------ plain forms
def _scores(case, logits):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _select(case, key):
    """[n, k] experts by key, the largest first, a tie to the lower expert, out of the kept groups."""
    n, experts = key.shape
    groups, kept = case["groups"], case["kept"]
    size = experts // groups
    at = torch.arange(experts, device=key.device).expand(n, experts)
    if kept < groups:
        by = key.view(n, groups, size)
        if case["group_score"] == "top2" and size > 1:
            score = by.topk(2, 2).values.sum(2)
        else:
            score = by.amax(2)
        best = score.sort(dim=1, descending=True, stable=True).indices[:, :kept].sort(1).values
        at = (best[:, :, None] * size + torch.arange(size, device=key.device)).flatten(1)
        key = key.gather(1, at)
    return at.gather(1, key.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]])


def _weights(case, s):
    if case["renorm"]:
        s = s / s.sum(1, keepdim=True).clamp_min(CLAMP)
    return case["scale"] * s


def _route_plain(st):
    case = st["case"]
    s = _scores(case, st["logits"])
    ids = _select(case, s + st["bias"])
    return ids.int(), _weights(case, s.gather(1, ids))


def _route_backward_plain(st):
    case, ids = st["case"], st["ids"].long()
    s = _scores(case, st["logits"])
    t = s.gather(1, ids)
    dw = st["dw"] * case["scale"]
    if case["renorm"]:
        total = t.sum(1, keepdim=True)
        d = total.clamp_min(CLAMP)
        dt = (dw - (total > CLAMP) * (dw * t).sum(1, keepdim=True) / d) / d
    else:
        dt = dw
    ds = torch.zeros_like(s).scatter_(1, ids, dt)
    if case["score"] == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _pow2(e):
    """2^e for whole e in [-126, 127], put together from its bits: exact on every device."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e; 0 for a block of zeros."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(-126, 127)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _pad(x, rows, cols):
    out = x.new_zeros(*x.shape[:-2], rows, cols)
    out[..., :x.shape[-2], :x.shape[-1]] = x
    return out


def _quantize_rows_plain(x):
    """[n, c] in 32 bits -> e4m3 values and scale bytes [words, n, 4]."""
    n, c = x.shape
    blocks = _pad(x, n, 512 * _words(c)).view(n, -1, 128)
    e = _exponent(blocks.abs().amax(2))
    q = (blocks * _pow2(-e)[..., None]).to(F8)
    return (q.view(n, -1)[:, :c].contiguous(),
            (e + 127).to(torch.uint8).view(n, -1, 4).permute(1, 0, 2).contiguous())


def _quantize_weights_plain(x):
    m, r, c = x.shape
    blocks = _pad(x, 128 * _blocks(r), 512 * _words(c)).view(m, _blocks(r), 128, -1, 128)
    e = _exponent(blocks.abs().amax((2, 4)))
    q = (blocks * _pow2(-e)[:, :, None, :, None]).to(F8)
    return q.view(m, 128 * _blocks(r), -1)[:, :r, :c].contiguous(), (e + 127).to(torch.uint8)


def _rows_f32(q, scales):
    """The values of quantised rows."""
    n, c = q.shape
    s = _pow2(scales.int() - 127).permute(1, 0, 2).reshape(n, -1)
    return q.float() * s.repeat_interleave(128, 1)[:, :c]


def _matrix_f32(q, scales):
    r, c = q.shape
    s = _pow2(scales.int() - 127)
    return q.float() * s.repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :c]


def _expert_gemm_plain(st):
    a = _rows_f32(st["a"], st["a_scales"])
    out = torch.empty(a.shape[0], st["w"].shape[1], dtype=_dtype(st["case"]), device=a.device)
    for e, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if hi > lo:
            out[lo:hi] = (a[lo:hi] @ _matrix_f32(st["w"][e], st["w_scales"][e]).T).to(out.dtype)
    return out


def _expert_ffn_plain(st):
    q, s = _quantize_rows_plain(st["z"].float())
    z = _rows_f32(q, s)
    out = torch.empty(st["perm"].numel(), z.shape[1], dtype=_dtype(st["case"]), device=z.device)
    for e, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if hi > lo:
            x = z[st["perm"][lo:hi].long()]
            a = x @ _matrix_f32(st["w_g"][e], st["w_g_scales"][e]).T
            c = x @ _matrix_f32(st["w_u"][e], st["w_u_scales"][e]).T
            h = BETA1 * torch.tanh(a / BETA1) / (1.0 + torch.exp(-a)) * (BETA2 * torch.tanh(c / BETA2))
            h = _rows_f32(*_quantize_rows_plain(h))
            out[lo:hi] = (h @ _matrix_f32(st["w_o"][e], st["w_o_scales"][e]).T).to(out.dtype)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "route":
        return _route_plain(state)
    if op == "route_backward":
        return _route_backward_plain(state)
    if op == "quantize":
        if state["case"]["what"] == "rows":
            return _quantize_rows_plain(state["x"][state["index"].long()].float())
        return _quantize_weights_plain(state["x"].float())
    if op == "expert_gemm":
        return _expert_gemm_plain(state)
    return _expert_ffn_plain(state)


def _run_own(op, st):
    import sigmoid_top_routing_latentmoe_b200 as lm
    out = st["out"]
    if op == "route":
        lm.moe_route_logits(st["dims"], st["rule"], st["logits"], st["bias"], *out)
    elif op == "route_backward":
        lm.moe_route_logits_backward(st["dims"], st["rule"], st["logits"], st["ids"], st["dw"], out)
    elif op == "quantize":
        if st["case"]["what"] == "rows":
            lm.quantize_rows_fp8(st["x"], *out, index=st["index"])
        else:
            lm.quantize_weights_fp8(st["x"], *out)
    elif op == "expert_gemm":
        lm.moe_expert_gemm_fp8(st["dims"], st["a"], st["a_scales"], st["offsets"], st["w"], st["w_scales"], out,
                               st["ws"])
    else:
        lm.moe_expert_ffn_fp8(st["dims"], st["z"], st["perm"], st["offsets"], st["w_g"], st["w_g_scales"],
                              st["w_u"], st["w_u_scales"], st["w_o"], st["w_o_scales"], out, st["ws"])
    return out


# ------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once."""
    op = case["op"]
    if op in ("route", "route_backward"):
        n, experts, k = case["n"], case["experts"], case["k"]
        if op == "route":
            return {"bytes": 4 * n * experts + 4 * experts + 8 * n * k, "flops": 6 * n * experts}
        read = 4 * n * experts if case["score"] == "softmax" else 4 * n * k
        return {"bytes": read + 8 * n * k + 4 * n * experts, "flops": 6 * n * experts}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "quantize":
        if case["what"] == "rows":
            n, c = case["rows"], case["cols"]
            return {"bytes": size * min(n, case["src"]) * c + 4 * n + n * c + 4 * n * _words(c), "flops": 3 * n * c}
        m, r, c = case["mats"], case["rows"], case["cols"]
        return {"bytes": (size + 1) * m * r * c + 4 * m * _blocks(r) * _words(c), "flops": 3 * m * r * c}
    n, experts, k = case["n"], case["experts"], case["k"]
    pairs = n * k
    # experts that get a row, for evenly spread routings
    used = experts * (1.0 - (1.0 - k / experts) ** n)
    if op == "expert_gemm":
        k_in, n_out = case["n_in"], case["n_out"]
        return {"bytes": int(used * k_in * n_out) + pairs * (k_in + size * n_out), "flops": 2 * pairs * k_in * n_out}
    latent, ff = case["latent"], case["ff"]
    return {"bytes": int(used * 3 * latent * ff) + n * latent * size + pairs * latent * size,
            "flops": 6 * pairs * latent * ff}


# ------------------------------------------------------------------ exact
def _exact_route(case, logits, bias):
    """Scores, chosen experts and their scores, in 64 bits (the inputs hold no near ties)."""
    x = logits.double()
    if case["score"] == "sigmoid":
        s = torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))
    else:
        s = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    key = s + bias.double()
    n, experts = key.shape
    if case["kept"] < case["groups"]:
        desc = key.view(n, case["groups"], -1).sort(2, descending=True).values
        take = min(2, desc.shape[2]) if case["group_score"] == "top2" else 1
        score = sum(desc[..., i] for i in range(take))
        least = score.topk(case["kept"], 1).values[:, -1:]
        key = torch.where((score >= least).repeat_interleave(experts // case["groups"], 1), key, -math.inf)
    ids = key.topk(case["k"], 1).indices
    return s, ids


def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(v):
    """Round to the nearest e4m3 value, a tie to the even one; |v| <= 448."""
    ulp = _exact_pow2(torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent - 4)
    return torch.round(v / ulp) * ulp


def _exact_blocks(x, rows, cols):
    """x / scale rounded, and the scales' exponents, for blocks of `rows` x `cols` of the last two axes."""
    r, c = x.shape[-2:]
    b = _pad(x, -(-r // rows) * rows, -(-c // cols) * cols).unflatten(-1, (-1, cols)).unflatten(-3, (-1, rows))
    amax = b.abs().amax((-3, -1), keepdim=True)
    m, e = torch.frexp(amax.clamp_min(2.0 ** -140) / 448)
    e = torch.where(m > 0.5, e, e - 1).clamp_min(-126)  # the ceiling of log2
    e = torch.where(amax > 0, e, 0)
    q = _exact_e4m3(b * _exact_pow2(-e))
    return (q.flatten(-2).flatten(-3, -2)[..., :r, :c], e.squeeze(-1).squeeze(-2),
            (q * _exact_pow2(e)).flatten(-2).flatten(-3, -2)[..., :r, :c])


def _exact_matrix(q, scales):
    r, c = q.shape
    i, j = torch.arange(r, device=DEV) // 128, torch.arange(c, device=DEV) // 128
    return q.double() * _exact_pow2(scales.long()[i][:, j] - 127)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        s, ids = _exact_route(case, st["logits"], st["bias"])
        p = s.gather(1, ids)
        if case["renorm"]:
            p = p / torch.maximum(p.sum(1, keepdim=True), p.new_tensor(CLAMP))
        return ids.int(), p * case["scale"]
    if op == "route_backward":
        s, _ = _exact_route(case, st["logits"], st["bias"])
        ids, g = st["ids"].long(), st["dw"].double() * case["scale"]
        p = s.gather(1, ids)
        if case["renorm"]:
            total = p.sum(1, keepdim=True)
            g = g / total - (g * p).sum(1, keepdim=True) / total ** 2
        full = torch.zeros_like(s).scatter(1, ids, g)
        if case["score"] == "sigmoid":
            return full * s * (1 - s)
        return full * s - s * (full * s).sum(1, keepdim=True)
    if op == "quantize":
        if case["what"] == "rows":
            x = st["x"].double()[st["index"].long()]
            q, e, _ = _exact_blocks(x, 1, 128)
            scales = torch.full((x.shape[0], 4 * _words(case["cols"])), 127, dtype=torch.uint8, device=DEV)
            scales[:, :e.shape[1]] = (e + 127).to(torch.uint8)
            return q, scales.view(x.shape[0], -1, 4).transpose(0, 1).contiguous()
        x = st["x"].double()
        q, e, _ = _exact_blocks(x, 128, 128)
        scales = torch.full((x.shape[0], e.shape[1], 4 * _words(case["cols"])), 127, dtype=torch.uint8, device=DEV)
        scales[..., :e.shape[2]] = (e + 127).to(torch.uint8)
        return q, scales
    bounds, pairs = st["bounds"], case["n"] * case["k"]
    if op == "expert_gemm":
        j = torch.arange(case["n_in"], device=DEV) // 128
        out = torch.empty(pairs, case["n_out"], dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            rows = slice(bounds[e], bounds[e + 1])
            if bounds[e + 1] > bounds[e]:
                a = st["a"][rows].double() * _exact_pow2(st["a_scales"][j // 4, rows, j % 4].T.long() - 127)
                out[rows] = a @ _exact_matrix(st["w"][e], st["w_scales"][e]).T
        return out
    out = torch.empty(pairs, case["latent"], dtype=torch.float64, device=DEV)
    z = _exact_blocks(st["z"].double(), 1, 128)[2]
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        x = z[st["perm"][lo:hi].long()]
        a = x @ _exact_matrix(st["w_g"][e], st["w_g_scales"][e]).T
        c = x @ _exact_matrix(st["w_u"][e], st["w_u_scales"][e]).T
        h = BETA1 * torch.tanh(a / BETA1) * torch.sigmoid(a) * BETA2 * torch.tanh(c / BETA2)
        out[lo:hi] = _exact_blocks(h, 1, 128)[2] @ _exact_matrix(st["w_o"][e], st["w_o_scales"][e]).T
    return out
