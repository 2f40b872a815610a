"""Routing under a rule with groups of experts, its gradient, and the whole 8-bit path, on
the GPU against 64-bit references.

ids have to be equal: the rows that are compared have no decisive gap under 1e-6 (32-bit keys
are off by at most a few 2^-24), or exact ties.  Weights: a score is off by at most 8
roundings (expf 2, the sum and the division; a softmax's sum of R terms another R / 32 + 5),
the weight by 8 + k more."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")

U = 2.0 ** -24


def rule_of(score="sigmoid", groups=1, kept=1, top2=True, renorm=True, scale=1.0):
    return lm.make_route_rule(lm.SCORE_SIGMOID if score == "sigmoid" else lm.SCORE_SOFTMAX, groups, kept,
                              lm.GROUP_TOP2 if top2 else lm.GROUP_MAX, renorm, scale)


def dims_of(n, R, k):
    return lm.make_dims(n, 128, 128, R, k, 0, 128, 0, dtype=torch.float32)


def run_route(logits, bias, k, rule):
    n, R = logits.shape
    ids = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), -7.0, device="cuda")
    lm.moe_route_logits(dims_of(n, R, k), rule, logits, bias, ids, w)
    return ids.cpu().numpy(), w.double().cpu().numpy()


def draw(rng, n, R, k, bias_std, args):
    """Logits and bias without near ties: rows that have one are drawn again."""
    bias = (rng.standard_normal(R) * bias_std).astype(np.float32)
    logits = (1.5 * rng.standard_normal((n, R))).astype(np.float32)
    for _ in range(20):
        gap = ref.route(logits, bias, k, *args)[2]
        bad = gap < 1e-6
        if not bad.any():
            return logits, bias
        logits[bad] = 1.5 * rng.standard_normal((int(bad.sum()), R))
    raise AssertionError("near ties left")


CASES = [  # n, R, k, bias, (score, groups, kept, top2, renorm, scale)
    (1, 1, 1, 0.1, ("sigmoid", 1, 1, True, True, 1.0)),
    (3, 6, 3, 0.1, ("sigmoid", 3, 2, True, True, 2.5)),
    (65, 16, 2, 0.1, ("softmax", 1, 1, False, False, 1.0)),
    (40, 64, 8, 0.05, ("sigmoid", 8, 4, True, True, 2.5)),
    (33, 64, 8, 0.01, ("softmax", 8, 3, False, False, 16.0)),
    (21, 100, 7, 0.1, ("sigmoid", 5, 2, False, False, 1.0)),
    (17, 256, 8, 0.1, ("sigmoid", 8, 4, True, True, 2.5)),
    (9, 896, 16, 0.1, ("sigmoid", 14, 7, True, True, 1.0)),
    (9, 896, 16, 0.0, ("softmax", 7, 3, True, True, 1.0)),
    (5, 130, 40, 0.1, ("sigmoid", 1, 1, True, True, 1.0)),     # more than 32 slots
    (4, 70, 70, 0.1, ("softmax", 1, 1, True, False, 3.0)),     # every expert
    (5, 96, 20, 0.1, ("sigmoid", 96, 30, False, True, 1.0)),   # groups of one expert
    (5, 96, 20, 0.1, ("sigmoid", 48, 17, True, True, 1.0)),    # more groups than lanes
    (2, 4096, 32, 0.1, ("sigmoid", 64, 9, True, True, 1.0)),
    (2, 4096, 5, 0.1, ("sigmoid", 2048, 9, True, True, 1.0)),
]


@pytest.mark.parametrize("n,R,k,bias_std,args", CASES)
def test_route_logits(n, R, k, bias_std, args):
    rng = np.random.default_rng(R + k)
    if args[0] == "softmax":
        bias_std /= R
    if R == 4096 or k > 32:   # too many keys for random ones to stay apart
        logits = np.stack([rng.permutation(np.linspace(-3, 3, R)) for _ in range(n)]).astype(np.float32)
        bias = None
        assert (ref.route(logits, bias, k, *args)[2] >= 1e-6).all()
    else:
        logits, bias = draw(rng, n, R, k, bias_std, args)
    ids, w, _ = ref.route(logits, bias, k, *args)
    pad = torch.full((n, R + 5), float("nan"))          # another row stride
    pad[:, 2:2 + R] = torch.from_numpy(logits)
    for l in (torch.from_numpy(logits).cuda(), pad.cuda()[:, 2:2 + R]):
        got_ids, got_w = run_route(l, None if bias is None else torch.from_numpy(bias).cuda(), k, rule_of(*args))
        np.testing.assert_array_equal(got_ids, ids)
        tol = U * (16 + k + (R / 32 + 5 if args[0] == "softmax" else 0)) * np.abs(w)
        assert (np.abs(got_w - w) <= tol).all(), (np.abs(got_w - w) / np.abs(w)).max() / U


@pytest.mark.parametrize("R,k,groups,kept", [(8, 3, 1, 1), (64, 8, 8, 2), (200, 16, 4, 2), (200, 40, 2, 2)])
def test_route_ties_go_to_the_lower_index(R, k, groups, kept):
    """Every key the same; then two values only, in the wrong order."""
    logits = torch.zeros(2, R, device="cuda")
    logits[1, R // 2:] = 1.0
    ids, _ = run_route(logits, None, k, rule_of(groups=groups, kept=kept))
    np.testing.assert_array_equal(ids[0], np.arange(k))
    np.testing.assert_array_equal(ids, ref.route(logits.cpu().numpy(), None, k, "sigmoid", groups, kept)[0])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("R,groups,kept", [(16, 1, 1), (16, 4, 2), (160, 5, 2)])
def test_route_closed_experts_and_bad_logits(score, R, groups, kept):
    k = 4
    rng = np.random.default_rng(R)
    logits = np.stack([rng.permutation(np.linspace(-3, 3, R)) for _ in range(6)]).astype(np.float32)
    bias = np.zeros(R, np.float32)
    bias[::2] = -np.inf                                 # closed
    logits[1] = -np.inf                                 # no expert open
    logits[2, 3:] = -np.inf
    logits[3, 5] = np.nan
    logits[4] = np.nan
    logits[5, 7] = np.inf
    rule = rule_of(score, groups, kept)
    got_ids, got_w = run_route(torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda(), k, rule)
    ids, w, _ = ref.route(logits, bias, k, score, groups, kept)
    np.testing.assert_array_equal(got_ids, ids)
    np.testing.assert_allclose(got_w, w, rtol=U * (32 + R), atol=0)   # NaN where the reference has it
    for row in got_ids:                                 # always k distinct experts
        assert len(set(row)) == k and row.min() >= 0 and row.max() < R


def test_route_lowest_finite_values():
    """Masks of the type's lowest value: the masked experts come last, in order."""
    R, k = 48, 6
    low = torch.finfo(torch.float32).min
    logits = torch.full((2, R), low)
    logits[0, 20] = 1.0
    bias = torch.zeros(R)
    bias[:4] = low
    for score in ("sigmoid", "softmax"):
        got_ids, got_w = run_route(logits.cuda(), bias.cuda(), k, rule_of(score, 6, 3, renorm=False))
        ids, w, _ = ref.route(logits.numpy(), bias.numpy(), k, score, 6, 3, True, False)
        np.testing.assert_array_equal(got_ids, ids)
        np.testing.assert_allclose(got_w, w, rtol=64 * U, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_groups_of_one_expert(score):
    """As many groups as experts, to the largest number: the same as no groups, NaN and ties included."""
    rng = np.random.default_rng(41)
    for R, k, kept in ((4096, 32, 4095), (4096, 7, 7), (3600, 40, 50), (2, 1, 1)):
        logits = np.stack([rng.permutation(np.linspace(-3, 3, R)) for _ in range(6)]).astype(np.float32)
        logits[1] = 0.0
        if R > 2:
            logits[2, 5:9] = np.nan if score == "sigmoid" else -np.inf
        l = torch.from_numpy(logits).cuda()
        got = run_route(l, None, k, rule_of(score, R, kept))
        want = run_route(l, None, k, rule_of(score))
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])
        np.testing.assert_array_equal(got[0], ref.route(logits, None, k, score, R, kept)[0])


# --------------------------------------------------------------- gradient
def backward_ref(logits, ids, dw, score, renorm, scale):
    s = ref.route_keys(logits, None, score)[0]
    p, g = np.take_along_axis(s, ids, 1), scale * np.asarray(dw, np.float64)
    if renorm:
        tot = p.sum(1, keepdims=True)
        d = np.maximum(tot, 1e-9)
        g = (g - (tot > 1e-9) * (g * p).sum(1, keepdims=True) / d) / d
    ds = np.zeros_like(s)
    np.put_along_axis(ds, ids, g, 1)
    if score == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdims=True))


def run_backward(logits, ids, dw, rule, out=None):
    n, R = logits.shape
    k = ids.shape[1]
    out = torch.full((n, R), 9.0, device="cuda") if out is None else out
    lm.moe_route_logits_backward(dims_of(n, R, k), rule, logits, ids, dw, out)
    return out


@pytest.mark.parametrize("n,R,k,bias_std,args", CASES)
def test_route_backward(n, R, k, bias_std, args):
    score, groups, kept, top2, renorm, scale = args
    rng = np.random.default_rng(R * k + 1)
    logits = (1.5 * rng.standard_normal((n, R))).astype(np.float32)
    ids = ref.route(logits, None, k, *args)[0]
    dw = rng.standard_normal((n, k)).astype(np.float32)
    got = run_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
                       torch.from_numpy(dw).cuda(), rule_of(*args)).double().cpu().numpy()
    want = backward_ref(logits, ids, dw, score, renorm, scale)
    # every term of a difference is off by (32 + k + R / 32) roundings of the largest of them
    s = ref.route_keys(logits, None, score)[0]
    tot = np.take_along_axis(s, ids, 1).sum(1, keepdims=True) if renorm else 1.0
    size = s * scale * np.abs(dw).max(1, keepdims=True) * (2 / tot if renorm else 1 + s.sum(1, keepdims=True))
    assert (np.abs(got - want) <= U * (32 + k + R / 32) * size).all()


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_route_backward_against_differences(score, renorm):
    rng = np.random.default_rng(12)
    n, R, k = 4, 24, 5
    logits = rng.standard_normal((n, R)).astype(np.float32)
    ids = ref.route(logits, None, k, score)[0]
    dw = rng.standard_normal((n, k)).astype(np.float32)
    got = run_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
                       torch.from_numpy(dw).cuda(), rule_of(score, renorm=renorm, scale=1.7)).double().cpu().numpy()

    def loss(l):
        w = np.take_along_axis(ref.route_keys(l, None, score)[0], ids, 1)
        if renorm:
            w = w / np.maximum(w.sum(1, keepdims=True), 1e-9)
        return (1.7 * w * dw).sum(1)

    h = 1e-5                                            # central differences in 64 bits: off by ~h^2
    for e in range(R):
        step = np.zeros(R)
        step[e] = h
        diff = (loss(logits.astype(float) + step) - loss(logits.astype(float) - step)) / (2 * h)
        np.testing.assert_allclose(got[:, e], diff, atol=2e-6)


def test_route_backward_floor_strays_and_stride():
    """A sum at its floor, ids outside the experts, a strided gradient whose padding stays."""
    rng = np.random.default_rng(13)
    n, R, k = 5, 40, 3
    logits = rng.standard_normal((n, R)).astype(np.float32)
    logits[1] -= 60.0                                   # sigmoid sums under 1e-9
    ids = ref.route(logits, None, k)[0]
    dw = rng.standard_normal((n, k)).astype(np.float32)
    wide = torch.full((n, R + 6), 3.0, device="cuda")
    stray = ids.copy().astype(np.int32)
    stray[3, 1], stray[4, 0] = -1, R
    run_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(stray).cuda(), torch.from_numpy(dw).cuda(),
                 rule_of(renorm=True), wide[:, 3:3 + R])
    got = wide.double().cpu().numpy()
    assert (got[:, :3] == 3.0).all() and (got[:, 3 + R:] == 3.0).all()
    want = backward_ref(logits[:3], ids[:3], dw[:3], "sigmoid", True, 1.0)
    np.testing.assert_allclose(got[:3, 3:3 + R], want, rtol=64 * U, atol=64 * U)
    for t, keep in ((3, [0, 2]), (4, [1, 2])):
        part = backward_ref(logits[t:t + 1], ids[t:t + 1, keep], dw[t:t + 1, keep], "sigmoid", True, 1.0)
        np.testing.assert_allclose(got[t, 3:3 + R], part[0], rtol=64 * U, atol=64 * U)


def test_route_forward_and_backward_in_one_graph():
    """Captured and replayed with new logits, and the same bits as called directly."""
    rng = np.random.default_rng(31)
    n, R, k = 130, 96, 6
    rule, d = rule_of("sigmoid", 8, 4, True, True, 2.5), dims_of(n, R, k)
    logits, bias = (torch.from_numpy(a).cuda() for a in draw(rng, n, R, k, 0.1, ("sigmoid", 8, 4, True, True, 2.5)))
    dw = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).cuda()
    ids, w, dl = (torch.zeros(n, c, dtype=t, device="cuda") for c, t in ((k, torch.int32), (k, torch.float32), (R, torch.float32)))

    def step():
        lm.moe_route_logits(d, rule, logits, bias, ids, w)
        lm.moe_route_logits_backward(d, rule, logits, ids, dw, dl)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (32, 33):
        rng = np.random.default_rng(seed)
        logits.copy_(torch.from_numpy(rng.standard_normal((n, R)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (ids, w, dl)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, (ids, w, dl)))


# ------------------------------------------------------- from x, and together
@pytest.mark.parametrize("R,groups,kept,k,dtype", [(16, 4, 2, 2, torch.bfloat16), (96, 8, 4, 6, torch.bfloat16),
                                                   (16, 4, 2, 2, torch.float32), (64, 4, 2, 4, torch.float32)])
def test_route_grouped_from_x(R, groups, kept, k, dtype):
    """The same routing as from the logits that the call leaves in the workspace; logits near x W_r^T."""
    rng = np.random.default_rng(R)
    n, d = 150, 256
    dims = lm.make_dims(n, d, 128, R, k, 0, 128, 0, dtype=dtype)
    x = torch.from_numpy(rng.standard_normal((n, d))).to(dtype).cuda()
    w = torch.from_numpy(rng.standard_normal((R, d)) * 0.1).to(dtype).cuda()
    bias = torch.from_numpy((0.1 * rng.standard_normal(R)).astype(np.float32)).cuda()
    rule = rule_of("sigmoid", groups, kept, True, True, 2.5)
    ws = lm.alloc_workspace(dims)
    ids = torch.zeros(n, k, dtype=torch.int32, device="cuda")
    p = torch.zeros(n, k, device="cuda")
    lm.moe_route_grouped(dims, rule, x, w, bias, ids, p, ws)
    assert lm.get_device_status(ws) == lm.OK
    logits = lm.workspace_views(dims, ws)["logits"]
    want = x.double() @ w.double().T
    size = x.double().abs() @ w.double().abs().T
    assert ((logits.double() - want).abs() <= d * 2.0 ** -23 * size).all()
    ids2, p2 = torch.zeros_like(ids), torch.zeros_like(p)
    lm.moe_route_logits(dims, rule, logits, bias, ids2, p2)
    assert torch.equal(ids, ids2) and torch.equal(p, p2)


def test_route_dispatch_experts_combine():
    """The path as a user runs it: grouped routing of x, dispatch, 8-bit experts, combine."""
    rng = np.random.default_rng(21)
    n, d, L, F, R, k = 260, 256, 272, 144, 24, 4
    dims = lm.make_dims(n, d, L, R, k, 0, F, 0)
    bf = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()
    x, w_r = bf(rng.standard_normal((n, d))), bf(0.1 * rng.standard_normal((R, d)))
    z = bf(rng.standard_normal((n, L)))
    bias = torch.from_numpy((0.1 * rng.standard_normal(R)).astype(np.float32)).cuda()
    rms = torch.from_numpy((1 + 0.1 * rng.standard_normal(L)).astype(np.float32)).cuda()
    ws = lm.alloc_workspace(dims)
    e = lambda *s, dtype=torch.int32: torch.empty(*s, dtype=dtype, device="cuda")
    ids, p = e(n, k), e(n, k, dtype=torch.float32)
    counts, offsets, perm, inv = e(R), e(R + 1), e(n * k), e(n, k)
    eo, u = e(n * k, L, dtype=torch.bfloat16), e(n, L, dtype=torch.bfloat16)
    q = {}
    for name, r, c in (("g", F, L), ("u", F, L), ("o", L, F)):
        w = bf(0.05 * rng.standard_normal((R, r, c)))
        q[name] = (e(R, r, c, dtype=torch.float8_e4m3fn),
                   e(*lm.fp8_weight_scales_shape(R, r, c), dtype=torch.uint8))
        lm.quantize_weights_fp8(w, *q[name])
        q[name + "v"] = ref.quantize_blocks(w.double().cpu().numpy(), 128, 128)[2]
    lm.moe_route_grouped(dims, rule_of("sigmoid", 6, 3, True, True, 2.5), x, w_r, bias, ids, p, ws)
    lm.moe_dispatch(dims, ids, counts, offsets, perm, inv, ws)
    lm.check_dispatch(dims, ids, counts, offsets, perm, inv, ws)
    lm.moe_expert_ffn_fp8(dims, z, perm, offsets, *q["g"], *q["u"], *q["o"], eo, ws)
    lm.moe_combine(dims, eo, inv, p, rms, u)
    assert lm.get_device_status(ws) == lm.OK
    want, bound = ref.ffn(z.double().cpu().numpy(), perm.cpu().numpy(), offsets.cpu().numpy(),
                          q["gv"], q["uv"], q["ov"], 4.0, 25.0)
    got = eo.double().cpu().numpy()
    bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    assert (np.abs(got - want) <= bound).all()
    # the combine of what the experts gave (its inputs are the experts' rounded rows)
    iv, pv = inv.cpu().numpy(), p.double().cpu().numpy()
    ut = (pv[:, :, None] * got[iv]).sum(1)
    norm = ut / np.sqrt((ut ** 2).mean(1, keepdims=True) + dims.rms_eps) * rms.double().cpu().numpy()
    assert (np.abs(u.double().cpu().numpy() - norm) <= 2.0 ** -8 * np.abs(norm) + 64 * U * np.abs(norm).max()).all()
