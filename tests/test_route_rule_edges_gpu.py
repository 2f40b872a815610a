"""Routing under a rule where it can go wrong: a NaN among the chosen experts, logits a
single step apart far from zero, calls from several host threads at once."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")

U = 2.0 ** -24


def rule_of(score="sigmoid", groups=1, kept=1, renorm=True, scale=1.0):
    return lm.make_route_rule(lm.SCORE_SIGMOID if score == "sigmoid" else lm.SCORE_SOFTMAX, groups, kept,
                              lm.GROUP_TOP2, renorm, scale)


def dims_of(n, R, k):
    return lm.make_dims(n, 128, 128, R, k, 0, 128, 0, dtype=torch.float32)


def route(logits, bias, k, rule):
    n, R = logits.shape
    ids = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), -7.0, device="cuda")
    lm.moe_route_logits(dims_of(n, R, k), rule, logits, bias, ids, w)
    return ids, w


# (R, k, groups, kept): every expert chosen, on each path of the selection; and as many experts as the kept
# groups hold
NAN_CASES = [(3, 3, 1, 1), (64, 32, 1, 1), (40, 40, 1, 1), (70, 70, 1, 1), (96, 32, 3, 1), (96, 64, 3, 2)]


def nan_rows(R, k, groups, kept, seed):
    """Row 0 plain; row 1 a NaN in an expert that is chosen all the same (the others are closed by the bias, or
    there are no more than k); row 2 the same, elsewhere; row 3 NaN everywhere."""
    rng = np.random.default_rng(seed)
    logits = np.stack([rng.permutation(np.linspace(-3, 3, R)) for _ in range(4)]).astype(np.float32)
    bias = np.zeros(R, np.float32)
    if groups == 1:
        bias[k - 1:] = -np.inf          # k - 1 experts open; a NaN ranks with the closed ones, lower index first
        if k < R:
            logits[1, k - 1] = logits[2, k - 1] = np.nan
        else:
            logits[1, 0] = logits[2, k // 2] = np.nan
    else:
        size = R // groups
        bias[kept * size:] = -10.0      # the first `kept` groups, which hold k experts
        logits[1, 0], logits[2, kept * size - 1] = np.nan, np.nan
    logits[3] = np.nan
    return logits, bias


@pytest.mark.parametrize("R,k,groups,kept", NAN_CASES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_nan_among_the_chosen(R, k, groups, kept, score, renorm):
    """The sum of the weights is NaN then, and so is every weight that is divided by it."""
    logits, bias = nan_rows(R, k, groups, kept, R + k)
    ids, w = (t.cpu().numpy() for t in route(torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda(), k,
                                             rule_of(score, groups, kept, renorm, 2.5)))
    want_ids, want, _ = ref.route(logits, bias, k, score, groups, kept, True, renorm, 2.5)
    if score == "sigmoid":
        np.testing.assert_array_equal(ids, want_ids)
        chosen_nan = np.isnan(np.take_along_axis(logits, ids.astype(np.int64), 1))
        assert chosen_nan[1].sum() == 1 and chosen_nan[2].sum() == 1 and not chosen_nan[0].any()
        assert np.isnan(w[1:]).all() if renorm else (np.isnan(w) == chosen_nan).all()
    else:
        assert np.isnan(w[1:]).all()
    np.testing.assert_array_equal(ids[0], want_ids[0])
    np.testing.assert_allclose(w[0], want[0], rtol=U * (32 + R), atol=0)


@pytest.mark.parametrize("R,k,groups,kept", NAN_CASES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_nan_among_the_chosen_backward(R, k, groups, kept, score, renorm):
    """A NaN sum reaches every selected expert's gradient; without the sum only its own expert's."""
    logits, bias = nan_rows(R, k, groups, kept, R + k)
    ids = ref.route(logits, bias, k, score, groups, kept, True, renorm)[0]
    rng = np.random.default_rng(k)
    dw = rng.standard_normal((4, k)).astype(np.float32)
    out = torch.full((4, R), 9.0, device="cuda")
    lm.moe_route_logits_backward(dims_of(4, R, k), rule_of(score, groups, kept, renorm),
                                 torch.from_numpy(logits).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
                                 torch.from_numpy(dw).cuda(), out)
    got = out.cpu().numpy()
    assert np.isfinite(got[0]).all()
    if score == "softmax":                      # every score of the row is NaN
        assert np.isnan(got[1:]).all()
        return
    for t in (1, 2, 3):
        chosen = np.zeros(R, bool)
        chosen[ids[t]] = True
        want = chosen if renorm else chosen & np.isnan(logits[t])
        np.testing.assert_array_equal(np.isnan(got[t]), want)
        assert (got[t][~chosen] == 0.0).all()


@pytest.mark.parametrize("grouped", [False, True])
def test_host_threads_side_by_side(grouped):
    """Calls of two sizes, both with more shared memory than a kernel gets unasked, from four threads."""
    k, results = 5, []

    def work(R):
        rng = np.random.default_rng(R)
        logits = np.stack([rng.permutation(np.linspace(-3, 3, R)) for _ in range(3)]).astype(np.float32)
        groups, kept = (R // 2, 9) if grouped else (1, 1)
        rule, d, l = rule_of("sigmoid", groups, kept), dims_of(3, R, k), torch.from_numpy(logits).cuda()
        ids, w = torch.zeros(3, k, dtype=torch.int32, device="cuda"), torch.zeros(3, k, device="cuda")
        stream = torch.cuda.Stream()
        args = (ctypes.byref(d), ctypes.byref(rule), l.data_ptr(), R, None, ids.data_ptr(), w.data_ptr(),
                stream.cuda_stream)
        torch.cuda.synchronize()
        refused = sum(lm._lib.moe_route_logits(*args) != lm.OK for _ in range(5000))
        stream.synchronize()
        want = ref.route(logits, None, k, "sigmoid", groups, kept)[0]
        results.append((R, refused, bool((ids.cpu().numpy() == want).all())))

    threads = [threading.Thread(target=work, args=(R,)) for R in (4096, 2600, 4096, 2600)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(results) == [(2600, 0, True)] * 2 + [(4096, 0, True)] * 2, results


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_neighbouring_logits_far_from_zero(score):
    """Two logits one step of fp32 apart, at -8 and beyond, the larger one behind: it comes first.  A step of a
    logit there is 2^-20 or more and changes its score by that factor; a 32-bit score is off by at most 5 * 2^-24
    (exponential 2, sum 1, reciprocal 2; softmax: exponential 2, product 1), so the two do not change places."""
    low = -np.geomspace(8.0, 86.0, 6000).astype(np.float32)
    n = len(low)
    near = np.stack([low, np.nextafter(low, np.float32(0.0))], 1)
    logits = torch.from_numpy(near if score == "sigmoid" else np.concatenate([np.zeros((n, 1), np.float32), near], 1))
    R = logits.shape[1]
    ids, _ = route(logits.cuda(), None, R, rule_of(score))
    want = [1, 0] if score == "sigmoid" else [0, 2, 1]
    wrong = (ids.cpu().numpy() != np.array(want)).any(1)
    assert not wrong.any(), (int(wrong.sum()), low[wrong][:5])
    # the same behind more experts than stay in registers, whose scores are far lower
    wide = torch.full((n, 96), -200.0)
    wide[:, 40:40 + R] = logits
    ids, _ = route(wide.cuda(), None, R, rule_of(score))
    assert not (ids.cpu().numpy() != 40 + np.array(want)).any()
