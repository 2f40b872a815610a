"""What routing under a rule and the 8-bit experts refuse, before anything touches a device."""
import ctypes

import pytest
import torch

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")

FAKE = 1 << 20                                           # never dereferenced: checks fail first
DIMS = lm.make_dims(8, 64, 128, 24, 4, 0, 256, 0)


def rule(**kw):
    r = lm.make_route_rule(n_groups=6, topk_groups=2)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def route(dims=DIMS, r=None, logits=FAKE, ld=24, bias=None, ids=FAKE, probs=FAKE):
    r = rule() if r is None else r
    return lm._lib.moe_route_logits(ctypes.byref(dims), ctypes.byref(r), logits, ld, bias, ids, probs, None)


@pytest.mark.parametrize("change", [
    dict(score=2), dict(group_score=5), dict(renormalise=2), dict(n_groups=0), dict(n_groups=5),
    dict(topk_groups=0), dict(topk_groups=7), dict(topk_groups=0x7fffffff), dict(n_groups=24, topk_groups=3),
    dict(scale=float("nan")), dict(scale=float("inf")),
])
def test_bad_rules(change):
    assert route(r=rule(**change)) == lm.EINVAL
    assert lm._lib.lmoe_last_error()


def test_route_arguments():
    assert route(logits=None) == lm.EINVAL
    assert route(ld=23) == lm.EINVAL
    assert route(logits=FAKE + 2) == lm.EINVAL
    assert route(ids=None) == lm.EINVAL
    assert route(probs=FAKE + 8) == lm.EINVAL
    assert route(bias=FAKE + 4) == lm.EINVAL
    assert lm._lib.moe_route_logits(ctypes.byref(DIMS), None, FAKE, 24, None, FAKE, FAKE, None) == lm.EINVAL
    r = rule()
    back = lambda **kw: lm._lib.moe_route_logits_backward(ctypes.byref(DIMS), ctypes.byref(r), *{
        **dict(logits=FAKE, ld=24, ids=FAKE, dprobs=FAKE, dlogits=FAKE, ldd=24, stream=None), **kw}.values())
    for bad in (dict(logits=None), dict(dlogits=None), dict(ldd=8), dict(ids=FAKE + 4), dict(dprobs=None)):
        assert back(**bad) == lm.EINVAL
    grouped = lambda ws, n: lm._lib.moe_route_grouped(ctypes.byref(DIMS), ctypes.byref(r), FAKE, FAKE, None, FAKE,
                                                      FAKE, ws, n, None)
    assert grouped(FAKE + 16, 1 << 30) == lm.EINVAL
    assert grouped(FAKE, 64) == lm.EWORKSPACE


def test_quantizer_arguments():
    rows = lambda **kw: lm._lib.lmoe_quantize_rows_fp8(*{
        **dict(x=FAKE, dtype=lm.BF16, n_src=4, ld=64, index=None, rows=4, cols=64, q=FAKE, s=FAKE, stream=None),
        **kw}.values())
    for bad in (dict(dtype=7), dict(cols=8), dict(cols=24), dict(cols=0), dict(ld=60), dict(ld=68), dict(ld=48),
                dict(rows=5), dict(rows=-1), dict(x=None), dict(x=FAKE + 8), dict(q=FAKE + 4), dict(s=None),
                dict(index=FAKE + 2, rows=9), dict(n_src=1 << 31, rows=1 << 31)):
        assert rows(**bad) == lm.EINVAL, bad
    assert rows(rows=0, n_src=0, x=None, q=None, s=None) == lm.OK
    w = lambda **kw: lm._lib.lmoe_quantize_weights_fp8(*{
        **dict(w=FAKE, dtype=lm.F32, mats=2, rows=3, cols=64, q=FAKE, s=FAKE, stream=None), **kw}.values())
    for bad in (dict(dtype=-1), dict(mats=-1), dict(rows=0), dict(cols=40), dict(w=None), dict(q=FAKE + 1),
                dict(s=FAKE + 4)):
        assert w(**bad) == lm.EINVAL, bad
    assert w(mats=1 << 30, rows=1 << 12) == lm.EUNSUPPORTED
    assert w(mats=0) == lm.OK


def test_expert_arguments():
    gemm = lambda **kw: lm._lib.moe_expert_gemm_fp8(*{
        **dict(dims=ctypes.byref(DIMS), n_in=128, n_out=64, a=FAKE, a_s=FAKE, off=FAKE, w=FAKE, w_s=FAKE, out=FAKE,
               ws=FAKE, n=1 << 30, stream=None), **kw}.values())
    for bad in (dict(dims=None), dict(n_in=24), dict(n_in=0), dict(n_out=4), dict(n_out=12), dict(a=None),
                dict(a_s=FAKE + 4), dict(off=None), dict(w=None), dict(w_s=None), dict(out=FAKE + 2), dict(ws=None)):
        assert gemm(**bad) == lm.EINVAL, bad
    assert gemm(n=128) == lm.EWORKSPACE
    ptrs = [FAKE] * 6
    ffn = lambda dims=DIMS, w=lm.Fp8Experts(*ptrs), z=FAKE, n=1 << 30: lm._lib.moe_expert_ffn_fp8(
        ctypes.byref(dims), z, FAKE, FAKE, ctypes.byref(w), FAKE, FAKE, n, None)
    assert ffn(z=None) == lm.EINVAL
    assert ffn(n=8) == lm.EWORKSPACE
    for i in range(6):
        assert ffn(w=lm.Fp8Experts(*[FAKE if j != i else None for j in range(6)])) == lm.EINVAL
    assert ffn(dims=lm.make_dims(8, 64, 136, 24, 4, 0, 256, 0)) == lm.EINVAL      # latent % 16
    assert ffn(dims=lm.make_dims(8, 64, 128, 24, 4, 0, 264, 0)) == lm.EINVAL      # ff_routed % 16


def test_binding_refuses_host_tensors():
    x, q = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(lm.fp8_row_scales_shape(4, 64), dtype=torch.uint8)
    with pytest.raises(lm.LmoeError):
        lm.quantize_rows_fp8(x, q, s)
    with pytest.raises(lm.LmoeError):
        lm.quantize_weights_fp8(x[None], q[None], s)
    with pytest.raises(lm.LmoeError):
        lm.quantize_rows_fp8(x.half(), q, s)
    with pytest.raises(lm.LmoeError):
        lm.moe_route_logits(DIMS, rule(), torch.zeros(8, 24), None, None, None)


def test_scale_shapes():
    assert lm.fp8_row_scales_shape(5, 16) == (1, 5, 4)
    assert lm.fp8_row_scales_shape(5, 528) == (2, 5, 4)
    assert lm.fp8_weight_scales_shape(3, 129, 512) == (3, 2, 4)


def test_backward_refuses_a_gradient_over_the_logits():
    """The gradient is written before the last logits are read: a call in place would be wrong.
    Matrices beside each other in the columns of one buffer do not overlap."""
    r, n, R = rule(), 8, 24
    def back(logits, ld, dlogits, ldd, n=n):
        dims = lm.make_dims(n, 64, 128, R, 4, 0, 256, 0)
        status = lm._lib.moe_route_logits_backward(ctypes.byref(dims), ctypes.byref(r), logits, ld, None, None,
                                                   dlogits, ldd, None)
        assert status == lm.EINVAL               # without ids no call gets as far as a launch
        return b"overlap" in lm._lib.lmoe_last_error()
    def touch(a, lda, b, ldb):   # shared elements, counted one by one
        at = lambda p, ld: {p // 4 + t * ld + e for t in range(n) for e in range(R)}
        return bool(at(a, lda) & at(b, ldb))
    for shift in (0, 4, 4 * 23, 4 * 24, 4 * 26, 4 * 27, 4 * 49, 4 * 50, 4 * 51, 4 * (7 * 50 + 23), 4 * (7 * 50 + 24)):
        for a, b in ((FAKE, FAKE + shift), (FAKE + shift, FAKE)):
            assert back(a, 50, b, 50) == touch(a, 50, b, 50), (shift, a < b)
    assert back(FAKE, 24, FAKE, 24) and not back(FAKE, 24, FAKE + 4 * 24 * n, 24)
    assert back(FAKE, 24, FAKE + 4 * 24 * (n - 1), 30)      # other strides: the ranges decide
    assert back(FAKE, 24, FAKE, 24, n=1) and not back(FAKE, 24, FAKE + 4 * 24, 24, n=1)
