"""8-bit routed experts on the GPU: quantisers, ragged product and expert FFN against
64-bit references.

The quantisers have to agree value for value: dividing by a power of two is exact and each
element is rounded once.  Products: K 2^-23 of the sum of magnitudes (every addend rounded or
cut once in 32 bits) and the rounding of the output, 2^-8 of the value in bfloat16 and 2^-24
in float32.  The FFN's bound is derived in fp8_ref.ffn."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")

F8 = torch.float8_e4m3fn
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(params=["0", "1"], ids=["single", "pairs"])
def tiles(request, monkeypatch):
    """Single CTAs over 128-row tiles, CTA pairs over 256-row ones."""
    monkeypatch.setenv("LMOE_FP8_PAIRS", request.param)


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def dims_of(n, R, k, latent=128, ff=128, dtype=torch.bfloat16):
    return lm.make_dims(n, 128, latent, R, k, 0, ff, 0, dtype=dtype)


def quantized_weights(rng, R, rows, cols, std=0.02):
    """(values in 64 bits, e4m3 tensor, scales) as the reference quantises them."""
    w = rng.standard_normal((R, rows, cols)) * std
    q, e, v = ref.quantize_blocks(w, 128, 128)
    return v, ref.f8(q).cuda(), gpu(ref.weight_scales(e, cols))


def quantized_rows(rng, n, cols):
    x = rng.standard_normal((n, cols)) * np.exp(rng.standard_normal((n, 1)))
    q, e, v = ref.quantize_blocks(x, 1, 128)
    return v, ref.f8(q).cuda(), gpu(ref.row_scales(e, n, cols))


def offsets_of(rng, pairs, R, skew=1.0):
    """Random bounds of R experts over all pairs, some of them empty."""
    p = np.exp(skew * rng.standard_normal(R))
    return np.concatenate([[0], np.cumsum(rng.multinomial(pairs, p / p.sum()))]).astype(np.int32)


# ------------------------------------------------------------- quantisers
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,cols", [(1, 16), (3, 128), (130, 144), (257, 528), (9, 2064)])
def test_quantize_rows(n, cols, dtype):
    rng = np.random.default_rng(n * 1000 + cols)
    x = torch.from_numpy(rng.standard_normal((n, cols)) * 10.0 ** rng.integers(-6, 6, (n, 1))).to(dtype)
    x[0, : cols // 2] = 0.0
    if n > 2:
        x[1] = 0.0                                      # a row of zeros
        x[2, ::7] = 448.0                               # ties and exact powers of two
        x[2, 1::7] = 2.0 ** -7
    q = torch.zeros(n, cols, dtype=F8, device="cuda")
    s = torch.zeros(lm.fp8_row_scales_shape(n, cols), dtype=torch.uint8, device="cuda")
    lm.quantize_rows_fp8(x.cuda(), q, s)
    want_q, want_e, _ = ref.quantize_blocks(x.double().numpy(), 1, 128)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want_q)
    np.testing.assert_array_equal(s.cpu().numpy(), ref.row_scales(want_e, n, cols))


def test_quantize_rows_index_and_stride():
    rng = np.random.default_rng(1)
    n_src, cols = 37, 272
    wide = torch.from_numpy(rng.standard_normal((n_src, cols + 24))).to(torch.bfloat16).cuda()
    x = wide[:, 8:8 + cols]                             # rows 16-byte aligned, not neighbours
    index = rng.integers(0, n_src, 300).astype(np.int32)
    index[[5, 70]] = [-1, n_src]                        # no such rows: zeros
    index[100:104] = 7                                  # the same row again
    q = torch.ones(300, cols, dtype=torch.float32).to(F8).cuda()
    s = torch.zeros(lm.fp8_row_scales_shape(300, cols), dtype=torch.uint8, device="cuda")
    lm.quantize_rows_fp8(x, q, s, index=gpu(index))
    rows = x.double().cpu().numpy()[np.clip(index, 0, n_src - 1)]
    rows[[5, 70]] = 0.0
    want_q, want_e, _ = ref.quantize_blocks(rows, 1, 128)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want_q)
    np.testing.assert_array_equal(s.cpu().numpy(), ref.row_scales(want_e, 300, cols))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_extremes(dtype):
    """NaN and infinities become NaN and leave the scale alone; the smallest and the largest values."""
    x = np.zeros((6, 256))
    x[0, :4] = [np.nan, np.inf, -np.inf, 3.0]
    x[1] = np.nan
    x[2, :3] = [2.0 ** -126, 2.0 ** -130, -(2.0 ** -133)]
    x[3, :2] = [3.0e38, -1.0]
    x[4, 128:] = np.inf
    x[5, :3] = [449.0, -0.0, 1e-3]
    xt = torch.from_numpy(x).to(dtype)
    q = torch.zeros(6, 256, dtype=F8, device="cuda")
    s = torch.zeros(lm.fp8_row_scales_shape(6, 256), dtype=torch.uint8, device="cuda")
    lm.quantize_rows_fp8(xt.cuda(), q, s)
    want_q, want_e, _ = ref.quantize_blocks(xt.double().numpy(), 1, 128)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want_q)
    np.testing.assert_array_equal(s.cpu().numpy(), ref.row_scales(want_e, 6, 256))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,r,c", [(1, 1, 16), (3, 128, 128), (2, 200, 528), (5, 8, 1040)])
def test_quantize_weights(m, r, c, dtype):
    rng = np.random.default_rng(m + r + c)
    w = torch.from_numpy(rng.standard_normal((m, r, c)) * 0.02).to(dtype)
    w[0, 0, 3] = float("nan")
    q = torch.zeros(m, r, c, dtype=F8, device="cuda")
    s = torch.zeros(lm.fp8_weight_scales_shape(m, r, c), dtype=torch.uint8, device="cuda")
    lm.quantize_weights_fp8(w.cuda(), q, s)
    want_q, want_e, _ = ref.quantize_blocks(w.double().numpy(), 128, 128)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want_q)
    np.testing.assert_array_equal(s.cpu().numpy(), ref.weight_scales(want_e, c))


# ---------------------------------------------------------------- product
def run_gemm(dims, a, a_s, offsets, w, w_s, n_out, fill=7.0, stream=None):
    P = dims.n_tokens * dims.top_k
    ws = lm.alloc_workspace(dims)
    out = torch.full((P, n_out), fill, dtype=lm._act(dims), device="cuda")
    lm.moe_expert_gemm_fp8(dims, a, a_s, None if offsets is None else gpu(offsets), w, w_s, out, ws,
                           stream=stream)
    assert lm.get_device_status(ws) == lm.OK
    return out.double().cpu().numpy()


def check_gemm(got, av, wv, offsets, dtype, fill=7.0):
    seen = np.zeros(len(got), bool)
    for e in range(len(wv)):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        seen[lo:hi] = True
        want = av[lo:hi] @ wv[e].T
        tol = av.shape[1] * 2.0 ** -23 * (np.abs(av[lo:hi]) @ np.abs(wv[e]).T) + ROUND[dtype] * np.abs(want)
        assert (np.abs(got[lo:hi] - want) <= tol).all(), (e, np.abs(got[lo:hi] - want).max())
    assert (got[~seen] == fill).all()                   # rows of no expert: as they were


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,R,k,n_in,n_out", [
    (1, 1, 1, 16, 8),            # one token, less than one block
    (3, 4, 2, 128, 128),
    (33, 3, 2, 144, 264),        # a block and a piece; a column past two tiles
    (200, 5, 3, 528, 136),       # more than four blocks: a second word of scales
    (129, 2, 1, 2064, 520),
    (640, 300, 2, 256, 256),     # more experts than some of them have rows
])
def test_expert_gemm(tiles, n, R, k, n_in, n_out, dtype):
    rng = np.random.default_rng(n + n_in)
    av, a, a_s = quantized_rows(rng, n * k, n_in)
    wv, w, w_s = quantized_weights(rng, R, n_out, n_in)
    offsets = offsets_of(rng, n * k, R)
    got = run_gemm(dims_of(n, R, k, dtype=dtype), a, a_s, offsets, w, w_s, n_out)
    check_gemm(got, av, wv, offsets, dtype)


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 127, 128, 129, 256, 257, 1000])
def test_expert_gemm_dense(tiles, rows):
    rng = np.random.default_rng(rows)
    av, a, a_s = quantized_rows(rng, rows, 400)
    wv, w, w_s = quantized_weights(rng, 1, 392, 400)
    d = dims_of(rows, 1, 1)
    got = run_gemm(d, a, a_s, None, w, w_s, 392)
    check_gemm(got, av, wv, [0, rows], torch.bfloat16)
    np.testing.assert_array_equal(got, run_gemm(d, a, a_s, np.array([0, rows], np.int32), w, w_s, 392))


@pytest.mark.parametrize("lo,hi", [(0, 0), (5, 300), (-3, 100), (290, 1 << 30), (200, 100)])
def test_expert_gemm_one_expert_with_bounds(tiles, lo, hi):
    """A single expert's rows from its two offsets, clamped to the rows there are."""
    rng = np.random.default_rng(15)
    av, a, a_s = quantized_rows(rng, 300, 256)
    wv, w, w_s = quantized_weights(rng, 1, 264, 256)
    got = run_gemm(dims_of(300, 1, 1), a, a_s, np.array([lo, hi], np.int32), w, w_s, 264)
    lo = min(max(lo, 0), 300)
    check_gemm(got, av, wv, [lo, min(max(hi, lo), 300)], torch.bfloat16)


def test_expert_gemm_rows_of_no_expert(tiles):
    rng = np.random.default_rng(5)
    av, a, a_s = quantized_rows(rng, 400, 256)
    wv, w, w_s = quantized_weights(rng, 3, 256, 256)
    offsets = np.array([10, 10, 160, 333], np.int32)    # rows before the first and behind the last
    got = run_gemm(dims_of(200, 3, 2), a, a_s, offsets, w, w_s, 256)
    check_gemm(got, av, wv, offsets, torch.bfloat16)


def test_expert_gemm_bad_offsets_stay_inside(tiles):
    """Offsets outside the rows or out of order are clamped: no row out of range is touched."""
    rng = np.random.default_rng(6)
    av, a, a_s = quantized_rows(rng, 300, 128)
    wv, w, w_s = quantized_weights(rng, 4, 128, 128)
    got = run_gemm(dims_of(150, 4, 2), a, a_s, np.array([-5, 100, 60, 100000, 200], np.int32), w, w_s, 128)
    # expert 0: [0, 100); 1: nothing; 2: [60, 300); 3: nothing (its rows were expert 2's)
    want = np.where(np.arange(300)[:, None] < 60, av @ wv[0].T, av @ wv[2].T)
    sure = np.r_[0:60, 100:300]
    tol = 128 * 2.0 ** -23 * (np.abs(av) @ np.abs(wv).max(0).T) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol)[sure].all()


def test_expert_gemm_scales_over_the_range(tiles):
    """Row and weight scales far from 1, each block with its own."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((150, 640)) * np.repeat(2.0 ** rng.integers(-60, 60, (150, 5)), 128, 1)
    q, e, av = ref.quantize_blocks(x, 1, 128)
    w = rng.standard_normal((2, 256, 640)) * np.repeat(2.0 ** rng.integers(-30, 30, (2, 1, 5)), 128, 2)
    wq, we, wv = ref.quantize_blocks(w, 128, 128)
    offsets = np.array([0, 70, 150], np.int32)
    got = run_gemm(dims_of(150, 2, 1, dtype=torch.float32), ref.f8(q).cuda(), gpu(ref.row_scales(e, 150, 640)),
                   offsets, ref.f8(wq).cuda(), gpu(ref.weight_scales(we, 640)), 256)
    check_gemm(got, av, wv, offsets, torch.float32)


def test_expert_gemm_nan_stays_in_its_row(tiles):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((140, 256))
    x[130, 5] = np.nan
    q, e, av = ref.quantize_blocks(x, 1, 128)
    wv, w, w_s = quantized_weights(rng, 1, 256, 256)
    got = run_gemm(dims_of(140, 1, 1), ref.f8(q).cuda(), gpu(ref.row_scales(e, 140, 256)), None, w, w_s, 256)
    assert np.isnan(got[130]).all()
    ok = np.arange(140) != 130
    check_gemm(got[ok], av[ok], wv, [0, 139], torch.bfloat16)


def test_expert_gemm_input_gradient(tiles):
    """dA = dOut W: the same product with the transposed weights and scales."""
    rng = np.random.default_rng(10)
    R, n_out, n_in, P = 3, 272, 400, 260
    wv, w, w_s = quantized_weights(rng, R, n_out, n_in)
    offsets = offsets_of(rng, P, R)
    dv, dq, d_s = quantized_rows(rng, P, n_out)
    wt = w.transpose(1, 2).contiguous()
    wt_s = torch.full(lm.fp8_weight_scales_shape(R, n_in, n_out), 127, dtype=torch.uint8, device="cuda")
    cb, rb = (n_in + 127) // 128, (n_out + 127) // 128
    wt_s[:, :, :rb] = w_s[:, :, :cb].transpose(1, 2)
    got = run_gemm(dims_of(P, R, 1, dtype=torch.float32), dq, d_s, offsets, wt, wt_s, n_in)
    check_gemm(got, dv, wv.transpose(0, 2, 1), offsets, torch.float32)
    # against differences of <dOut, A W^T>, which is linear in A
    r, c, h = 17, 33, 0.25
    e = int(np.searchsorted(offsets, r, side="right") - 1)
    diff = dv[r] @ (wv[e] @ (h * np.eye(n_in)[c])) / h
    assert abs(got[r, c] - diff) <= n_out * 2.0 ** -23 * (np.abs(dv[r]) @ np.abs(wv[e][:, c])) + 2.0 ** -24 * abs(diff)


# -------------------------------------------------------------------- FFN
def ffn_case(rng, n, R, k, latent, ff, dtype, skew=1.0, w_std=0.05):
    z = torch.from_numpy(rng.standard_normal((n, latent))).to(dtype)
    offsets = offsets_of(rng, n * k, R, skew)
    perm = rng.integers(0, n, n * k).astype(np.int32)
    ws = [quantized_weights(rng, R, r, c, w_std) for r, c in ((ff, latent), (ff, latent), (latent, ff))]
    return z, perm, offsets, ws


def run_ffn(dims, z, perm, offsets, weights, fill=7.0, ws=None, out=None, stream=None):
    ws = lm.alloc_workspace(dims) if ws is None else ws
    if out is None:
        out = torch.full((dims.n_tokens * dims.top_k, dims.latent), fill, dtype=lm._act(dims), device="cuda")
    flat = [t for _, q, s in weights for t in (q, s)]
    lm.moe_expert_ffn_fp8(dims, z, perm, offsets, *flat, out, ws, stream=stream)
    return out, ws


def check_ffn(got, z, perm, offsets, weights, dtype, b1=4.0, b2=25.0, fill=7.0):
    want, bound = ref.ffn(z.double().numpy(), perm, offsets, *[v for v, _, _ in weights], b1, b2)
    tol = bound + ROUND[dtype] * (np.abs(want) + bound)
    inside = np.zeros(len(want), bool)
    inside[offsets[0]:offsets[-1]] = True
    err = np.abs(got - want)
    assert (err <= tol)[inside].all(), (err / np.maximum(tol, 1e-300))[inside].max()
    assert (got[~inside] == fill).all()


@pytest.mark.parametrize("n,R,k,latent,ff,dtype", [
    (1, 1, 1, 16, 16, torch.bfloat16),
    (1, 8, 4, 128, 128, torch.bfloat16),
    (5, 3, 2, 48, 144, torch.float32),
    (70, 5, 3, 528, 272, torch.bfloat16),
    (300, 16, 2, 384, 768, torch.bfloat16),
    (64, 100, 4, 272, 1040, torch.float32),
    (500, 2, 2, 640, 528, torch.bfloat16),
])
def test_expert_ffn(tiles, n, R, k, latent, ff, dtype):
    rng = np.random.default_rng(n + latent)
    z, perm, offsets, weights = ffn_case(rng, n, R, k, latent, ff, dtype)
    d = dims_of(n, R, k, latent, ff, dtype)
    out, ws = run_ffn(d, z.cuda(), gpu(perm), gpu(offsets), weights)
    assert lm.get_device_status(ws) == lm.OK
    check_ffn(out.double().cpu().numpy(), z, perm, offsets, weights, dtype)


def test_expert_ffn_wide_activations(tiles):
    """Pre-activations over +-15: the saturated ends of the gate, other caps than the defaults."""
    rng = np.random.default_rng(3)
    z, perm, offsets, weights = ffn_case(rng, 60, 4, 2, 256, 256, torch.bfloat16, w_std=0.4)
    d = lm.make_dims(60, 128, 256, 4, 2, 0, 256, 0, beta1=2.0, beta2=7.0)
    out, _ = run_ffn(d, z.cuda(), gpu(perm), gpu(offsets), weights)
    check_ffn(out.double().cpu().numpy(), z, perm, offsets, weights, torch.bfloat16, 2.0, 7.0)


def test_expert_ffn_nan_stays_in_its_rows(tiles):
    """A NaN (or an infinity, which 8 bits do not hold) in a token reaches its pairs only."""
    rng = np.random.default_rng(16)
    z, perm, offsets, weights = ffn_case(rng, 90, 3, 2, 256, 272, torch.bfloat16)
    z[17, 3], z[40, 200] = float("nan"), float("inf")
    out, ws = run_ffn(dims_of(90, 3, 2, 256, 272), z.cuda(), gpu(perm), gpu(offsets), weights)
    assert lm.get_device_status(ws) == lm.OK
    got = out.double().cpu().numpy()
    bad = np.isin(perm, (17, 40))
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    z[17], z[40] = 0.0, 0.0
    want, bound = ref.ffn(z.double().numpy(), perm, offsets, *[v for v, _, _ in weights], 4.0, 25.0)
    assert (np.abs(got - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound))[~bad].all()


def test_expert_ffn_dropped_rows_and_stray_tokens(tiles):
    """Sorted slots behind the last expert keep what they held; perm entries there are not read as rows."""
    rng = np.random.default_rng(4)
    z, perm, offsets, weights = ffn_case(rng, 100, 3, 2, 128, 256, torch.bfloat16)
    offsets = np.minimum(offsets, 150).astype(np.int32)
    perm[150:] = np.array([-1, 1 << 30] * 25, np.int32)
    out, ws = run_ffn(dims_of(100, 3, 2, 128, 256), z.cuda(), gpu(perm), gpu(offsets), weights)
    assert lm.get_device_status(ws) == lm.OK
    check_ffn(out.double().cpu().numpy(), z, perm, offsets, weights, torch.bfloat16)


def test_expert_ffn_repeats_streams_and_graphs(tiles):
    """The same bits on every call, on another stream and from a replayed graph with new inputs."""
    rng = np.random.default_rng(11)
    z, perm, offsets, weights = ffn_case(rng, 200, 6, 2, 384, 272, torch.bfloat16)
    d = dims_of(200, 6, 2, 384, 272)
    zd, pd, od = z.cuda(), gpu(perm), gpu(offsets)
    first, ws = run_ffn(d, zd, pd, od, weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                       # its buffers are made there too
        again, _ = run_ffn(d, zd, pd, od, weights)
    side.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(first)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run_ffn(d, zd, pd, od, weights, ws=ws, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    z2 = torch.from_numpy(rng.standard_normal(z.shape)).to(z.dtype)
    off2 = offsets_of(rng, 400, 6)
    zd.copy_(z2)
    od.copy_(torch.from_numpy(off2))
    graph.replay()
    torch.cuda.synchronize()
    check_ffn(out.double().cpu().numpy(), z2, perm, off2, weights, torch.bfloat16)


@pytest.mark.parametrize("n,R,k,latent,ff", [(3000, 5, 4, 1536, 512), (2500, 9, 8, 1024, 528)])
def test_expert_ffn_many_rows(n, R, k, latent, ff):
    """Enough to quantise once per token and sort, and for the tile rule to take pairs; a sample of
    the rows is compared."""
    rng = np.random.default_rng(n)
    z = torch.from_numpy(rng.standard_normal((n, latent))).to(torch.bfloat16)
    offsets = offsets_of(rng, n * k, R, 0.5)
    offsets[-1] -= 7                                    # dropped rows at the end
    perm = rng.integers(0, n, n * k).astype(np.int32)
    perm[-7:] = -1
    weights = [quantized_weights(rng, R, r, c, 0.05) for r, c in ((ff, latent), (ff, latent), (latent, ff))]
    out, ws = run_ffn(dims_of(n, R, k, latent, ff), z.cuda(), gpu(perm), gpu(offsets), weights)
    assert lm.get_device_status(ws) == lm.OK
    got = out.double().cpu().numpy()
    assert (got[-7:] == 7.0).all()
    for e in range(R):
        lo, hi = offsets[e], offsets[e + 1]
        if hi == lo:
            continue
        rows = np.unique(np.r_[lo, (lo + hi) // 2, hi - 1, rng.integers(lo, hi, 6)])
        want, bound = ref.ffn(z.double().numpy(), perm[rows], [0, len(rows)], *[v[e:e + 1] for v, _, _ in weights],
                              4.0, 25.0)
        assert (np.abs(got[rows] - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all(), e


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^31 and 2^32."""
    rng = np.random.default_rng(2)
    n, cols = 290_000, 16384                            # 4.75e9 quantised bytes
    x = torch.from_numpy(rng.standard_normal((64, cols))).to(torch.bfloat16).cuda()
    index = torch.arange(n, dtype=torch.int32, device="cuda") % 64
    q = torch.empty(n, cols, dtype=F8, device="cuda")
    s = torch.empty(lm.fp8_row_scales_shape(n, cols), dtype=torch.uint8, device="cuda")
    lm.quantize_rows_fp8(x, q, s, index=index)
    want = torch.empty(64, cols, dtype=F8, device="cuda"), torch.empty(cols // 512, 64, 4, dtype=torch.uint8, device="cuda")
    lm.quantize_rows_fp8(x, *want)
    tail = slice(n - 64, n)
    order = index[tail].long()
    assert torch.equal(q[tail].view(torch.uint8), want[0].view(torch.uint8)[order])
    assert torch.equal(s[:, tail], want[1][:, order])
    # a product that reads them, and one that writes past 2^32 bytes
    wv, w, w_s = quantized_weights(rng, 1, 8, cols)
    d = dims_of(n, 1, 1)
    ws = lm.alloc_workspace(d)
    out = torch.empty(n, 8, dtype=torch.bfloat16, device="cuda")
    lm.moe_expert_gemm_fp8(d, q, s, None, w, w_s, out, ws)
    av = ref.quantize_blocks(x.double().cpu().numpy(), 1, 128)[2][order.cpu().numpy()]
    check_gemm(out[tail].double().cpu().numpy(), av, wv, [0, 64], torch.bfloat16)
    del q, s, out
    av, a, a_s = quantized_rows(rng, 64, 16)
    rows = index[:150_000].long()
    wv, w, w_s = quantized_weights(rng, 1, cols, 16)
    d = dims_of(150_000, 1, 1)
    big = torch.empty(150_000, cols, dtype=torch.bfloat16, device="cuda")
    lm.moe_expert_gemm_fp8(d, a.view(torch.uint8)[rows].view(F8), a_s[:, rows].contiguous(), None, w, w_s, big,
                           lm.alloc_workspace(d))
    check_gemm(big[-64:].double().cpu().numpy(), av[rows[-64:].cpu().numpy()], wv, [0, 64], torch.bfloat16)


def test_two_streams_at_once():
    """Calls that run side by side, each with its own workspace."""
    rng = np.random.default_rng(14)
    z, perm, offsets, weights = ffn_case(rng, 300, 6, 2, 256, 256, torch.bfloat16)
    d = dims_of(300, 6, 2, 256, 256)
    zd, pd, od = z.cuda(), gpu(perm), gpu(offsets)
    want, _ = run_ffn(d, zd, pd, od, weights)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(4)], []
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(run_ffn(d, zd, pd, od, weights))
    torch.cuda.synchronize()
    for out, ws in outs:
        assert lm.get_device_status(ws) == lm.OK and torch.equal(out, want)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_other_device_is_refused():
    x = torch.zeros(4, 64, device="cuda:1")
    with pytest.raises(lm.LmoeError):
        lm.quantize_rows_fp8(x, torch.zeros(4, 64, dtype=F8, device="cuda:1"),
                             torch.zeros(1, 4, 4, dtype=torch.uint8, device="cuda:1"))


def test_binding_refuses_wrong_tensors():
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
    q, s = z(4, 64, dtype=F8), z(1, 4, 4, dtype=torch.uint8)
    for bad in ((z(4, 64).half(), q, s), (z(4, 64), z(4, 32, dtype=F8), s), (z(4, 64), q, z(2, 4, 4, dtype=torch.uint8)),
                (z(64, 4).t(), q, s), (z(4, 66)[:, 1:65], q, s)):
        with pytest.raises(lm.LmoeError):
            lm.quantize_rows_fp8(*bad)
    with pytest.raises(lm.LmoeError):
        lm.quantize_rows_fp8(z(4, 64), q, s, index=z(4, dtype=torch.int64))
    d = dims_of(4, 2, 1)
    w, w_s = z(2, 128, 64, dtype=F8), z(*lm.fp8_weight_scales_shape(2, 128, 64), dtype=torch.uint8)
    off, out, ws = z(3, dtype=torch.int32), z(4, 128, dtype=torch.bfloat16), lm.alloc_workspace(d)
    lm.moe_expert_gemm_fp8(d, q, s, off, w, w_s, out, ws)
    for bad in ((q, s, None, w, w_s, out), (q, s, off, w, w_s, out.float()), (q, s, off, w[:1], w_s, out),
                (q, s, off.long(), w, w_s, out), (q, s, off, w, w_s, z(128, 4, dtype=torch.bfloat16).t())):
        with pytest.raises(lm.LmoeError):
            lm.moe_expert_gemm_fp8(d, *bad, ws)


def test_no_tokens():
    d = dims_of(0, 4, 2)
    ws = lm.alloc_workspace(d)
    rng = np.random.default_rng(0)
    _, w, w_s = quantized_weights(rng, 4, 128, 128)
    e = lambda *s, dtype=torch.int32: torch.empty(*s, dtype=dtype, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    out = e(0, 128, dtype=torch.bfloat16)
    lm.moe_expert_gemm_fp8(d, e(0, 128, dtype=F8), e(1, 0, 4, dtype=torch.uint8), off, w, w_s, out, ws)
    lm.moe_expert_ffn_fp8(d, out, e(0), off, w, w_s, w, w_s, w, w_s, out, ws)
    lm.quantize_rows_fp8(out, e(0, 128, dtype=F8), e(1, 0, 4, dtype=torch.uint8))
    assert lm.get_device_status(ws) == lm.OK
