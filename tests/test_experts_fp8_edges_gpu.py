"""8-bit routed experts where they can go wrong: offsets that do not ascend, calls one
behind the other, hidden units next to rounding borders, the accumulator
of the products."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")

U = 2.0 ** -24


@pytest.fixture(params=["0", "1"], ids=["single", "pairs"])
def tiles(request, monkeypatch):
    """Single CTAs over 128-row tiles, CTA pairs over 256-row ones."""
    monkeypatch.setenv("LMOE_FP8_PAIRS", request.param)


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def quantized(x, br):
    """(values in 64 bits, e4m3 tensor, scales) of rows (br = 1) or stacked matrices (br = 128)."""
    q, e, v = ref.quantize_blocks(x, br, 128)
    return v, ref.f8(q).cuda(), gpu(ref.row_scales(e, *x.shape) if br == 1 else ref.weight_scales(e, x.shape[2]))


def ascending(offsets, rows):
    return np.maximum.accumulate(np.clip(offsets, 0, rows))


BAD_OFFSETS = {
    "back": (4, [-5, 100, 60, 100000, 200]),
    "all to the first": (7, [0, 300] + [0, 300] * 3),
    "falling": (5, [300, 250, 130, 70, 20, 0]),
    "none": (3, [400, -1, 17, 12]),
    "many": (600, np.random.default_rng(3).integers(-50, 400, 601)),     # more experts than a block scans at a time
}


@pytest.mark.parametrize("name", BAD_OFFSETS)
def test_offsets_that_do_not_ascend(tiles, name):
    """Each row has one expert: bounds are the running maximum of the clamped offsets.  The product and the FFN
    give the same bits as with those bounds."""
    R, offsets = BAD_OFFSETS[name]
    rng = np.random.default_rng(R)
    P, L, F = 300, 128, 144
    bounds = ascending(offsets, P).astype(np.int32)
    av, a, a_s = quantized(rng.standard_normal((P, L)), 1)
    (wv, w, w_s), (_, wu, wu_s), (_, wo, wo_s) = (quantized(0.05 * rng.standard_normal((R, r, c)), 128)
                                                   for r, c in ((F, L), (F, L), (L, F)))
    d = lm.make_dims(P, 128, L, R, 1, 0, F, 0, dtype=torch.float32)
    z, perm = gpu(rng.standard_normal((P, L)).astype(np.float32)), gpu(np.arange(P, dtype=np.int32))

    def run(off):
        off, ws = gpu(np.asarray(off, np.int32)), lm.alloc_workspace(d)
        out, eo = torch.full((P, F), 7.0, device="cuda"), torch.full((P, L), 7.0, device="cuda")
        lm.moe_expert_gemm_fp8(d, a, a_s, off, w, w_s, out, ws)
        lm.moe_expert_ffn_fp8(d, z, perm, off, w, w_s, wu, wu_s, wo, wo_s, eo, ws)
        assert lm.get_device_status(ws) == lm.OK
        return out, eo

    got, want = run(offsets), run(bounds)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = got[0].double().cpu().numpy()
    outside = np.ones(P, bool)
    for e in range(R):
        r = slice(bounds[e], bounds[e + 1])
        outside[r] = False
        tol = (L / 32 + 2) * 2.0 ** -23 * (np.abs(av[r]) @ np.abs(wv[e]).T)     # a rounding for each step of 32
        assert (np.abs(out[r] - av[r] @ wv[e].T) <= tol).all(), e
    assert (out[outside] == 7.0).all()


def test_calls_one_behind_the_other(tiles):
    """Products of other shapes in turn, each started beside the end of the one before: the same bits every time."""
    rng = np.random.default_rng(12)
    runs = []
    for n, R, n_in, n_out in ((700, 2, 128, 256), (1500, 3, 640, 264), (300, 1, 2064, 520)):
        _, a, a_s = quantized(rng.standard_normal((n, n_in)), 1)
        _, w, w_s = quantized(0.05 * rng.standard_normal((R, n_out, n_in)), 128)
        d = lm.make_dims(n, 128, 128, R, 1, 0, 128, 0, dtype=torch.float32)
        off = gpu(np.linspace(0, n, R + 1).astype(np.int32))
        runs.append((d, a, a_s, off, w, w_s, lm.alloc_workspace(d)))

    def outputs():
        outs = [torch.empty(r[0].n_tokens, r[4].shape[1], device="cuda") for r in runs]
        for r, out in zip(runs, outs):
            lm.moe_expert_gemm_fp8(*r[:6], out, r[6])
        return outs

    want = outputs()
    for outs in [outputs() for _ in range(60)]:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(lm.get_device_status(r[6]) == lm.OK for r in runs)


def border_case(gate, b1, b2, near, rng):
    """128 up projections c (multiples of 2^-20 below 16) whose hidden units with gate projection `gate` lie `near`
    roundings above or below the middle between two e4m3 values; the first unit sets the block's scale."""
    g = b1 * np.tanh(gate / b1) / (1.0 + np.exp(-gate))
    c = np.empty(128)
    c[0] = 16.0 - 2.0 ** -20
    e = int(ref.exponents(abs(g) * b2 * np.tanh(c[0] / b2)))
    top, least = (abs(g) * b2 * np.tanh(v / b2) * 2.0 ** -e for v in (c[0], 4.0))
    borders = np.concatenate([(np.arange(8, 16) + 0.5) * 2.0 ** x for x in range(-4, 6)])
    borders = borders[(borders > 1.001 * least) & (borders < 0.999 * top)]
    m = rng.choice(borders, 127) * (1.0 + near * U * rng.choice([-1.0, 1.0], 127))
    c[1:] = np.round(b2 * np.arctanh(m * 2.0 ** e / abs(g) / b2) * 2.0 ** 20) * 2.0 ** -20
    return c


@pytest.mark.parametrize("b1,b2", [(4.0, 25.0), (64.0, 40.0), (2.0, 1e6)])
def test_hidden_units_next_to_rounding_borders(tiles, b1, b2):
    """Hidden units beta1 tanh(a / beta1) sigmoid(a) beta2 tanh(c / beta2) for exact a from -80 to 80 and exact c,
    each some 28 roundings (2^-24) from the middle between two e4m3 values: an activation in 32 bits puts them on
    the right side.  Its error is at most 25 roundings.  By polynomials (|a| <= 5.5): e^-a 8 (ex2 4, its argument up
    to 8 4), 1 + e^-a 1, the reciprocal 2, numerators 6 and 4, products 2.  Beyond: e^-a 5 (the argument's rest is
    made up for), 1 + e^-a 1, denominators 1 + t 2 and their products 2, the reciprocal 2, numerators b - b t 2 and
    2, t itself (ex2 4, argument 1) 1 and 6 on the quotients at |x| = 1.5 and 0.5, products 2."""
    rng = np.random.default_rng(7)
    p, q = rng.integers(8, 16, 60), rng.integers(8, 16, 60)
    size = p * q * 2.0 ** rng.integers(-6, 0, 60)               # 1 ... 113, four bits by four bits
    gates = np.where(rng.random(60) < 0.75, -1.0, 1.0) * np.where(size > 80, size / 2, size)
    R, F, L = len(gates), 128, 384
    cs = np.stack([border_case(g, b1, b2, 28.0, rng) for g in gates])
    # gate row: z[256] W_g[256] = a.  up row: six digits of c to the base 16, each in an MMA step of its own
    z, wg, wu, wo = np.zeros((R, L)), np.zeros((R, F, L)), np.zeros((R, F, L)), np.zeros((R, L, F))
    mant = np.where(size > 80, 0.5, 1.0) * size / (p * q)
    z[:, 256], wg[:, :, 256] = np.sign(gates) * p * mant, q[:, None]
    left = cs.copy()
    for i in range(6):
        z[:, 32 * i] = 2.0 ** (-4 * i)
        wu[:, :, 32 * i] = np.floor(left * 2.0 ** (4 * i))
        left -= wu[:, :, 32 * i] * z[0, 32 * i]
    assert (left == 0).all() and wu.max() <= 15
    wo[:, np.arange(F), np.arange(F)] = 1.0
    zq = ref.quantize_blocks(z, 1, 128)[2]
    ws = [quantized(w, 128) for w in (wg, wu, wo)]
    assert (zq == z).all() and all((v == w).all() for (v, _, _), w in zip(ws, (wg, wu, wo)))
    h = (b1 * np.tanh(gates / b1) / (1 + np.exp(-gates)))[:, None] * b2 * np.tanh(cs / b2)
    want_q, want_e, want = ref.quantize_blocks(h, 1, 128)
    scaled = np.abs(h) * np.exp2(-want_e.astype(float))
    ulp = np.exp2(np.floor(np.log2(scaled)) - 3)
    off = np.abs(scaled / ulp - np.floor(scaled / ulp) - 0.5) * ulp / scaled / U
    assert (off[:, 1:] > 25).all() and (off[:, 1:] < 34).all()
    d = lm.make_dims(R, 128, L, R, 1, 0, F, 0, beta1=b1, beta2=b2, dtype=torch.float32)
    work, out = lm.alloc_workspace(d), torch.zeros(R, L, device="cuda")
    lm.moe_expert_ffn_fp8(d, gpu(z.astype(np.float32)), gpu(np.arange(R, dtype=np.int32)),
                          gpu(np.arange(R + 1, dtype=np.int32)), *[t for _, q8, s in ws for t in (q8, s)], out, work)
    assert lm.get_device_status(work) == lm.OK
    got = out.double().cpu().numpy()
    wrong = got[:, :F] != want
    assert not wrong.any(), (int(wrong.sum()), np.unique(gates[wrong.any(1)]))
    assert (got[:, F:] == 0).all()


def test_rows_beside_saturated_ones(tiles):
    """A row's bits do not depend on the rows beside it: the same alone and among rows whose units saturate."""
    rng = np.random.default_rng(19)
    n, L, F = 96, 256, 272
    z = rng.standard_normal((n, L)).astype(np.float32)
    wild = z.copy()
    wild[::2] *= 200.0
    ws = [quantized(0.08 * rng.standard_normal((1, r, c)), 128) for r, c in ((F, L), (F, L), (L, F))]
    flat = [t for _, q, s in ws for t in (q, s)]
    d = lm.make_dims(n, 128, L, 1, 1, 0, F, 0, dtype=torch.float32)
    outs = []
    for rows in (z, wild):
        out, work = torch.zeros(n, L, device="cuda"), lm.alloc_workspace(d)
        lm.moe_expert_ffn_fp8(d, gpu(rows), gpu(np.arange(n, dtype=np.int32)), gpu(np.array([0, n], np.int32)), *flat,
                              out, work)
        outs.append(out)
    assert torch.equal(outs[0][1::2], outs[1][1::2])
    assert torch.isfinite(outs[1]).all() and not torch.equal(outs[0][::2], outs[1][::2])


def product(a, w):
    """a w^T and what 32-bit sums may be off by: each MMA adds the 32 products of a step to the accumulator, rounded
    or cut at 2^-23 of the larger of the accumulator and of the step's magnitudes.  (Random signs keep the
    accumulator far below the sum of all magnitudes; positive terms do not.)"""
    acc, tol = np.zeros((len(a), len(w))), 0.0
    for s in range(0, a.shape[1], 32):
        at, wt = a[:, s:s + 32], w[:, s:s + 32].T
        tol = tol + 2 * U * (np.abs(acc) + np.abs(at) @ np.abs(wt))
        acc = acc + at @ wt
    return acc, tol


@pytest.mark.parametrize("sign", ["either", "positive"])
@pytest.mark.parametrize("K", [16, 144, 528, 2064, 4096])
def test_product_keeps_a_32_bit_accumulator(tiles, K, sign):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((150, K)) * np.exp(rng.standard_normal((150, 1)))
    w = rng.standard_normal((2, 264, K)) * 0.02
    if sign == "positive":
        x, w = np.abs(x), np.abs(w)
    av, a, a_s = quantized(x, 1)
    wv, wq, w_s = quantized(w, 128)
    offsets = np.array([0, 70, 150], np.int32)
    d = lm.make_dims(150, 128, 128, 2, 1, 0, 128, 0, dtype=torch.float32)
    out = torch.empty(150, 264, device="cuda")
    lm.moe_expert_gemm_fp8(d, a, a_s, gpu(offsets), wq, w_s, out, lm.alloc_workspace(d))
    got = out.double().cpu().numpy()
    for e in range(2):
        r = slice(offsets[e], offsets[e + 1])
        want, tol = product(av[r], wv[e])
        assert (np.abs(got[r] - want) <= tol).all(), (np.abs(got[r] - want) / tol).max()


@pytest.mark.parametrize("n,L,F,std", [(120, 528, 272, 0.05), (90, 2064, 144, 0.05), (60, 256, 1040, 0.4)])
def test_ffn_keeps_32_bits(tiles, n, L, F, std):
    """The FFN with the bounds of `product`: a hidden unit may take the next e4m3 value (or its block the next
    scale) only where it lies within 25 roundings and the projections' errors of that border.  The gate changes by
    at most |gate'| da + da^2 (|gate''| < 2), up by at most dc."""
    rng = np.random.default_rng(L)
    z = rng.standard_normal((n, L)).astype(np.float32)
    zq = ref.quantize_blocks(z, 1, 128)[2]
    ws = [quantized(std * rng.standard_normal((1, r, c)), 128) for r, c in ((F, L), (F, L), (L, F))]
    (a, da), (c, dc) = (product(zq, v[0]) for v, _, _ in ws[:2])
    h = ref.situ(a, c, 4.0, 25.0)
    sig, cap = 1 / (1 + np.exp(-a)), 4.0 * np.tanh(a / 4.0)
    d_gate = np.abs(sig / np.cosh(a / 4.0) ** 2 + cap * sig * (1 - sig)) * da + da ** 2
    d_up, up = dc, np.abs(25.0 * np.tanh(c / 25.0))
    dh = up * d_gate + np.abs(cap * sig) * d_up + d_gate * d_up + 25 * U * np.abs(h)
    q, e, hq = ref.quantize_blocks(h, 1, 128)
    s = np.exp2(np.repeat(e, 128, 1)[:, :F].astype(float))
    ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(h) / s, 2.0 ** -20))), -6) - 3) * s
    err = np.where(np.abs(np.abs(h - hq) - ulp / 2) <= dh, ulp, 0.0)
    pad = np.zeros((2, n, e.shape[1] * 128))
    pad[0, :, :F], pad[1, :, :F] = np.abs(h), dh
    top, d_top = pad.reshape(2, n, -1, 128).max(3)
    edge = (ref.exponents(top + d_top) != e) | (ref.exponents(np.maximum(top - d_top, 0)) != e)
    err = np.where(np.repeat(edge, 128, 1)[:, :F], 2 * ulp, err)
    assert (err > 0).mean() < 0.01                      # few units are left that open
    wo = ws[2][0][0]
    want, tol = product(hq, wo)
    tol = tol + err @ np.abs(wo).T * (1 + 2 * (F / 32 + 1) * U)
    d = lm.make_dims(n, 128, L, 1, 1, 0, F, 0, dtype=torch.float32)
    out, work = torch.zeros(n, L, device="cuda"), lm.alloc_workspace(d)
    lm.moe_expert_ffn_fp8(d, gpu(z), gpu(np.arange(n, dtype=np.int32)), gpu(np.array([0, n], np.int32)),
                          *[t for _, q8, sc in ws for t in (q8, sc)], out, work)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
