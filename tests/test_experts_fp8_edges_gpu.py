"""8-bit routed experts where they can go wrong: offsets that do not ascend, calls one
behind the other."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

lm = pytest.importorskip("sigmoid_top_routing_latentmoe_b200")


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
