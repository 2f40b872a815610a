"""64-bit references of the 8-bit routed experts and of routing under a rule."""
import numpy as np
import torch

F8 = torch.float8_e4m3fn


def exponents(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e; 0 for a block of zeros."""
    amax = np.asarray(amax, np.float64)
    m, x = np.frexp(np.where(amax > 0, amax, 1.0) / 448.0)   # in [0.5, 1) * 2^x
    return np.where(amax > 0, np.maximum(np.where(m > 0.5, x, x - 1), -126), 0).astype(np.int64)


def e4m3(v):
    """Round-to-nearest-even e4m3 of float64 values with |v| <= 448 (NaN and infinities: NaN)."""
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -20))), -6.0) - 3.0)
        return np.where(np.isfinite(v), np.round(v / ulp) * ulp, np.nan)


def quantize_blocks(x, br, bc):
    """(q values, exponents, dequantised values) of x [..., r, c] in blocks of br x bc."""
    x = np.asarray(x, np.float64)
    r, c = x.shape[-2:]
    rp, cp = -(-r // br) * br, -(-c // bc) * bc
    b = np.zeros(x.shape[:-2] + (rp, cp))
    b[..., :r, :c] = x
    b = b.reshape(x.shape[:-2] + (rp // br, br, cp // bc, bc))
    amax = np.where(np.isfinite(b), np.abs(b), 0.0).max((-3, -1))
    e = exponents(amax)
    s = np.exp2(e.astype(np.float64))[..., :, None, :, None]
    q = e4m3(b / s)
    back = lambda t: t.reshape(x.shape[:-2] + (rp, cp))[..., :r, :c]
    return back(q), e, back(q * s)


def row_scales(e, n, cols):
    """Scale bytes [words, n, 4] of exponents e [n, blocks]."""
    full = np.full((n, 4 * ((cols + 511) // 512)), 127, np.uint8)
    full[:, :e.shape[1]] = e + 127
    return np.ascontiguousarray(full.reshape(n, -1, 4).transpose(1, 0, 2))


def weight_scales(e, cols):
    """Scale bytes [m, row blocks, 4 words] of exponents e [m, row blocks, blocks]."""
    full = np.full(e.shape[:2] + (4 * ((cols + 511) // 512),), 127, np.uint8)
    full[..., :e.shape[2]] = e + 127
    return full


def f8(q):
    """Values on the e4m3 grid as a tensor."""
    return torch.from_numpy(np.asarray(q, np.float32)).to(F8)


def situ(a, c, b1, b2):
    with np.errstate(over="ignore"):
        return b1 * np.tanh(a / b1) / (1 + np.exp(-a)) * b2 * np.tanh(c / b2)


def ffn(z, perm, offsets, wg, wu, wo, b1, b2):
    """(out, bound) of the routed experts with 8-bit products, from the values the quantised
    weights stand for.  The bound covers what 32-bit arithmetic may change:

    * a product of K terms in 32 bits is off by at most K 2^-23 sum |terms| (each addend is
      rounded or cut once at the size of the sum of magnitudes);
    * a hidden unit h = gate(a) up(c) is then off by |gate'| <= 1.1 times |up| da, |gate| dc
      (|up'| <= 1) and 16 roundings of its own;
    * where that reaches a midpoint of two e4m3 values the hidden unit may be off by one step,
      and where a block's maximum lies that near to 448 scales, the whole block may be
      quantised at twice the scale;
    * the last product as the first two.
    """
    K, F = z.shape[1], wg.shape[1]
    zq = quantize_blocks(z, 1, 128)[2]
    out = np.zeros((len(perm), wo.shape[1]))
    bound = np.zeros_like(out)
    for e in range(wg.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        x = zq[perm[lo:hi]]
        a, c = x @ wg[e].T, x @ wu[e].T
        da, dc = (K * 2.0 ** -23 * (np.abs(x) @ np.abs(w[e]).T) for w in (wg, wu))
        h = situ(a, c, b1, b2)
        gate = np.abs(b1 * np.tanh(a / b1) / (1 + np.exp(-a)))
        dh = 1.1 * b2 * np.abs(np.tanh(c / b2)) * da + gate * dc + 16 * 2.0 ** -24 * np.abs(h)
        q, ex, hq = quantize_blocks(h, 1, 128)
        s = np.exp2(np.repeat(ex, 128, 1)[:, :F].astype(float))
        ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(h) / s, 2.0 ** -20))), -6) - 3) * s
        slack = np.abs(np.abs(h - hq) - ulp / 2)     # distance to the midpoint
        err = np.where(slack <= dh, ulp, 0.0)
        pad = np.zeros((hi - lo, ex.shape[1] * 128))
        for t, u in ((np.abs(h), 0), (dh, 1)):
            pad[:, :F] = t
            m = pad.reshape(hi - lo, -1, 128).max(2)
            amax, d = (m, None) if u == 0 else (amax, m)
        edge = (exponents(amax + d) != ex) | (exponents(np.maximum(amax - d, 0)) != ex)
        err = np.where(np.repeat(edge, 128, 1)[:, :F], 2 * ulp, err)
        out[lo:hi] = hq @ wo[e].T
        bound[lo:hi] = err @ np.abs(wo[e]).T + F * 2.0 ** -23 * ((np.abs(hq) + err) @ np.abs(wo[e]).T)
    return out, bound


def route_keys(logits, bias, score):
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            top = np.max(l, 1, keepdims=True)
            ex = np.exp(l - np.where(np.isneginf(top), 0.0, top))
            tot = ex.sum(1, keepdims=True)
            s = ex / np.where(tot == 0, 1.0, tot)
        key = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    return s, np.where(np.isnan(key), -np.inf, key)


def route(logits, bias, k, score="sigmoid", groups=1, kept=1, top2=True, renorm=True, scale=1.0):
    """(ids, weights, smallest decisive gap of each row)."""
    s, key = route_keys(logits, bias, score)
    n, R = key.shape
    size = R // groups
    ids = np.zeros((n, k), np.int64)
    gap = np.full(n, np.inf)
    with np.errstate(invalid="ignore"):
        for t in range(n):
            by = -np.sort(-key[t].reshape(groups, size), 1)
            gs = by[:, 0] + by[:, 1] if top2 and size > 1 else by[:, 0]
            gs = np.where(np.isnan(gs), -np.inf, gs)
            order = np.lexsort((np.arange(groups), -gs))
            if kept < groups:
                gap[t] = gs[order[kept - 1]] - gs[order[kept]]
            experts = np.sort(np.concatenate([np.arange(g * size, (g + 1) * size) for g in order[:kept]]))
            best = experts[np.lexsort((experts, -key[t, experts]))]
            ids[t] = best[:k]
            d = -np.diff(key[t, best[:k + 1]])
            if d.size:
                gap[t] = np.fmin(gap[t], np.nanmin(np.where(np.isnan(d), np.inf, d)))
        w = np.take_along_axis(s, ids, 1)
        if renorm:
            w = w / np.maximum(w.sum(1, keepdims=True), 1e-9)
    return ids, scale * w, gap
