"""Plain implementations in 64 bits of the operators around the routed
experts, from their definitions in include/moe.h (numpy; the tests compare the
CUDA kernels against these)."""
import numpy as np

from streamed_quantized_expert_b200.synth import bf16_bits_to_f32, to_bf16_bits

U32 = 2.0 ** -24  # half a step of fp32, relative
UBF = 2.0 ** -8   # half a step of bf16, relative


def round_to(a, f32: bool):
    """fp32 values rounded to the type they are kept in."""
    a = np.ascontiguousarray(a, np.float32)
    return a if f32 else bf16_bits_to_f32(to_bf16_bits(a))


def route(logits, k, sigmoid, bias=None, G=1, top=1, gtop=1, renorm=True, scale=1.0, L=0.0, table=None):
    """(ids, w, c): c is the score that chooses, -inf for experts that are off."""
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    off = np.isneginf(l)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            u = np.exp(l - l.max(axis=1, keepdims=True))
            u[off] = 0.0
            tot = u.sum(axis=1, keepdims=True)
            s = np.where(tot > 0, u / np.where(tot > 0, tot, 1.0), 0.0)
    s[off] = 0.0
    c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    c[off] = -np.inf
    if L > 0:
        hi = np.where(off, -np.inf, c).max(axis=1)
        lo = np.where(off, np.inf, c).min(axis=1)
        # c + L (hi - lo), from hi downwards: at L = 1 the lowest meets hi exactly
        with np.errstate(invalid="ignore"):
            up = hi[:, None] + ((c - lo[:, None]) + (np.float64(np.float32(L)) - 1.0) * (hi - lo)[:, None])
        c = np.where((np.asarray(table)[:E] >= 0)[None, :] & ~off & (hi > lo)[:, None], up, c)
    m = E // G
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        groups = range(G)
        if top < G:
            score = [c[t, g * m:(g + 1) * m].max() for g in range(G)]
            for g in range(G) if gtop == 2 else ():
                # scores, biases and lifts each for itself: what is equal over the reals is equal here
                e1, e2 = g * m + np.argsort(-c[t, g * m:(g + 1) * m], kind="stable")[:2]
                score[g] = -np.inf
                if not (off[t, e1] or off[t, e2]):
                    score[g] = s[t, e1] + s[t, e2] + (0.0 if bias is None else np.float64(bias[e1]) + np.float64(bias[e2]))
                    n = 0 if L == 0 or not hi[t] > lo[t] else int(table[e1] >= 0) + int(table[e2] >= 0)
                    if n:
                        down = (np.float64(np.float32(L)) - 1.0) * (hi[t] - lo[t])
                        score[g] = n * hi[t] + ((score[g] - n * lo[t]) + n * down)
            groups = sorted(range(G), key=lambda g: (-score[g], g))[:top]
        cand = [e for g in groups for e in range(g * m, (g + 1) * m)]
        cand.sort(key=lambda e: (-c[t, e], -l[t, e], e))
        ids[t] = cand[:k]
        w[t] = s[t, ids[t]]
        den = w[t].sum() if renorm else 1.0
        w[t] = scale * w[t] / den if den > 0 else 0.0
    return ids, w, c


def codes(p):
    """(q, a, t): codes and largest magnitudes of the rows of p, and 127 p / a
    itself; rows of zeros or with a non-finite value have codes 0."""
    p = np.asarray(p, np.float64)
    with np.errstate(invalid="ignore"):
        a = np.abs(p).max(axis=1)
        ok = np.isfinite(p).all(axis=1) & (a > 0)
        t = np.where(ok[:, None], 127.0 * np.where(ok[:, None], p, 0.0) / np.where(ok, a, 1.0)[:, None], 0.0)
    a = np.where(np.isfinite(p).all(axis=1), a, np.nan)
    return np.rint(t).astype(np.int8), a, t


def add_norm(h, h_f32, delta, gamma, eps):
    """(h', x, p, r) of moe_add_norm_quant for values already in their types."""
    hn = np.asarray(h, np.float32)
    if delta is not None:
        with np.errstate(invalid="ignore", over="ignore"):
            hn = round_to(hn + np.asarray(delta, np.float32), h_f32)
    h64, g = hn.astype(np.float64), np.asarray(gamma, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        r = 1.0 / np.sqrt((h64 ** 2).mean(axis=1) + np.float64(np.float32(eps)))
        p = hn * np.asarray(gamma, np.float32)[None, :]  # fp32, as the codes are defined
        return hn, h64 * r[:, None] * g, p, r


def swiglu(gu):
    gu = np.asarray(gu, np.float64)
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def int_matmul(xq, xs, wq, ws, add=None, row_w=None):
    """(y, the product alone), both in 64 bits."""
    acc = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T  # below 2^53: exact
    prod = acc * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :]
    if row_w is not None:
        prod = prod * np.asarray(row_w, np.float64)[:, None]
    return (prod if add is None else prod + np.asarray(add, np.float64)), prod
