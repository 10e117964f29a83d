"""Plain 64-bit references of the router, the 4-bit products and the expert
layer, with bounds on what fp32 evaluation may differ by.

Bounds: u32 = 2^-24 is half a step of fp32. An MFMA adds 32 exact products to
its accumulator; it is taken to round at most 8 times, each time by at most a
whole step (2 u32) of the sum of the magnitudes so far. The terms of a sum of
K inputs then cost at most K / 32 * 8 * 2 u32 of the sum of |w x|, its join
over the waves up to 16 u32 more.
"""
import numpy as np

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": U32}  # half a step of the output type
FP4 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def bf16(a):
    """float64 values rounded to bf16 (nearest even), as float32."""
    u = np.asarray(a, np.float32).view(np.uint32)
    u = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return u.view(np.float32)


def bits(a):
    return (np.ascontiguousarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)


# ----------------------------------------------------------------- router

def route(l, K, bias=None, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
          scale=1.0):
    T, E = l.shape
    l = np.asarray(l, np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    ids, out = np.full((T, K), -1, np.int32), np.zeros((T, K))
    for t in range(T):
        row, live = l[t], l[t] > -np.inf
        with np.errstate(over="ignore"):
            if scoring == "sigmoid":
                s = np.where(live, 1 / (1 + np.exp(-np.where(live, row, 0))), 0)
            else:
                e = np.where(live, np.exp(row - (row.max() if live.any() else 0)), 0)
                s = e / max(e.sum(), 1e-300)
        c = row if bias is None else s + np.asarray(bias, np.float64)
        c = np.where(live & ~np.isnan(c), c, -np.inf)
        if n_group > 1:
            per = np.sort(c.reshape(n_group, -1), 1)[:, ::-1]
            v = per[:, 0].copy()
            if bias is not None and per.shape[1] > 1:
                v += np.where(per[:, 1] > -np.inf, per[:, 1], 0)
            keep = np.zeros(n_group, bool)
            keep[np.argsort(-v, kind="stable")[:topk_group]] = True
            c = np.where(np.repeat(keep, E // n_group), c, -np.inf)
        order = np.argsort(-c, kind="stable")[:K]
        order = order[c[order] > -np.inf]
        w = s[order]
        if renormalize and len(order):
            if scoring == "softmax":
                w = np.exp(row[order] - row[order].max())
                w = w / w.sum()
            else:
                w = w / (w.sum() + 1e-20)
        ids[t, :len(order)] = order
        out[t, :len(order)] = w * scale
    return ids, out


def route_scores(l, ids, scoring, renormalize, scale):
    """Scores of given ids (all valid), differentiable numerically."""
    l = np.asarray(l, np.float64)
    if scoring == "sigmoid":
        s = 1 / (1 + np.exp(-l))
        w = np.take_along_axis(s, ids, 1)
        if renormalize:
            w = w / (w.sum(1, keepdims=True) + 1e-20)
    else:
        x = np.take_along_axis(l, ids, 1) if renormalize else l
        e = np.exp(x - x.max(1, keepdims=True))
        w = e / e.sum(1, keepdims=True)
        if not renormalize:
            w = np.take_along_axis(w, ids, 1)
    return w * scale


def route_grad(l, ids, d, scoring, renormalize, scale):
    l = np.asarray(l, np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        row = l[t]
        ok = np.array([0 <= i < l.shape[1] and row[i] > -np.inf for i in ids[t]])
        j, g = ids[t][ok], scale * np.asarray(d[t], np.float64)[ok]
        if scoring == "sigmoid":
            x = np.exp(-np.abs(row[j]))
            s = np.where(row[j] >= 0, 1, x) / (1 + x)
            if renormalize:
                D = s.sum() + 1e-20
                g = (g - (g * (s / D)).sum()) / D
            np.add.at(out[t], j, g * x / (1 + x) ** 2)
        elif renormalize:
            if len(j):
                e = np.exp(row[j] - row[j].max())
                w = e / e.sum()
                np.add.at(out[t], j, w * (g - (g * w).sum()))
        else:
            live = row > -np.inf
            e = np.where(live, np.exp(row - (row.max() if live.any() else 0)), 0)
            s = e / max(e.sum(), 1e-300)
            out[t] = -s * (g * s[j]).sum()
            np.add.at(out[t], j, s[j] * g)
    return out


# ------------------------------------------------------------ 4-bit weights

def decode(codes, scales, zeros, group, kind):
    """[E,N,K] float64 values."""
    K = codes.shape[2]
    s = np.repeat(np.asarray(scales, np.float64), group, 2)[:, :, :K]
    if kind == "fp4":
        return FP4[codes] * s
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 2)[:, :, :K]
    return (codes.astype(np.float64) - z) * s


def product_slack(mag, K):
    """Bound of an fp32 sum of K products of total magnitude `mag`."""
    return mag * ((K / 32 + 4) * 16 + 16) * U32


def matvec(x, w, ids, first, mask, out, per_route=False):
    """x [T,K] or [T,R,K]; returns (y float64, touched)."""
    T, R = ids.shape
    y, hit = np.array(out, np.float64), np.zeros((T, R), bool)
    for t in range(T):
        for r in range(R):
            e = int(ids[t, r]) - first
            if 0 <= e < w.shape[0] and (mask is None or mask[t, r]):
                y[t, r] = w[e] @ (x[t, r] if per_route else x[t]).astype(np.float64)
                hit[t, r] = True
    return y, hit


def layer(x, ids, scores, w13, w2, first, mask, mag13=None, mag2=None):
    """(out, bound) in float64. mag13 / mag2: magnitudes of the weights as
    they are multiplied (|w|, or larger where an offset is taken out)."""
    x = x.astype(np.float64)
    T, K = ids.shape
    E, H, I = w2.shape
    mag13 = np.abs(w13) if mag13 is None else mag13
    mag2 = np.abs(w2) if mag2 is None else mag2
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        terms = 0
        for k in range(K):
            e = int(ids[t, k]) - first
            if not 0 <= e < E or (mask is not None and not mask[t, k]):
                continue
            terms += 1
            gu = w13[e] @ x[t]
            dgu = product_slack(mag13[e] @ np.abs(x[t]), H)
            g, u, dg, du = gu[:I], gu[I:], dgu[:I], dgu[I:]
            with np.errstate(over="ignore"):
                sl = g / (1 + np.exp(-g))
            h = sl * u
            # |silu'| < 1.1; silu itself to 8 u32, its product to 1, two
            # bf16 halves to 2^-16
            dh = (1.1 * dg + 8 * U32 * np.abs(sl)) * (np.abs(u) + du) + np.abs(sl) * du
            dh = dh + np.abs(h) * 2.0 ** -16
            s = abs(float(scores[t, k]))
            out[t] += float(scores[t, k]) * (w2[e] @ h)
            bound[t] += s * (mag2[e] @ dh + product_slack(mag2[e] @ (np.abs(h) + dh), I))
            bound[t] += s * 4 * U32 * np.abs(w2[e] @ h)
        bound[t] += 16 * max(terms, 1) * U32 * bound[t] + terms * U32 * np.abs(out[t])
    return out, bound
