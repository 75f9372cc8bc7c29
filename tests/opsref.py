"""Definitions in 64 bits of the router, the gradients of dispatch and combine
and the experts' products with 4-bit weights, for the tests: numpy on the CPU,
sharing nothing with the library."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(bytes_u8):
    """The values of e4m3fn bytes."""
    b = bytes_u8.astype(np.int64)
    ex, man = (b >> 3) & 15, b & 7
    mag = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    mag = np.where((b & 127) == 127, np.nan, mag)
    return np.where(b >> 7, -mag, mag)


def route(l, K, score, bias, renorm, scale):
    """(ids, weights, weight before scaling) of logits l, float64 [T, E]."""
    l = np.where(l == np.inf, np.finfo(np.float32).max, l)
    T, E = l.shape
    with np.errstate(over="ignore"):
        p = 1.0 / (1.0 + np.exp(-l))
    key = l if bias is None else p + bias[None, :]
    key = np.where(np.isnan(l) | (l == -np.inf) | np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    ok = np.take_along_axis(key, ids, 1) > -np.inf
    if score == "softmax":
        top = np.max(np.where(np.isnan(l), -np.inf, l), axis=1, keepdims=True)
        p = np.exp(l - np.where(np.isfinite(top), top, 0.0))
        total = np.nansum(p, axis=1, keepdims=True)
        p = p / np.where(total > 0, total, 1.0)
    q = np.where(ok, np.take_along_axis(p, ids, 1), 0.0)
    if renorm:
        s = q.sum(1, keepdims=True)
        q = q / np.where(s > 0, s, 1.0)
    q = np.where(ok & np.isnan(l).any(1, keepdims=True), np.nan, q)
    return np.where(ok, ids, -1).astype(np.int32), scale * q, q


def route_grad(l, ids, g, score, renorm, scale):
    """(gradient, sum of the absolute terms) for the choices ids; masked ids take no part."""
    l = np.where(l == np.inf, np.finfo(np.float32).max, l)
    T, E = l.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    g = np.where(ok, g, 0.0)
    lk = np.where(ok, np.take_along_axis(l, at, 1), -np.inf)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    with np.errstate(over="ignore"):
        pk = np.where(ok, 1.0 / (1.0 + np.exp(-lk)), 0.0)
        rk = np.where(ok, 1.0 / (1.0 + np.exp(np.where(ok, lk, 0.0))), 0.0)
    if score == "softmax":
        top = l.max(1, keepdims=True) if not renorm else lk.max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        e = np.where(lk > -np.inf, np.exp(lk - top), 0.0)
        z = (e if renorm else np.exp(l - top)).sum(1, keepdims=True)
        q = e / np.where(z > 0, z, 1.0)
        dot, mag = (g * q).sum(1, keepdims=True), (abs(g) * q).sum(1, keepdims=True)
        if not renorm:
            pe = np.exp(l - top) / np.where(z > 0, z, 1.0)
            out, size = -scale * pe * dot, abs(scale) * pe * mag
        dk = scale * q * (g - dot) if renorm else scale * q * g
        sk = abs(scale) * q * (abs(g) + (mag if renorm else 0.0))
    elif renorm:
        s = pk.sum(1, keepdims=True)
        q = pk / np.where(s > 0, s, 1.0)
        dot, mag = (g * q).sum(1, keepdims=True), (abs(g) * q).sum(1, keepdims=True)
        dk, sk = scale * q * rk * (g - dot), abs(scale) * q * rk * (abs(g) + mag)
    else:
        dk, sk = scale * g * pk * rk, abs(scale * g) * pk * rk
    for k in range(ids.shape[1]):
        t = np.nonzero(ok[:, k])[0]
        out[t, at[t, k]] += dk[t, k]
        size[t, at[t, k]] += sk[t, k]
    return out, size


def expert(x, off, codes, scales, act):
    """(result, bound of the accumulated magnitude terms) of the rows below off[E].

    x float64 [rows, C] (scales of fp8 rows applied), codes uint8 [E, N, C/2],
    scales [E, N, C/128].  Returns per row the outputs and, for the error
    bounds, (acc, sum of |terms|) of every product column."""
    rows, C = x.shape
    E, N = codes.shape[:2]
    acc, mag = np.zeros((rows, N)), np.zeros((rows, N))
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        w = np.empty((N, C))
        w[:, 0::2], w[:, 1::2] = E2M1[codes[e] & 15], E2M1[codes[e] >> 4]
        w *= np.repeat(scales[e].astype(np.float64), 128, axis=1)
        acc[a:b] = x[a:b] @ w.T
        mag[a:b] = abs(x[a:b]) @ abs(w).T
    if act == "none":
        return acc, acc, mag
    D = N // 2
    g, u = acc[:, :D], acc[:, D:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u, acc, mag
