"""Plain fp64 forms of the linear attention and query/key norms, and the bounds that their tests use.

Each linear-attention walk also gives `bound`: the sum of the absolute values of everything that is added up in
an output.  A rounding of relative size u anywhere in such a sum moves the output by at most u * bound, so a
kernel with c roundings between inputs and output is off by at most c * u * bound.
"""
import numpy as np

U32 = 2.0 ** -24       # half a step, relative
UBF = 2.0 ** -8


def walk(query, key, value, g, S, back):
    """Token by token for one sequence: query, key, value [T, H, d] fp64, g [H], S [H, d, d].  Returns (out, S)."""
    a = np.exp(np.asarray(g, dtype=np.float64))[:, None, None]
    S = S.copy()
    out = np.zeros_like(value)
    T = query.shape[0]
    for t in (range(T - 1, -1, -1) if back else range(T)):
        if not back:
            S = a * S
        S = S + value[t][:, :, None] * key[t][:, None, :]
        out[t] = np.einsum("hij,hj->hi", S, query[t])
        if back:
            S = a * S
    return out, S


def sequences(cu, total):
    return [(int(b), int(e)) for b, e in zip(cu[:-1], cu[1:])]


def both(query, key, value, g, S, back, cu):
    """walk() for every sequence, and for the absolute values: (out, S_end, out_bound, S_bound)."""
    out, bound = np.zeros_like(value), np.zeros_like(value)
    end, send = np.zeros_like(S), np.zeros_like(S)
    for n, (b, e) in enumerate(sequences(cu, query.shape[0])):
        out[b:e], end[n] = walk(query[b:e], key[b:e], value[b:e], g, S[n], back)
        bound[b:e], send[n] = walk(np.abs(query[b:e]), np.abs(key[b:e]), np.abs(value[b:e]), g, np.abs(S[n]), back)
    return out, end, bound, send


def forward(q, k, v, g, S0, cu):
    return both(q, k, v, g, S0, False, cu)


def backward(q, k, v, g, S0, do, dST, cu):
    """dq, dk, dv, dS0 as (value, bound) pairs."""
    t = lambda x: np.swapaxes(x, -1, -2)  # noqa: E731
    dq, _, dqb, _ = both(do, v, k, g, t(S0), False, cu)
    dv, dS0, dvb, dS0b = both(k, q, do, g, dST, True, cu)
    dk, _, dkb, _ = both(v, do, q, g, t(dST), True, cu)
    return (dq, dqb), (dk, dkb), (dv, dvb), (dS0, dS0b)


def roundings32(longest, d):
    """fp32 roundings between inputs and an output, at most: the decay (its exp and up to `longest` products of it, or
    one exp of a rounded exponent, which counts as many), one addition for each token, one for each channel."""
    return 4 * longest + d + 16


def turn(x, pos, inv_freq, rot, interleaved):
    """R(pos) x: x [T, H, d] fp64, pos [T], inv_freq [rot / 2] (as the fp32 numbers that they are)."""
    y = x.copy()
    if rot == 0:
        return y
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rotate(x, w, pos, inv_freq, rot, interleaved, kind, eps, scale):
    n = x.shape[-1] if kind == "rms" else 1
    r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    y = x * r
    if w is not None:
        y = y * np.asarray(w, dtype=np.float64)
    return scale * turn(y, pos, inv_freq, rot, interleaved)


def norm_rotate_backward(x, w, pos, inv_freq, rot, interleaved, kind, eps, scale, dy):
    """dx, dw and dw's bound (the sum of the absolute terms)."""
    n = x.shape[-1] if kind == "rms" else 1
    r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    xh = x * r
    u = scale * turn(dy, -np.asarray(pos) if pos is not None else None, inv_freq, rot, interleaved)
    h = u if w is None else u * np.asarray(w, dtype=np.float64)
    dx = r * (h - xh * ((xh * h).sum(-1, keepdims=True) / n))
    return dx, (u * xh).sum((0, 1)), np.abs(u * xh).sum((0, 1))
