"""Plain 64-bit implementations of the operators around the experts' step (numpy), with bounds of what 32-bit sums and
the outputs' roundings may change, for the tests."""
import math

import numpy as np

import ref8

U = 2.0 ** -24  # half a step of 32-bit numbers, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133}  # a step below the normal numbers
# a 32-bit sum of squares over a row: up to 64 terms a thread one after another, 5 + 4 exchanges, the mean, the root and
# the quotient; the root halves the sums' part.  In units of U.
NORM = 64 / 2 + 9 + 4


def sigmoid(x):
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1, e) / (1 + e)


def norm(x, w=None, eps=1e-6):
    with np.errstate(all="ignore"):
        y = x / np.sqrt((x * x).mean(1, keepdims=True) + np.float64(np.float32(eps)))
        return y if w is None else y * w


def add_norm(y, res, post=False, w_post=None, gate=None, sig=False, scale=1.0, res_scale=1.0, w=None, eps=1e-6):
    """(sum, its bound, norm, its bound) before the outputs' roundings."""
    scale, res_scale = np.float64(np.float32(scale)), np.float64(np.float32(res_scale))
    v = norm(y, w_post, eps) if post else y
    if gate is not None:
        v = v * (sigmoid(gate) if sig else gate)
    s = res_scale * res + scale * v
    # norm, weight, sigmoid (exponential 2 steps, sum, quotient), gate, two products and the sum
    ds = (np.abs(scale * v) * ((NORM + 2 if post else 0) + 10) + np.abs(res_scale * res) * 2 + np.abs(s)) * U
    out = norm(s, w, eps)
    inv = norm(np.ones_like(s), None, eps)
    rms = np.sqrt((s * s).mean(1, keepdims=True) + eps)
    drms = np.sqrt((ds * ds).mean(1, keepdims=True)) / rms  # relative change of the root by the sums' errors
    dout = ds / rms * (1 if w is None else np.abs(w)) + np.abs(out) * (drms + (NORM + 2) * U)
    del inv
    return s, ds, out, dout


def check(got, ref, bound, kind, what=""):
    """got (64-bit copies of a tensor of type `kind`) within `bound` and half a step of ref; what is not finite alike."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    top = 3.4028235677973366e38 if kind == "f32" else 3.3961775292304601e38  # from here on a value rounds to infinity
    ref = np.where(np.abs(ref) >= top, np.sign(ref) * np.inf, ref)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), what
    with np.errstate(invalid="ignore"):
        room = np.broadcast_to(bound, ref.shape) * (1 + HALF[kind]) + np.abs(ref) * HALF[kind] + TINY[kind]
        bad = fine & ~(np.abs(got - ref) <= room)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], np.broadcast_to(room, ref.shape)[bad][:4])


def check_e4m3(q, s, ref, bound, what=""):
    """q, s (bytes) as quant8 gives them for some values within `bound` of ref."""
    t, h = ref.shape
    for b in range(s.shape[1]):
        at = slice(128 * b, min(h, 128 * b + 128))
        y, d = ref[:, at], np.broadcast_to(bound, ref.shape)[:, at]
        fine = np.isfinite(y)
        a = np.where(fine, np.abs(y), 0)
        lo, hi = np.where(fine, np.maximum(a - d, 0), 0).max(1), np.where(fine, a + d, 0).max(1)
        hi = np.where(a.max(1) == 0, 0, hi)  # zeros are exact
        for r in range(t):
            e = int(s[r, b]) - 127
            ok = {ref8.scale_exponent(lo[r]), ref8.scale_exponent(hi[r])}
            assert e in ok, (what, r, b, e, ok)
            f = 2.0 ** -e
            with np.errstate(invalid="ignore"):
                c0, c1 = (ref8.E4M3[ref8.round_e4m3(np.clip(v * f, -448, 448))] for v in (y[r] - d[r], y[r] + d[r]))
            g = ref8.E4M3[q[r, at]]
            ok = np.where(fine[r], (g >= c0) & (g <= c1), np.isnan(g))
            assert ok.all(), (what, r, b, np.argwhere(~ok)[:3].tolist())


def act(name, z):
    if name == "silu":
        return z * sigmoid(z)
    if name == "gelu":
        return z * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "relu":
        return np.where(z > 0, z, 0.0) + np.where(np.isnan(z), z, 0.0)
    return sigmoid(z) if name == "sigmoid" else z


def logprobs(x, tokens, k, scale=1.0):
    """(logp, entropy, top ids, their logp, bound of log Z's error) of rows x in 64 bits."""
    scale = np.float64(np.float32(scale))
    t, v = x.shape
    with np.errstate(all="ignore"):
        live = x > -np.inf  # false for NaN
        top = np.where(live.any(1), np.where(live, x, -np.inf).max(1), 0.0)[:, None]
        d = np.where(live, np.where(x == top, 0.0, scale * (x - top)), -np.inf)
        e = np.exp(d)
        z = e.sum(1, keepdims=True)
        lp = d - np.log(z)
        lp[~live] = -np.inf
        p = e / z
        ent = np.where(live.any(1), -np.where(p > 0, p * lp, 0.0).sum(1), 0.0)
        spread = np.where(live.any(1), np.where(p > 0, p * np.abs(d), 0.0).sum(1), 0.0)
    # terms: the exponent's rounding (its size, weighted), the exponential (2^-22), a thread's own sum, the tree
    dz = (max(64, v // 128) + 40 + 8 * spread / math.log(2)) * U
    inside = (tokens >= 0) & (tokens < v)
    given = np.where(inside, np.take_along_axis(lp, np.where(inside, tokens, 0), 1), -np.inf)
    order = np.argsort(np.where(live, -x, np.inf), axis=1, kind="stable")[:, :k]
    none = ~np.take_along_axis(live, order, 1)
    return given, ent, np.where(none, -1, order), np.where(none, -np.inf, np.take_along_axis(lp, order, 1)), dz[:, None]


def act_bound(name, x, h):
    """What 32 bits may change in h = act(x): exponentials and quotients of two steps each, and their arguments' roundings."""
    own = {"none": 0, "relu": 0, "silu": 16, "sigmoid": 16, "gelu": 32 + 4 * x * x,
           "gelu_tanh": 32 + 8 * (1.6 * np.abs(x) + 0.072 * np.abs(x) ** 3)}[name]
    return np.abs(h) * own * U


def mm16(a, b, gated=False, a_act="none", bias=None, row_scale=None, res=None):
    """(out, bound before the output's rounding) in 64 bits.  Sums: every term of a 16-wide step may lose what lies below
    2^-23 of the sum, in all k 2^-23 of the terms' magnitudes; the activations: exponentials and quotients of two steps
    each, and what their arguments' roundings do."""
    k = a.shape[1]
    z, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    dz = (k + 2) * 2.0 ** -23 * mag
    n = b.shape[0] // 2 if gated else b.shape[0]
    x, dx = z[:, :n], dz[:, :n]
    h = act(a_act, x)
    dh = dx * 1.2 + act_bound(a_act, x, h)
    if gated:
        u, du = z[:, n:], dz[:, n:]
        h, dh = h * u, dh * np.abs(u) + np.abs(h) * du + dh * du + np.abs(h * u) * U
    if row_scale is not None:
        h, dh = h * row_scale[:, None], dh * np.abs(row_scale[:, None]) + np.abs(h * row_scale[:, None]) * U
    if res is not None:
        h = h + res
        dh = dh + np.abs(h) * U
    return h, dh
