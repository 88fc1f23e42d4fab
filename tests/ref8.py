"""Plain 64-bit implementations of the 8-bit expert operators (numpy, loops over experts and groups), for the tests.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinity, NaN 0x7f / 0xff.  E8M0: byte e is 2^(e - 127)."""
import numpy as np


def _table():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if (b & 127) == 127 else (-x if b & 128 else x)
    return v


E4M3 = _table()
_POS = E4M3[:127]  # 0 .. 448, ascending


def round_e4m3(x):
    """Bytes of the nearest e4m3 values of |x| <= 448, ties to the even code; what is not finite is NaN (0x7f)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.minimum(np.searchsorted(_POS, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def scale_exponent(a):
    """Least e >= -127 with a <= 448 * 2^e (0 for a == 0)."""
    if a == 0:
        return 0
    e = -127
    while a > 448 * 2.0 ** e:
        e += 1
    return e


def quant8(x, block_rows=1):
    """(q bytes, s bytes) of x [rows][cols]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    q = np.empty((rows, cols), np.uint8)
    s = np.empty((-(-rows // block_rows), -(-cols // 128)), np.uint8)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            b = x[at]
            f = np.abs(b[np.isfinite(b)])
            e = scale_exponent(f.max() if f.size else 0.0)
            s[i, j] = e + 127
            with np.errstate(invalid="ignore"):
                q[at] = round_e4m3(b * 2.0 ** -e)
    return q, s


def dequant8(q, s, block_rows=1):
    f = np.exp2(s.astype(np.float64) - 127)
    f = np.repeat(np.repeat(f, block_rows, axis=0)[: q.shape[0]], 128, axis=1)[:, : q.shape[1]]
    return E4M3[q] * f


def mm8(a, sa, b, sb):
    """(product, sum of the terms' magnitudes) in 64 bits."""
    x, w = dequant8(a, sa, 1), dequant8(b, sb, 128)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def gate(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0):
    t, e = logits.shape
    idx = np.full((t, k), -1, np.int64)
    w = np.zeros((t, k))
    for r in range(t):
        x = logits[r].astype(np.float64)
        b = np.zeros(e) if bias is None else bias.astype(np.float64)
        live = ~np.isnan(x) & (x > -np.inf) & ~np.isnan(b) & (b > -np.inf)
        seen = ~np.isnan(x) & (x > -np.inf)  # the softmax runs over every expert with a logit
        p = np.zeros(e)
        if score == "sigmoid":
            p[seen] = [1 / (1 + np.exp(-v)) if v > -700 else np.exp(v) for v in x[seen]]
        elif seen.any():
            m = x[seen].max()
            z = np.where(x[seen] == m, 1.0, 0.0) if np.isinf(m) else np.exp(x[seen] - m)
            p[seen] = z / z.sum()
        sel = p + b
        order = sel if bias is not None else x
        allowed = live.copy()
        if groups > 1 and top_groups < groups:
            gs, best = e // groups, []
            by = order if group_top == 1 else sel  # one expert's score orders as its logit does
            for g in range(groups):
                v = sorted(by[g * gs:(g + 1) * gs][live[g * gs:(g + 1) * gs]], reverse=True)[:group_top]
                best.append((-sum(v), g) if v else (np.inf, g))
            keep = {g for _, g in sorted(best)[:top_groups]}
            allowed &= np.array([i // gs in keep for i in range(e)])
        ids = sorted(np.nonzero(allowed)[0], key=lambda i: (-order[i], i))[:k]
        idx[r, : len(ids)] = ids
        if len(ids):
            if renorm and score == "sigmoid":
                top = x[ids].max()
                q = np.exp(x[ids] - top) if top < -60 else p[ids]
                w[r, : len(ids)] = q / q.sum()
            elif renorm:
                top = x[ids].max()
                q = np.where(x[ids] == top, 1.0, 0.0) if np.isinf(top) else np.exp(x[ids] - top)
                w[r, : len(ids)] = q / q.sum()
            else:
                w[r, : len(ids)] = p[ids]
    return idx, w * scale


def experts8(x, gu, gus, dn, dns, idx, w, out_step, whole=False):
    """(out, allowance) in 64 bits.  The allowance bounds what 32-bit sums, the roundings of the outputs
    (relative out_step, once per entry and once at the end) and e4m3 roundings of h that those sums can push
    over a border may change.  whole: the partial sums of the first product are exact in 32 bits."""
    t, hid = x.shape
    e, i = gu.shape[0], gu.shape[1] // 2
    out, allow = np.zeros((t, hid)), np.zeros((t, hid))
    q, s = quant8(x)
    for r in range(t):
        for j, ex in enumerate(idx[r]):
            if not 0 <= ex < e:
                continue
            v, mag = mm8(q[r:r + 1], s[r:r + 1], gu[ex], gus[ex])
            g, u = v[0, :i], v[0, i:]
            d = mag[0] * (0 if whole else hid) * 2.0 ** -23  # each step of a 32-wide product may truncate 33 terms at 2^-23 of their sum
            h = g / (1 + np.exp(-g)) * u
            # |silu'| <= 1.1, |silu(g)| <= |g|; the division, exponential and product: 2^-20 of h
            dh = 1.1 * d[:i] * np.abs(u) + np.abs(g) * d[i:] + 1.1 * d[:i] * d[i:] + np.abs(h) * 2.0 ** -20
            hq, hs = quant8(h[None])
            lo, los = quant8(h[None] - dh)
            hi, his = quant8(h[None] + dh)
            hv = dequant8(hq, hs)[0]
            # rounding is monotone: under one scale the kernel's value is between those of h - dh and h + dh
            a, b = E4M3[round_e4m3((h - dh) / np.repeat(np.exp2(hs[0] - 127.0), 128))], \
                E4M3[round_e4m3((h + dh) / np.repeat(np.exp2(hs[0] - 127.0), 128))]
            f = np.repeat(np.exp2(hs[0] - 127.0), 128)
            flip = np.maximum(np.abs(a * f - hv), np.abs(b * f - hv))
            # a block whose largest value is within reach of the next scale: a whole step of either scale
            amax = np.abs(h).reshape(-1, 128).max(1)
            am = np.abs(h).reshape(-1, 128).argmax(1) + 128 * np.arange(i // 128)
            for kb in range(i // 128):
                if scale_exponent(amax[kb] + dh[am[kb]]) != scale_exponent(max(amax[kb] - dh[am[kb]], 0)):
                    sl = slice(kb * 128, kb * 128 + 128)
                    flip[sl] = np.abs(h[sl]) / 8 + f[sl.start] * 2.0 ** -8
            y, ymag = mm8(hq, hs, dn[ex], dns[ex])
            wd = np.abs(dequant8(dn[ex], dns[ex], 128))
            dy = wd @ flip + ymag[0] * i * 2.0 ** -23 + np.abs(y[0]) * out_step
            out[r] += w[r, j] * y[0]
            allow[r] += np.abs(w[r, j]) * dy + np.abs(w[r, j] * y[0]) * 34 * 2.0 ** -24
    return out, allow + np.abs(out) * out_step + allow * out_step
