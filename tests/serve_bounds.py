"""How far the serving calls are from their definition when every rounding goes its own way: bounds of the
size of the real error, beside the worst cases of serve_ref.

Model.  A result is out = sum_t w_t v_t, w = softmax(z).  Independent errors with standard deviations
sz_t of the logits, sw of the weights and sv of the values' coordinates (both relative) give it a random error
whose squared norm over the coordinates is, on average,
    E^2 = sum_t w_t^2 (|v_t - out|^2 sz_t^2 + |v_t|^2 (sw^2 + sv^2)),
and a token's weight one of w_t (sz_t + its mean).  The final rotation keeps norms.  A rounding to fp16 is at
most 2^-11 of the value and spread evenly: 2^-11 / sqrt(3) at most in the root mean square.  A rounding of each
coordinate of one factor of a dot product is sqrt(sum of squared terms) times that.
"""
from __future__ import annotations

import math

import numpy as np

U16 = 2.0 ** -11 / math.sqrt(3)
U32 = 2.0 ** -24

# Errors of one kernel's operands: query and key coordinates, the sign part as a whole, weights, value
# coordinates; `sum`: of the 32-bit sums and functions, relative to the terms' root of squares.
#  many: the many-row kernel on a prefix.  Query rows and ||v|| c rounded to fp16
#  ragged: two fp16 halves of a query; fp16 values and weights
#  f32: fp16 pairs or fp32 throughout, 2^-20 and better
# and the fp16 tables of the centroids (keys: 2^-19 up to 2 bits, 5e-5 at 3).
FORMS = {
    "many": dict(query=U16, key=lambda bits: table(bits), sign=0.0, weight=U16,
                 value=lambda bits: math.hypot(U16, value_table(bits)), sum=2.0 ** -20),
    "ragged": dict(query=2.0 ** -22, key=lambda bits: table(bits), sign=0.0, weight=U16,
                   value=lambda bits: value_table(bits), sum=2.0 ** -20),
    "f32": dict(query=2.0 ** -22, key=lambda bits: 2.0 ** -20 if bits != 3 else 2.0 ** -19, sign=0.0,
                weight=2.0 ** -20, value=lambda bits: 2.0 ** -20, sum=2.0 ** -20),
}
SIGMAS = 6.0  # of a normal error: 2e-9 to be beyond, at some 10^6 rows and weights in all


def table(bits):
    """Largest relative error of a key centroid of a `bits`-bit parameter set (the keys' codes have one less)."""
    return {2: 2.0 ** -23, 3: 2.0 ** -19, 4: 5e-5}[bits]


def value_table(bits):
    """Largest relative error of fp16 value centroids of a `bits`-bit parameter set."""
    return {2: 2.0 ** -19, 3: 5e-5, 4: 2.0 ** -11}[bits]


def forms(dtype, d, m, B, Hkv, rows, t_prefix, t_cap):
    """The forms of the prefix's and the own caches' products (the library's choice by sizes)."""
    if d not in (64, 128, 256) or m != d // 2 or dtype == "f32":
        return "f32", "f32"
    many = B * rows > 8 and (t_cap == 0 or B * Hkv * rows * t_prefix >= 40000000 // d)
    return "many" if many else "ragged", "ragged"


def attend(q, R, S, caches, Hkv, scale, bits):
    """As serve_ref.attend, without its bounds, for caches (Cache, stride, shared, lens, form).  Returns (out,
    E per row [B, Hq, Nq], weights of the last cache, their error)."""
    B, Hq, Nq, d = q.shape
    m, G = S.shape[0], Hq // Hkv
    R, S = R.astype(np.float64), S.astype(np.float64)
    out, err = np.zeros((B, Hq, Nq, d)), np.zeros((B, Hq, Nq))
    stride = caches[-1][1]
    weights, werr = np.zeros((B, Hkv, stride)), np.zeros((B, Hkv, stride))
    parts = [c[0].dequantized() for c in caches]
    gam = math.sqrt(math.pi / 2) / m
    rot = math.sqrt(d) * U32  # a rotated coordinate, relative to |q|
    for b in range(B):
        for h in range(Hkv):
            x = q[b, h * G:(h + 1) * G].reshape(G * Nq, d)
            qr, qs = x @ R.T, x @ S.T
            norm2 = (x ** 2).sum(1, keepdims=True)
            K, Z, V, EW, n = [], [], [], [], 0
            for (c, st, shared, lens, form), (kc, sg, v) in zip(caches, parts):
                f = FORMS[form]
                n = st if lens is None else int(lens[b])
                r0 = (h if shared else b * Hkv + h) * st
                kc, sg, v = kc[r0:r0 + n], sg[r0:r0 + n], v[r0:r0 + n]
                kn = c.kn[r0:r0 + n].astype(np.float64)
                rho = c.kr[r0:r0 + n].astype(np.float64) * gam
                sign = rho * (qs @ sg.T)
                K.append(kn * (qr @ kc.T + sign) * scale)
                code2 = qr ** 2 @ (kc ** 2).T
                sign2 = rho ** 2 * (qs ** 2).sum(1, keepdims=True)
                # the rotation's own rounding: rot |q| in a coordinate of R q, rot |q| |S row| of S q
                turn = rot ** 2 * norm2 * ((kc ** 2).sum(1) + rho ** 2 * d * m)
                var = (code2 * (f["query"] ** 2 + f["key"](bits) ** 2 + f["sum"] ** 2) +
                       sign2 * (f["query"] ** 2 + f["sum"] ** 2) + (f["sign"] * sign) ** 2 + turn)
                # a logit and the exponent it goes into are rounded to fp32 (base 2, with the value's norm)
                Z.append(var * (kn * scale) ** 2 + (4 * U32 * (np.abs(K[-1]) + 16)) ** 2)
                V.append(v)
                EW.append(np.full(n, f["weight"] ** 2 + f["value"](bits) ** 2 + f["sum"] ** 2))
            z, sz2, v, ew = np.concatenate(K, 1), np.concatenate(Z, 1), np.concatenate(V), np.concatenate(EW)
            T = z.shape[1]
            if T == 0:
                continue
            w = np.exp(z - z.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            o = w @ v
            v2 = (v ** 2).sum(1)
            away = np.maximum(v2 - 2 * o @ v.T + (o ** 2).sum(1, keepdims=True), 0.0)
            e2 = (w ** 2 * (away * sz2 + v2 * ew)).sum(1) + (rot ** 2) * (o ** 2).sum(1)
            out[b, h * G:(h + 1) * G] = (o @ R).reshape(G, Nq, d)
            err[b, h * G:(h + 1) * G] = np.sqrt(e2).reshape(G, Nq)
            mean = np.sqrt((w ** 2 * sz2).sum(1, keepdims=True))
            weights[b, h, :n] = w[:, T - n:].sum(0)
            werr[b, h, :n] = (w * (np.sqrt(sz2) + mean + 2.0 ** -21))[:, T - n:].sum(0)
    return out, err, weights, werr


def out_of_bounds(got, want, err, half_step):
    """Rows whose error is beyond SIGMAS of its model, after the output's own rounding."""
    g = np.asarray(got, np.float64).reshape(want.shape)
    off = np.linalg.norm(g - want, axis=-1)
    d = want.shape[-1]
    lim = SIGMAS * err * (1 + half_step) + half_step * np.linalg.norm(want, axis=-1) + 1e-37
    if half_step == 2.0 ** -11:
        lim = lim + math.sqrt(d) * 2.0 ** -25  # fp16's smallest numbers
    return ~(off <= lim)


def typical(got, want, err, half_step):
    """Whether the error's root mean square over all rows is that of the model and the output's rounding: of
    the errors' own size, where out_of_bounds leaves six times that for the worst row."""
    g = np.asarray(got, np.float64).reshape(want.shape)
    size = (want ** 2).sum(-1).mean()
    return ((g - want) ** 2).sum(-1).mean() <= (err ** 2).mean() + half_step ** 2 / 3 * size


def weights_out_of_bounds(got, want, werr, before):
    """Weights beyond SIGMAS of their model; `before`: what the call added to."""
    g = np.asarray(got, np.float64)
    return ~(np.abs(g - (before + want)) <= SIGMAS * werr + 2.0 ** -23 * np.abs(before + want) + 1e-37)
