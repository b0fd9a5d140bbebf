"""Plain 64-bit implementations of the serving operators over packed records, and how far fp32 and
16-bit arithmetic may be from them.

Caches are made of random code and sign words (every record layout is a valid one) with random
norms, some of them zero, so that no test depends on a compression step.
"""
from __future__ import annotations

import math

import numpy as np

import oracle
from kv_cache_vector_compress_b200 import synth

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Cache:
    """n random records on the host (numpy), and their dequantized parts in 64 bits."""

    def __init__(self, n, d, m, bits, seed, zero=0.02):
        rng = np.random.default_rng(seed)
        word = lambda k: rng.integers(0, 1 << 32, size=(n, k), dtype=np.uint64).astype(np.uint32)  # noqa: E731
        self.kc, self.ks, self.vc = word((bits - 1) * d // 32), word(m // 32), word(bits * d // 32)
        self.kn = (np.sqrt(d) * rng.uniform(0.7, 1.4, n)).astype(np.float16)
        self.kr = rng.uniform(0.1, 0.4, n).astype(np.float16)
        self.vn = (np.sqrt(d) * np.exp(rng.uniform(-2, 2, n))).astype(np.float16)
        self.kn[rng.random(n) < zero] = 0
        self.vn[rng.random(n) < zero] = 0
        self.n, self.d, self.m, self.bits = n, d, m, bits

    @staticmethod
    def bits_of(words):
        return (words[..., None] >> np.arange(32, dtype=np.uint32)) & 1

    def dequantized(self):
        """(centroids of the keys [n, d], signs [n, m], centroids of the values times the norms [n, d])."""
        kcen = oracle.codebook_f32(self.d, self.bits - 1)[1].astype(np.float64)
        vcen = oracle.codebook_f32(self.d, self.bits)[1].astype(np.float64)

        def idx(w, beta):
            b = self.bits_of(w.reshape(self.n, -1, beta))
            return sum(b[:, :, p].astype(np.int64) << p for p in range(beta)).reshape(self.n, self.d)

        sign = 2.0 * self.bits_of(self.ks).reshape(self.n, self.m) - 1.0
        v = vcen[idx(self.vc, self.bits)] * self.vn.astype(np.float64)[:, None]
        return kcen[idx(self.kc, self.bits - 1)], sign, v

    def device(self, dev="cuda"):
        """(keys, values) tuples of tensors as the binding takes them."""
        import torch
        t = lambda a, ty: torch.from_numpy(np.ascontiguousarray(a).view(ty)).to(dev)  # noqa: E731
        return ((t(self.kc, np.int32), t(self.ks, np.int32), t(self.kn, np.float16), t(self.kr, np.float16)),
                (t(self.vc, np.int32), t(self.vn, np.float16)))


def matrices(d, m, seed):
    return synth.rotation(d, seed), synth.gaussian(m, d, seed + 1)


def attend(q, R, S, caches, Hkv, scale, operand=0.0):
    """The reference of one call.  q: [B, Hq, Nq, d] in 64 bits.  caches: a list of (Cache, stride,
    shared, lens): records [Hkv, stride] if shared, else [B, Hkv, stride], of which lens[b] (or
    stride) are attended.  Returns (out, the largest error allowed per element before its last
    rounding, softmax weights [B, Hkv, stride] of the last cache, allowed error of the weights).

    `operand` is the relative rounding of a 16-bit operand of a product (0: 32 bits).  Scores: a
    product of n = d + m terms in fp32 is off by at most (n + 8) 2^-24 sum |terms| (each of its
    operations rounds by half a step; 8 for the rotation's own roundings, the norms and the scale),
    and the rotation of the query by d 2^-24 |q| |R| in each coordinate; a rounded operand adds
    2 operand sum |terms|.  A logit that is off by e multiplies its weight by at most exp(e) and
    the normaliser by as much: 2 e relative, to first order.  Sums over T tokens: the weights are
    added with at most (T + 16) 2^-24 relative error, and value products with rounded operands
    (weight and centroid) add 2 operand.  The final rotation: d 2^-24 sum |R| |o|.
    """
    B, Hq, Nq, d = q.shape
    m, G = S.shape[0], Hq // Hkv
    R, S = R.astype(np.float64), S.astype(np.float64)
    out, tol = np.zeros((B, Hq, Nq, d)), np.zeros((B, Hq, Nq, d))
    last, stride = caches[-1][0], caches[-1][1]
    weights, wtol = np.zeros((B, Hkv, stride)), np.zeros((B, Hkv, stride))
    parts = [c[0].dequantized() for c in caches]
    gam = math.sqrt(math.pi / 2) / m
    u = 2.0 ** -24
    for b in range(B):
        for h in range(Hkv):
            K, E, V, T = [], [], [], 0
            x = q[b, h * G:(h + 1) * G].reshape(G * Nq, d)
            qr, qs = x @ R.T, x @ S.T
            # what the fp32 rotation of the query may be off by, in each coordinate
            er, es = d * u * (np.abs(x) @ np.abs(R.T)), d * u * (np.abs(x) @ np.abs(S.T))
            for (c, st, shared, lens), (kc, sg, v) in zip(caches, parts):
                n = st if lens is None else int(lens[b])
                r0 = (h if shared else b * Hkv + h) * st
                sl = slice(r0, r0 + n)
                kn, rho = c.kn[sl].astype(np.float64), c.kr[sl].astype(np.float64) * gam
                s = kn * (qr @ kc[sl].T + rho * (qs @ sg[sl].T))
                mag = kn * (np.abs(qr) @ np.abs(kc[sl]).T + rho * np.abs(qs).sum(1, keepdims=True))
                e = mag * ((d + m + 8) * u + 2 * operand)
                e += kn * (er @ np.abs(kc[sl]).T + rho * es.sum(1, keepdims=True))
                K.append(s * scale)
                E.append(e * scale)
                V.append(v[sl])
            z, e, v = np.concatenate(K, 1), np.concatenate(E, 1), np.concatenate(V, 0)
            T = z.shape[1]
            if T == 0:
                continue
            w = np.exp(z - z.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            rel = 2 * e.max(1, keepdims=True) + (T + 16) * u
            rel = np.expm1(np.minimum(rel, 50.0)) + 4 * u * np.abs(z).max(1, keepdims=True)  # a logit itself is rounded to fp32
            o = w @ v
            # 16-bit weights and values.  A weight is held relative to at least 2^-8 of the largest, a
            # value to its tile's largest, and fp16's numbers are 2^-24 apart at the low end.
            eo = (w @ np.abs(v)) * (rel + 2 * operand)
            if operand:
                eo += T * u * w.max(1, keepdims=True) * np.abs(v).max()
            out[b, h * G:(h + 1) * G] = (o @ R).reshape(G, Nq, d)
            tol[b, h * G:(h + 1) * G] = ((eo + d * u * np.abs(o)) @ np.abs(R)).reshape(G, Nq, d)
            n = z.shape[1] - sum(k.shape[1] for k in K[:-1])
            weights[b, h, :n] = w[:, T - n:].sum(0)
            wtol[b, h, :n] = (w * rel)[:, T - n:].sum(0)
    return out, tol, weights, wtol


def evict(weights, lens, budget, recent):
    """Kept slots of every slice: a list [B][Hkv] of ascending index arrays."""
    B, Hkv, _ = weights.shape
    kept = []
    for b in range(B):
        n, row = int(lens[b]), []
        for h in range(Hkv):
            w = weights[b, h, :n].astype(np.float64)
            w = np.where(np.isnan(w), np.inf, w)
            tier = np.where(np.isnan(weights[b, h, :n]), 1, 0)
            tier[max(0, n - recent):] = 2
            order = np.lexsort((np.arange(n), -w, -tier))
            row.append(np.sort(order[:budget]))
        kept.append(row)
    return kept
