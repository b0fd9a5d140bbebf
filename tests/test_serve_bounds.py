"""The bounds of serve_bounds on the CPU: arithmetic with the kernels' roundings stays inside them, and results
with something missing or a little wrong do not."""
import math

import numpy as np
import pytest

from . import serve_bounds as sb
from . import serve_ref as ref

MANY = [(d, bits, B) for d in (64, 128, 256) for bits in (2, 3, 4) for B in (5, 16)]
WEIGH = [(64, 2), (64, 4), (128, 2), (128, 3), (128, 4), (256, 2), (256, 3), (256, 4)]


def rounded(x, eps):
    """x to a mantissa of half step eps."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m / eps) * eps, e)


def to_type(x, dtype):
    return rounded(x, ref.HALF_STEP[dtype])


class Host:
    """The problem that the GPU tests make, without a GPU."""

    def __init__(self, dtype, d, bits, B, Hq, Hkv, t_prefix, t_cap, lens=None, seed=0):
        self.__dict__.update(dtype=dtype, d=d, m=d // 2, bits=bits, B=B, Hq=Hq, Hkv=Hkv, t_prefix=t_prefix, t_cap=t_cap)
        rng = np.random.default_rng(1000 + seed)
        self.R, self.S = ref.matrices(d, self.m, 40 + d)
        self.q = to_type(rng.standard_normal((B, Hq, 1, d)), dtype)
        self.lens = np.asarray(lens if lens is not None else rng.integers(0, t_cap + 1, B), np.int32)
        self.pre = ref.Cache(Hkv * t_prefix, d, self.m, bits, seed + 1) if t_prefix else None
        self.own = ref.Cache(B * Hkv * t_cap, d, self.m, bits, seed + 2)

        # (as if the prefix had many rows)
        self.form = sb.forms(dtype, d, self.m, B, Hkv, Hq // Hkv, t_prefix, 0 if t_prefix else t_cap)

    def attend(self, q=None, lens=None, skip=0, no_sign=False):
        """The definition; with other queries or lengths, without the prefix's last `skip` tokens or the signs."""
        fp, fo = self.form
        caches = []
        if self.pre:
            caches.append((cut(self.pre, self.Hkv, skip, no_sign), self.t_prefix - skip, True, None, fp))
        caches.append((cut(self.own, 1, 0, no_sign), self.t_cap, False, self.lens if lens is None else lens, fo))
        return sb.attend(self.q if q is None else q, self.R, self.S, caches, self.Hkv, 1 / math.sqrt(self.d), self.bits)

    def refused(self, out, want, err):
        return sb.out_of_bounds(to_type(out, self.dtype), want, err, ref.HALF_STEP[self.dtype]).any()


def cut(c, heads, skip, no_sign):
    x = ref.Cache(0, c.d, c.m, c.bits, 0)
    x.n = c.n - heads * skip
    for name in ("kc", "ks", "vc", "kn", "kr", "vn"):
        a = getattr(c, name)
        a = a.reshape(heads, -1, *a.shape[1:])
        setattr(x, name, a[:, :a.shape[1] - skip].reshape(x.n, *a.shape[2:]))
    if no_sign:
        x.kr = np.zeros_like(x.kr)
    return x


def emulated(p, norms_in_operands=False):
    """The attention with each operand rounded as the kernels round it (the sums in 64 bits).  Or with the key
    norms multiplied into the many-row kernel's operands before they are rounded."""
    form = dict(zip(("pre", "own"), p.form))
    eps = 2.0 ** -11
    R, S, G = p.R.astype(np.float64), p.S.astype(np.float64), p.Hq // p.Hkv
    gam, scale = math.sqrt(math.pi / 2) / p.m, 1 / math.sqrt(p.d)
    out = np.zeros(p.q.shape)
    for b in range(p.B):
        for h in range(p.Hkv):
            x = p.q[b, h * G:(h + 1) * G, 0]
            qr, qs = x @ R.T, gam * (x @ S.T)
            Z, V = [], []
            for name, c, r0, n in (("pre", p.pre, h * p.t_prefix, p.t_prefix),
                                   ("own", p.own, (b * p.Hkv + h) * p.t_cap, int(p.lens[b]))):
                if c is None or n == 0:
                    continue
                kc, sg, v = (t[r0:r0 + n] for t in c.dequantized())
                kn, rho = (t[r0:r0 + n].astype(np.float64) for t in (c.kn, c.kr))
                if form[name] == "many":
                    if norms_in_operands:
                        kc, rho, kn = rounded(kn[:, None] * kc, eps), rounded(kn * rho, eps), 1.0
                    Z.append(scale * kn * (rounded(qr, eps) @ kc.T + rounded(qs, eps) @ (sg * rho[:, None]).T))
                    V.append(rounded(v, eps))
                else:
                    Z.append(scale * kn * (qr @ kc.T + qs @ (sg * rho[:, None]).T))
                    V.append(rounded(v, eps) if form[name] == "ragged" else v)
            if not Z:
                continue
            z, v = np.concatenate(Z, 1), np.concatenate(V)
            w = np.exp(z - z.max(1, keepdims=True))
            num = rounded(w, eps) if p.dtype != "f32" else w
            out[b, h * G:(h + 1) * G, 0] = (num @ v) / w.sum(1, keepdims=True) @ R
    return out


def mistakes(p):
    """(what, a result with that mistake)."""
    out = p.attend()[0]
    yield "zeros", 0 * out
    yield "times 0.9", 0.9 * out
    yield "the last own token left out", p.attend(lens=np.maximum(p.lens - 1, 0))[0]
    yield "own caches left out", p.attend(lens=0 * p.lens)[0]
    yield "no sign sketch", p.attend(no_sign=True)[0]
    if p.pre:
        yield "the last ten prefix tokens left out", p.attend(skip=10)[0]
        yield "the last tile left out", p.attend(skip=p.t_prefix % 128)[0]
    if p.dtype == "f32":
        yield "queries rounded to fp16", p.attend(q=rounded(p.q, 2.0 ** -11))[0]


@pytest.mark.parametrize("d,bits,B", MANY)
def test_many_rows(d, bits, B):
    p = Host("bf16" if B % 2 else "f16", d, bits, B, 8, 2, 419, 12, seed=B + d)
    want, err, _, _ = p.attend()
    assert not p.refused(want, want, err) and not p.refused(emulated(p), want, err)
    for what, bad in mistakes(p):
        assert p.refused(bad, want, err), what


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,bits", WEIGH)
def test_own_caches(d, bits, dtype):
    p = Host(dtype, d, bits, 3, 8, 2, 0, 150, lens=[150, 0, 37], seed=d + bits)
    want, err, w, werr = p.attend()
    assert not p.refused(want, want, err) and not p.refused(emulated(p), want, err)
    for what, bad in mistakes(p):
        assert p.refused(bad, want, err), what
    # the weights: of the other 150 tokens when one is left out; a row less; queries in fp16
    before = np.ones_like(w)
    assert not sb.weights_out_of_bounds(before + w, w, werr, before).any()
    for bad in (p.attend(lens=np.maximum(p.lens - 1, 0))[2], 0.75 * w, p.attend(q=rounded(p.q, 2.0 ** -11))[2]):
        if not np.array_equal(bad, w):  # (a 16-bit query is one already)
            assert sb.weights_out_of_bounds(before + bad, w, werr, before).any()


@pytest.mark.parametrize("d", [128, 256])
def test_typical_error_of_many_rows(d):
    """At 2 bits half of a logit is its sign sketch: ||k|| rho rounded to fp16 moves all of a token's signs
    together and is the largest error by far.  The key norms stay out of the operands."""
    p = sketchy(Host("f16", d, 2, 32, 8, 2, 700, 1, lens=[0] * 32, seed=d))
    want, err, _, _ = p.attend()
    good, bad = emulated(p), emulated(p, norms_in_operands=True)
    assert sb.typical(to_type(good, "f16"), want, err, ref.HALF_STEP["f16"])
    assert not sb.typical(to_type(bad, "f16"), want, err, ref.HALF_STEP["f16"])


def sketchy(p):
    """Norms as 2-bit keys have them: ||k|| near sqrt(d), residuals of 0.6."""
    rng = np.random.default_rng(5)
    p.pre.kn[:] = np.sqrt(p.d) * rng.uniform(0.9, 1.1, p.pre.n)
    p.pre.kr[:] = rng.uniform(0.58, 0.62, p.pre.n)
    return p
