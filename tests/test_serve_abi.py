"""Refusals of the serving calls (no GPU: every call returns before a launch; fake device addresses
are never dereferenced), and the sizes their helpers give."""
import ctypes

import pytest

from .test_abi import _Params

FAKE = 0x10000
P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from kv_cache_vector_compress_b200 import build
    L = ctypes.CDLL(build.build())
    L.tq_workspace_bytes.restype = SZ
    for n in ("tq_attend_shared_scratch_bytes", "tq_attend_weigh_scratch_bytes", "tq_evict_scratch_bytes"):
        getattr(L, n).restype = SZ
    L.tq_attend_shared_scratch_bytes.argtypes = [P, I, I, I, I, I, I64, I64]
    L.tq_attend_weigh_scratch_bytes.argtypes = [P, I, I, I, I, I, I64]
    L.tq_evict_scratch_bytes.argtypes = [P, I, I, I64, I64]
    L.tq_attend_shared.argtypes = [P, P, I, I, I, I, I, I64] + [P] * 7 + [I64] + [P] * 6 + [F, P, P, SZ, P, P]
    L.tq_attend_weigh.argtypes = [P, P, I, I, I, I, I, P, I64] + [P] * 6 + [F, P, P, P, SZ, P, P]
    L.tq_evict.argtypes = [P, I, I, P, I64] + [P] * 7 + [I64] * 3 + [P] * 9 + [P, SZ, P, P]
    return L


def params(L, dim=128, bits=3, m=64, cut=0):
    return _Params(dim, bits, m, FAKE, FAKE, FAKE, L.tq_workspace_bytes(dim, bits, m) - cut)


def shared(L, prm, dtype=0, B=2, Hq=4, Hkv=2, Nq=1, tp=10, cap=8, q=FAKE, pre=FAKE, own=FAKE, lens=FAKE, scale=0.0,
           out=FAKE, scratch=FAKE, sb=1 << 50):
    return L.tq_attend_shared(ctypes.byref(prm) if prm else None, q, dtype, B, Hq, Hkv, Nq, tp, *[pre] * 6, lens, cap,
                              *[own] * 6, scale, out, scratch, sb, None, None)


def weigh(L, prm, dtype=0, B=2, Hq=4, Hkv=2, Nq=1, cap=8, lens=FAKE, own=FAKE, weights=FAKE, out=FAKE, sb=1 << 50):
    return L.tq_attend_weigh(ctypes.byref(prm), FAKE, dtype, B, Hq, Hkv, Nq, lens, cap, *[own] * 6, 0.0, weights, out,
                             FAKE, sb, None, None)


def test_shared_refusals(lib):
    g = params(lib)
    bad = [dict(dtype=3), dict(dtype=-1), dict(B=0), dict(Hq=3), dict(Nq=0), dict(Hkv=0), dict(tp=-1), dict(cap=-1),
           dict(tp=0, cap=0), dict(q=None), dict(q=FAKE + 8), dict(pre=None), dict(pre=FAKE + 4), dict(own=None),
           dict(own=FAKE + 2), dict(lens=None), dict(lens=FAKE + 4), dict(out=None), dict(out=FAKE + 8),
           dict(scratch=None), dict(sb=64), dict(scale=float("nan"))]
    for kw in bad:
        assert shared(lib, g, **kw) == 1, kw
    assert shared(lib, None) == 1
    assert shared(lib, params(lib, dim=100)) == 1
    assert shared(lib, params(lib, bits=1)) == 1      # keys need a projection and a code bit
    assert shared(lib, params(lib, cut=1)) == 1
    assert shared(lib, params(lib, dim=96)) == 2
    assert shared(lib, g, tp=2 ** 31) == 2
    assert shared(lib, g, cap=2 ** 31 - 1) == 2
    assert shared(lib, g, B=1 << 17, Hq=4) == 2


def test_weigh_refusals(lib):
    g = params(lib)
    for kw in [dict(dtype=9), dict(B=-1), dict(Hq=5), dict(cap=0), dict(lens=None), dict(own=None), dict(own=FAKE + 8),
               dict(weights=None), dict(weights=FAKE + 4), dict(out=None), dict(sb=64)]:
        assert weigh(lib, g, **kw) == 1, kw
    assert weigh(lib, g, cap=2 ** 31) == 2


def evict(L, prm, B=2, Hkv=2, cap=100, lens=1 << 20, budget=50, recent=10, out_cap=60, src=None, dst=None,
          kept=1 << 21, out_lens=1 << 22, weights=None, sb=1 << 20):
    s = src or [(1 << 30) + (i << 24) for i in range(7)]
    d = dst or [(1 << 32) + (i << 24) for i in range(7)]
    if weights is not None:
        s = s[:6] + [weights]
    return L.tq_evict(ctypes.byref(prm), B, Hkv, lens, cap, *s, budget, recent, out_cap, *d, kept, out_lens, 1 << 23, sb,
                      None, None)


def test_evict_refusals(lib):
    g = params(lib)
    s = [(1 << 30) + (i << 24) for i in range(7)]
    d = [(1 << 32) + (i << 24) for i in range(7)]
    for kw in [dict(B=0), dict(cap=0), dict(budget=0), dict(budget=101), dict(recent=-1), dict(recent=51),
               dict(out_cap=49), dict(lens=None), dict(lens=(1 << 20) + 4), dict(kept=None), dict(out_lens=None),
               dict(sb=0), dict(weights=(1 << 30) + 4), dict(out_lens=1 << 20),
               dict(dst=s),                                     # in place
               dict(dst=d[:3] + [s[3] + 16] + d[4:]),           # one array overlaps its source
               dict(dst=[s[4]] + d[1:]),                        # ... or another array's source
               dict(kept=s[0] + 16)]:
        assert evict(lib, g, **kw) == 1, kw
    assert evict(lib, params(lib, dim=96)) == 2
    assert evict(lib, g, cap=2 ** 31, budget=2) == 2


def test_scratch_sizes(lib):
    g = params(lib)
    p = ctypes.byref(g)
    assert lib.tq_attend_shared_scratch_bytes(p, 0, 2, 3, 2, 1, 5, 5) == 0
    assert lib.tq_attend_shared_scratch_bytes(p, 0, 2, 4, 2, 1, 0, 0) == 0
    assert lib.tq_attend_shared_scratch_bytes(p, 7, 2, 4, 2, 1, 5, 5) == 0
    small = lib.tq_attend_weigh_scratch_bytes(p, 0, 2, 4, 2, 1, 100)
    big = lib.tq_attend_weigh_scratch_bytes(p, 0, 2, 4, 2, 1, 10000)
    assert big - small >= 4 * 2 * 4 * 9900  # a score for each row and slot
    assert lib.tq_evict_scratch_bytes(p, 4, 2, 100, 50) >= 4 * 8
    assert lib.tq_evict_scratch_bytes(p, 4, 2, 100, 101) == 0
