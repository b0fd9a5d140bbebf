"""The serving calls within the bounds of serve_bounds, which are of the size of their rounding errors: the
shapes of test_serve_gpu, whose bounds are worst cases."""
import math

import numpy as np
import pytest

from . import serve_bounds as sb
from . import serve_ref as ref
from .test_serve_bounds import sketchy
from .test_serve_gpu import Problem, tq  # noqa: F401  (tq: the fixture)

pytestmark = pytest.mark.gpu


def reference(pr):
    fp, fo = sb.forms(pr.dtype, pr.d, pr.m, pr.B, pr.Hkv, pr.Hq // pr.Hkv * pr.Nq, pr.t_prefix, pr.t_cap)
    caches = [(pr.pre, pr.t_prefix, True, None, fp)] if pr.pre else []
    caches += [(pr.own, pr.t_cap, False, pr.lens, fo)] if pr.own else []
    return sb.attend(pr.q64, pr.R, pr.S, caches, pr.Hkv, pr.scale, pr.bits)


def hold(pr, out, want, err, what):
    bad = sb.out_of_bounds(out.double().cpu().numpy(), want, err, ref.HALF_STEP[pr.dtype])
    off = np.linalg.norm(out.double().cpu().numpy().reshape(want.shape) - want, axis=-1)
    assert not bad.any(), (what, int(bad.sum()), bad.size, float((off / (err + 1e-37))[bad].max()))


def shared(tq, **kw):  # noqa: F811
    pr = Problem(tq, **kw)
    hold(pr, pr.shared(tq), *reference(pr)[:2], kw)


def weigh(tq, **kw):  # noqa: F811
    import torch
    pr = Problem(tq, **kw)
    want, err, w, werr = reference(pr)
    weights = torch.from_numpy(pr.w0).cuda()
    hold(pr, pr.weigh(tq, weights), want, err, kw)
    bad = sb.weights_out_of_bounds(weights.cpu().numpy(), w, werr, pr.w0.astype(np.float64))
    assert not bad.any(), (kw, int(bad.sum()), bad.size)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("B", [5, 16, 33, 70])
def test_many_rows(tq, d, bits, B):  # noqa: F811
    kw = dict(dtype="bf16" if B % 2 else "f16", d=d, bits=bits, B=B, Hq=8, Hkv=2, seed=B + d)
    shared(tq, t_prefix=419, t_cap=12, **kw)
    shared(tq, t_prefix=419, t_cap=0, **kw)


@pytest.mark.parametrize("d,bits", [(128, 2), (256, 2), (64, 3), (128, 3), (256, 3)])
def test_typical_error_of_many_rows(tq, d, bits):  # noqa: F811
    pr = sketchy(Problem(tq, dtype="f16", d=d, bits=bits, B=32, Hq=8, Hkv=2, t_prefix=700, t_cap=0, seed=d))
    pr.pk, pr.pv = pr.pre.device()
    want, err = reference(pr)[:2]
    out = pr.shared(tq)
    hold(pr, out, want, err, (d, bits))
    assert sb.typical(out.double().cpu().numpy(), want, err, ref.HALF_STEP["f16"])


@pytest.mark.parametrize("d,B,t_prefix", [(64, 41, 1907), (128, 41, 953), (256, 41, 477), (128, 9, 4341), (256, 70, 1000)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_many_rows_with_own_caches(tq, d, B, t_prefix, dtype):  # noqa: F811
    """At and past the size from which the prefix and the own caches have kernels of their own, and just below."""
    for tp in (t_prefix, t_prefix - 2):
        shared(tq, dtype=dtype, d=d, bits=3, B=B, Hq=8, Hkv=2, t_prefix=tp, t_cap=40, seed=B + d)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,bits", [(d, b) for d in (64, 128, 256) for b in (2, 3, 4)])
def test_types_and_widths(tq, d, bits, dtype):  # noqa: F811
    weigh(tq, dtype=dtype, d=d, bits=bits, B=3, Hq=8, Hkv=2, t_cap=150, lens=[150, 0, 37], seed=d + bits)
    shared(tq, dtype=dtype, d=d, bits=bits, B=2, Hq=8, Hkv=2, t_prefix=333, t_cap=50, lens=[50, 1], seed=d + bits)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("d,m,bits", [(32, 32, 2), (512, 256, 3), (1024, 512, 4), (128, 32, 3), (64, 96, 4)])
def test_other_shapes(tq, d, m, bits, dtype):  # noqa: F811
    weigh(tq, dtype=dtype, d=d, m=m, bits=bits, B=2, Hq=4, Hkv=2, t_cap=70, lens=[70, 33], seed=3)
    shared(tq, dtype=dtype, d=d, m=m, bits=bits, B=2, Hq=6, Hkv=2, Nq=2, t_prefix=131, t_cap=5, lens=[0, 5], seed=4)


@pytest.mark.parametrize("t_prefix,t_cap,lens", [(1, 1, [0, 1, 1]), (31, 33, [33, 32, 1]), (127, 3, [0, 0, 0]),
                                                 (129, 64, [64, 1, 0]), (640, 20, [3, 20, 0]),
                                                 (2049, 100, [100, 99, 98]), (5000, 1000, [1000, 0, 517])])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_lengths(tq, t_prefix, t_cap, lens, dtype):  # noqa: F811
    shared(tq, dtype=dtype, B=3, Hq=8, Hkv=2, t_prefix=t_prefix, t_cap=t_cap, lens=lens, seed=t_prefix)
    weigh(tq, dtype=dtype, B=3, Hq=8, Hkv=2, t_cap=t_cap, lens=lens, seed=t_prefix)


@pytest.mark.parametrize("Hq,Hkv,Nq", [(1, 1, 1), (2, 2, 3), (5, 1, 1), (8, 1, 1), (9, 1, 1), (14, 2, 3), (16, 1, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows(tq, Hq, Hkv, Nq, dtype):  # noqa: F811
    weigh(tq, dtype=dtype, B=2, Hq=Hq, Hkv=Hkv, Nq=Nq, t_cap=90, lens=[90, 41], seed=Hq)
    shared(tq, dtype=dtype, B=2, Hq=Hq, Hkv=Hkv, Nq=Nq, t_prefix=77, t_cap=90, lens=[90, 41], seed=Hq)


@pytest.mark.parametrize("d,B,Hq", [(64, 150, 16), (128, 101, 8), (128, 110, 16), (256, 51, 16), (512, 83, 8)])
def test_batches(tq, d, B, Hq):  # noqa: F811
    lens = [(17 * b) % 41 for b in range(B)]
    weigh(tq, dtype="f16", d=d, B=B, Hq=Hq, Hkv=1, t_cap=40, lens=lens, seed=B)
    shared(tq, dtype="f16", d=d, B=B, Hq=Hq, Hkv=1, t_prefix=70, t_cap=40, lens=lens, seed=B)


@pytest.mark.parametrize("q_scale", [0.0, 1e-4, 3.0, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_query_sizes(tq, q_scale, dtype):  # noqa: F811
    kw = dict(dtype=dtype, B=9, Hq=8, Hkv=1, t_cap=100, lens=[100] * 9, q_scale=q_scale, seed=7)
    weigh(tq, **kw)
    shared(tq, t_prefix=300, **kw)
    shared(tq, t_prefix=4400, **kw)


@pytest.mark.parametrize("d,bits", [(64, 3), (128, 2), (256, 4), (512, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_takes_it_all(tq, d, bits, dtype):  # noqa: F811
    """Queries of 3e4 along one token's key each: the output is that token's value, its weight one a row."""
    import torch
    B, Hq, Hkv, tp, cap = 6, 8, 2, 13100, 100
    pr = Problem(tq, dtype=dtype, d=d, bits=bits, B=B, Hq=Hq, Hkv=Hkv, t_prefix=tp, t_cap=cap, lens=[cap] * B, seed=8)
    R, S, G = pr.R.astype(np.float64), pr.S.astype(np.float64), Hq // Hkv
    rng = np.random.default_rng(9)

    def keys(c):
        kc, sg, v = c.dequantized()
        rho = c.kr.astype(np.float64)[:, None] * math.sqrt(math.pi / 2) / pr.m
        return kc @ R + rho * (sg @ S), c.kn.astype(np.float64), v @ R

    pre, own = keys(pr.pre), keys(pr.own)
    for use_prefix in (False, True):
        q, want, token = np.zeros((B, Hq, 1, d)), np.zeros((B, Hq, 1, d)), np.zeros((B, Hkv, cap))
        for b in range(B):
            for r in range(Hq):
                h = r // G
                (dirs, kn, v), base, n = (pre, h * tp, tp) if use_prefix else (own, (b * Hkv + h) * cap, cap)
                t = base + int(rng.choice(np.argsort(-kn[base:base + n])[:n // 3]))
                q[b, r, 0] = 3e4 * math.sqrt(d) * dirs[t] / np.linalg.norm(dirs[t])
                want[b, r, 0] = v[t]
                if not use_prefix:
                    token[b, h, t - base] += 1
                # it leads by far, over the prefix and the own tokens
                z = np.concatenate([pre[1][h * tp:(h + 1) * tp] * (pre[0][h * tp:(h + 1) * tp] @ q[b, r, 0]),
                                    own[1][(b * Hkv + h) * cap:][:cap] *
                                    (own[0][(b * Hkv + h) * cap:][:cap] @ q[b, r, 0])])
                z = np.sort(z) / math.sqrt(d)
                assert z[-1] > 1.2 * z[-2] > 0
        pr.q = torch.from_numpy(q).to(pr.q.dtype).cuda()
        forms = sb.forms(dtype, d, pr.m, B, Hkv, G, tp, cap)
        f = sb.FORMS[forms[0 if use_prefix else 1]]
        err = np.linalg.norm(want, axis=-1) * math.sqrt(f["weight"] ** 2 + f["value"](bits) ** 2 + f["sum"] ** 2)
        hold(pr, pr.shared(tq), want, err, (d, bits, use_prefix))
        if not use_prefix:
            w = torch.zeros(B, Hkv, cap, device="cuda")
            hold(pr, pr.weigh(tq, w), want, err, (d, bits, "weigh"))
            np.testing.assert_allclose(w.cpu().numpy(), token, rtol=1e-5, atol=0)


@pytest.mark.parametrize("d,bits,B,dtype", [(64, 3, 3, "f32"), (128, 3, 3, "f32"), (128, 4, 3, "f16"), (256, 3, 300, "f16")])
def test_law_of_the_codebook(tq, d, bits, B, dtype):  # noqa: F811
    import oracle
    import torch
    plain = oracle.codebook_f32
    pr = Problem(tq, dtype=dtype, d=d, bits=bits, B=B, Hq=4, Hkv=1, t_prefix=150, t_cap=60, seed=43)
    pr.p = tq.Params(d, bits, d // 2, torch.from_numpy(pr.R).cuda(), torch.from_numpy(pr.S).cuda(), law="beta")
    out, weights = pr.shared(tq), torch.from_numpy(pr.w0).cuda()
    out2 = pr.weigh(tq, weights)
    try:
        oracle.codebook_f32 = lambda dim, bits: plain(dim, bits, law="beta")
        want, err, _, _ = reference(pr)
        pr.pre = None
        want2, err2, w, werr = reference(pr)
    finally:
        oracle.codebook_f32 = plain
    hold(pr, out, want, err, "shared")
    hold(pr, out2, want2, err2, "weigh")
    assert not sb.weights_out_of_bounds(weights.cpu().numpy(), w, werr, pr.w0.astype(np.float64)).any()
