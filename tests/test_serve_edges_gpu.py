"""Edges of the serving operators: weights across an eviction, orders, bad numbers, scratch contents."""
import numpy as np
import pytest

from . import serve_ref as ref
from .test_serve_gpu import Problem, tq  # noqa: F401  (tq: the fixture)

pytestmark = pytest.mark.gpu


def test_weights_of_tokens_to_come_are_zero(tq):  # noqa: F811
    """After an eviction into a cache of the binding's own, new tokens start from no weight (memory that
    nobody has written holds NaN here)."""
    import torch
    B, Hkv, cap, budget = 3, 2, 96, 30
    pr = Problem(tq, dtype="f32", B=B, Hq=4, Hkv=Hkv, t_cap=cap, lens=[96, 50, 10], seed=61)
    w = torch.from_numpy(pr.w0).cuda()
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # fills new memory with NaN
    try:
        k, v, w, _, lens = tq.tq_evict(pr.p, pr.k, pr.v, w, pr.dlens, Hkv, cap, budget, 4, cap)
    finally:
        torch.use_deterministic_algorithms(before)
    assert lens.tolist() == [30, 30, 10]
    for b, n in enumerate(lens.tolist()):
        assert torch.count_nonzero(w[b, :, n:]) == 0 and torch.count_nonzero(w[b, :, :n]) > 0
    # the next tokens: records of the old cache, in the slots behind the kept ones
    for dst, src in zip((*k, *v), (*pr.k, *pr.v)):
        dst.view(B, Hkv, cap, -1)[:, :, 30:40] = src.view(B, Hkv, cap, -1)[:, :, 50:60]
    pr.dlens = torch.tensor([40, 40, 10], dtype=torch.int32, device="cuda")
    before = w.sum(-1)
    tq.tq_attend_weigh(pr.p, pr.q, k, v, pr.dlens, Hkv, cap, w)
    torch.testing.assert_close(w.sum(-1) - before, torch.full((B, Hkv), 2.0, device="cuda"), rtol=0, atol=1e-4)


@pytest.mark.parametrize("d,m,bits", [(32, 32, 2), (128, 64, 3), (128, 32, 3), (512, 256, 4), (256, 128, 2)])
@pytest.mark.parametrize("where", ["query", "key norms", "key norm", "value norm"])
def test_nan_is_not_lost(tq, d, m, bits, where):  # noqa: F811
    """A NaN reaches every row that it concerns, whatever kernel the shape has, and no other row: in a query;
    in the norms of a slice's last 200 records; in the one record of a short slice; in one value norm."""
    import torch
    B, Hq, Hkv, cap = 3, 4, 2, 1500
    pr = Problem(tq, dtype="f32", d=d, m=m, bits=bits, B=B, Hq=Hq, Hkv=Hkv, t_cap=cap, lens=[1500, 900, 1], seed=62)
    want, wantw = pr.shared(tq), torch.from_numpy(pr.w0).cuda()
    pr.weigh(tq, wantw)
    bad = np.zeros((B, Hq), bool)
    slot = lambda b, h, t: (b * Hkv + h) * cap + t  # noqa: E731
    if where == "query":
        pr.q[1, 3] = float("nan")
        bad[1, 3] = True
    elif where == "key norms":
        pr.own.kn[slot(0, 1, 1300):slot(0, 1, 1500)] = np.nan
        bad[0, 2:] = True
    elif where == "key norm":
        pr.own.kn[slot(2, 0, 0)] = np.nan
        bad[2, :2] = True
    else:
        pr.own.vn[slot(1, 0, 333)] = np.nan
        bad[1, :2] = True
    pr.k, pr.v = pr.own.device()
    w = torch.from_numpy(pr.w0).cuda()
    bad = torch.from_numpy(bad).cuda()
    for out in (pr.shared(tq), pr.weigh(tq, w)):
        nan = torch.isnan(out).flatten(2)
        assert nan[bad].all() and not nan[~bad].any()
        torch.testing.assert_close(out[~bad], want[~bad], rtol=1e-4, atol=1e-5)
    heads = bad.view(B, Hkv, -1).any(-1)
    there = torch.arange(cap, device="cuda") < pr.dlens[:, None, None]
    assert torch.isnan(w)[heads[..., None] & there].all()
    torch.testing.assert_close(w[~heads], wantw[~heads], rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("d,bits", [(64, 3), (128, 3), (256, 2)])
@pytest.mark.parametrize("G", [1, 5, 7])
def test_results_do_not_depend_on_the_scratch(tq, dtype, d, bits, G):  # noqa: F811
    """Rows that fill no block of four or eight: the same bits whatever the scratch held (zeros, ordinary and
    large numbers, infinities, NaN).  The value norms of a stage's second 16 tokens are 2^8.1 times those of
    the first: just what moves the reference of a row whose logits are all 0, and of few others."""
    import torch
    B, Hkv, tp, cap = 2, 1, 320, 1600
    pr = Problem(tq, dtype=dtype, d=d, bits=bits, B=B, Hq=G * Hkv, Hkv=Hkv, t_prefix=tp if B * G <= 8 else 0,
                 t_cap=cap, lens=[1600, 1111], seed=63, q_scale=0.3)
    for c in (pr.pre, pr.own):
        if c is not None:
            c.vn[:] = np.where(np.arange(c.n) % 32 < 16, 2.0 ** -5, 2.0 ** 3.1)
    if pr.pre:
        pr.pk, pr.pv = pr.pre.device()
    pr.k, pr.v = pr.own.device()
    need = max(tq.tq_attend_shared_scratch_bytes(pr.p, pr.q.dtype, B, G, Hkv, 1, pr.t_prefix, cap),
               tq.tq_attend_weigh_scratch_bytes(pr.p, pr.q.dtype, B, G, Hkv, 1, cap))
    got = []
    for fill in (0x0000, 0x3C00, 0x7BFF, 0x7C00, 0xFC00, 0xFFFF, 0x55AA):
        fill = fill - 0x10000 if fill >= 0x8000 else fill
        scratch = torch.full((need // 2 + 8,), fill, dtype=torch.int16, device="cuda")
        w = torch.from_numpy(pr.w0).cuda()
        a = pr.shared(tq, scratch=scratch)
        scratch.fill_(fill)
        got.append((a, pr.weigh(tq, w, scratch=scratch), w))
    assert not any(torch.isnan(t).any() for t in got[0])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def two_kinds(tq, dtype, d, bits, B, Hq, t_prefix, t_cap, z_top, z_low, seed):  # noqa: F811
    """A Problem whose records are of two kinds, the query the same in every row: logits z_top and z_low (to
    the rounding of the query).  Returns it, the two records and the exact (logits [2], values [2, d])."""
    import math
    import torch
    pr = Problem(tq, dtype=dtype, d=d, bits=bits, B=B, Hq=Hq, Hkv=1, t_prefix=0, t_cap=1, seed=seed)
    two = ref.Cache(2, d, pr.m, bits, seed, zero=0.0)
    two.kc[1] = two.kc[0]
    two.kn[:] = 8.0, 8.0 * z_low / z_top
    two.kr[:] = 0
    two.vn[:] = 8.0
    kc, _, v = two.dequantized()
    R = pr.R.astype(np.float64)
    q = R.T @ kc[0] * (z_top * math.sqrt(d) / (8.0 * (kc[0] ** 2).sum()))
    pr.q = torch.from_numpy(q).to(pr.q.dtype).expand(B, Hq, 1, d).contiguous().cuda()
    q = pr.q[0, 0, 0].double().cpu().numpy()
    pr.t_prefix, pr.t_cap = t_prefix, t_cap
    z = two.kn.astype(np.float64) * ((R @ q) @ kc[0]) / math.sqrt(d)
    return pr, two.device(), z, v @ R


def test_light_tokens_of_a_long_prefix_count(tq):  # noqa: F811
    """Four million tokens, 2^-25.3 of the two heaviest ones' weight each, make up 5% of the softmax: too
    light for fp16 beside a weight of 1.  A weight is held to half a step of fp16 at 2^7 times that, 2^-32 of
    the largest, so that half the prefix (one of its two splits) is off by 2^21 2^-32."""
    import torch
    d, T, rows = 64, 1 << 22, 128 * 74
    pr, (k2, v2), z, v = two_kinds(tq, "f16", d, 2, rows // 64, 64, T, 0, 35.0, 17.5, 64)
    kind = torch.ones(T, dtype=torch.long, device="cuda")
    kind[0] = kind[T // 2] = 0
    pr.pk, pr.pv = tuple(t[kind].contiguous() for t in k2), tuple(t[kind].contiguous() for t in v2)
    out = pr.shared(tq).double().cpu().numpy().reshape(rows, d)
    light = (T - 2) * np.exp(z[1] - z[0])
    assert 0.05 < light < 0.2
    want = (2 * v[0] + light * v[1]) / (2 + light)
    # logits of operands rounded to fp16 (query and key) are off by 2 2^-11 of themselves and move the light
    # share by as much as their difference; the sums' operands (weight and value) by 2 2^-11, the output by 2^-11.
    # The 32-bit sum takes 16 tokens at a time, 2^17 times, and each time may lose 2^-23 of what it holds
    tol = (light / (2 + light) * 2 * 2.0 ** -11 * (abs(z[0]) + abs(z[1])) + 2.0 ** 21 * 2.0 ** -32 + 3 * 2.0 ** -11
           + 2.0 ** 17 * 2.0 ** -23)
    err = np.linalg.norm(out - want, axis=1)
    assert err.max() <= tol * np.linalg.norm(v, axis=1).max(), (err.max(), tol)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("d,m", [(128, 64), (128, 32)])
def test_out_may_be_the_queries(tq, dtype, d, m):  # noqa: F811
    import torch
    pr = Problem(tq, dtype=dtype, d=d, m=m, B=9, Hq=8, Hkv=2, t_prefix=300, t_cap=200, seed=66)
    a, w1, w2 = pr.shared(tq), torch.from_numpy(pr.w0).cuda(), torch.from_numpy(pr.w0).cuda()
    b = pr.weigh(tq, w1)
    q = pr.q
    pr.q = q.clone()
    assert torch.equal(a, pr.shared(tq, out=pr.q))
    pr.q = q.clone()
    assert torch.equal(b, pr.weigh(tq, w2, out=pr.q)) and torch.equal(w1, w2)


def test_what_is_missing_is_named(tq):  # noqa: F811
    import torch
    pr = Problem(tq, dtype="f16", t_prefix=10, t_cap=20, seed=67)
    w = torch.from_numpy(pr.w0).cuda()
    for name, call in [
            ("lens", lambda: tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, None, 2, 20, w)),
            ("weights", lambda: tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, pr.dlens, 2, 20, None)),
            ("own keys", lambda: tq.tq_attend_weigh(pr.p, pr.q, None, pr.v, pr.dlens, 2, 20, w)),
            ("lens", lambda: tq.tq_attend_shared(pr.p, pr.q, pr.pk, pr.pv, pr.k, pr.v, None, 2, 10, 20)),
            ("prefix keys", lambda: tq.tq_attend_shared(pr.p, pr.q, None, None, pr.k, pr.v, pr.dlens, 2, 10, 20)),
            ("own keys", lambda: tq.tq_attend_shared(pr.p, pr.q, pr.pk, pr.pv, None, None, pr.dlens, 2, 10, 20)),
            ("lens", lambda: tq.tq_evict(pr.p, pr.k, pr.v, w, None, 2, 20, 5, 1, 5)),
            ("weights", lambda: tq.tq_evict(pr.p, pr.k, pr.v, None, pr.dlens, 2, 20, 5, 1, 5))]:
        with pytest.raises(TypeError, match=name):
            call()


@pytest.mark.parametrize("bits,m,serves", [(4, 64, True), (2, 32, True), (3, 0, False), (1, 64, False)])
def test_tables_are_made_for_sets_that_serve(tq, bits, m, serves):  # noqa: F811
    """The search of the serving tables takes the host a third of tq_prepare: not done, and their place at the
    end of the workspace left alone, for a parameter set that the serving calls refuse."""
    import torch
    R, S = ref.matrices(128, max(m, 32), 3)
    p = tq.Params(128, bits, m, torch.from_numpy(R).cuda(), torch.from_numpy(S).cuda() if m else None, prepare=False)
    p.workspace.fill_(0xAB)
    tq.tq_prepare(p)
    assert bool((p.workspace[-256:-144] != 0xAB).any()) == serves
    assert tq._lib.tq_evict_scratch_bytes(p.ref, 1, 1, 8, 4) == (256 if serves else 0)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_all_rows_see_all_tokens(tq, dtype):  # noqa: F811
    """Three rows a sequence in one call: as calls of one row each at the same lengths.  At a row's own
    lengths those are the causal order, which the one call does not have."""
    import torch
    pr = Problem(tq, dtype=dtype, B=3, Hq=4, Hkv=2, Nq=3, t_cap=90, lens=[90, 41, 7], seed=68)
    w = torch.zeros(3, 2, 90, device="cuda")
    out, q, tol = pr.weigh(tq, w), pr.q, 2e-3 if dtype == "f16" else 1e-5
    total = torch.zeros_like(w)
    for i in range(3):
        pr.q = q[:, :, i:i + 1].contiguous()
        one = pr.weigh(tq, total)
        torch.testing.assert_close(out[:, :, i:i + 1], one, rtol=tol, atol=tol)
        if i < 2:
            causal = tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, (pr.dlens - 2 + i).int(), 2, 90, torch.zeros_like(w))
            assert not torch.allclose(out[:, :, i:i + 1], causal, rtol=tol, atol=tol)
    torch.testing.assert_close(w, total, rtol=1e-5, atol=1e-6)
