"""The serving calls against their 64-bit definitions, at the lengths, layouts and masks where they
can go wrong.  Tolerances are derived in serve_ref.attend."""
import math

import numpy as np
import pytest

from . import serve_ref as ref

pytestmark = pytest.mark.gpu

OPERAND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -11, "f32": 0.0}


@pytest.fixture(scope="module")
def tq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kv_cache_vector_compress_b200 import tq as _tq
    return _tq


def torch_type(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


class Problem:
    def __init__(self, tq, dtype="f32", d=128, m=None, bits=3, B=2, Hq=4, Hkv=2, Nq=1, t_prefix=0, t_cap=64,
                 lens=None, seed=0, q_scale=1.0):
        import torch
        m = d // 2 if m is None else m
        self.__dict__.update(dtype=dtype, d=d, m=m, bits=bits, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, t_prefix=t_prefix,
                             t_cap=t_cap)
        rng = np.random.default_rng(1000 + seed)
        self.R, self.S = ref.matrices(d, m, 40 + d)
        self.p = tq.Params(d, bits, m, torch.from_numpy(self.R).cuda(), torch.from_numpy(self.S).cuda())
        q = torch.from_numpy(rng.standard_normal((B, Hq, Nq, d)) * q_scale).to(torch_type(dtype))
        self.q = q.cuda()
        self.q64 = q.double().numpy()
        self.lens = np.asarray(lens if lens is not None else rng.integers(0, t_cap + 1, B), np.int32)
        self.scale = 1 / math.sqrt(d)
        self.pre = ref.Cache(Hkv * t_prefix, d, m, bits, seed + 1) if t_prefix else None
        self.own = ref.Cache(B * Hkv * t_cap, d, m, bits, seed + 2) if t_cap else None
        self.pk, self.pv = self.pre.device() if self.pre else (None, None)
        self.k, self.v = self.own.device() if self.own else (None, None)
        self.dlens = torch.from_numpy(self.lens).cuda()
        self.w0 = rng.uniform(0, 2, (B, Hkv, max(t_cap, 1))).astype(np.float32)

    def reference(self, operand):
        caches = [(self.pre, self.t_prefix, True, None)] if self.pre else []
        caches += [(self.own, self.t_cap, False, self.lens)] if self.own else []
        return ref.attend(self.q64, self.R, self.S, caches, self.Hkv, self.scale, operand)

    def shared(self, tq, **kw):
        return tq.tq_attend_shared(self.p, self.q, self.pk, self.pv, self.k, self.v, self.dlens, self.Hkv,
                                   self.t_prefix, self.t_cap, **kw)

    def weigh(self, tq, weights, **kw):
        return tq.tq_attend_weigh(self.p, self.q, self.k, self.v, self.dlens, self.Hkv, self.t_cap, weights, **kw)


def check(got, want, tol, half_step, what):
    g = got.double().cpu().numpy().reshape(want.shape)
    err, lim = np.abs(g - want), tol + half_step * (np.abs(want) + tol) + 1e-38
    if half_step == 2.0 ** -11:
        lim = lim + 2.0 ** -25  # fp16 outputs: half the distance of its smallest numbers
    bad = ~(err <= lim)
    assert not bad.any(), (what, int(bad.sum()), bad.size, float((err - lim).max()), float(err.max()))


def run_shared(tq, **kw):
    pr = Problem(tq, **kw)
    want, tol, _, _ = pr.reference(OPERAND[pr.dtype])
    check(pr.shared(tq), want, tol, ref.HALF_STEP[pr.dtype], kw)
    return pr


def run_weigh(tq, **kw):
    import torch
    pr = Problem(tq, **kw)
    want, tol, w, wtol = pr.reference(OPERAND[pr.dtype])
    # the weights' scores keep 32 bits, but for the 3-bit key centroids behind 16-bit rows: the best
    # fp16 table of the four magnitudes has relative errors of 3.06e-5, 1.1e-5, 7.3e-6 and 0
    _, _, _, wtol = pr.reference(1.55e-5 if pr.bits == 4 and pr.dtype != "f32" else 0.0)
    weights = torch.from_numpy(pr.w0).cuda()
    out = pr.weigh(tq, weights)
    check(out, want, tol, ref.HALF_STEP[pr.dtype], kw)
    check(weights, pr.w0.astype(np.float64) + w, wtol, 2.0 ** -23, kw)
    # behind the last token: left as it was
    got = weights.cpu().numpy()
    for b in range(pr.B):
        assert np.array_equal(got[b, :, pr.lens[b]:], pr.w0[b, :, pr.lens[b]:])
    return pr


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,bits", [(64, 2), (64, 4), (128, 2), (128, 3), (128, 4), (256, 2), (256, 3), (256, 4)])
def test_weigh_types_and_widths(tq, dtype, d, bits):
    run_weigh(tq, dtype=dtype, d=d, bits=bits, B=3, Hq=8, Hkv=2, t_cap=150, lens=[150, 0, 37], seed=d + bits)


@pytest.mark.parametrize("d,m", [(32, 32), (512, 256), (1024, 512), (128, 32), (64, 96)])
def test_other_shapes(tq, d, m):
    run_weigh(tq, dtype="bf16", d=d, m=m, B=2, Hq=4, Hkv=2, t_cap=70, lens=[70, 33], seed=3)
    run_shared(tq, dtype="f32", d=d, m=m, B=2, Hq=6, Hkv=2, Nq=2, t_prefix=131, t_cap=5, lens=[0, 5], seed=4)


@pytest.mark.parametrize("t_cap,lens", [(1, [1, 0, 1]), (2, [2, 1, 0]), (31, [31, 30, 1]), (32, [32, 31, 0]),
                                        (33, [33, 32, 31]), (65, [64, 65, 33]), (129, [129, 128, 127]),
                                        (1000, [1000, 0, 999]), (5, [0, 0, 0])])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_weigh_lengths(tq, t_cap, lens, dtype):
    run_weigh(tq, dtype=dtype, B=3, Hq=6, Hkv=2, t_cap=t_cap, lens=lens, seed=t_cap)


@pytest.mark.parametrize("Hq,Hkv,Nq", [(1, 1, 1), (2, 2, 3), (5, 1, 1), (7, 1, 1), (8, 1, 1), (9, 1, 1), (14, 2, 3),
                                       (16, 1, 4), (3, 3, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows(tq, Hq, Hkv, Nq, dtype):
    run_weigh(tq, dtype=dtype, B=2, Hq=Hq, Hkv=Hkv, Nq=Nq, t_cap=90, lens=[90, 41], seed=Hq)
    run_shared(tq, dtype=dtype, B=2, Hq=Hq, Hkv=Hkv, Nq=Nq, t_prefix=77, t_cap=90, lens=[90, 41], seed=Hq)


@pytest.mark.parametrize("t_prefix,t_cap,lens", [(1, 0, None), (500, 0, None), (0, 40, [40, 0, 7]), (1, 1, [0, 1, 1]),
                                                 (31, 33, [33, 32, 1]), (127, 3, [0, 0, 0]), (129, 64, [64, 1, 0]),
                                                 (640, 20, [3, 20, 0]), (2049, 100, [100, 99, 98])])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_shared_lengths(tq, t_prefix, t_cap, lens, dtype):
    run_shared(tq, dtype=dtype, B=3, Hq=8, Hkv=2, t_prefix=t_prefix, t_cap=t_cap, lens=lens, seed=t_prefix)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("B", [5, 16, 33, 70])
def test_shared_many_rows(tq, d, bits, B):
    """Rows below, at and past the tiles of query rows, a prefix that ends inside a tile of tokens."""
    run_shared(tq, dtype="bf16" if B % 2 else "f16", d=d, bits=bits, B=B, Hq=8, Hkv=2, t_prefix=419, t_cap=12,
               seed=B + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_rows_past_eight(tq, d, bits, dtype):
    """Blocks of eight rows, the last one not full."""
    run_weigh(tq, dtype=dtype, d=d, bits=bits, B=3, Hq=22, Hkv=2, t_cap=170, lens=[170, 0, 45], seed=d * bits)


@pytest.mark.parametrize("d,B,Hq", [(64, 150, 16), (128, 101, 8), (128, 110, 16), (256, 51, 16), (512, 83, 8)])
def test_batches_of_many_rows(tq, d, B, Hq):
    """Merges of 8 and 16 rows a CTA and preparations of 16, the last of each not full."""
    lens = [(17 * b) % 41 for b in range(B)]
    run_weigh(tq, dtype="bf16", d=d, B=B, Hq=Hq, Hkv=1, t_cap=40, lens=lens, seed=B)
    run_shared(tq, dtype="bf16", d=d, B=B, Hq=Hq, Hkv=1, t_prefix=70, t_cap=40, lens=lens, seed=B)


def test_eight_rows_over_many_stages(tq):
    """Long enough for blocks of eight rows where there are no more than eight."""
    run_weigh(tq, dtype="f16", d=64, bits=2, B=48, Hq=16, Hkv=2, t_cap=2400, lens=[2400] * 24 + [1000] * 24, seed=5)


@pytest.mark.parametrize("op", ["weigh", "shared"])
@pytest.mark.parametrize("q_scale", [0.0, 1e-4, 30.0, 3e4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_query_sizes(tq, op, q_scale, dtype):
    """Zero queries (equal weights), tiny ones, and ones whose softmax picks one token."""
    run = run_weigh if op == "weigh" else run_shared
    run(tq, dtype=dtype, B=9, Hq=8, Hkv=1, t_prefix=0 if op == "weigh" else 300, t_cap=100, lens=[100] * 9,
        q_scale=q_scale, seed=7)


def test_value_norms_of_all_sizes(tq):
    """Value norms over fp16's whole range in one context: no weight overflows, the small ones vanish."""
    import torch
    for dtype, op in [("f16", "weigh"), ("bf16", "shared"), ("f32", "weigh")]:
        pr = Problem(tq, dtype=dtype, B=20, Hq=8, Hkv=1, t_prefix=300 if op == "shared" else 0, t_cap=200,
                     lens=[200] * 20, seed=11)
        for c in (pr.pre, pr.own):
            if c is not None:
                c.vn[:] = np.exp2(np.random.default_rng(1).uniform(-24, 6, c.n)).astype(np.float16)
        if pr.pre:
            pr.pk, pr.pv = pr.pre.device()
        pr.k, pr.v = pr.own.device()
        want, tol, _, _ = pr.reference(OPERAND[dtype])
        out = pr.weigh(tq, torch.from_numpy(pr.w0).cuda()) if op == "weigh" else pr.shared(tq)
        check(out, want, tol, ref.HALF_STEP[dtype], (dtype, op))
        # all values zero: exactly zero
        for c in (pr.pre, pr.own):
            if c is not None:
                c.vn[:] = 0
        if pr.pre:
            pr.pk, pr.pv = pr.pre.device()
        pr.k, pr.v = pr.own.device()
        out = pr.weigh(tq, torch.from_numpy(pr.w0).cuda()) if op == "weigh" else pr.shared(tq)
        assert torch.count_nonzero(out) == 0


def test_records_behind_the_length_do_not_matter(tq):
    """Infinities and NaN norms behind lens[b] change nothing, bit for bit."""
    import torch
    for op in ("weigh", "shared"):
        pr = Problem(tq, dtype="bf16", B=3, Hq=8, Hkv=2, t_prefix=0 if op == "weigh" else 50, t_cap=100,
                     lens=[100, 40, 0], seed=5)
        w1, w2 = torch.from_numpy(pr.w0).cuda(), torch.from_numpy(pr.w0).cuda()
        a = pr.weigh(tq, w1) if op == "weigh" else pr.shared(tq)
        behind = np.arange(100)[None, None, :] >= pr.lens[:, None, None]
        behind = np.broadcast_to(behind, (3, 2, 100)).reshape(-1)
        pr.own.kn[behind], pr.own.kr[behind], pr.own.vn[behind] = np.nan, np.inf, np.nan
        pr.k, pr.v = pr.own.device()
        b = pr.weigh(tq, w2) if op == "weigh" else pr.shared(tq)
        assert torch.equal(a, b) and torch.equal(w1, w2)


def test_a_bad_record_stays_in_its_rows(tq):
    """A NaN norm inside the length makes the rows that attend it NaN, and no others."""
    import torch
    pr = Problem(tq, dtype="f16", B=3, Hq=8, Hkv=2, t_cap=100, lens=[100, 60, 20], seed=6)
    pr.own.kn[(1 * 2 + 0) * 100 + 30] = np.nan
    pr.k, pr.v = pr.own.device()
    out = pr.weigh(tq, torch.from_numpy(pr.w0).cuda())
    bad = torch.isnan(out).flatten(2).any(-1).cpu().numpy()
    assert bad[1, :4].all() and not bad[1, 4:].any() and not bad[0].any() and not bad[2].any()


def test_lengths_outside_are_clamped_and_reported(tq):
    import torch
    for op in ("weigh", "shared"):
        pr = Problem(tq, dtype="f32", B=3, Hq=4, Hkv=2, t_prefix=0 if op == "weigh" else 40, t_cap=50,
                     lens=[50, 0, 20], seed=8)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        w1, w2 = torch.from_numpy(pr.w0).cuda(), torch.from_numpy(pr.w0).cuda()
        a = pr.weigh(tq, w1, dev_status=st) if op == "weigh" else pr.shared(tq, dev_status=st)
        assert st.item() == 0
        pr.dlens = torch.tensor([2 ** 31 - 1, -5, 20], dtype=torch.int32, device="cuda")
        b = pr.weigh(tq, w2, dev_status=st) if op == "weigh" else pr.shared(tq, dev_status=st)
        assert st.item() == tq.TQ_ERR_INVALID_ARG
        assert torch.equal(a, b) and torch.equal(w1, w2)


def test_shared_agrees_with_a_copied_prefix(tq):
    """A prefix shared by the batch is the same as a copy of it at the head of every own cache."""
    import torch
    pr = Problem(tq, dtype="f32", B=4, Hq=8, Hkv=2, t_prefix=60, t_cap=30, lens=[30, 10, 0, 1], seed=9)
    a = pr.shared(tq)
    B, Hkv, n = 4, 2, 90

    def join(p, o):
        p = p.view(1, Hkv, 60, -1).expand(B, -1, -1, -1)
        return torch.cat([p, o.view(B, Hkv, 30, -1)], 2).reshape(B * Hkv * n, -1).contiguous()

    k, v = tuple(map(join, pr.pk, pr.k)), tuple(map(join, pr.pv, pr.v))
    w = torch.zeros(B, Hkv, n, device="cuda")
    b = tq.tq_attend_weigh(pr.p, pr.q, k, v, (pr.dlens + 60).int(), Hkv, n, w)
    torch.testing.assert_close(a, b, rtol=1e-4, atol=1e-5)
    # every row's weights add up to one
    torch.testing.assert_close(w.sum(-1), torch.full((B, Hkv), 4.0, device="cuda"), rtol=1e-5, atol=0)


def test_runs_are_bit_identical_and_streams_hold(tq):
    import torch
    pr = Problem(tq, dtype="bf16", B=8, Hq=8, Hkv=2, t_prefix=700, t_cap=400, seed=10)
    w = [torch.from_numpy(pr.w0).cuda() for _ in range(3)]
    torch.cuda.synchronize()
    a, b = pr.shared(tq), pr.weigh(tq, w[0])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):  # two calls at once, each with its own scratch
        a1, b1 = pr.shared(tq), pr.weigh(tq, w[1])
    with torch.cuda.stream(s2):
        a2, b2 = pr.shared(tq), pr.weigh(tq, w[2])
    torch.cuda.synchronize()
    assert torch.equal(a, a1) and torch.equal(a, a2) and torch.equal(b, b1) and torch.equal(b, b2)
    assert torch.equal(w[0], w[1]) and torch.equal(w[0], w[2])


def test_graph_follows_the_lengths(tq):
    """A captured call reads queries, lengths and caches when it is replayed."""
    import torch
    pr = Problem(tq, dtype="f16", B=4, Hq=8, Hkv=2, t_prefix=100, t_cap=200, lens=[1, 2, 3, 4], seed=12)
    B, Hkv = 4, 2
    need = tq.tq_attend_shared_scratch_bytes(pr.p, pr.q.dtype, B, 8, Hkv, 1, 100, 200)
    need = max(need, tq.tq_attend_weigh_scratch_bytes(pr.p, pr.q.dtype, B, 8, Hkv, 1, 200),
               tq.tq_evict_scratch_bytes(pr.p, B, Hkv, 200, 120))
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    w = torch.from_numpy(pr.w0).cuda()
    o1, o2 = torch.empty_like(pr.q), torch.empty_like(pr.q)
    ev = tq.tq_evict(pr.p, pr.k, pr.v, w, pr.dlens, Hkv, 200, 120, 10, 130)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pr.shared(tq, out=o1, scratch=scratch)
        pr.weigh(tq, w, out=o2, scratch=scratch)
        tq.tq_evict(pr.p, pr.k, pr.v, w, pr.dlens, Hkv, 200, 120, 10, 130, out_keys=ev[0], out_values=ev[1],
                    out_weights=ev[2], kept=ev[3], out_lens=ev[4], scratch=scratch)
    for lens in ([200, 0, 131, 7], [0, 0, 0, 0], [150, 200, 200, 120]):
        w.copy_(torch.from_numpy(pr.w0))
        pr.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        pr.q.mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        w2 = torch.from_numpy(pr.w0).cuda()
        assert torch.equal(o1, pr.shared(tq)) and torch.equal(o2, pr.weigh(tq, w2)) and torch.equal(w, w2)
        assert ev[4].tolist() == [min(n, 120) for n in lens]


def test_offsets_past_32_bits(tq):
    """Caches whose arrays are longer than 2^31 words and 2^32 bytes: the last sequence's records lie
    behind both (only the tokens in use are ever written)."""
    import torch
    B, d, bits, cap, n = 3, 256, 4, 46_000_000, 100
    pr = Problem(tq, dtype="bf16", d=d, bits=bits, B=B, Hq=2, Hkv=1, t_cap=n, lens=[40, 100, 71], seed=41)
    assert 2 * cap * pr.p.key_words() > 2 ** 31

    def spread(t):
        big = torch.empty((B * cap, *t.shape[1:]), dtype=t.dtype, device="cuda")
        big.view(B, cap, *t.shape[1:])[:, :n] = t.view(B, n, *t.shape[1:])
        return big

    k, v = tuple(map(spread, pr.k)), tuple(map(spread, pr.v))
    w = torch.zeros(B, 1, cap, device="cuda")
    out = tq.tq_attend_weigh(pr.p, pr.q, k, v, pr.dlens, 1, cap, w)
    want, tol, ws, wtol = pr.reference(OPERAND["bf16"])
    check(out, want, tol, ref.HALF_STEP["bf16"], "weigh")
    got = tq.tq_attend_shared(pr.p, pr.q, None, None, k, v, pr.dlens, 1, 0, cap)
    check(got, want, tol, ref.HALF_STEP["bf16"], "shared")
    _, _, _, wtol = pr.reference(1.55e-5)  # as in run_weigh
    check(w[:, :, :n].contiguous(), ws, wtol, 2.0 ** -23, "weights")
    assert torch.count_nonzero(w[:, :, n:]) == 0
    ok, ov, ow, kept, lens = tq.tq_evict(pr.p, k, v, w, pr.dlens, 1, cap, 50, 5, 60)
    keep = ref.evict(w[:, :, :n].cpu().numpy(), pr.lens, 50, 5)
    for b in range(B):
        s = keep[b][0]
        assert kept[b, 0, :len(s)].tolist() == s.tolist() and lens[b].item() == len(s)
        for dst, src in zip((*ok, *ov), (*pr.k, *pr.v)):
            assert torch.equal(dst.view(B, 60, -1)[b, :len(s)], src.view(B, n, -1)[b, torch.from_numpy(s).cuda()])


@pytest.mark.parametrize("dtype,B", [("bf16", 40), ("f32", 3)])
def test_law_of_the_codebook(tq, dtype, B):
    """The codebooks of the exact coordinate law go through the same tables."""
    import oracle
    import torch
    pr = Problem(tq, dtype=dtype, d=64, bits=3, B=B, Hq=4, Hkv=1, t_prefix=150, t_cap=20, seed=43)
    gaussian = pr.shared(tq)
    pr.p = tq.Params(64, 3, 32, torch.from_numpy(pr.R).cuda(), torch.from_numpy(pr.S).cuda(), law="beta")
    out = pr.shared(tq)
    assert not torch.equal(out, gaussian)
    plain = oracle.codebook_f32
    try:
        oracle.codebook_f32 = lambda dim, bits: plain(dim, bits, law="beta")
        want, tol, _, _ = pr.reference(OPERAND[dtype])
    finally:
        oracle.codebook_f32 = plain
    check(out, want, tol, ref.HALF_STEP[dtype], (dtype, B))


def test_softmax_scale(tq):
    import torch
    pr = Problem(tq, dtype="f32", B=12, Hq=4, Hkv=2, t_prefix=90, t_cap=30, seed=44)
    pr.scale = 0.7
    for op in ("shared", "weigh"):
        if op == "weigh":
            pr.pre = None
        want, tol, _, _ = pr.reference(0.0)
        out = pr.shared(tq, scale=0.7) if op == "shared" else pr.weigh(tq, torch.from_numpy(pr.w0).cuda(), scale=0.7)
        check(out, want, tol, ref.HALF_STEP["f32"], op)


# ------------------------------------------------------------------- eviction

def run_evict(tq, weights, lens, budget, recent, out_cap, d=128, bits=3, seed=0):
    import torch
    B, Hkv, cap = weights.shape
    m = max(32, d // 2)
    R, S = ref.matrices(d, m, 5)
    p = tq.Params(d, bits, m, torch.from_numpy(R).cuda(), torch.from_numpy(S).cuda())
    src, dst = ref.Cache(B * Hkv * cap, d, m, bits, seed), ref.Cache(B * Hkv * out_cap, d, m, bits, seed + 1)
    (k, v), (ok, ov) = src.device(), dst.device()
    w = torch.from_numpy(weights).cuda()
    ow = torch.full((B, Hkv, out_cap), -3.0, device="cuda")
    kept = torch.full((B, Hkv, budget), -7, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (*ok, *ov, ow, kept)]
    source = [t.clone() for t in (*k, *v, w)]
    ol = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    tq.tq_evict(p, k, v, w, dl, Hkv, cap, budget, recent, out_cap, out_keys=ok, out_values=ov, out_weights=ow,
                kept=kept, out_lens=ol)
    want = ref.evict(weights, lens, budget, recent)
    assert ol.tolist() == [min(int(n), budget) for n in lens]
    got = [t.cpu().numpy().reshape(B, Hkv, out_cap, -1) for t in (*ok, *ov, ow)]
    old = [t.cpu().numpy().reshape(B, Hkv, out_cap, -1) for t in before[:-1]]
    data = [t.cpu().numpy().reshape(B, Hkv, cap, -1) for t in source]
    for now, was in zip((*k, *v, w), source):
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8)), "the source changed"
    kn = kept.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            s = want[b][h]
            assert np.array_equal(kn[b, h, :len(s)], s), (b, h)
            assert (kn[b, h, len(s):] == -7).all()
            for g, o, x in zip(got, old, data):
                assert g[b, h, :len(s)].tobytes() == x[b, h, s].tobytes(), (b, h)
                assert g[b, h, len(s):].tobytes() == o[b, h, len(s):].tobytes(), (b, h)


@pytest.mark.parametrize("cap,budget,recent", [(1, 1, 0), (1, 1, 1), (2, 1, 0), (2, 1, 1), (33, 32, 5), (100, 1, 1),
                                               (100, 99, 0), (100, 100, 10), (100, 50, 50), (1025, 1024, 0),
                                               (2500, 700, 64), (5000, 4999, 4999)])
def test_evict_sizes(tq, cap, budget, recent):
    rng = np.random.default_rng(cap)
    w = np.exp(2 * rng.standard_normal((3, 2, cap))).astype(np.float32)
    run_evict(tq, w, [cap, max(0, cap // 2), 0], budget, recent, budget + 3, seed=cap)


@pytest.mark.parametrize("d,bits", [(32, 2), (64, 2), (64, 3), (128, 4), (256, 3), (1024, 4)])
def test_evict_widths(tq, d, bits):
    w = np.random.default_rng(d).random((2, 2, 90)).astype(np.float32)
    run_evict(tq, w, [90, 61], 40, 7, 40, d=d, bits=bits)


def test_evict_ties_and_odd_weights(tq):
    """Equal weights go to the smaller slot; zeros of both signs are equal; negative numbers,
    denormals, infinities and NaN have their place."""
    w = np.zeros((6, 1, 3000), np.float32)
    w[1, 0] = 1.0
    w[2, 0, ::2] = -0.0
    rng = np.random.default_rng(3)
    w[3, 0] = rng.integers(0, 4, 3000)
    w[4, 0] = rng.standard_normal(3000)
    w[4, 0, [5, 900, 2990]] = np.inf, -np.inf, np.nan
    w[4, 0, 17] = -np.nan
    w[5, 0] = rng.integers(0, 3000, 3000) * np.float32(1e-45)
    for budget, recent in [(1, 0), (3, 1), (1500, 100), (2999, 0)]:
        run_evict(tq, w, [3000] * 6, budget, recent, budget)


def test_evict_one_long_slice(tq):
    w = np.random.default_rng(9).random((1, 1, 200_003)).astype(np.float32)
    run_evict(tq, w, [200_003], 100_001, 777, 100_001, d=32, bits=2)


@pytest.mark.parametrize("cap", [24_577, 51_201])
def test_evict_many_long_slices(tq, cap):
    rng = np.random.default_rng(cap)
    w = rng.integers(0, 200, (50, 3, cap)).astype(np.float32)  # ties everywhere
    lens = rng.integers(0, cap + 1, 50)
    lens[:4] = cap, 0, 1, 300
    run_evict(tq, w, lens, 300, 20, 301, d=32, bits=2)


@pytest.mark.parametrize("cap", [51_200, 51_201])  # the longest slice held on chip, and one more
def test_evict_few_long_slices(tq, cap):
    w = np.random.default_rng(cap).standard_normal((1, 3, cap)).astype(np.float32)
    run_evict(tq, w, [cap], 20_000, 20_000 - 1, 20_000, d=32, bits=2)


# ------------------------------------------------------------------- together

def test_a_generation_with_a_shared_prompt_and_a_bounded_cache(tq):
    """A batch decodes with ragged caches: prompts compressed, every step appends a token, attends
    with weights, and caches that reach their capacity are cut to the budget in a second buffer;
    the attention over what was kept, with the shared prompt before it, matches its definition."""
    import torch
    d, m, bits, B, Hq, Hkv, cap, budget, recent, tp = 128, 64, 3, 3, 8, 2, 48, 24, 6, 70
    pr = Problem(tq, dtype="bf16", d=d, bits=bits, B=B, Hq=Hq, Hkv=Hkv, t_prefix=tp, t_cap=cap, lens=[20, 33, 1], seed=21)
    p, lens, w = pr.p, pr.dlens, torch.zeros(B, Hkv, cap, device="cuda")
    k, v = pr.k, pr.v
    g = torch.Generator(device="cuda").manual_seed(3)
    total = np.zeros((B, Hkv, cap))
    for step in range(20):
        x = torch.randn(2, B * Hkv, d, generator=g, device="cuda").half()
        rec = (*tq.tq_compress_keys(p, x[0]), *tq.tq_compress_values(p, x[1]))
        at = (torch.arange(B * Hkv, device="cuda") * cap + lens.long().repeat_interleave(Hkv))
        for dst, src in zip((*k, *v), rec):
            dst.index_copy_(0, at, src)
        lens += 1
        q = torch.randn(B, Hq, 1, d, generator=g, device="cuda").bfloat16()
        out = tq.tq_attend_weigh(p, q, k, v, lens, Hkv, cap, w)
        # the definition, over the records as they stand
        c = ref.Cache(B * Hkv * cap, d, m, bits, 0)
        c.kc, c.ks, c.vc = (t.cpu().numpy().view(np.uint32) for t in (k[0], k[1], v[0]))
        c.kn, c.kr, c.vn = (t.cpu().numpy() for t in (k[2], k[3], v[1]))
        ln = lens.cpu().numpy()
        want, tol, ws, wtol = ref.attend(q.double().cpu().numpy(), pr.R, pr.S, [(c, cap, False, ln)], Hkv, pr.scale,
                                         2.0 ** -11)
        check(out, want, tol, ref.HALF_STEP["bf16"], step)
        total += ws
        check(w, total, (step + 1) * (wtol + 1e-6), 2.0 ** -20, step)
        both, tol2, _, _ = ref.attend(q.double().cpu().numpy(), pr.R, pr.S,
                                      [(pr.pre, tp, True, None), (c, cap, False, ln)], Hkv, pr.scale, 2.0 ** -11)
        got = tq.tq_attend_shared(p, q, pr.pk, pr.pv, k, v, lens, Hkv, tp, cap)
        check(got, both, tol2, ref.HALF_STEP["bf16"], step)
        if int(ln.max()) == cap - 1:
            before = w.cpu().numpy()
            keep = ref.evict(before, ln, budget, recent)
            k, v, w, kept, lens = tq.tq_evict(p, k, v, w, lens, Hkv, cap, budget, recent, cap)
            w = torch.where(torch.arange(cap, device="cuda") < lens[:, None, None], w, 0.0)
            total2 = np.zeros_like(total)
            for b in range(B):
                for h in range(Hkv):
                    s = keep[b][h]
                    assert kept[b, h, :len(s)].tolist() == s.tolist()
                    assert set(range(int(ln[b]) - min(recent, int(ln[b])), int(ln[b]))) <= set(s.tolist())
                    total2[b, h, :len(s)] = total[b, h, s]
            total = total2
    assert int(lens.max()) < cap


def test_binding_checks(tq):
    import torch
    pr = Problem(tq, dtype="bf16", t_prefix=10, t_cap=20, seed=30)
    w = torch.from_numpy(pr.w0).cuda()
    with pytest.raises(TypeError):
        tq.tq_attend_weigh(pr.p, pr.q.double(), pr.k, pr.v, pr.dlens, 2, 20, w)
    with pytest.raises(TypeError):
        tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, pr.dlens.long(), 2, 20, w)
    with pytest.raises(ValueError):
        tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, pr.dlens, 2, 21, w)      # a larger capacity than the arrays'
    with pytest.raises(ValueError):
        tq.tq_attend_weigh(pr.p, pr.q[..., :64], pr.k, pr.v, pr.dlens, 2, 20, w)
    with pytest.raises(ValueError):
        tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, pr.dlens.cpu(), 2, 20, w)
    with pytest.raises(tq.TQError):
        tq.tq_attend_weigh(pr.p, pr.q, pr.k, pr.v, pr.dlens, 2, 20, w, scratch=w[:1, :1, :1])
    with pytest.raises(ValueError):
        tq.tq_attend_weigh(pr.p, pr.q.repeat(1, 1, 2, 1).transpose(1, 2).contiguous().transpose(1, 2), pr.k, pr.v,
                           pr.dlens, 2, 20, w)
    with pytest.raises(ValueError):
        tq.tq_attend_shared(pr.p, pr.q, pr.pk, pr.pv, pr.k, pr.v, pr.dlens, 2, 11, 20)
    with pytest.raises(ValueError):
        tq.tq_evict(pr.p, pr.k, pr.v, w[:, :, :10].contiguous(), pr.dlens, 2, 20, 5, 1, 5)
    with pytest.raises(tq.TQError):
        tq.tq_evict(pr.p, pr.k, pr.v, w, pr.dlens, 2, 20, 20, 1, 20, out_keys=pr.k, out_values=pr.v)
