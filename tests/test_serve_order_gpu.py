"""Long runs of the kernels that hand results to one another inside a launch or from launch to launch:
against the 64-bit definition, and the same bits every time."""
import numpy as np
import pytest

from . import serve_ref as ref
from .test_serve_gpu import OPERAND, Problem, check, tq  # noqa: F401  (tq: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,bits", [(64, 2), (64, 4), (128, 3), (256, 2), (256, 4)])
def test_many_tiles_of_one_prefix(tq, d, bits):  # noqa: F811
    """One KV head and 37 rows over some 130 splits of five tiles and more each: every tile's scores take
    the place of the weights of an earlier one (two score buffers up to d = 128, one at 256)."""
    import torch
    pr = Problem(tq, dtype="bf16", d=d, bits=bits, B=1, Hq=37, Hkv=1, t_prefix=148 * 128 * 5 + 77, t_cap=0, seed=71)
    got = pr.shared(tq)
    for _ in range(20):
        assert torch.equal(got, pr.shared(tq))
    want, tol, _, _ = pr.reference(OPERAND["bf16"])
    check(got, want, tol, ref.HALF_STEP["bf16"], (d, bits))
    # ... and of the size that rounding gives: the output's own, 2^-8 / sqrt(3) of it in the root mean
    # square, and those of queries, keys, weights and values, 2^-11 / sqrt(3) each of sums of random signs
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.sqrt((err ** 2).mean()) <= 2.0 ** -8 * np.sqrt((want ** 2).mean())


@pytest.mark.parametrize("d,Hq,dtype", [(128, 8, "bf16"), (256, 4, "f16"), (64, 2, "f32"), (128, 2, "f16")])
def test_calls_that_follow_on_one_scratch(tq, d, Hq, dtype):  # noqa: F811
    """Calls with other queries and lengths in turn on one scratch, none waited for: each launch of a call
    reads what this call's preparation wrote, never what the call before left in its place."""
    import torch
    B, Hkv, tp, cap = 24, 2, 4000, 300
    rng = np.random.default_rng(d)
    pr = Problem(tq, dtype=dtype, d=d, B=B, Hq=Hq, Hkv=Hkv, t_prefix=tp, t_cap=cap, seed=72)
    need = max(tq.tq_attend_shared_scratch_bytes(pr.p, pr.q.dtype, B, Hq, Hkv, 1, tp, cap),
               tq.tq_attend_weigh_scratch_bytes(pr.p, pr.q.dtype, B, Hq, Hkv, 1, cap))
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    w0 = torch.from_numpy(pr.w0).cuda()
    sets = []
    for k in range(4):
        lens = rng.integers(0, cap + 1, B) if k else np.zeros(B)
        lens = torch.from_numpy(lens.astype(np.int32)).cuda()
        q = (pr.q * (1 + 3 * k)).contiguous()
        pr.q, pr.dlens, w = q, lens, w0.clone()
        sets.append((q, lens, pr.shared(tq), pr.weigh(tq, w), w))
        torch.cuda.synchronize()
    got = []
    for i in range(60):
        pr.q, pr.dlens = sets[i % 4][:2]
        w = w0.clone()
        got.append((pr.shared(tq, scratch=scratch), pr.weigh(tq, w, scratch=scratch), w))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for a, b in zip(g, sets[i % 4][2:]):
            assert torch.equal(a, b), i
