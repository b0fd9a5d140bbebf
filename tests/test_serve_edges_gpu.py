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
