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
