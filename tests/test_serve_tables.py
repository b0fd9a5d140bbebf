"""How near fp16 operand tables come to the centroids, for both laws: the bounds that the serving calls
document.  (The search of the library, restated: of 1024 scales that put the largest centroid on an fp16
number in [8, 16), the one with the least squared error by cell mass.)"""
import numpy as np
import pytest

import oracle


def half(v):
    return np.asarray(v, np.float32).astype(np.float16).astype(np.float64)


def table_errors(dim, bits, law):
    """Largest relative error of a centroid (hi alone, hi + lo)."""
    b, c = (np.asarray(t, np.float64) for t in oracle.codebook_f32(dim, bits, law=law))
    h = len(c) // 2
    mag = c[h:]
    lo = np.concatenate([[0.0], b[h:]])[:h]
    up = np.concatenate([b[h:], [2 * mag[-1] - lo[-1]]])
    mass = (up - lo) * np.exp(-0.5 * dim * mag ** 2)
    scale = mag[-1] / (8 * (1 + np.arange(1024) / 1024))
    e = ((mag / scale[:, None] - half(mag / scale[:, None])) * scale[:, None]) ** 2 @ mass
    s = np.float64(np.float32(scale[e.argmin()]))
    hi = half(mag / s)
    return np.abs(hi * s / mag - 1).max(), np.abs((hi + half(mag / s - hi)) * s / mag - 1).max()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("law,bits,hi_bound", [
    ("gaussian", 1, 2.0 ** -23), ("gaussian", 2, 2.0 ** -21), ("gaussian", 3, 3.1e-5), ("gaussian", 4, 2.0 ** -11),
    ("beta", 1, 2.0 ** -23), ("beta", 2, 2.0 ** -19), ("beta", 3, 5e-5), ("beta", 4, 2.0 ** -11)])
def test_documented_bounds(law, bits, hi_bound, dim):
    hi, both = table_errors(dim, bits, law)
    assert hi <= hi_bound and both <= 2.0 ** -20
