"""The training operators' 64-bit forms against differences: every gradient of
training_ref.backward is the slope of <dy, y> in float64.  Runs on the CPU."""
import numpy as np
import pytest

import training_ref as ref


def loss(x, dy, w, wgu, wd):
    i = wd.shape[0]
    gu = x @ wgu
    h = gu[:, :i] * ref.sigmoid(gu[:, :i]) * gu[:, i:]
    return float((w[:, None] * dy * (h @ wd)).sum())


@pytest.mark.parametrize("rows,d,i", [(1, 3, 2), (4, 5, 3)])
def test_gradients_are_slopes(rows, d, i):
    rng = np.random.default_rng(rows + d)
    x, dy, w = rng.standard_normal((rows, d)), rng.standard_normal((rows, d)), rng.standard_normal(rows)
    wgu, wd = rng.standard_normal((d, 2 * i)), rng.standard_normal((i, d))
    gu = x @ wgu
    (dx, _), (dwgu, _), (dwd, _), (dot, _) = ref.backward(x, dy, w, gu[:, :i], gu[:, i:], wgu, wd, "f32")
    eps = 1e-6
    for a, grad in ((x, dx), (wgu, dwgu), (wd, dwd), (w, dot)):
        for at in np.ndindex(a.shape):
            old = a[at]
            a[at] = old + eps
            up = loss(x, dy, w, wgu, wd)
            a[at] = old - eps
            down = loss(x, dy, w, wgu, wd)
            a[at] = old
            # the difference's own error: third derivatives (of size one here) times eps^2, and 2^-52 / eps of the loss
            assert abs((up - down) / (2 * eps) - grad[at]) <= 1e-7 * (1 + abs(grad[at]))


def test_codes_checker_sees_mistakes():
    """A planted mistake in codes, in scales and in their order is found."""
    rng = np.random.default_rng(5)
    v = rng.standard_normal((3, 128))
    s = ref.scales(v)
    q = np.round(v / np.repeat(s, 64, 1)).astype(np.int8)
    zero = np.zeros_like(v)
    ref.check_codes(q, s, v, zero)
    assert np.max(np.abs(ref.values(q, s) - v)) <= 0.5 * s.max() * (1 + 1e-12)
    for bad_q, bad_s in ((q + np.eye(3, 128, 7, dtype=np.int8), s), (q, s * 1.001), (np.roll(q, 64, 1), s)):
        with pytest.raises(AssertionError):
            ref.check_codes(bad_q, bad_s, v, zero)
