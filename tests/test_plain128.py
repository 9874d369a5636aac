"""The plain definitions the kernels with 128-element scales are compared with:
their FP8 codes against torch's conversions, the norm's gradient against
differences."""

import numpy as np
import pytest
import torch

import plain128 as P

TORCH = {1: torch.float8_e4m3fn, 2: torch.float8_e5m2}


@pytest.mark.parametrize("fmt", [1, 2])
def test_every_code_decodes_as_torch_does(fmt):
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(TORCH[fmt]).double().numpy()
    assert np.array_equal(P.decode(c, fmt), want, equal_nan=True)


@pytest.mark.parametrize("fmt", [1, 2])
def test_every_code_and_every_tie_encodes(fmt):
    """Codes map to themselves; halfway points go to the even code; floats just
    beside them to the nearer one."""
    c = np.arange(0x7F if fmt == 1 else 0x7C, dtype=np.uint8)
    v = P.decode(c, fmt)
    for sign in (1.0, -1.0):
        bit = 0x80 if sign < 0 else 0
        assert np.array_equal(P.encode(sign * v, fmt), c | bit)
        mid = (v[:-1] + v[1:]) / 2
        even = np.where(c[:-1] % 2 == 0, c[:-1], c[1:])
        assert np.array_equal(P.encode(sign * mid, fmt), even | bit)
        assert np.array_equal(P.encode(sign * mid * (1 + 2 ** -23), fmt), c[1:] | bit)
        assert np.array_equal(P.encode(sign * mid * (1 - 2 ** -23), fmt), c[:-1] | bit)
    x = np.random.default_rng(0).standard_normal(4096).astype(np.float32) * 30
    want = torch.from_numpy(x).to(TORCH[fmt]).view(torch.uint8).numpy()
    assert np.array_equal(P.encode(x, fmt), want)


@pytest.mark.parametrize("fmt", [1, 2])
def test_power_of_two_scales_hold_the_maximum_and_no_smaller_one_does(fmt):
    rng = np.random.default_rng(1)
    a = np.concatenate([2.0 ** rng.uniform(-100, 100, 1000), P.MAXV[fmt] * 2.0 ** np.arange(-20, 20),
                        np.nextafter(P.MAXV[fmt] * 2.0 ** np.arange(-20, 20), np.inf)])
    s = P.scale_of(a, fmt, True).astype(np.float64)
    assert np.all(np.frexp(s)[0] == 0.5)
    assert np.all(a <= P.MAXV[fmt] * s) and np.all(a > P.MAXV[fmt] * s / 2)
    assert P.scale_of(np.array([0.0]), fmt, True)[0] == P.TINY


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, w, gy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    eps, d = 1e-3, 1e-6
    gh, gw = P.norm_bwd(gy, x, w, eps, None)

    def loss(x, w):
        return (P.norm(x, None, w, eps)[1] * gy).sum()

    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = d
            # central differences: error O(d^2) and rounding 2^-52 / d
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - gh[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros_like(w)
        e[j] = d
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - gw[j]) < 1e-7
