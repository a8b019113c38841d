"""Microscaled matrices where a hair decides a code: SwiGLU's values next to the border between two codes."""

import numpy as np
import pytest
import test_gpu_mx as base

from oracle import mx

pytestmark = pytest.mark.gpu

F32 = base.F32


@pytest.fixture
def lib(qw):
    return qw.qw


def _digits(v, bits):
    """Rows of a product's weights, one run of 32 columns for each digit of v (24 bits, most significant first), whose sum by a
    row of ones in the runs' first columns is v exactly: 4-bit digits are e4m3 codes, 2-bit digits e2m1 codes."""
    size = 4 if bits == 8 else 2
    n = 24 // size
    f, ex = np.frexp(np.abs(v))
    whole = np.rint(f * 2.0 ** 24).astype(np.int64)
    assert (whole * 2.0 ** (ex - 24.0) == np.abs(v)).all()
    w = np.zeros((len(v), n * 32))
    for j in range(n):
        digit = (whole >> (24 - size * (j + 1))) & ((1 << size) - 1)
        w[:, 32 * j] = np.sign(v) * digit * 2.0 ** (ex - size * (j + 1.0))
    return w


def _next_to_borders(rng, gates, bits, delta):
    """For each gate a run of 32 features: u in 24 bits so that silu(g) u is `delta` or a little more off the border between two
    codes of the run; the first has the run's largest, off any border."""
    v = np.unique(np.abs(mx.code_values(bits)[np.isfinite(mx.code_values(bits))]))
    mid = (v[1:] + v[:-1]) / 2
    mid = mid[mid >= mx.TOP[bits] / 28]  # 4 binades: u keeps its 24 bits, whatever the border
    s = gates / (1 + np.exp(-gates))
    e = np.floor(np.log2(np.abs(s)))
    y = rng.choice(mid, (len(gates), 32)) * (1 + delta * 1.15 * rng.choice([-1.0, 1.0], (len(gates), 32)))
    y[:, 0] = mx.TOP[bits] * (1 - 2.0 ** -10)
    u = (y / (s / 2.0 ** e)[:, None]).astype(np.float32).astype(np.float64)
    h = s[:, None] * u
    q = np.abs(h / 2.0 ** e[:, None])
    assert (np.abs(q[..., None] / mid - 1).min(-1) >= delta).all()
    return np.repeat(gates, 32), u.reshape(-1), h.reshape(-1)


@pytest.mark.parametrize("T", [1, 3, 16, 40, 64, 70, 300])
@pytest.mark.parametrize("xb,wb,ob", [(8, 8, 8), (8, 4, 8), (4, 4, 8), (8, 8, 4)])
def test_swiglu_next_to_borders(lib, T, xb, wb, ob):
    """Every code is that of silu(g) u where that is 2^-21 relative off a border. The exponential is within one unit of the last
    place (2^-23), the reciprocal within 2^-23, and 1 + e, g r and the product with u are rounded once each (2^-24): 7 2^-24 < 2^-21.
    The sums are exact: each gate and u comes in digits."""
    rng = np.random.default_rng(T)
    gates = -np.concatenate([np.linspace(0.01, 6, 20), np.linspace(6, 88, 30), [-0.5, -3, -17, -60]])
    gates = gates.astype(np.float32).astype(np.float64)
    g, u, h = _next_to_borders(rng, gates, ob, 2.0 ** -21)
    wg, wu = _digits(g, wb), _digits(u, wb)
    ones = np.zeros((T, wg.shape[1]))
    ones[:, ::32] = 1.0
    x, mg, mu = (base.Matrix.of(lib, a, b) for a, b in ((ones, xb), (wg, wb), (wu, wb)))
    assert (mg.held == wg).all() and (mu.held == wu).all()
    for m, want in ((mg, g), (mu, u)):
        np.testing.assert_array_equal(base._linear(lib, x, m, F32).double().cpu().numpy(), np.tile(want, (T, 1)))
    base._swiglu(lib, x, mg, mu, ob).check(*mx.quantize(np.tile(h, (T, 1)), ob))
