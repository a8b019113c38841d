"""The microscaled matrices' oracle against closed forms and torch's e4m3 conversion, and what the
library's calls refuse. No GPU: every refused call returns before it touches a device."""

import ctypes

import numpy as np
import pytest

from oracle import mx


def test_code_values():
    np.testing.assert_array_equal(mx.code_values(4), [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
    import torch
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(mx.code_values(8), v)


def test_nearest_goes_to_even():
    y = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 0.2501, -2.5, -0.1])
    np.testing.assert_array_equal(mx.code_values(4)[mx.nearest(y, 4)], [0, 1, 1, 2, 2, 4, 4, 6, 0.5, -2, 0])
    import torch
    y = np.random.default_rng(0).normal(0, 60, 4000).clip(-448, 448).astype(np.float32)
    y = np.concatenate([y, [0, 2.0 ** -10, 2.0 ** -9, 3 * 2.0 ** -10, 17, 19, 21, 447, 448, 432]]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(mx.code_values(8)[mx.nearest(y.astype(np.float64), 8)], want)


@pytest.mark.parametrize("bits,top", [(8, 448.0), (4, 6.0)])
def test_exponent_is_the_smallest(bits, top):
    x = np.zeros((6, 32))
    x[0, 3], x[1, 3], x[2, 3] = top, np.nextafter(top, 1e9), -top * 2.0 ** -20
    x[3, 0], x[4, 0] = 2.0 ** -149, np.inf
    e = mx.quantize(x, bits)[1][:, 0]
    np.testing.assert_array_equal(e, [0, 1, -20, -127, mx.NAN_E, -127])
    r = np.random.default_rng(1).normal(0, 1, (50, 40)) * 2.0 ** np.arange(-25, 25)[:, None]
    c, e = mx.quantize(r, bits)
    a = np.abs(np.pad(r, ((0, 0), (0, 24))).reshape(50, 2, 32)).max(-1)
    assert (a <= top * 2.0 ** e).all() and (a > top * 2.0 ** (e - 1.0)).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_held_values_are_near_and_held_again(bits):
    x = np.random.default_rng(2).normal(0, 1, (9, 77))
    h = mx.held(x, bits)
    a = np.abs(np.pad(x, ((0, 0), (0, 19))).reshape(9, 3, 32)).max(-1).repeat(32, 1)[:, :77]
    step = 2.0 ** -4 if bits == 8 else 2.0 ** -2  # half a code's step, and half the smallest step under the run's scale
    small = 2.0 ** -10 * 2 / 448 if bits == 8 else 0.25 * 2 / 6
    assert (np.abs(h - x) <= np.maximum(step * np.abs(x), small * a)).all()
    np.testing.assert_array_equal(mx.held(h, bits), h)


@pytest.mark.parametrize("rows,cols,bits", [(1, 1, 8), (130, 129, 4), (257, 300, 8)])
def test_pack_and_unpack(rows, cols, bits):
    x = np.random.default_rng(rows).normal(0, 1, (rows, cols))
    c, e = mx.quantize(x, bits)
    cb, sb = mx.pack(c, e, bits)
    atoms = -(-cols // 128)
    assert cb.size == rows * atoms * 16 * bits and sb.size == -(-rows // 128) * atoms * 512
    c2, e2 = mx.unpack(cb, sb, rows, cols, bits)
    np.testing.assert_array_equal(c2[:, :e.shape[1]], c)
    np.testing.assert_array_equal(e2[:, :e.shape[1]], e)
    assert (c2[:, e.shape[1]:] == 0).all() and (e2[:, e.shape[1]:] == -127).all()
    # the documented place of one exponent
    r, j = rows - 1, e.shape[1] - 1
    assert sb.reshape(-1, atoms, 512)[r // 128, j // 4, 16 * (r % 32) + 4 * (r // 32 % 4) + j % 4] == e[r, j] + 127


def test_norm_and_products_closed_forms():
    np.testing.assert_allclose(mx.rmsnorm(np.full((1, 8), 3.0), 2.0, 7.0), 2 * 3 / 4 * np.ones((1, 8)))
    x, g, u = np.array([[1.0, 2.0]]), np.array([[0.0, 0.0], [1.0, 1.0]]), np.array([[1.0, 1.0], [1.0, 0.0]])
    np.testing.assert_allclose(mx.swiglu(x, g, u), [[0.0, 3 / (1 + np.exp(-3))]])
    np.testing.assert_allclose(mx.linear(x, u), [[3.0, 1.0]])


# ---- refusals ---------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def qw():
    import decode_qwen3_decoder_gb300 as pkg
    pkg._build_lib()
    pkg.qw.load()
    return pkg.qw


P = 4096  # an aligned address that no refused call touches


def _m(qw, **kw):
    a = dict(codes_ptr=P, scales_ptr=P, rows=3, cols=256, bits=8)
    a.update(kw)
    return qw.qw_mx_view(**a)


def _ref(m):
    return None if m is None else ctypes.byref(m)


BAD = [(dict(bits=6), -7), (dict(bits=0), -7), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=(1 << 20) + 1), -1),
       (dict(rows=(1 << 31) - 1, cols=1 << 20), -1), (dict(codes_ptr=0), -1), (dict(scales_ptr=0), -1),
       (dict(codes_ptr=P + 16), -1), (dict(scales_ptr=P + 16), -1)]


def test_bytes(qw):
    assert qw.qw_mx_code_bytes(8, 3, 1) == 384 and qw.qw_mx_code_bytes(4, 3, 129) == 384
    assert qw.qw_mx_scale_bytes(128, 128) == 512 and qw.qw_mx_scale_bytes(129, 129) == 2048
    assert [qw.qw_mx_code_bytes(b, r, c) for b, r, c in ((6, 1, 1), (8, -1, 1), (8, 1, 0), (8, 1, 1 << 21), (8, 0, 5))] == [0] * 5
    assert qw.qw_mx_code_bytes(8, 1 << 24, 1 << 20) == 1 << 44
    assert qw.qw_mx_scale_bytes(-1, 1) == qw.qw_mx_scale_bytes(1, 0) == 0


@pytest.mark.parametrize("name", ["qw_mx_quantize", "qw_mx_read"])
def test_quantize_and_read_refuse(qw, name):
    def call(m, x=P, ld=256, dtype=0):
        return getattr(qw.load(), name)(_ref(m), x, ld, dtype, None)
    for kw, want in BAD:
        assert call(_m(qw, **kw)) == want, kw
        assert "mx_" in qw.qw_last_error()
    for kw in (dict(x=None), dict(x=P + 8), dict(ld=255), dict(ld=252), dict(ld=260), dict(ld=258, dtype=2), dict(dtype=3), dict(dtype=-1)):
        assert call(_m(qw), **kw) == -1, kw
    assert call(None) == -1
    assert call(_m(qw, rows=0, codes_ptr=0, scales_ptr=0), x=None) == 0  # nothing to do


def test_rmsnorm_refuses(qw):
    def call(m, **kw):
        a = dict(x=P, ld_x=256, x_dtype=2, add=P + 1024, ld_add=256, add_dtype=1, sum=P, ld_sum=256, w=P, eps=1e-6)
        a.update(kw)
        return qw.load().qw_mx_rmsnorm(_ref(m), a["x"], a["ld_x"], a["x_dtype"], a["add"], a["ld_add"], a["add_dtype"],
                                       a["sum"], a["ld_sum"], a["w"], a["eps"], None)
    for kw, want in BAD:
        assert call(_m(qw, **kw)) == want, kw
    for kw in (dict(x=None), dict(x=P + 4), dict(ld_x=255), dict(ld_x=258), dict(x_dtype=7), dict(add=P + 2), dict(ld_add=252),
               dict(add_dtype=5), dict(sum=P + 8), dict(ld_sum=128), dict(ld_sum=260), dict(sum=P + 1024), dict(w=None),
               dict(w=P + 2), dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(_m(qw), **kw) == -1, kw
        assert "mx_rmsnorm" in qw.qw_last_error()
    assert call(_m(qw, rows=0), x=None, sum=None, w=None) == 0


def test_linear_refuses(qw):
    def call(x, w, **kw):
        a = dict(out=P, ld=8, dtype=0, status=P)
        a.update(kw)
        return qw.load().qw_mx_linear(_ref(x), _ref(w), a["out"], a["ld"], a["dtype"], a["status"], None)
    for kw, want in BAD:
        assert call(_m(qw, **kw), _m(qw)) == want, kw
        assert call(_m(qw), _m(qw, **kw)) == want, kw
    assert call(None, _m(qw)) == call(_m(qw), None) == -1
    assert call(_m(qw, cols=255), _m(qw)) == -1
    assert call(_m(qw, bits=4), _m(qw)) == -7
    for kw in (dict(out=None), dict(out=P + 8), dict(ld=2), dict(ld=12), dict(ld=6, dtype=2), dict(dtype=4), dict(status=None)):
        assert call(_m(qw), _m(qw), **kw) == -1, kw
        assert "mx_linear" in qw.qw_last_error()
    assert call(_m(qw, rows=0), _m(qw), out=None) == 0
    assert call(_m(qw), _m(qw, rows=0), out=None) == 0
    big = dict(rows=(1 << 31) - 1, cols=128)
    assert call(_m(qw, **big), _m(qw, **big), ld=1 << 31) == -7


def test_swiglu_refuses(qw):
    def call(x, g, u, o, status=P):
        return qw.load().qw_mx_swiglu(_ref(x), _ref(g), _ref(u), _ref(o), status, None)
    ok = lambda: [_m(qw, rows=5), _m(qw, rows=7), _m(qw, rows=7), _m(qw, rows=5, cols=7)]  # noqa: E731
    for i in range(4):
        for kw, want in BAD:
            a = ok()
            base = dict(rows=a[i].rows, cols=a[i].cols)
            base.update(kw)
            a[i] = _m(qw, **base)
            assert call(*a) == want, (i, kw)
        a = ok()
        a[i] = None
        assert call(*a) == -1
    for i, kw in ((0, dict(rows=5, cols=200)), (1, dict(rows=6)), (2, dict(rows=7, cols=200)), (2, dict(rows=7, bits=4)),
                  (3, dict(rows=4, cols=7)), (3, dict(rows=5, cols=8))):
        a = ok()
        a[i] = _m(qw, **kw)
        assert call(*a) == -1, (i, kw)
        assert "mx_swiglu" in qw.qw_last_error()
    a = ok()
    a[0] = _m(qw, rows=5, bits=4)
    assert call(*a) == -7
    a = ok()
    a[1] = a[2] = _m(qw, rows=0)
    assert call(*a) == -1
    assert call(*ok(), status=None) == -1
    a = ok()
    a[0], a[3] = _m(qw, rows=0), _m(qw, rows=0, cols=7)
    assert call(*a) == 0
