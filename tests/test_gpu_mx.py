"""GPU parity of the microscaled matrices' operators (qw_mx_quantize, _read, _rmsnorm, _linear, _swiglu) with
the fp64 oracle.

Quantise, read and rmsnorm are exact: each code and exponent is that of the real number. Products:
see _check_product and _check_swiglu for the tolerances."""

import numpy as np
import pytest

from oracle import mx

pytestmark = pytest.mark.gpu

F16, BF16, F32 = "f16", "bf16", "f32"
TYPES = [F16, BF16, F32]
HALF = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}  # half a step, relative
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}  # half a subnormal step


def _dt(name):
    import torch
    return {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}[name]


def _ty(qw, name):
    return {F16: qw.QW_F16, BF16: qw.QW_BF16, F32: qw.QW_F32}[name]


def _rows(x, dtype, pad=0):
    """A tensor on the GPU whose rows are x's, 16-byte aligned, with NaN up to the next row."""
    import torch
    x = torch.as_tensor(x)
    ld = -(-x.shape[1] // 8) * 8 + pad
    t = torch.full((x.shape[0], ld), float("nan"), dtype=_dt(dtype))
    t[:, :x.shape[1]] = x.to(_dt(dtype))
    return t.cuda()


class Matrix:
    """A matrix in device memory: every byte set, 64 guard bytes after codes and scales."""

    def __init__(self, qw, rows, cols, bits, fill=0xAB):
        import torch
        self.qw, self.rows, self.cols, self.bits = qw, rows, cols, bits
        self.nc, self.ns = qw.qw_mx_code_bytes(bits, rows, cols), qw.qw_mx_scale_bytes(rows, cols)
        self.codes = torch.full((self.nc + 64,), fill, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((self.ns + 64,), fill, dtype=torch.uint8, device="cuda")
        self.view = qw.qw_mx_view(self.codes.data_ptr(), self.scales.data_ptr(), rows, cols, bits)
        self.fill, self.written = fill, False

    @classmethod
    def of(cls, qw, x, bits):
        """The oracle's quantisation of x; scale bytes of rows that are not there are NaN."""
        import torch
        m = cls(qw, x.shape[0], x.shape[1], bits)
        c, e = mx.quantize(x, bits)
        cb, sb = mx.pack(c, e, bits)
        m.codes[:m.nc] = torch.from_numpy(cb).cuda()
        m.scales[:m.ns] = torch.from_numpy(sb).cuda()
        m.held, m.written = mx.values(c, e, bits, x.shape[1]), True
        return m

    def get(self):
        """Codes, exponents (padding included); checks the guards and the scale bytes of rows that are not there."""
        c, s = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        assert (c[self.nc:] == self.fill).all() and (s[self.ns:] == self.fill).all()
        unused = mx.unpack_scales(s[:self.ns], self.cols)[self.rows:]
        assert self.written or (unused == self.fill).all()
        return mx.unpack(c[:self.nc], s[:self.ns], self.rows, self.cols, self.bits)

    def values(self):
        return mx.values(*self.get(), self.bits, self.cols)

    def check(self, codes, e):
        """Equal to the oracle's, values and exponents (the sign of a zero aside), and the padding."""
        c2, e2 = self.get()
        n = e.shape[1]
        np.testing.assert_array_equal(e2[:, :n], e)
        fin = e != mx.NAN_E
        v = mx.code_values(self.bits)
        np.testing.assert_array_equal(v[c2[:, :n]][fin], v[codes][fin])
        assert (c2[:, n:] == 0).all() and (e2[:, n:] == -127).all()
        tail = n * 32 - self.cols
        if tail:
            assert (v[c2[:, n - 1, 32 - tail:]][fin[:, -1]] == 0).all()


@pytest.fixture
def lib(qw):
    return qw.qw


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


SHAPES = [(1, 1), (1, 32), (3, 33), (5, 127), (129, 128), (257, 1000), (64, 2048), (2, 5001), (128, 256)]


def _awkward(rng, rows, cols, dtype):
    """Normal values, with rows of zeros, of powers of two, of ties, of tiny and huge values and of NaN and infinities."""
    import torch
    x = rng.normal(0, 1, (rows, cols)) * 2.0 ** rng.integers(-8, 8, (rows, 1))
    kinds = [lambda n: np.zeros(n), lambda n: 2.0 ** -rng.integers(0, 12, n).astype(float), lambda n: np.resize([6, 5, 3.5, 2.5, 1.75, .25, .75, 1.25], n),
             lambda n: rng.normal(0, 2.0 ** -20, n), lambda n: np.where(np.arange(n) == n // 2, np.nan, 1.0), lambda n: np.where(np.arange(n) == n - 1, -np.inf, 2.0),
             lambda n: np.resize([448, 432, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -21], n), lambda n: np.resize([65504.0, -1e-7], n)]
    if dtype != F16:
        kinds += [lambda n: np.resize([3.3e38, -1.0], n), lambda n: rng.normal(0, 1e-38, n), lambda n: np.resize([2.0 ** -149, 2.0 ** -126], n)]
    for i, k in enumerate(kinds):
        if rows > i + 1:
            x[i + 1] = k(cols)
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(_dt(dtype))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_read(lib, rows, cols, dtype, bits):
    import torch
    x = _awkward(np.random.default_rng(rows * 7 + cols), rows, cols, dtype)
    t = _rows(x, dtype, pad=8)
    m = Matrix(lib, rows, cols, bits)
    lib.qw_mx_quantize(m.view, t.data_ptr(), t.stride(0), _ty(lib, dtype))
    c, e = mx.quantize(x.double().numpy(), bits)
    m.check(c, e)
    for out in TYPES:
        o = torch.full((rows, t.stride(0)), 7.0, dtype=_dt(out), device="cuda")
        lib.qw_mx_read(m.view, o.data_ptr(), o.stride(0), _ty(lib, out))
        want = torch.from_numpy(mx.values(c, e, bits, cols))
        if out == F16:
            want = want.clamp(-65504, 65504)
        assert torch.equal(o[:, :cols].cpu().nan_to_num(nan=123.0), want.float().to(_dt(out)).nan_to_num(nan=123.0))
        assert (o[:, cols:] == 7.0).all()


def test_read_any_scale(lib):
    """Every exponent byte of a matrix that the caller wrote."""
    import torch
    e = (np.arange(256) - 127).reshape(2, 128)
    c = np.random.default_rng(0).integers(0, 127, (2, 128, 32)).astype(np.uint8)
    m = Matrix(lib, 2, 4096, 8)
    cb, sb = mx.pack(c, e, 8)
    m.codes[:m.nc], m.scales[:m.ns] = torch.from_numpy(cb).cuda(), torch.from_numpy(sb).cuda()
    o = torch.empty((2, 4096), device="cuda")
    lib.qw_mx_read(m.view, o.data_ptr(), 4096, lib.QW_F32)
    want = torch.from_numpy(mx.values(c, e, 8, 4096)).float()
    assert torch.equal(o.cpu().nan_to_num(nan=-1.0, posinf=-2.0), want.nan_to_num(nan=-1.0, posinf=-2.0))


def _norm(lib, x, add, w, bits, dtype, add_type, eps=1e-6, want_sum=True, inplace=False, stream=None):
    import torch
    rows, cols = x.shape
    t = _rows(x, dtype)
    a = _rows(add, add_type, pad=8) if add is not None else None
    wt = torch.as_tensor(w).to(torch.bfloat16).cuda()
    s = t if inplace else torch.full((rows, t.stride(0) + 8), 7.0, dtype=_dt(dtype), device="cuda")
    m = Matrix(lib, rows, cols, bits)
    lib.qw_mx_rmsnorm(m.view, t.data_ptr(), t.stride(0), _ty(lib, dtype), a.data_ptr() if a is not None else 0,
                      a.stride(0) if a is not None else 0, _ty(lib, add_type) if a is not None else 0,
                      s.data_ptr() if want_sum else 0, s.stride(0), wt.data_ptr(), eps, stream)
    xs = x.to(_dt(dtype))
    want = xs if add is None else (xs.float() + add.to(_dt(add_type)).float()).to(_dt(dtype))
    torch.cuda.synchronize()
    if want_sum:
        assert torch.equal(s[:, :cols].cpu().nan_to_num(nan=77.0), want.nan_to_num(nan=77.0))
        if not inplace:
            assert (s[:, cols:] == 7.0).all()
    return m, want.double().numpy(), wt.double().cpu().numpy()


def _norm_rows(rng, rows, cols):
    import torch
    x = rng.normal(0, 1, (rows, cols)) * (1 + 7 * (np.arange(cols) % 61 == 7)) * 2.0 ** rng.uniform(-3, 6, (rows, 1))
    return torch.from_numpy(x.astype(np.float32))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,cols,dtype,add", [
    (1, 1, F32, None), (3, 40, F16, BF16), (200, 1024, F32, BF16), (200, 1024, BF16, F32), (65, 1000, BF16, None),
    (7, 2048, F16, F16), (33, 2049, F32, F32), (5, 8192, F32, F16), (3, 16384, BF16, BF16), (2, 16385, F32, BF16), (2, 40000, F16, None)])
def test_rmsnorm(lib, rows, cols, dtype, add, bits):
    import torch
    rng = np.random.default_rng(cols)
    x = _norm_rows(rng, rows, cols)
    a = torch.from_numpy(rng.normal(0, 1, (rows, cols)).astype(np.float32)) if add else None
    w = 1 + 0.1 * rng.normal(0, 1, cols)
    m, s, wf = _norm(lib, x, a, w, bits, dtype, add)
    m.check(*mx.quantize(mx.rmsnorm(s, wf, float(np.float32(1e-6))), bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("cols", [96, 1024, 3000, 20000])
def test_rmsnorm_borders(lib, cols, bits):
    """Rows whose values lie a hair off the border between two codes: s = 1 gives y = w (1 - eps / 2), and the
    weights are the borders. Rounded to fp32 some are on them."""
    import torch
    v = np.unique(np.abs(mx.code_values(bits)[np.isfinite(mx.code_values(bits))]))
    mid = (v[1:] + v[:-1]) / 2
    w = np.resize(mid[mid > 0.01], cols)
    w = torch.from_numpy(w).to(torch.bfloat16).double().numpy()  # exact in bf16
    x = torch.ones((4, cols))
    x[1:] = torch.tensor([2.0, -4.0, 3.0])[:, None]
    for eps in (1e-6, 3e-8, 1e-10):
        m, s, wf = _norm(lib, x, None, w, bits, F32, None, eps=eps)
        np.testing.assert_array_equal(wf, w)
        m.check(*mx.quantize(mx.rmsnorm(s, wf, float(np.float32(eps))), bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("cols", [64, 1024, 20000])
def test_rmsnorm_odd_rows(lib, cols, bits):
    """Zeros, sizes whose squares leave fp32, a NaN, an infinity; no sum, and the sum over x."""
    import torch
    rng = np.random.default_rng(cols)
    x = _norm_rows(rng, 9, cols)
    for i, f in enumerate([0.0, 1e-25, 1e-38, 1e25, 1e-12, 1e18]):
        x[i] *= f / float(x[i].abs().max())
    x[6, cols // 2], x[7, 1] = float("nan"), float("inf")
    w = 1 + 0.1 * rng.normal(0, 1, cols)
    for kw in (dict(), dict(want_sum=False), dict(inplace=True)):
        m, s, wf = _norm(lib, x, None, w, bits, F32, None, **kw)
        with np.errstate(invalid="ignore"):
            m.check(*mx.quantize(mx.rmsnorm(s, wf, float(np.float32(1e-6))), bits))


@pytest.mark.parametrize("rows,cols", [(4099, 200), (4096, 256), (4097, 31)])
def test_rmsnorm_many_short_rows(lib, rows, cols):
    """Rows of one warp, several a CTA: ordinary ones beside ones in doubt, of odd sizes, a NaN."""
    import torch
    rng = np.random.default_rng(cols)
    x = _norm_rows(rng, rows, cols)
    x[5] *= 1e-30
    x[6] *= 1e25
    x[7, 3], x[rows - 1] = float("nan"), 0.0
    a = torch.from_numpy(rng.normal(0, 1, (rows, cols)).astype(np.float32)) * (torch.arange(rows) > 7)[:, None]
    w = 1 + 0.1 * rng.normal(0, 1, cols)
    m, s, wf = _norm(lib, x, a, w, 8, F32, BF16)
    with np.errstate(invalid="ignore"):
        m.check(*mx.quantize(mx.rmsnorm(s, wf, float(np.float32(1e-6))), 8))


@pytest.mark.parametrize("eps", [1e-30, 1.0, 1e20, 1e30, 3e38])
def test_rmsnorm_any_eps(lib, eps):
    """eps far above the squares and far below, rows on both sides of what pairs of floats hold (2^90)."""
    rng = np.random.default_rng(0)
    x = _norm_rows(rng, 8, 1000)
    for i, f in enumerate([1e-11, 1e-3, 1.0, 1e9, 1e13, 3e13, 1e14, 1e18]):
        x[i] *= f / float(x[i].abs().max())
    w = 2.0 ** 60 * (1 + 0.1 * rng.normal(0, 1, 1000))
    m, s, wf = _norm(lib, x, None, w, 8, F32, None, eps=eps)
    m.check(*mx.quantize(mx.rmsnorm(s, wf, float(np.float32(eps))), 8))


@pytest.mark.parametrize("cols", [40, 1027, 20000])
def test_rmsnorm_fp16_sums_stop(lib, cols):
    """fp16 sums beyond 65504 stop there, in what is written and in what is normalised; infinities that were there stay."""
    import torch
    x = torch.full((4, cols), 60000.0)
    x[0], x[1, 5], x[2, 3], x[3, 4] = -1.0, float("inf"), float("nan"), -60000.0
    a = torch.full((4, cols), 9000.0)
    a[3, 4] = -9000.0
    xs, s = x.half().cuda(), torch.empty((4, -(-cols // 8) * 8), dtype=torch.float16, device="cuda")
    t, b = _rows(x, F16), _rows(a, F32)
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    m = Matrix(lib, 4, cols, 8)
    lib.qw_mx_rmsnorm(m.view, t.data_ptr(), t.stride(0), lib.QW_F16, b.data_ptr(), b.stride(0), lib.QW_F32, s.data_ptr(), s.stride(0),
                      w.data_ptr(), 1e-6)
    v = xs.float() + a.cuda()
    want = torch.where(v.isfinite(), v.clamp(-65504, 65504), v).half().cpu()
    assert torch.equal(s[:, :cols].cpu().nan_to_num(nan=7.0, posinf=8.0), want.nan_to_num(nan=7.0, posinf=8.0))
    assert float(want[0, 0]) == 9000.0 and float(want[3, 4]) == -65504.0 and float(want[1, 0]) == 65504.0
    with np.errstate(invalid="ignore"):
        m.check(*mx.quantize(mx.rmsnorm(want.double().numpy(), np.ones(cols), float(np.float32(1e-6))), 8))


def _weights(rng, M, K):
    return rng.normal(0, 1, (M, K)) / np.sqrt(K) * 2.0 ** rng.integers(-3, 3, (M, 1))


def _acts(rng, T, K):
    return rng.normal(0, 1, (T, K)) * (1 + 7 * (np.arange(K) % 61 == 7)) * 2.0 ** rng.integers(-3, 3, (T, 1))


def _sum_error(x, w):
    """Products are exact and a step adds 32 or more of them to an fp32 sum, each addition within a whole step
    (truncation) of the largest magnitude, at most sum|x w|: two a step, and 16 for joining parts."""
    steps = 2 * (-(-x.shape[1] // 32)) + 16
    return steps * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def _check_product(got, x, w, dtype):
    want = x @ w.T
    if dtype == F16:
        want = want.clip(-65504, 65504)
    err = _sum_error(x, w)
    tol = err + HALF[dtype] * (np.abs(want) + err) + TINY[dtype]
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / tol))


FORMATS = [(8, 4), (4, 4), (8, 8)]


def _linear(lib, mx_x, mx_w, dtype, stream=None, status=None, out=None):
    import torch
    T, M = mx_x.rows, mx_w.rows
    st = status if status is not None else _status()
    o = out if out is not None else torch.full((T + 2, -(-M // 8) * 8 + 8), 7.0, dtype=_dt(dtype), device="cuda")
    lib.qw_mx_linear(mx_x.view, mx_w.view, o.data_ptr(), o.stride(0), _ty(lib, dtype), st.data_ptr(), stream)
    if stream is None and status is None:
        assert int(st.item()) == 0
        assert (o[T:] == 7.0).all() and (o[:T, M:] == 7.0).all()
    return o[:T, :M]


@pytest.mark.parametrize("xb,wb", FORMATS)
@pytest.mark.parametrize("T,K,M,dtype", [
    (1, 1, 1, F32), (1, 1024, 300, F16), (2, 32, 127, BF16), (3, 100, 128, F32), (16, 1024, 1024, F16), (17, 129, 129, BF16),
    (31, 256, 255, F16), (33, 384, 256, F32), (64, 640, 257, BF16), (65, 2048, 512, F16), (100, 1000, 1000, F32), (127, 128, 600, F32),
    (128, 512, 640, BF16), (129, 4096, 300, F32), (300, 513, 1025, F16), (700, 96, 2000, BF16), (1, 8192, 256, F32), (5, 2500, 4500, BF16)])
def test_linear(lib, T, K, M, dtype, xb, wb):
    rng = np.random.default_rng(T + K + M)
    x, w = Matrix.of(lib, _acts(rng, T, K), xb), Matrix.of(lib, _weights(rng, M, K), wb)
    got = _linear(lib, x, w, dtype).double().cpu().numpy()
    _check_product(got, x.held, w.held, dtype)


def _device_matrix(lib, rows, cols, bits, seed):
    """A random matrix quantised on the GPU, and a function that reads some of its rows back in 64 bits."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, -(-cols // 8) * 8), generator=gen, device="cuda", dtype=torch.float16)
    m = Matrix(lib, rows, cols, bits)
    lib.qw_mx_quantize(m.view, x.data_ptr(), x.stride(0), lib.QW_F16)
    v = torch.empty_like(x, dtype=torch.float32)
    lib.qw_mx_read(m.view, v.data_ptr(), v.stride(0), lib.QW_F32)
    m.keep, m.written = x, True
    return m, lambda idx: v[torch.as_tensor(idx, device="cuda")][:, :cols].double().cpu().numpy()


@pytest.mark.parametrize("xb,wb", FORMATS)
@pytest.mark.parametrize("T,K,M", [(1, 130, 70000), (16, 260, 45000), (17, 384, 50001), (64, 128, 90001), (65, 300, 30000),
                                   (2600, 260, 2300), (1500, 1100, 4000)])
def test_linear_many_tiles(lib, T, K, M, xb, wb):
    """More tiles than places: CTAs walk several, with their rings and accumulators wrapping. Some columns against 64 bits."""
    x, xr = _device_matrix(lib, T, K, xb, 1)
    w, wr = _device_matrix(lib, M, K, wb, 2)
    for dtype in (F32, BF16):
        got = _linear(lib, x, w, dtype)
        t = np.unique(np.linspace(0, T - 1, 40).astype(int))
        m = np.unique(np.concatenate([np.linspace(0, M - 1, 500).astype(int), np.arange(max(0, M - 140), M)]))
        _check_product(got[t][:, m].double().cpu().numpy(), xr(t), wr(m), dtype)
        assert bool(got.isfinite().all())


@pytest.mark.parametrize("xb,wb", FORMATS)
@pytest.mark.parametrize("T,K,I", [(1, 130, 45000), (16, 256, 40001), (17, 128, 20000), (2600, 260, 1200)])
def test_swiglu_many_tiles(lib, T, K, I, xb, wb):
    x, xr = _device_matrix(lib, T, K, xb, 1)
    g, gr = _device_matrix(lib, I, K, wb, 2)
    u, ur = _device_matrix(lib, I, K, wb, 3)
    m = _swiglu(lib, x, g, u, 8)
    c, e = m.get()
    runs = np.unique(np.concatenate([np.linspace(0, I // 32 - 1, 30).astype(int), [-(-I // 32) - 1]]))
    t = np.unique(np.linspace(0, T - 1, 30).astype(int))
    for j in runs:  # a run of 32 features at a time
        f = np.arange(32 * j, min(32 * j + 32, I))
        part = type("Part", (), {"bits": 8, "values": lambda self: mx.values(c[t][:, j:j + 1], e[t][:, j:j + 1], 8, len(f))})()
        _check_swiglu(part, xr(t), gr(f), ur(f))


@pytest.mark.parametrize("xb,wb", FORMATS)
@pytest.mark.parametrize("T", [2, 40, 200])
def test_linear_nan_stays_in_its_row(lib, T, xb, wb):
    """A NaN run of x spoils its row of the output, one of w its column, and nothing else; a run whose scale is the
    largest or the smallest spoils none."""
    rng = np.random.default_rng(T)
    xf, wf = _acts(rng, T, 300), _weights(rng, 150, 300)
    xf[1, 7], wf[133, 299] = np.nan, np.inf
    x, w = Matrix.of(lib, xf, xb), Matrix.of(lib, wf, wb)
    got = _linear(lib, x, w, F32).double().cpu().numpy()
    bad = np.zeros((T, 150), bool)
    bad[1], bad[:, 133] = True, True
    assert (np.isnan(got) == bad).all()
    keep_t, keep_m = np.arange(T) != 1, np.arange(150) != 133
    _check_product(got[keep_t][:, keep_m], x.held[keep_t], w.held[keep_m], F32)


def test_linear_fp16_stops(lib):
    x, w = Matrix.of(lib, np.full((3, 64), 400.0), 8), Matrix.of(lib, np.stack([np.full(64, 400.0), np.full(64, -400.0)]), 8)
    got = _linear(lib, x, w, F16).float().cpu().numpy()
    np.testing.assert_array_equal(got, np.tile([65504.0, -65504.0], (3, 1)))


def _check_swiglu(m, x, g, u, exact=False):
    """q(h'), h' the fp32 value: |h' - h| follows from the products' errors (|silu'| <= 1.1, |silu(v)| <= |v|) and 2^-20
    relative, 2^-23 |g| more where g < 0 (the exponent -g log2 e is rounded, by 2^-24 relative at most, and log2 e itself by
    2^-26: an error of |g| (2^-24 + 2^-26) in the logarithm of the exponential); half a code's step of h' on top, of the smallest codes half of theirs under a scale below 2 amax / L."""
    got, bits = m.values(), m.bits
    gv, uv, h = x @ g.T, x @ u.T, mx.swiglu(x, g, u)
    eg, eu = (0.0, 0.0) if exact else (_sum_error(x, g), _sum_error(x, u))
    d = 1.1 * eg * (np.abs(uv) + eu) + (np.abs(gv) + eg) * eu + (2.0 ** -20 + 2.0 ** -23 * np.maximum(-gv, 0)) * np.abs(h)
    pad = -h.shape[1] % 32
    top = np.pad(np.abs(h) + d, ((0, 0), (0, pad))).reshape(h.shape[0], -1, 32).max(-1).repeat(32, 1)[:, :h.shape[1]]
    half, small = (2.0 ** -4, 2.0 ** -10) if bits == 8 else (2.0 ** -2, 0.25)
    tol = d + np.maximum(half * (np.abs(h) + d), small * 2 * top / mx.TOP[bits]) + 2.0 ** -140
    assert (np.abs(got - h) <= tol).all(), float(np.max(np.abs(got - h) / tol))
    # a code changes only where h is within d of a border: rarely
    near = np.mean(got != mx.held(h, bits))
    assert near <= 0.005 + 2.0 / h.size, near


def _swiglu(lib, x, g, u, bits, status=None, stream=None, out=None):
    st = status if status is not None else _status()
    m = out or Matrix(lib, x.rows, g.rows, bits)
    lib.qw_mx_swiglu(x.view, g.view, u.view, m.view, st.data_ptr(), stream)
    if status is None:
        assert int(st.item()) == 0
    return m


@pytest.mark.parametrize("xb,wb", FORMATS)
@pytest.mark.parametrize("T,K,M,dtype", [(65, 4096, 1000, BF16), (128, 4100, 260, F32), (100, 8192, 130, F16), (127, 4096, 20001, F32), (128, 16000, 1, BF16)])
def test_linear_long_columns(lib, T, K, M, dtype, xb, wb):
    """65 to 128 rows: shared by clusters of 8, 4, and a stream of more tiles than CTAs."""
    rng = np.random.default_rng(T + K + M)
    x, w = Matrix.of(lib, _acts(rng, T, K), xb), Matrix.of(lib, _weights(rng, M, K), wb)
    _check_product(_linear(lib, x, w, dtype).double().cpu().numpy(), x.held, w.held, dtype)


@pytest.mark.parametrize("xb,wb,ob", [(8, 4, 8), (4, 4, 4), (8, 8, 4), (4, 4, 8)])
@pytest.mark.parametrize("T,K,I", [(17, 8192, 130), (64, 8100, 256), (33, 8192, 4800)])
def test_swiglu_long_columns(lib, T, K, I, xb, wb, ob):
    rng = np.random.default_rng(T + K + I)
    x, g, u = Matrix.of(lib, _acts(rng, T, K), xb), Matrix.of(lib, _weights(rng, I, K), wb), Matrix.of(lib, _weights(rng, I, K), wb)
    _check_swiglu(_swiglu(lib, x, g, u, ob), x.held, g.held, u.held)


@pytest.mark.parametrize("xb,wb,ob", [(8, 4, 8), (4, 4, 4), (8, 8, 8), (8, 4, 4), (4, 4, 8)])
@pytest.mark.parametrize("T,K,I", [(1, 1, 1), (1, 1024, 640), (3, 100, 33), (16, 512, 128), (20, 129, 200), (64, 1024, 384), (65, 640, 129),
                                   (128, 256, 1000), (200, 2048, 256), (300, 96, 2000), (2, 4096, 300)])
def test_swiglu(lib, T, K, I, xb, wb, ob):
    rng = np.random.default_rng(T + K + I)
    x, g, u = Matrix.of(lib, _acts(rng, T, K), xb), Matrix.of(lib, _weights(rng, I, K), wb), Matrix.of(lib, _weights(rng, I, K), wb)
    m = _swiglu(lib, x, g, u, ob)
    _check_swiglu(m, x.held, g.held, u.held)
    c, e = m.get()  # the padding, as the next product reads it
    n = -(-I // 32)
    assert (c[:, n:] == 0).all() and (e[:, n:] == -127).all()
    assert (mx.code_values(ob)[c].reshape(T, -1)[:, I:] == 0).all()


def test_swiglu_nan_row_and_large_gates(lib):
    """A NaN row of x gives NaN runs there only; gates beyond +-88 give u g and 0."""
    xf = np.ones((4, 32))
    xf[2, 3] = np.nan
    gf, uf = np.zeros((64, 32)), np.full((64, 32), 0.5)
    gf[:32], gf[32:] = 4.0, -4.0  # g = 128, -128
    x, g, u = Matrix.of(lib, xf, 8), Matrix.of(lib, gf, 4), Matrix.of(lib, uf, 4)
    v = _swiglu(lib, x, g, u, 8).values()
    assert np.isnan(v[2]).all()
    for t in (0, 1, 3):
        np.testing.assert_array_equal(v[t], np.repeat([2048.0, 0.0], 32))


def test_swiglu_negative_gates(lib):
    """Gates from -2 to -86, up to u = 2^20: SiLU falls to 2^-117 and u's factor keeps; a run holds one gate's size. The sums of 32
    codes of one exponent are exact."""
    rng = np.random.default_rng(5)
    xf, uf = np.ones((5, 32)), 2.0 ** rng.integers(0, 15, (640, 1)) * rng.uniform(0.5, 1, (640, 32))
    gf = -np.linspace(2, 86, 20).repeat(32)[:, None] / 32 * np.ones((1, 32))
    x, g, u = Matrix.of(lib, xf, 8), Matrix.of(lib, gf, 8), Matrix.of(lib, uf, 8)
    _check_swiglu(_swiglu(lib, x, g, u, 8), x.held, g.held, u.held, exact=True)


class Layer:
    """Two branches of a layer as they would be used: attention's output projection, norm, SwiGLU, down, norm."""

    def __init__(self, lib, T, D, A, I, xb, wb, seed=0):
        import torch
        rng = np.random.default_rng(seed)
        self.lib, self.T, self.D, self.A, self.I, self.xb = lib, T, D, A, I, xb
        q = lambda r, c: self._quantize(torch.from_numpy(rng.normal(0, c ** -0.5, (r, c)).astype(np.float32)), wb)  # noqa: E731
        self.wo, self.wg, self.wu, self.wd = q(D, A), q(I, D), q(I, D), q(D, I)
        self.n1, self.n2 = (torch.from_numpy(1 + 0.1 * rng.normal(0, 1, D)).to(torch.bfloat16).cuda() for _ in range(2))
        self.attn = torch.from_numpy(rng.normal(0, 1, (T, A)).astype(np.float32)).half().cuda()
        self.x = torch.from_numpy(rng.normal(0, 4, (T, D)).astype(np.float32)).cuda()
        self.qa, self.q1, self.qh, self.q2 = (Matrix(lib, T, c, xb) for c in (A, D, I, D))
        self.s1, self.s2 = torch.empty_like(self.x), torch.empty_like(self.x)
        self.b1, self.b2 = (torch.empty((T, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.status = _status()
        torch.cuda.synchronize()

    def _quantize(self, x, bits):
        t = _rows(x, BF16)
        m = Matrix(self.lib, x.shape[0], x.shape[1], bits)
        self.lib.qw_mx_quantize(m.view, t.data_ptr(), t.stride(0), self.lib.QW_BF16)
        return m

    def run(self, stream=None):
        L, D, st = self.lib, self.D, self.status.data_ptr()
        L.qw_mx_quantize(self.qa.view, self.attn.data_ptr(), self.A, L.QW_F16, stream)
        L.qw_mx_linear(self.qa.view, self.wo.view, self.b1.data_ptr(), D, L.QW_BF16, st, stream)
        L.qw_mx_rmsnorm(self.q1.view, self.x.data_ptr(), D, L.QW_F32, self.b1.data_ptr(), D, L.QW_BF16, self.s1.data_ptr(), D,
                        self.n1.data_ptr(), 1e-6, stream)
        L.qw_mx_swiglu(self.q1.view, self.wg.view, self.wu.view, self.qh.view, st, stream)
        L.qw_mx_linear(self.qh.view, self.wd.view, self.b2.data_ptr(), D, L.QW_BF16, st, stream)
        L.qw_mx_rmsnorm(self.q2.view, self.s1.data_ptr(), D, L.QW_F32, self.b2.data_ptr(), D, L.QW_BF16, self.s2.data_ptr(), D,
                        self.n2.data_ptr(), 1e-6, stream)

    def outputs(self):
        import torch
        torch.cuda.synchronize()
        return [t.cpu().clone() for t in (self.qa.codes, self.b1, self.s1, self.q1.codes, self.q1.scales[:0], self.qh.codes, self.b2, self.s2, self.q2.codes)]

    def check(self):
        """Each step from what the step before left."""
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        eps = float(np.float32(1e-6))
        self.qa.check(*mx.quantize(f(self.attn), self.xb))
        _check_product(f(self.b1), self.qa.values(), self.wo.values(), BF16)
        np.testing.assert_array_equal(f(self.s1), f(self.x.cpu() + self.b1.cpu().float()))
        self.q1.check(*mx.quantize(mx.rmsnorm(f(self.s1), f(self.n1), eps), self.xb))
        _check_swiglu(self.qh, self.q1.values(), self.wg.values(), self.wu.values())
        _check_product(f(self.b2), self.qh.values(), self.wd.values(), BF16)
        self.q2.check(*mx.quantize(mx.rmsnorm(f(self.s2), f(self.n2), eps), self.xb))
        assert int(self.status.item()) == 0


@pytest.mark.parametrize("xb,wb", FORMATS)
@pytest.mark.parametrize("T", [1, 7, 64, 150, 600])
def test_layer(lib, T, xb, wb):
    layer = Layer(lib, T, 512, 384, 1000, xb, wb, seed=T)
    layer.run()
    layer.check()


@pytest.mark.parametrize("T", [1, 64, 300])
def test_layer_captured_and_repeated(lib, T):
    """Equal bits run to run, from a graph, and with new inputs in a replayed graph."""
    import torch
    layer = Layer(lib, T, 512, 384, 1000, 8, 4, seed=5)
    layer.run()
    first = layer.outputs()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.run(torch.cuda.current_stream())
    for _ in range(3):
        for t in (layer.b1, layer.s1, layer.b2, layer.s2):
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, layer.outputs()))
    layer.x.mul_(2)
    layer.attn.copy_(layer.attn.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    layer.check()


def test_two_streams_and_threads(lib):
    """Two layers at once from two host threads, each on its stream, many times."""
    import threading

    import torch
    layers = [Layer(lib, t, 512, 384, 1000, xb, 4, seed=t) for t, xb in ((200, 8), (30, 4))]
    want = []
    for layer in layers:
        layer.run()
        want.append(layer.outputs())
    errors = []

    def work(layer):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                layer.run(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(layer,)) for layer in layers]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for layer, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(w, layer.outputs()))


def test_beside_a_model(qw):
    """A model's prefill and decode on one stream, a layer of products on another: kernels that share SMs and their
    tensor memory, clusters among them."""
    import threading

    import torch

    import synth
    from gpu_util import Run, engine
    lib = qw.qw
    layers = [Layer(lib, t, 512, 384, 1000, 8, 4, seed=t) for t in (3, 600)]
    want = []
    for layer in layers:
        layer.run()
        want.append(layer.outputs())
    eng = engine(qw, synth.ONE_BLOCK, max_tokens=256, max_batch=16, max_context=512, kv_pages=256)
    r = Run(qw, eng)
    prompt = [list(np.random.default_rng(b).integers(0, synth.ONE_BLOCK.vocab, 16)) for b in range(12)]
    errors = []

    def work():
        try:
            s = torch.cuda.Stream()
            for _ in range(30):
                for layer in layers:
                    layer.run(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    th = threading.Thread(target=work)
    th.start()
    for i in range(4):
        r.prefill(list(range(12)), prompt, debug=False, logits=False, reserve_extra=8)
        for _ in range(4):
            r.decode(list(range(12)), [5] * 12, debug=False, logits=False)
        lib.qw_kv_reset(eng.kv, -1, eng.stream)
    th.join()
    assert not errors
    for layer, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(w, layer.outputs()))
        assert int(layer.status.item()) == 0
    eng.close()


def test_rows_do_not_depend_on_the_others(lib):
    """A row's codes after quantise and norm are those of the row alone; nothing is written without rows."""
    import torch
    x = _norm_rows(np.random.default_rng(3), 300, 777)
    w = np.ones(777)
    whole = _norm(lib, x, None, w, 8, F32, None)[0].get()
    one = _norm(lib, x[133:134], None, w, 8, F32, None)[0].get()
    np.testing.assert_array_equal(whole[0][133], one[0][0])
    np.testing.assert_array_equal(whole[1][133], one[1][0])
    empty = lib.qw_mx_view(0, 0, 0, 777, 8)
    lib.qw_mx_quantize(empty, 0, 0, lib.QW_F16)
    lib.qw_mx_linear(empty, empty, 0, 0, lib.QW_F16, _status().data_ptr())
    torch.cuda.synchronize()


def test_large_offsets(lib):
    """Elements, codes and outputs past 2^32 bytes and 2^31 elements."""
    import torch
    rows, cols = 2_200_000, 1024
    t = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    x = torch.from_numpy(np.random.default_rng(0).normal(0, 1, (300, cols))).half()
    t[-300:] = x.cuda()
    m = Matrix(lib, rows, cols, 8)
    lib.qw_mx_quantize(m.view, t.data_ptr(), cols, lib.QW_F16)
    o = torch.full((rows, cols), 3.0, dtype=torch.float16, device="cuda")
    lib.qw_mx_read(m.view, o.data_ptr(), cols, lib.QW_F16)
    want = torch.from_numpy(mx.held(x.double().numpy(), 8)).half()
    assert torch.equal(o[-300:].cpu(), want) and float(o[:-300].abs().max()) == 0.0
    # its last rows by a few weights: the output's last row starts past 2^31 elements
    w = Matrix.of(lib, _weights(np.random.default_rng(1), 40, cols), 4)
    out = torch.full((rows, 1024), 5.0, dtype=torch.bfloat16, device="cuda")
    st = _status()
    lib.qw_mx_linear(m.view, w.view, out.data_ptr(), 1024, lib.QW_BF16, st.data_ptr())
    got = out[-300:, :40].double().cpu().numpy()
    _check_product(got, mx.held(x.double().numpy(), 8), w.held, BF16)
    assert int(st.item()) == 0 and float(out[:-300, :40].abs().max()) == 0.0 and bool((out[:, 40:] == 5.0).all())
