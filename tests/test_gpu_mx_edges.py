"""Microscaled matrices where a hair decides a code: SwiGLU's values and RMSNorm's next to the border between two
codes, runs that are tiny or huge beside their row."""

import numpy as np
import pytest
import test_gpu_mx as base

from oracle import mx

pytestmark = pytest.mark.gpu

F32, BF16 = base.F32, base.BF16


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
    y = rng.choice(mid, (len(gates), 32)) * (1 + (1.02 * delta + 2.0 ** -24) * rng.choice([-1.0, 1.0], (len(gates), 32)))
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
    place (2^-23), the reciprocal within 2^-23, and 1 + e, the quotient and the product with u are rounded once each (2^-24).
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


@pytest.mark.parametrize("T", [2, 50, 200])
@pytest.mark.parametrize("xb,wb,ob", [(8, 8, 8), (8, 4, 4), (4, 4, 8)])
def test_swiglu_rounds_as_fp32(lib, T, xb, wb, ob):
    """The same 5 2^-24 off a border: the exponential 2^-23, and one rounding each of the sum, the quotient and the product. Gates of
    both signs."""
    rng = np.random.default_rng(T + 1)
    gates = np.concatenate([-np.geomspace(1e-3, 88, 40), np.geomspace(1e-3, 60, 30)]).astype(np.float32).astype(np.float64)
    g, u, h = _next_to_borders(rng, gates, ob, 5 * 2.0 ** -24)
    wg, wu = _digits(g, wb), _digits(u, wb)
    ones = np.zeros((T, wg.shape[1]))
    ones[:, ::32] = 1.0
    x, mg, mu = (base.Matrix.of(lib, a, b) for a, b in ((ones, xb), (wg, wb), (wu, wb)))
    base._swiglu(lib, x, mg, mu, ob).check(*mx.quantize(np.tile(h, (T, 1)), ob))


@pytest.mark.parametrize("T", [2, 50, 200])
@pytest.mark.parametrize("xb,wb", base.FORMATS)
def test_swiglu_no_less_exact_than_fp32(lib, T, xb, wb):
    """Values as near to borders as u's 24 bits allow, where any rounding may decide: as many codes are those of the 64-bit values as
    with fp32 arithmetic on the same sums (a hundredth more may miss: where the two round differently, it is chance which is right)."""
    import torch
    rng = np.random.default_rng(T + 2)
    gates = np.concatenate([-np.geomspace(1e-2, 80, 300), np.geomspace(1e-2, 10, 100)]).astype(np.float32).astype(np.float64)
    g, u, h = _next_to_borders(rng, gates, 8, 0.0)
    wg, wu = _digits(g, wb), _digits(u, wb)
    ones = np.zeros((T, wg.shape[1]))
    ones[:, ::32] = 1.0
    x, mg, mu = (base.Matrix.of(lib, a, b) for a, b in ((ones, xb), (wg, wb), (wu, wb)))
    got = base._swiglu(lib, x, mg, mu, 8).values()
    gt, ut = (torch.from_numpy(v).float().cuda() for v in (g, u))
    plain = (gt / (1 + torch.exp(-gt)) * ut).double().cpu().numpy()
    want, plain = mx.held(h[None], 8)[0], mx.held(plain[None], 8)[0]
    miss, most = (got != want).mean(), (plain != want).mean()
    assert (got == got[0]).all() and miss <= most + 0.01, (miss, most)


def _check_norm(lib, x, add, w, bits, dtype, add_type, eps=1e-6, **kw):
    """Codes and exponents are those of the real numbers; a |y| above fp32's range makes its run NaN."""
    m, s, wf = base._norm(lib, x, add, w, bits, dtype, add_type, eps=eps, **kw)
    y = mx.rmsnorm(s, wf, float(np.float32(eps)))
    m.check(*mx.quantize(np.where(np.abs(y) > 3.4028234663852886e38, np.inf, y), bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("cols", [96, 1024, 3000, 10000, 20000])
def test_rmsnorm_tiny_runs(lib, cols, bits):
    """Runs that are tiny beside their row, each value as near to a border between two codes of 2^-127 as an fp32 x can be: the
    products by 1 / sqrt are subnormal, or their roundings' rests are."""
    import torch
    rng = np.random.default_rng(cols)
    rows = 6
    x = base._norm_rows(rng, rows, cols).double().numpy()
    tiny = np.arange(cols) // 32 % 3 == 1
    x[:, tiny] = 0.0
    w = np.ones(cols)
    w[32:64] = 2.0 ** -20  # and where it is the weight that makes them tiny
    step = 2.0 ** -127 * (2.0 ** -9 if bits == 8 else 0.5)
    for r in range(rows):
        rstd = 1 / np.sqrt((x[r] * x[r]).mean() + float(np.float32(1e-6)))  # the tiny runs add nothing to it in 64 bits
        n = tiny.sum()
        border = (rng.integers(0, 8, (n, 200)) + 0.5) * step
        c = border / rstd / w[tiny][:, None]
        c32 = c.astype(np.float32).astype(np.float64)
        off = np.abs(c32 / c - 1)
        best = off.argmin(1)
        x[r, tiny] = c32[np.arange(n), best] * rng.choice([-1.0, 1.0], n)
    x[1, tiny] *= 2.0 ** rng.integers(0, 60)  # and a row whose tiny runs are less so
    _check_norm(lib, torch.from_numpy(x.astype(np.float32)), None, w, bits, F32, None)
    b = base._norm_rows(rng, rows, cols).to(torch.bfloat16)  # sums that cancel to a tiny rest, over x and unwritten
    b[:, torch.from_numpy(tiny)] = 0
    for kw in (dict(inplace=True), dict(want_sum=False)):
        _check_norm(lib, torch.from_numpy(x.astype(np.float32)), b.float(), w, bits, F32, BF16, **kw)
    xb = torch.from_numpy(x).float().to(torch.bfloat16).float()
    _check_norm(lib, xb, None, w, bits, BF16, None)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("cols", [96, 1024, 3000, 20000])
def test_rmsnorm_huge_and_tiny_weights(lib, cols, bits):
    """Weights from 2^-133 to 2^127 before values from 2^-149 to the row's largest: y = 2^-17 with s / sqrt subnormal, y next to the
    end of fp32 and beyond it."""
    import torch
    rng = np.random.default_rng(cols)
    x = base._norm_rows(rng, 8, cols).double().numpy()
    run = np.arange(cols) // 32 % 6
    w = 1 + 0.1 * rng.normal(0, 1, cols)
    w[run == 1] *= 2.0 ** 120
    x[:, run == 1] = rng.integers(-5000, 5000, (8, (run == 1).sum())) * 2.0 ** -149
    w[run == 2] *= 2.0 ** rng.integers(-130, -20, (run == 2).sum()).astype(float)
    w[run == 4] *= 2.0 ** 77
    x[:, run == 4] *= 2.0 ** -100
    w[0] = 2.0 ** 127
    if cols > 200:
        w[64:96] = 2.0 ** 126
    w = torch.from_numpy(w).to(torch.bfloat16).double().numpy()
    _check_norm(lib, torch.from_numpy(x.astype(np.float32)), None, w, bits, F32, None)


@pytest.mark.parametrize("bits", [8, 4])
def test_rmsnorm_end_of_fp32(lib, bits):
    """Rows of equal values, y = w s / sqrt(s^2 + eps): the largest |y| some 2^-24 around fp32's largest number."""
    import torch
    w = np.zeros(128)
    w[0], w[40] = 2.0 ** 127 * (2 - 2.0 ** -7), 2.0 ** 127  # the largest bf16: y up to it, below fp32's largest
    x = np.zeros((64, 128))
    # y_0 = w_0 x_0 / sqrt(mean): mean = (x_0^2 + x_40^2) / 128; x_40 sets how far y_0 is from the end
    end = 3.4028234663852886e38
    for r in range(64):
        x[r, 0] = 1.0
        want = end * (1 + (r - 32) * 2.0 ** -25)
        x[r, 40] = np.sqrt(128 * (w[0] / want) ** 2 - 1)
    x = torch.from_numpy(x.astype(np.float32))
    _check_norm(lib, x, None, w, bits, F32, None, eps=1e-20)


def test_operands_in_one_buffer(lib):
    """Column slices of one buffer share no element: x, the branch, the sum and a product's output side by side, and codes next to
    one another."""
    import torch
    rng = np.random.default_rng(0)
    T, D = 70, 256
    buf = torch.from_numpy(rng.normal(0, 1, (T, 4 * D))).float().cuda()
    x, add, s, o = (buf[:, D * i:D * (i + 1)] for i in range(4))
    want = (x + add).cpu()
    nc, ns = lib.qw_mx_code_bytes(8, T, D), lib.qw_mx_scale_bytes(T, D)
    codes, scales = torch.empty(2 * nc, dtype=torch.uint8, device="cuda"), torch.empty(2 * ns, dtype=torch.uint8, device="cuda")
    a, b = (lib.qw_mx_view(codes.data_ptr() + nc * i, scales.data_ptr() + ns * i, T, D, 8) for i in range(2))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    lib.qw_mx_rmsnorm(a, x.data_ptr(), 4 * D, lib.QW_F32, add.data_ptr(), 4 * D, lib.QW_F32, s.data_ptr(), 4 * D, w.data_ptr(), 1e-6)
    m = base.Matrix.of(lib, rng.normal(0, 0.1, (D, D)), 8)
    st = base._status()
    lib.qw_mx_linear(a, m.view, o.data_ptr(), 4 * D, lib.QW_F32, st.data_ptr())
    lib.qw_mx_swiglu(a, m.view, m.view, b, st.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(s.cpu(), want) and int(st.item()) == 0
    h = mx.values(*mx.quantize(mx.rmsnorm(want.double().numpy(), 1.0, float(np.float32(1e-6))), 8), 8, D)
    base._check_product(o.double().cpu().numpy(), h, m.held, F32)


@pytest.mark.parametrize("xb,wb", base.FORMATS)
@pytest.mark.parametrize("T", [2, 60, 120])
def test_tiles_around_what_clusters_fit(lib, T, xb, wb):
    """128 rows of w a tile, shared by as many CTAs as all tiles get at once: around 15, 36, 74 and 152 tiles."""
    K = 4096 if xb == 4 else 2100
    x, xr = base._device_matrix(lib, T, K, xb, 1)
    for tiles in (14, 15, 16, 18, 19, 20, 30, 31, 36, 37, 38, 39, 72, 73, 75, 76, 77, 152, 153):
        M = 128 * tiles - 5
        w, wr = base._device_matrix(lib, M, K, wb, tiles)
        m = np.unique(np.concatenate([np.arange(0, M, 97), np.arange(M - 130, M)]))
        base._check_product(base._linear(lib, x, w, F32)[:, m].double().cpu().numpy(), xr(np.arange(T)), wr(m), F32)


def test_first_calls_are_captured(qw):
    """A process whose first products are captured: what the calls ask of the device once is asked under capture."""
    import os
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import decode_qwen3_decoder_gb300 as pkg
import test_gpu_mx as base
pkg._build_lib()
lib = pkg.qw
lib.load()
rng = np.random.default_rng(0)
graphs = []
for T, K, M in ((2, 2048, 1200), (100, 2048, 2100), (200, 256, 300)):
    x, w = base.Matrix.of(lib, rng.normal(0, 1, (T, K)), 8), base.Matrix.of(lib, rng.normal(0, 1, (M, K)), 8)
    out, st = torch.zeros((T, -(-M // 8) * 8), device="cuda"), base._status()
    h = base.Matrix(lib, T, M, 8)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream()
        lib.qw_mx_linear(x.view, w.view, out.data_ptr(), out.stride(0), lib.QW_F32, st.data_ptr(), s)
        lib.qw_mx_swiglu(x.view, w.view, w.view, h.view, st.data_ptr(), s)
    graphs.append((g, x, w, out, st, h, M))
for g, x, w, out, st, h, M in graphs:
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    base._check_product(out[:, :M].double().cpu().numpy(), x.held, w.held, "f32")
    base._check_swiglu(h, x.held, w.held, w.held)
print("captured")
"""
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code % (os.path.dirname(tests), tests)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def _with_scales(lib, codes, exps, bits):
    """A matrix of codes [rows, runs, 32] under any exponents [rows, runs]."""
    import torch
    m = base.Matrix(lib, codes.shape[0], codes.shape[1] * 32, bits)
    cb, sb = mx.pack(codes, exps, bits)
    m.codes[:m.nc], m.scales[:m.ns] = torch.from_numpy(cb).cuda(), torch.from_numpy(sb).cuda()
    m.held, m.written = mx.values(codes, exps, bits, m.cols), True
    return m


@pytest.mark.parametrize("xb,wb", base.FORMATS)
@pytest.mark.parametrize("T", [1, 16, 60, 200])
def test_linear_any_scale(lib, T, xb, wb):
    """Codes that are not 0 under the smallest and largest powers of two, 2^-127 and 2^127, that cancel in the product: exponent
    bytes 0 to 254 in the tensor cores."""
    rng = np.random.default_rng(T)
    M, runs = 300, 24
    top = {8: 126, 4: 7}  # the codes' magnitudes; e4m3's 127 is NaN
    cx, cw = (np.where(rng.integers(0, 2, (r, runs, 32)) > 0, 1 << (b - 1), 0) | rng.integers(1, top[b] + 1, (r, runs, 32)) for r, b in ((T, xb), (M, wb)))
    e = np.tile([-127, -126, -125, 126, 127, 0, -64, 100], 3)
    ex, ew = np.tile(e, (T, 1)), np.tile(-e, (M, 1))
    ew[:, e == -127] = 126
    x, w = _with_scales(lib, cx.astype(np.uint8), ex, xb), _with_scales(lib, cw.astype(np.uint8), ew, wb)
    got = base._linear(lib, x, w, F32).double().cpu().numpy()
    base._check_product(got, x.held, w.held, F32)
    # and the same values under ordinary scales give the same bits
    x1, w1 = _with_scales(lib, cx.astype(np.uint8), ex * 0, xb), _with_scales(lib, cw.astype(np.uint8), ew + e, wb)
    np.testing.assert_array_equal(base._linear(lib, x1, w1, F32).double().cpu().numpy(), got)


@pytest.mark.parametrize("xb,wb,ob", [(8, 8, 8), (8, 4, 8), (4, 4, 4)])
@pytest.mark.parametrize("T", [1, 16, 64, 200, 2000])
def test_swiglu_codes_of_exact_sums(lib, T, xb, wb, ob):
    """Random gates and ups whose sums are exact in fp32 (integers below 2^24): codes differ from those of the 64-bit values only
    where the value lies within 2^-21 of a border."""
    rng = np.random.default_rng(T)
    K, I = 256, 640
    whole = lambda r, s: rng.integers(-3, 4, (r, K)) * s  # noqa: E731
    x, g, u = (base.Matrix.of(lib, a, b) for a, b in ((whole(T, 1.0), xb), (whole(I, 1 / 32), wb), (whole(I, 0.125), wb)))
    gv, uv = x.held @ g.held.T, x.held @ u.held.T
    h = gv / (1 + np.exp(-gv)) * uv
    c, e = base._swiglu(lib, x, g, u, ob).get()
    got = mx.values(c, e, ob, I)
    near = np.sort(np.stack([mx.held(h * (1 + s * 2.0 ** -21), ob) for s in (-1, 1)]), axis=0)
    assert ((got >= near[0]) & (got <= near[1])).all()
    # the inputs alone: how many codes are left open (the sums take few values, so that some come together)
    assert np.mean(near[0] != near[1]) < 1e-3
