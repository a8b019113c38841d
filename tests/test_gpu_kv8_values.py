"""Attention over the 8-bit cache at the ends of its types' ranges."""

import numpy as np
import pytest

from test_gpu_kv8 import BF16, F16, Case, _dt

pytestmark = pytest.mark.gpu


def _attn(c, q, starts, lens, G, dtype, scale, score=None):
    """qw_kv8_attn of the rows q [T, n_kv G hd]; out and lse."""
    torch, qw = c.torch, c.qw
    starts, lens = np.asarray(starts), np.asarray(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, Hq, mk, ml = int(cu[-1]), c.n_kv * G, int((starts + lens).max()), int(lens.max())
    out, lse = torch.empty((T, Hq, c.hd), dtype=_dt(dtype), device="cuda"), torch.empty((T, Hq), device="cuda")
    nb = qw.qw_kv8_attn_ws_bytes(c.view, c.B, T, ml, mk, Hq, score is not None)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    ds, dc = c.i32(starts), c.i32(cu)
    qw.qw_kv8_attn(c.view, c.B, T, ml, mk, ds.data_ptr(), dc.data_ptr(), q.data_ptr(), Hq * c.hd, Hq, getattr(qw, "QW_" + dtype.upper()),
                   scale, out.data_ptr(), Hq * c.hd, lse.data_ptr(), 0, score.data_ptr() if score is not None else 0,
                   score.shape[2] if score is not None else 0, ws.data_ptr(), nb, c.status.data_ptr())
    torch.cuda.synchronize()
    assert c.bits() == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _append(c, k, v):
    """K and V [n, n_kv, hd] fp16 arrays into every entry from position 0."""
    n = len(k)
    dk, dv = (c.torch.from_numpy(np.ascontiguousarray(np.concatenate([x] * c.B), np.float16)).cuda() for x in (k, v))
    ds, dc = c.i32([0] * c.B), c.i32(np.arange(c.B + 1) * n)
    ld = c.n_kv * c.hd
    c.qw.qw_kv8_append(c.view, c.B, n * c.B, n, ds.data_ptr(), dc.data_ptr(), dk.data_ptr(), ld, dv.data_ptr(), ld, c.qw.QW_F16,
                       c.status.data_ptr())
    for b in range(c.B):
        c.orc.append(c.table[b], 0, [x.astype(np.float16).astype(np.float64) for x in (k, v)])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,rows", [(60, 1), (1800, 1), (1800, 6), (90, 90), (3000, 40)])
def test_values_next_to_65504_stay_finite(qw, hd, n, rows):
    """65504 is held as 65536 and read back as 65504: an fp16 output made of it is 65504 too, in every
    kernel; bf16 holds 65536 itself."""
    c = Case(qw, [n], 2, hd, seed=5)
    sign = np.where(np.arange(hd) % 3 == 1, -1.0, 1.0)
    _append(c, c.rng.normal(0, 1, (n, 2, hd)), np.broadcast_to(65504.0 * sign, (n, 2, hd)))
    for dtype, top in ((F16, 65504.0), (BF16, 65536.0)):
        q = c.torch.from_numpy(c.rng.normal(0, 1, (rows, 4 * hd))).cuda().to(_dt(dtype))
        out, _ = _attn(c, q, [n - rows], [rows], 2, dtype, hd ** -0.5)
        assert np.all(out == top * sign)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,rows", [(20, 1), (40, 6), (90, 90), (400, 150)])
def test_logits_too_small_for_fp32_give_equal_weights(qw, hd, n, rows):
    """bf16 queries of zeros and of the smallest values, keys of zeros and a small scale: the factor of a
    logit underflows, every visible key gets the same weight and hidden ones none."""
    c = Case(qw, [n], 1, hd, seed=6)
    k, v = np.zeros((n, 1, hd)), c.rng.normal(0, 1, (n, 1, hd))
    k[n // 2:] = c.rng.normal(0, 1, (n - n // 2, 1, hd))
    _append(c, k, v)
    q = c.torch.zeros((rows, 2 * hd), device="cuda")
    q[:, hd:] = 2.0 ** -120
    q = q.to(c.torch.bfloat16)
    held = c.orc.rows(1, c.table[0], n)[:, 0]
    for scale in (1e-6, 1e-30):
        score = c.torch.zeros((1, 1, n), device="cuda")
        out, lse = _attn(c, q, [n - rows], [rows], 2, BF16, scale, score)
        want_s = np.zeros(n)
        for i in range(rows):
            m = n - rows + i + 1
            want, mag = held[:m].mean(0), np.abs(held[:m]).mean(0)
            # equal weights are powers of two, exact in fp16: fp32 sums of m terms and the output's rounding
            assert np.all(np.abs(out[i] - want) <= mag * (m + 8) * 2.0 ** -23 + np.abs(want) * 2.0 ** -8)
            assert np.all(np.abs(lse[i] - np.log(m)) <= (m + 8) * 2.0 ** -23 + np.log(m) * 2.0 ** -21)
            want_s[:m] += 2.0 / m
        got = score[0, 0].double().cpu().numpy()
        assert np.all(np.abs(got - want_s) <= want_s * (2 * rows + n + 16) * 2.0 ** -22)


@pytest.mark.parametrize("n,rows", [(20, 1), (40, 6), (90, 90)])
def test_bf16_queries_beyond_the_fp16_range(qw, n, rows):
    """Rows of any bf16 magnitude whose logits fit fp32: here the scale takes a power of two back."""
    hd = 64
    c = Case(qw, [n], 1, hd, seed=7)
    k, v = c.rng.normal(0, 1, (n, 1, hd)), c.rng.normal(0, 1, (n, 1, hd))
    _append(c, k, v)
    q0 = c.torch.from_numpy(c.rng.normal(0, 1, (rows, 2 * hd))).cuda().to(c.torch.bfloat16)
    want, wl = _attn(c, q0, [n - rows], [rows], 2, BF16, 0.125)
    for e in (-102, -90, 100, 110, 118, 120):  # the products are those of the first call
        q = (q0.float() * 2.0 ** e).to(c.torch.bfloat16)
        out, lse = _attn(c, q, [n - rows], [rows], 2, BF16, 0.125 * 2.0 ** -e)
        np.testing.assert_array_equal(out, want)
        np.testing.assert_array_equal(lse, wl)
