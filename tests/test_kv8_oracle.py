"""The 8-bit cache's oracle against closed forms and torch's e4m3, and the refusals of the library's
calls, which are decided on the host (no GPU needed)."""

import ctypes

import numpy as np
import pytest

from oracle import kv8


def test_e4m3_values_and_rounding_match_torch():
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(kv8.e4m3_values(), codes.view(torch.float8_e4m3fn).float().numpy())
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.02, 0.02, 4000), [0.0, 448, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(kv8.e4m3_round(x), want)


@pytest.mark.parametrize("amax,e", [(0.0, -32), (448.0, 0), (448.5, 1), (2.0 ** -24, -32), (65504.0, 8), (1.75, -8), (1.7510, -7)])
def test_exponent(amax, e):
    assert kv8.exponent(amax) == e


def test_append_is_idempotent_and_keeps_earlier_tokens():
    rng = np.random.default_rng(1)
    x = [rng.normal(0, 1, (40, 1, 64)).astype(np.float16).astype(np.float64) for _ in range(2)]
    x[0][30] *= 64  # the exponent of a page grows with a later token
    one, two = kv8.Cache(3, 1, 64), kv8.Cache(3, 1, 64)
    t = np.arange(3)
    one.append(t, 0, x)
    for a in range(40):
        two.append(t, a, [v[a:a + 1] for v in x])
    before = [v.copy() for v in two.x]
    two.append(t, 39, [v[39:] for v in x])
    for w in range(2):
        np.testing.assert_array_equal(before[w], two.x[w])
        np.testing.assert_array_equal(one.e[w], two.e[w])
        # Both are multiples of the subnormal step u = 2^-9 2^e where they differ. A second rounding
        # to that grid adds at most u / 2 to a first one of at most u / 2, and the direct one is
        # off by at most u / 2: below 1.5 u apart, so at most one step.
        bound = 2.0 ** -9 * 2.0 ** one.e[w][..., None, None]
        assert np.all(np.abs(one.x[w] - two.x[w]) <= bound)


def test_single_key_returns_its_value():
    rng = np.random.default_rng(2)
    c = kv8.Cache(1, 2, 64)
    c.append([0], 0, [rng.normal(0, 1, (1, 2, 64)).astype(np.float16) for _ in range(2)])
    out, lse, w, _ = c.attention([0], 0, rng.normal(0, 1, (1, 4, 64)), 0.125)
    np.testing.assert_allclose(out[0, [0, 2]], c.rows(1, [0], 1)[0], rtol=1e-14)
    np.testing.assert_array_equal(w, np.ones((4, 1, 1)))


def test_evict_keeps_recent_and_lowest_of_equals():
    c = kv8.Cache(8, 1, 64)
    c.append(np.arange(4), 0, [np.ones((50, 1, 64)) * np.arange(1, 51)[:, None, None] for _ in range(2)])
    s = np.zeros((1, 50), np.float32)
    s[0, [7, 20]] = 3
    kept, new = c.evict(np.arange(4), np.arange(4, 8), 50, 6, 2, s)
    np.testing.assert_array_equal(kept, [[0, 1, 7, 20, 48, 49]])
    np.testing.assert_array_equal(new[0, :6], [0, 0, 3, 3, 0, 0])
    # values 1, 2, 8, 21, 49 and 50 with 4 significant bits: 21 = 10.5 * 2 and 50 = 12.5 * 4 go to even
    np.testing.assert_array_equal(c.rows(0, np.arange(4, 8), 6)[:, 0, 0], [1, 2, 8, 20, 48, 48])


# ---- refusals ---------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def qw():
    import decode_qwen3_decoder_gb300 as pkg
    pkg._build_lib()
    pkg.qw.load()
    return pkg.qw


P = 4096  # an aligned address that no refused call touches


def _view(qw, **kw):
    a = dict(blocks_ptr=P, n_pages=8, n_kv_heads=2, head_dim=128, page_table_ptr=P, max_pages=4)
    a.update(kw)
    return qw.qw_kv8_view(**a)


def test_block_bytes(qw):
    assert [qw.qw_kv8_block_bytes(d) for d in (64, 128, 96, 0, -1)] == [2080, 4128, 0, 0, 0]


BAD_VIEWS = [(dict(blocks_ptr=0), -1), (dict(page_table_ptr=0), -1), (dict(blocks_ptr=P + 16), -1), (dict(n_pages=0), -1),
             (dict(max_pages=0), -1), (dict(n_kv_heads=0), -1), (dict(head_dim=96), -7)]


def _rows_call(qw, name, view, **kw):
    a = dict(B=2, T=4, max_len=3, start=P, cu=P, k=P, ld_k=256, v=P, ld_v=256, dtype=0, status=P)
    a.update(kw)
    L = qw.load()
    return getattr(L, name)(ctypes.byref(view), a["B"], a["T"], a["max_len"], a["start"], a["cu"], a["k"], a["ld_k"], a["v"],
                            a["ld_v"], a["dtype"], a["status"], None)


@pytest.mark.parametrize("name", ["qw_kv8_append", "qw_kv8_read"])
def test_append_and_read_refuse(qw, name):
    for kw, want in BAD_VIEWS:
        assert _rows_call(qw, name, _view(qw, **kw)) == want, kw
        assert qw.qw_last_error()
    for kw in (dict(B=0), dict(B=1025), dict(T=-1), dict(max_len=0), dict(start=None), dict(cu=None), dict(k=None),
               dict(v=None), dict(status=None), dict(dtype=3), dict(ld_k=255), dict(ld_v=248), dict(k=P + 8), dict(ld_v=260)):
        assert _rows_call(qw, name, _view(qw), **kw) == -1, kw
    assert getattr(qw.load(), name)(None, 1, 1, 1, P, P, P, 256, P, 256, 0, P, None) == -1
    assert _rows_call(qw, name, _view(qw), T=0) == 0  # nothing to do


def _attn_call(qw, view, **kw):
    a = dict(B=2, T=4, max_len=3, max_keys=64, n_heads=4, dtype=0, dev_start=P, dev_cu=P, dev_q=P, ld_q=512, scale=0.1,
             dev_out=P, ld_out=512, dev_lse=None, dev_score_in=None, dev_score_out=None, ld_score=0, dev_ws=P,
             ws_bytes=1 << 40, dev_status=P)
    a.update(kw)
    return qw.load().qw_kv8_attn(ctypes.byref(view), ctypes.byref(qw.qw_kv8_attn_args(**a)), None)


def test_attention_refuses(qw):
    for kw, want in BAD_VIEWS:
        assert _attn_call(qw, _view(qw, **kw)) == want, kw
    for kw in (dict(B=0), dict(T=-2), dict(max_len=0), dict(max_keys=0), dict(max_keys=65), dict(n_heads=3), dict(n_heads=1),
               dict(dtype=2), dict(dev_start=None), dict(dev_cu=None), dict(dev_q=None), dict(dev_out=None), dict(dev_ws=None),
               dict(dev_status=None), dict(ld_q=504), dict(ld_out=504), dict(dev_q=P + 2), dict(dev_out=P + 8),
               dict(ld_q=516), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0),
               dict(dev_score_in=P), dict(dev_score_out=P, ld_score=63), dict(ws_bytes=0), dict(dev_ws=P + 128)):
        assert _attn_call(qw, _view(qw), **kw) == -1, kw
        assert "attn" in qw.qw_last_error()
    assert _attn_call(qw, _view(qw), n_heads=34, ld_q=34 * 128, ld_out=34 * 128) == -7
    assert qw.load().qw_kv8_attn(ctypes.byref(_view(qw)), None, None) == -1
    assert _attn_call(qw, _view(qw), T=0) == 0
    assert qw.qw_kv8_attn_ws_bytes(_view(qw), 0, 1, 1, 1, 2, False) == 0
    assert qw.qw_kv8_attn_ws_bytes(_view(qw), 1, 1, 1, 1, 2, True) > 0


def test_attention_row_limit_and_workspace(qw):
    """65535 * 256 query rows of a KV head are one launch; the workspace follows the rows there are, not
    the bound on one entry times the entries."""
    big = _view(qw, max_pages=1 << 22, n_pages=1 << 22)
    n = 65535 * 256 // 2
    for T, want in ((n + 1, -7), (n, -1)):  # the second is refused for its workspace of 0 bytes only
        assert _attn_call(qw, big, B=1, T=T, max_len=T, max_keys=T, ws_bytes=0) == want
        assert (qw.qw_kv8_attn_ws_bytes(big, 1, T, T, T, 4, True) == 0) == (want == -7)
    loose = qw.qw_kv8_attn_ws_bytes(big, 1024, 8192, 8192, 8192, 4, True)
    assert loose < 1 << 30


def test_evict_refuses(qw):
    def call(view, **kw):
        a = dict(B=2, max_len=64, len=P, keep=8, recent=2, dst=None, score=P, out=P, ld=64, kept=P, new=P + 64, status=P)
        a.update(kw)
        return qw.load().qw_kv8_evict(ctypes.byref(view), a["B"], a["max_len"], a["len"], a["keep"], a["recent"], a["dst"],
                                      a["score"], a["out"], a["ld"], a["kept"], a["new"], a["status"], None)
    for kw, want in BAD_VIEWS:
        assert call(_view(qw, **kw)) == want, kw
    for kw in (dict(B=0), dict(max_len=0), dict(max_len=65), dict(len=None), dict(keep=0), dict(recent=-1), dict(recent=9),
               dict(score=None), dict(out=None), dict(ld=63), dict(kept=None), dict(new=None), dict(status=None), dict(new=P)):
        assert call(_view(qw), **kw) == -1, kw
        assert "evict" in qw.qw_last_error()
