"""The 8-bit attention's plans at the ends of what a launch can hold, decided on the host (no GPU needed)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def qw():
    import decode_qwen3_decoder_gb300 as pkg
    pkg._build_lib()
    pkg.qw.load()
    return pkg.qw


def test_logits_are_stored_only_as_far_as_a_launch_reaches(qw):
    """A decode with scores keeps its logits (8 bytes a key here) up to 65535 blocks of 1024 keys; past them
    the scores' own kernels run, whose workspace does not grow with the keys."""
    pages = 1 << 23
    view = qw.qw_kv8_view(4096, pages, 1, 64, 4096, pages)
    last = 65535 * 1024
    size = [qw.qw_kv8_attn_ws_bytes(view, 1, 1, 1, n, 2, True) for n in (last, last + 1, 16 * pages)]
    assert size[0] > 8 * last and size[1] == size[2] < 8 << 20


def test_a_call_without_rows_takes_empty_tensors(qw):
    """T = 0: nothing to do, whatever the tensors' addresses (torch gives an empty one's as 0)."""
    L, P = qw.load(), 4096
    view = qw.qw_kv8_view(P, 8, 2, 128, P, 4)
    for name in ("qw_kv8_append", "qw_kv8_read"):
        assert getattr(L, name)(ctypes.byref(view), 2, 0, 3, P, P, None, 0, None, 1, 0, P, None) == 0
        assert getattr(L, name)(ctypes.byref(view), 2, 1, 3, P, P, None, 256, None, 256, 0, P, None) == -1

    def attn(T, ld):
        a = qw.qw_kv8_attn_args(B=2, T=T, max_len=3, max_keys=64, n_heads=4, dtype=0, dev_start=P, dev_cu=P, dev_q=None, ld_q=ld,
                                scale=0.1, dev_out=None, ld_out=ld, dev_ws=P, ws_bytes=1 << 40, dev_status=P)
        return L.qw_kv8_attn(ctypes.byref(view), ctypes.byref(a), None)
    assert attn(0, 0) == 0 and attn(1, 512) == -1
