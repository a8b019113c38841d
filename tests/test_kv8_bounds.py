"""The 8-bit attention's plans at the ends of what a launch can hold, decided on the host (no GPU needed)."""

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
