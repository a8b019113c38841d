"""What the microscaled matrices' calls refuse beside the refusals of single arguments. No GPU: every refused call returns
before it touches a device."""

import pytest


@pytest.fixture(scope="module")
def qw():
    import decode_qwen3_decoder_gb300 as pkg
    pkg._build_lib()
    pkg.qw.load()
    return pkg.qw


def test_stall_refuses(qw):
    for barriers, us in ((-1, 0), (32, 0), (1, 99), (1, -1), (0, 2000001)):
        assert qw.load().qw_mx_test_stall(barriers, us) == -1, (barriers, us)
        assert "mx_test_stall" in qw.qw_last_error()
    assert qw.load().qw_mx_test_stall(31, 2000000) == qw.load().qw_mx_test_stall(0, 0) == 0
