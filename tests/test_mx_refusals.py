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


A = 1 << 20  # an aligned address that no refused call touches; operands of the calls below lie from here on


def _m(qw, codes, scales, rows, cols, bits):
    return qw.qw_mx_view(codes, scales, rows, cols, bits)


def test_operands_that_share_memory(qw):
    """An output over an input, over another output or over a part of one is refused."""
    import ctypes
    L, ref = qw.load(), ctypes.byref
    far = A << 4
    m = lambda codes, scales, rows=200, cols=256: ref(_m(qw, codes, scales, rows, cols, 8))  # noqa: E731
    nc, ns = 200 * 256, 2 * 2 * 512  # bytes of codes and scales
    x = far  # 200 rows of 256 fp32, 300 apart
    for codes, scales in ((x, A), (A, x), (x + 1024 - 32, A), (x - nc + 32, A), (x + 198 * 1200, A), (A, x + 198 * 1200 + 992), (x + 1024, A)):
        for call in (L.qw_mx_quantize, L.qw_mx_read):
            assert call(m(codes, scales), x, 300, 2, None) == -1, (codes - x, scales - x)
            assert "overlaps" in qw.qw_last_error()

    def norm(codes, scales, add, total, w):
        return L.qw_mx_rmsnorm(m(codes, scales), x, 300, 2, add, 600, 1, total, 300, w, 1e-6, None)
    clear = [A, 2 * A, 3 * A, 4 * A, 5 * A]
    for i, p in ((0, x), (1, x), (0, clear[2]), (0, clear[3]), (1, clear[4]), (3, x + 16), (3, x - 16), (3, clear[2] + 64), (3, clear[4] - 1008)):
        a = list(clear)
        a[i] = p
        assert norm(*a) == -1, (i, p)
        assert "overlaps" in qw.qw_last_error()

    for out in (A, A + nc - 16, 2 * A + ns - 16, 3 * A, 4 * A, 3 * A - 16):
        # x: codes at A, scales at 2 A; w [200][256]: 3 A, 4 A; out [200][200] bf16
        assert L.qw_mx_linear(m(A, 2 * A), m(3 * A, 4 * A), out, 200, 1, far, None) == -1, out
        assert "overlaps" in qw.qw_last_error()

    for codes, scales in ((A, 8 * A), (7 * A, A), (2 * A, 8 * A), (3 * A + 32, 8 * A), (7 * A, 6 * A), (7 * A, 5 * A + nc - 32)):
        st = L.qw_mx_swiglu(m(A, 2 * A), m(3 * A, 4 * A), m(5 * A, 6 * A), m(codes, scales, 200, 200), far, None)
        assert st == -1 and "overlaps" in qw.qw_last_error(), (codes, scales)


def test_status_alignment(qw):
    """The status word is written by a 32-bit atomic."""
    import ctypes
    L, ref = qw.load(), ctypes.byref
    m = lambda at, rows=3, cols=256: ref(_m(qw, at, at + 65536, rows, cols, 8))  # noqa: E731
    for off in (1, 2, 3):
        assert L.qw_mx_linear(m(A), m(2 * A), 3 * A, 8, 0, 4 * A + off, None) == -1
        assert "status" in qw.qw_last_error()
        assert L.qw_mx_swiglu(m(A), m(2 * A), m(3 * A), m(4 * A, 3, 3), 5 * A + off, None) == -1
        assert "status" in qw.qw_last_error()
