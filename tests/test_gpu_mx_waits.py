"""Products whose bounded waits run out: an arrival that never comes at one kind of barrier and a limit of a millisecond (no
trap, no fault). Every CTA comes to its end, the status says so, and the next call is right."""

import time

import pytest
import test_gpu_mx as base

pytestmark = pytest.mark.gpu

KINDS = ["FULL", "EMPTY", "SFULL", "ACCF", "ACCE"]


@pytest.fixture
def lib(qw):
    yield qw.qw
    qw.qw.qw_mx_test_stall(0, 0)


def _give_up(lib, run, reached):
    """run(status) -> tensors."""
    import torch
    st = base._status()
    want = [t.clone() for t in run(st)]
    assert int(st.item()) == 0
    for kind in KINDS:
        try:
            lib.qw_mx_test_stall(getattr(lib, "QW_MX_STALL_" + kind), 1000)
            st.zero_()
            t0 = time.perf_counter()
            got = run(st)
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 1.0
        finally:
            lib.qw_mx_test_stall(0, 0)
        assert int(st.item()) == (lib.QW_MX_TIMEOUT if kind in reached else 0), kind
        if kind not in reached:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), kind
        st.zero_()
        for t in got:
            t.zero_()
        got = run(st)
        assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in zip(got, want)), kind
        # the bit is set beside others and never cleared
        st.fill_(4)
        run(st)
        assert int(st.item()) == 4


ALWAYS = {"FULL", "SFULL", "ACCF"}


@pytest.mark.parametrize("xb,wb", base.FORMATS)
@pytest.mark.parametrize("T,K,M,reached", [
    (200, 130, 600, ALWAYS),                               # pairs of CTAs, a tile each of one or two stages
    (200, 4096, 600, ALWAYS | {"EMPTY"}),                  # ... whose ring goes round
    (2600, 2600, 2300, ALWAYS | {"EMPTY", "ACCE"}),        # ... and several tiles a pair
    (1, 300, 200, ALWAYS),                                 # few rows, a CTA a tile
    (3, 16384, 256, ALWAYS | {"EMPTY"}),                   # a cluster of 8, partial sums through its shared memory
    (40, 16384, 256, ALWAYS | {"EMPTY"}),
    (100, 16384, 256, ALWAYS | {"EMPTY"}),
    (16, 2100, 90001, ALWAYS | {"EMPTY", "ACCE"}),         # a stream of tiles, two accumulators
    (64, 2100, 90001, ALWAYS | {"EMPTY", "ACCE"}),
    (128, 4096, 60001, ALWAYS | {"EMPTY", "ACCE"})])
def test_linear_gives_up(lib, T, K, M, reached, xb, wb):
    import torch
    x, w = base._device_matrix(lib, T, K, xb, 1)[0], base._device_matrix(lib, M, K, wb, 2)[0]
    out = torch.zeros((T, -(-M // 8) * 8), dtype=torch.bfloat16, device="cuda")

    def run(st):
        lib.qw_mx_linear(x.view, w.view, out.data_ptr(), out.stride(0), lib.QW_BF16, st.data_ptr())
        return [out]
    _give_up(lib, run, reached)


@pytest.mark.parametrize("xb,wb", base.FORMATS)
@pytest.mark.parametrize("T,K,I,reached", [
    (200, 130, 600, ALWAYS), (2600, 2600, 1400, ALWAYS | {"EMPTY", "ACCE"}),
    (3, 16384, 256, ALWAYS | {"EMPTY"}), (64, 16384, 256, ALWAYS | {"EMPTY"}), (16, 2100, 90001, ALWAYS | {"EMPTY", "ACCE"})])
def test_swiglu_gives_up(lib, T, K, I, reached, xb, wb):
    x, g, u = (base._device_matrix(lib, r, K, b, s)[0] for r, b, s in ((T, xb, 1), (I, wb, 2), (I, wb, 3)))
    m = base.Matrix(lib, T, I, xb, fill=0)

    def run(st):
        lib.qw_mx_swiglu(x.view, g.view, u.view, m.view, st.data_ptr())
        return [m.codes, m.scales]
    _give_up(lib, run, reached)
