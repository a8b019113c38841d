"""A layer's chain of microscaled operators, every byte that it writes compared: each run starts from memory that holds nothing of
the run before, on the stream it runs on, and its outcome is compared there."""

import threading

import numpy as np
import pytest
import test_gpu_mx as base

from oracle import mx

pytestmark = pytest.mark.gpu


@pytest.fixture
def lib(qw):
    return qw.qw


def _used(m):
    """Which scale bytes belong to rows."""
    import torch
    rows = np.zeros((-(-m.rows // 128) * 128, -(-m.cols // 128) * 4), np.uint8)
    rows[:m.rows] = 1
    out = np.empty((rows.shape[0] // 128, rows.shape[1] // 4, 512), bool)
    for r in range(128):
        for j in range(4):
            out[:, :, 16 * (r % 32) + 4 * (r // 32) + j] = rows[r::128, j::4]
    pad = np.zeros(m.scales.numel() - out.size, bool)
    return torch.from_numpy(np.concatenate([out.reshape(-1), pad])).cuda()


class Chain(base.Layer):
    """A layer that knows all that it writes."""

    def __init__(self, lib, T, xb, wb, seed):
        import torch
        super().__init__(lib, T, 512, 384, 1000, xb, wb, seed=seed)
        self.mats, self.floats = [self.qa, self.q1, self.qh, self.q2], [self.b1, self.s1, self.b2, self.s2]
        self.masks = [_used(m) for m in self.mats]
        self.bad = torch.zeros((), dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        self.poison(0xAB)
        self.run()
        torch.cuda.synchronize()
        self.check()
        for m in self.mats:
            m.get()  # guards and the exponents of rows that are not there, as the poison left them
        self.want = [m.codes.clone() for m in self.mats] + [m.scales.clone() for m in self.mats] + [t.clone() for t in self.floats]

    def poison(self, byte):
        for m in self.mats:
            m.codes.fill_(byte)
            m.scales.fill_(byte)
        for t in self.floats:
            t.fill_(float("nan"))

    def compare(self, byte):
        """Counts, on the current stream, outputs that are not the first run's or bytes written beside them."""
        n = len(self.mats)
        for m, c, s, used in zip(self.mats, self.want[:n], self.want[n:], self.masks):
            self.bad += (m.codes[:m.nc] != c[:m.nc]).sum() + (m.codes[m.nc:] != byte).sum()
            self.bad += ((m.scales != s) & used).sum() + ((m.scales != byte) & ~used).sum()
        for t, w in zip(self.floats, self.want[2 * n:]):
            self.bad += (t != w).sum()

    def rounds(self, n, replay=None):
        """n runs on the current stream, each from poison of another byte."""
        import torch
        stream = torch.cuda.current_stream()
        for i in range(n):
            byte = (0xFF, 0x00, 0x5A)[i % 3]
            self.poison(byte)
            replay() if replay else self.run(stream)
            self.compare(byte)

    def assert_clean(self):
        import torch
        torch.cuda.synchronize()
        assert int(self.bad.item()) == 0 and int(self.status.item()) == 0


def test_a_wrong_byte_is_counted(lib):
    """The comparison itself: an exponent, a code, a value, and a byte beside them."""
    import torch
    c = Chain(lib, 70, 8, 4, seed=1)
    for spoil in (lambda: c.q2.scales[3].add_(1), lambda: c.q1.codes[77].add_(1), lambda: c.s2[69, 511].add_(1.0), lambda: c.qh.scales[-1].add_(1)):
        c.poison(0x5A)
        c.run(torch.cuda.current_stream())
        spoil()
        c.bad.zero_()
        c.compare(0x5A)
        assert int(c.bad.item()) == 1


@pytest.mark.parametrize("xb,wb", base.FORMATS)
@pytest.mark.parametrize("T", [1, 7, 64, 130, 600])
def test_chain_repeats_and_replays(lib, T, xb, wb):
    import torch
    c = Chain(lib, T, xb, wb, seed=T)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.rounds(6)
    c.assert_clean()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(torch.cuda.current_stream())
    c.rounds(6, graph.replay)
    c.assert_clean()


def test_chains_on_streams_and_threads(lib):
    """Three layers at once, each from its own host thread and stream."""
    import torch
    chains = [Chain(lib, t, xb, wb, seed=t) for t, xb, wb in ((200, 8, 4), (30, 4, 4), (1, 8, 8))]
    errors = []

    def work(c):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                c.rounds(30)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(c,)) for c in chains]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for c in chains:
        c.assert_clean()


def test_chains_beside_a_model(qw):
    """A model's prefill and decode on one stream, chains on another: kernels that share SMs and their tensor memory."""
    import torch

    import synth
    from gpu_util import Run, engine
    lib = qw.qw
    chains = [Chain(lib, t, 8, 4, seed=t) for t in (3, 600)]
    eng = engine(qw, synth.ONE_BLOCK, max_tokens=256, max_batch=16, max_context=512, kv_pages=256)
    r = Run(qw, eng)
    prompt = [list(np.random.default_rng(b).integers(0, synth.ONE_BLOCK.vocab, 16)) for b in range(12)]
    errors = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    for c in chains:
                        c.rounds(1)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    th = threading.Thread(target=work)
    th.start()
    first = None
    for _ in range(4):
        d = r.prefill(list(range(12)), prompt, debug=False, logits=False, reserve_extra=8)
        first = d["next"] if first is None else first
        np.testing.assert_array_equal(d["next"], first)
        for _ in range(4):
            r.decode(list(range(12)), [5] * 12, debug=False, logits=False)
        lib.qw_kv_reset(eng.kv, -1, eng.stream)
    th.join()
    assert not errors
    for c in chains:
        c.assert_clean()
    eng.close()
