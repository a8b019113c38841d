"""Life of a model's caches: freed and bound again, emptied after an eviction, stopped on the way."""

import numpy as np
import pytest

from gpu_util import LOGITS_ABS, Run, weights
from test_gpu_kv8_model import MAXC, S, Check, _tokens, model  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eng(qw):
    e = qw.qw.Engine(S, dict(weights(S).named()), max_tokens=256, max_batch=8, max_context=MAXC, kv_pages=200, max_seqs=8,
                     kv_bits=8, keep_scores=True)
    yield e
    e.close()


@pytest.fixture()
def run(qw, eng):
    qw.qw.qw_kv_reset(eng.kv, -1, eng.stream)
    return Run(qw, eng)


def test_caches_freed_and_bound_again(run):
    """Caches of every kind, one after another at the same host address as a rule (each is bound right after
    the one before is freed), decode the same batch into the same buffers: none replays the kernels that
    another was captured with. Pools stay allocated."""
    import torch
    qw, eng = run.qw, run.eng
    kinds = [("f16", False), ("8", False), ("f16", False), ("8", True), ("8", False), ("f16", False)]
    tok, nxt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    lg = torch.zeros((1, S.vocab), device="cuda")
    size = {k: qw.qw_kv_pool_bytes(eng.model, 6, 2) if k[0] == "f16" else qw.qw_kv8_pool_bytes(eng.model, 6, 2, k[1]) for k in kinds}
    pools = [torch.zeros(size[k], dtype=torch.uint8, device="cuda") for k in kinds]
    before, results, kv = [], [], None
    torch.cuda.synchronize()
    for i, k in enumerate(kinds):
        ptr, n = pools[i].data_ptr(), size[k]
        if kv is not None:
            qw.qw_free_kv(kv)
        kv = qw.qw_kv_alloc(eng.model, ptr, n, 2, eng.stream) if k[0] == "f16" else qw.qw_kv8_alloc(eng.model, ptr, n, 2, k[1], eng.stream)
        qw.qw_kv_reserve(kv, 0, 80, eng.stream)
        prompt = torch.tensor(_tokens(12, 900 + i // 3), dtype=torch.int32, device="cuda")  # the last three have another prompt
        torch.cuda.synchronize()
        qw.qw_prefill(eng.model, kv, [0], [12], prompt.data_ptr(), 0, nxt.data_ptr(), eng.stream)
        got = []
        for t in _tokens(3, 910):
            eng.stream.synchronize()
            tok.fill_(t)
            torch.cuda.synchronize()
            qw.qw_decode_step(eng.model, kv, [0], tok.data_ptr(), lg.data_ptr(), nxt.data_ptr(), eng.stream)
            assert qw.qw_sync_status(eng.model, eng.stream) == 0
            got.append(lg.cpu().numpy().astype(np.float64))
        results.append(np.concatenate(got))
        for p, was in zip(pools, before):  # nobody touched the pools of the freed caches
            assert torch.equal(p, was)
        before.append(pools[i].clone())
    qw.qw_free_kv(kv)
    assert np.abs(results[0] - results[2]).max() <= LOGITS_ABS  # the same kind and prompt
    np.testing.assert_array_equal(results[3], results[4])
    # the kinds differ by the 8-bit codes only, the prompts by much more
    assert np.abs(results[0] - results[3]).max() > 10 * LOGITS_ABS
    assert np.abs(results[0] - results[1]).max() < np.abs(results[0] - results[3]).max() / 3
    assert np.abs(results[5] - results[4]).max() < np.abs(results[0] - results[3]).max() / 3


def test_a_sequence_emptied_after_an_eviction_starts_again(run, model):  # noqa: F811
    """Truncated to nothing it begins at position 0 with the whole context ahead of it."""
    qw, eng = run.qw, run.eng
    qw.qw_kv_reserve(eng.kv, 2, MAXC, eng.stream)
    run.prefill([2], [_tokens(250, 1)], debug=False, reserve=False)
    qw.qw_kv_evict(eng.kv, 2, 60, 10, eng.stream)
    qw.qw_kv_truncate(eng.kv, 2, 0, eng.stream)
    c = Check(run, model)
    prompt = _tokens(20, 2)
    g = run.prefill([2], [prompt], reserve=False)
    c.after([2], [prompt], g)
    step = g["next"].tolist()
    c.after([2], [step], run.decode([2], step))
    for n in (250, MAXC - 21 - 250):  # up to the last position
        run.prefill([2], [_tokens(n, 3)], debug=False, reserve=False)
    assert qw.qw_kv_length(eng.kv, 2) == MAXC
    # generation into it: the prompt and the steps fill the context
    qw.qw_kv_evict(eng.kv, 2, 30, 10, eng.stream)
    qw.qw_kv_truncate(eng.kv, 2, 0, eng.stream)
    out = np.zeros((1, 13), np.int32)
    half = _tokens(250, 4)
    qw.qw_generate(eng.model, eng.kv, [2], [250], np.asarray(half, np.int32), 12, out, eng.stream)
    assert qw.qw_sync_status(eng.model, eng.stream) == 0 and qw.qw_kv_length(eng.kv, 2) == 262


@pytest.mark.parametrize("n", [3, 5])
def test_a_stopped_sequence_gives_no_more_weight(run, n):
    """After its EOS a sequence steps on with the batch; what its dropped tokens would have looked at is
    not counted: each of its tokens has spread a weight of one for each head of the group."""
    qw, eng, steps = run.qw, run.eng, 20
    seqs, lens = list(range(n)), [6 + 5 * i for i in range(n)]
    prompt = np.concatenate([np.asarray(_tokens(k, 400 + k), np.int32) for k in lens])

    def reset():
        qw.qw_kv_reset(eng.kv, -1, eng.stream)
        for s, k in zip(seqs, lens):
            qw.qw_kv_reserve(eng.kv, s, k + steps, eng.stream)
    reset()
    out = np.zeros((n, steps + 1), np.int32)
    qw.qw_generate(eng.model, eng.kv, seqs, lens, prompt, steps, out, eng.stream)
    c = Check(run, None)
    for b in range(n):
        np.testing.assert_allclose(c.scores(b).sum(-1), (lens[b] + steps) * S.n_heads / S.n_kv_heads, rtol=1e-5)
    stopped = set()
    for eos in (int(out[1, 4]), int(out[0, 11]), int(out[2, 0])):
        reset()
        cut, cnt = np.zeros((n, steps + 1), np.int32), np.zeros(n, np.int32)
        qw.qw_generate_eos(eng.model, eng.kv, seqs, lens, prompt, steps, eos, cut, cnt, eng.stream)
        for b in range(n):
            length = qw.qw_kv_length(eng.kv, b)
            sc = c.scores(b)
            stopped |= {b} if cnt[b] <= steps else set()
            np.testing.assert_allclose(sc.sum(-1), length * S.n_heads / S.n_kv_heads, rtol=1e-5)
            assert np.all(sc[..., length:] == 0)
    assert {0, 1, 2} <= stopped
    # the sequences go on afterwards, their weights with them
    more = [_tokens(3, 700 + b) for b in range(n)]
    before = [qw.qw_kv_length(eng.kv, b) for b in range(n)]
    for b in range(n):
        qw.qw_kv_reserve(eng.kv, b, before[b] + 6, eng.stream)
    g = run.prefill(seqs, more, debug=False, reserve=False)
    run.decode(seqs, g["next"].tolist(), debug=False)
    for b in range(n):
        np.testing.assert_allclose(c.scores(b).sum(-1), (before[b] + 4) * S.n_heads / S.n_kv_heads, rtol=1e-5)


def test_stopped_sequences_under_a_large_reservation(qw):
    """As above where the logits of a step's bound no longer fit the workspace and the scores' own kernels run."""
    B, steps = 24, 10
    e = qw.qw.Engine(S, dict(weights(S).named()), max_tokens=256, max_batch=B, max_context=90000, kv_pages=5700, max_seqs=B,
                     kv_bits=8, keep_scores=True)
    try:
        q, c = qw.qw, Check(Run(qw, e), None)
        seqs, lens = list(range(B)), [5 + b % 4 for b in range(B)]
        prompt = np.concatenate([np.asarray(_tokens(k, 500 + b), np.int32) for b, k in enumerate(lens)])
        eos = -1
        for _ in range(2):
            q.qw_kv_reset(e.kv, -1, e.stream)
            for s, k in zip(seqs, lens):
                q.qw_kv_reserve(e.kv, s, 88000 if s == 5 else k + steps, e.stream)
            out, cnt = np.zeros((B, steps + 1), np.int32), np.zeros(B, np.int32)
            if eos < 0:
                q.qw_generate(e.model, e.kv, seqs, lens, prompt, steps, out, e.stream)
                eos = int(out[7, 2])
            else:
                q.qw_generate_eos(e.model, e.kv, seqs, lens, prompt, steps, eos, out, cnt, e.stream)
                assert cnt[7] <= 3
            assert q.qw_sync_status(e.model, e.stream) == 0
            ptr, ld = q.qw_kv8_scores(e.kv)
            off = ptr - e.pool.data_ptr()
            sc = e.pool[off:off + 4 * B * S.n_layers * S.n_kv_heads * ld].view(c.run.torch.float32).view(B, S.n_layers * S.n_kv_heads, ld)
            for b in range(B):
                n = q.qw_kv_length(e.kv, b)
                np.testing.assert_allclose(sc[b].sum(-1).cpu().numpy(), n * S.n_heads / S.n_kv_heads, rtol=1e-5)
                assert not bool(sc[b, :, n:].any())
    finally:
        e.close()
