"""The model on an 8-bit KV cache with more than 512 tokens reserved: decode graphs take the reservation as
their bound on the keys, whatever a sequence holds. Oracle and tolerances as in test_gpu_kv8_model."""

import numpy as np
import pytest

from gpu_util import LOGITS_ABS, Run, check_token, weights
from test_gpu_kv8_model import S, _forward, _held, _tokens, model  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=[False, True], ids=["plain", "scores"])
def eng(qw, request):
    e = qw.qw.Engine(S, dict(weights(S).named()), max_tokens=1024, max_batch=4, max_context=2048, kv_pages=400, max_seqs=4,
                     kv_bits=8, keep_scores=request.param)
    yield e
    e.close()


@pytest.fixture()
def run(qw, eng):
    qw.qw.qw_kv_reset(eng.kv, -1, eng.stream)
    return Run(qw, eng)


@pytest.mark.parametrize("n", [5, 14, 530])
def test_decode_graphs_of_one_sequence(run, model, n):  # noqa: F811
    import torch
    qw, eng, steps = run.qw, run.eng, 20
    qw.qw_kv_reserve(eng.kv, 3, 1024, eng.stream)  # another sequence's prompt leaves its partials behind
    run.prefill([3], [_tokens(1000, 7)], debug=False, reserve=False)
    qw.qw_kv_reserve(eng.kv, 1, 1500, eng.stream)
    prompt = _tokens(n, 40 + n)
    g = run.prefill([1], [prompt], debug=False, reserve=False)
    first, at, ids = int(g["next"][0]), n, []
    for _ in range(steps):
        tok = int(g["next"][0])
        g = run.decode([1], [tok], debug=False)
        logits = _forward(model, [tok], at, 0, _held(run, 1, at + 1))[1]
        assert np.max(np.abs(g["logits"][0] - logits)) <= LOGITS_ABS, at
        check_token(g["next"][0], logits)
        ids.append(int(g["next"][0]))
        at += 1
    last = g["logits"].copy()
    # the same steps in one graph
    qw.qw_kv_reset(eng.kv, 1, eng.stream)
    qw.qw_kv_reserve(eng.kv, 1, 1500, eng.stream)
    assert int(run.prefill([1], [prompt], debug=False, reserve=False)["next"][0]) == first
    t = torch.tensor([first], dtype=torch.int32, device="cuda")
    out = torch.full((steps,), -7, dtype=torch.int32, device="cuda")
    qw.qw_decode_steps(eng.model, eng.kv, [1], steps - 1, t.data_ptr(), out.data_ptr(), eng.stream)
    assert qw.qw_sync_status(eng.model, eng.stream) == 0
    assert out[:steps - 1].tolist() == ids[:-1]
    np.testing.assert_array_equal(run.decode([1], [ids[-2]], debug=False)["logits"], last)


def test_short_chunk_over_a_long_cache(run, model):  # noqa: F811
    """A continuation of a few tokens, then steps, of a batch whose lengths lie far apart."""
    qw, eng, seqs, lens = run.qw, run.eng, [0, 2], [600, 30]
    for s, n in zip(seqs, lens):
        qw.qw_kv_reserve(eng.kv, s, 1200, eng.stream)
    run.prefill(seqs, [_tokens(n, 60 + n) for n in lens], debug=False, reserve=False)
    more = [_tokens(5, 81), _tokens(3, 82)]
    g = run.prefill(seqs, more, debug=False, reserve=False)
    at = list(lens)
    for toks in (more, None, None):
        if toks is None:
            toks = [[int(x)] for x in g["next"]]
            g = run.decode(seqs, [x[0] for x in toks], debug=False)
        for b, s in enumerate(seqs):
            logits = _forward(model, toks[b], at[b], 0, _held(run, s, at[b] + len(toks[b])))[1]
            assert np.max(np.abs(g["logits"][b] - logits)) <= LOGITS_ABS
            check_token(g["next"][b], logits)
            at[b] += len(toks[b])
