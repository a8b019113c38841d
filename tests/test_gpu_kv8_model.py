"""The model on an 8-bit KV cache (qw_kv8_alloc): prefill, chunks, decode steps, generation, the
accumulated attention weights and eviction.

The oracle's forward pass runs on the values that the GPU's cache holds, read back from its blocks,
so a code that rounded to the other side does not blur the comparison: hidden states keep the
tolerance of the fp16 cache. That the held values are the right ones is checked apart: they are
within half an e4m3 step (2^-4 of the value, half of 2^-9 2^e where codes are subnormal) of the
oracle's K and V, which the hidden states' tolerance moves by at most 4 times itself of the page's
largest value (two products and a norm on the way)."""

import ctypes

import numpy as np
import pytest

import oracle
import synth
from gpu_util import HIDDEN_REL, LOGITS_ABS, Run, check_token, rel_err, weights
from oracle import kv8
from oracle.qwen3 import _widen

pytestmark = pytest.mark.gpu

S = synth.Shape(n_layers=3, vocab=4096)
MAXC = 512


@pytest.fixture(scope="module")
def eng(qw):
    e = qw.qw.Engine(S, dict(weights(S).named()), max_tokens=256, max_batch=24, max_context=MAXC, kv_pages=400, max_seqs=24,
                     kv_bits=8, keep_scores=True)
    yield e
    e.close()


@pytest.fixture()
def run(qw, eng):
    qw.qw.qw_kv_reset(eng.kv, -1, eng.stream)
    return Run(qw, eng)


def _blocks(run):
    import torch
    ptr, none, n_pages = run.qw.qw_kv_pool_ptrs(run.eng.kv)
    assert none is None
    run.eng.stream.synchronize()
    blk = run.qw.qw_kv8_block_bytes(S.head_dim)
    off = ptr - run.eng.pool.data_ptr()
    n = S.n_layers * n_pages * S.n_kv_heads * blk
    return run.eng.pool[off:off + n].cpu().numpy().reshape(S.n_layers, n_pages, S.n_kv_heads, blk)


def _held(run, seq, n):
    """Per layer (K, V) [n, n_kv, hd] and exponents of positions 0 .. n - 1."""
    raw = _blocks(run)
    table = run.qw.qw_kv_page_table(run.eng.kv, seq)[:(n + 15) // 16]
    out = []
    for l in range(S.n_layers):
        c = kv8.Cache.from_blocks(raw[l][table], S.head_dim)
        ids = np.arange(len(table))
        out.append(([c.rows(w, ids, n) for w in range(2)], [np.repeat(c.e[w], 16, 0)[:n] for w in range(2)]))
    return out


def _forward(m, ids, slot0, shift, held):
    """The oracle's forward pass of tokens at slots slot0 .. over the held cache; hidden states, logits
    of the last token, K and V per layer, and each layer's attention weights [n_heads, n, keys]."""
    n = len(ids)
    pos = slot0 + shift + np.arange(n)
    x = m.embed_rows(ids)
    hid, kv, wts = [], [], []
    ang = oracle.rope_angles(pos, S.head_dim, S.rope_theta)
    for l in range(S.n_layers):
        lw = m.layer(l)
        h = oracle.rms_norm(x, lw.in_norm, S.rms_eps)
        q, k, v = ((h @ w.T).reshape(n, -1, S.head_dim).transpose(1, 0, 2) for w in (lw.wq, lw.wk, lw.wv))
        q = oracle.apply_rope(oracle.rms_norm(q, lw.q_norm, S.rms_eps), ang)
        k = oracle.apply_rope(oracle.rms_norm(k, lw.k_norm, S.rms_eps), ang)
        kv.append((k.transpose(1, 0, 2), v.transpose(1, 0, 2)))
        K, V = held[l][0]
        G = S.n_heads // S.n_kv_heads
        hidden = np.arange(slot0 + n)[None, :] > slot0 + np.arange(n)[:, None]
        o, w = np.zeros((n, S.n_heads, S.head_dim)), np.zeros((S.n_heads, n, slot0 + n))
        for i in range(S.n_heads):
            a = q[i] @ K[:slot0 + n, i // G].T * S.head_dim ** -0.5
            a[hidden] = -np.inf
            a = np.exp(a - a.max(1, keepdims=True))
            w[i] = a / a.sum(1, keepdims=True)
            o[:, i] = w[i] @ V[:slot0 + n, i // G]
        wts.append(w)
        x = x + o.reshape(n, -1) @ lw.wo.T
        x = x + oracle.ffn(oracle.rms_norm(x, lw.post_norm, S.rms_eps), lw.wg, lw.wu, lw.wd)
        hid.append(x)
    logits = m.lm_head(oracle.rms_norm(x[-1:], _widen(m.src.final_norm), S.rms_eps))[0]
    return np.stack(hid), logits, kv, wts


@pytest.fixture(scope="module")
def model():
    return oracle.Model(weights(S))


class Check:
    """Follows one engine's sequences through steps and checks each."""

    def __init__(self, run, model):
        self.run, self.m = run, model
        self.len, self.shift, self.score = {}, {}, {}

    def after(self, seqs, tokens, got, fresh=True):
        """tokens: per sequence the ids of this call; got: Run's output with debug dumps."""
        at = 0
        for b, s in enumerate(seqs):
            n, a = len(tokens[b]), self.len.get(s, 0)
            held = _held(self.run, s, a + n)
            hid, logits, kv, wts = _forward(self.m, tokens[b], a, self.shift.get(s, 0), held)
            for l in range(S.n_layers):
                for t in range(n):
                    assert rel_err(got["hidden"][l, at + t], hid[l, t]) <= HIDDEN_REL, (s, l, t)
                for w in range(2):
                    x, want, e = held[l][0][w][a:], kv[l][w], held[l][1][w][a:]
                    bound = np.abs(want) * 2.0 ** -4 + 2.0 ** (e[..., None] - 10.0) + 4 * HIDDEN_REL * np.abs(want).max()
                    assert np.all(np.abs(x - want) <= bound), (s, l, w)
                sc = self.score.setdefault(s, np.zeros((S.n_layers, S.n_kv_heads, MAXC)))
                sc[l, :, :a + n] += wts[l].reshape(S.n_kv_heads, -1, n, a + n).sum((1, 2))
            assert np.max(np.abs(got["logits"][b] - logits)) <= LOGITS_ABS
            check_token(got["next"][b], logits)
            assert np.all(got["pos"][at:at + n] == a + self.shift.get(s, 0) + np.arange(n))
            at += n
            self.len[s] = a + n
            assert self.run.qw.qw_kv_length(self.run.eng.kv, s) == a + n

    def scores(self, seq):
        ptr, ld = self.run.qw.qw_kv8_scores(self.run.eng.kv)
        off = ptr - self.run.eng.pool.data_ptr()
        per = S.n_layers * S.n_kv_heads * ld * 4
        x = self.run.eng.pool[off + seq * per:off + (seq + 1) * per].cpu().numpy().view(np.float32)
        return x.reshape(S.n_layers, S.n_kv_heads, ld)


def _tokens(n, seed):
    return synth.make_tokens(S.vocab, n, seed).tolist()


@pytest.mark.parametrize("lens", [[5], [3, 4], [40, 17, 9], [130, 1]])
def test_prefill_chunk_and_decode_match_the_oracle(run, model, lens):
    seqs = [2 * i + 1 for i in range(len(lens))]
    c = Check(run, model)
    prompts = [_tokens(n, 70 + i) for i, n in enumerate(lens)]
    for s, n in zip(seqs, lens):
        run.qw.qw_kv_reserve(run.eng.kv, s, n + 60, run.eng.stream)
    g = run.prefill(seqs, prompts, reserve=False)
    c.after(seqs, prompts, g)
    for _ in range(2):
        step = g["next"].tolist()
        g = run.decode(seqs, step)
        c.after(seqs, [[t] for t in step], g)
    more = [_tokens(1 + 7 * i, 90 + i) for i in range(len(lens))]  # a chunk over the cached prefix
    g = run.prefill(seqs, more, reserve=False)
    c.after(seqs, more, g)
    step = g["next"].tolist()
    c.after(seqs, [[t] for t in step], run.decode(seqs, step))
    for s in seqs:
        sc = c.scores(s)
        n = c.len[s]
        # every query spreads a weight of one for each head of the group
        total = n * S.n_heads / S.n_kv_heads
        np.testing.assert_allclose(sc[..., :n].sum(-1), total, rtol=1e-5)
        assert np.all(sc[..., n:] == 0)
        # the queries differ by the hidden states' tolerance; a weight by about |t| times that
        np.testing.assert_allclose(sc[..., :n], c.score[s][..., :n], rtol=0.15, atol=0.02)


def test_decode_of_a_larger_batch(run, model):
    seqs = list(range(20))
    c = Check(run, model)
    prompts = [_tokens(3 + b, 200 + b) for b in seqs]
    g = run.prefill(seqs, prompts, reserve_extra=4)
    c.after(seqs, prompts, g)
    step = g["next"].tolist()
    c.after(seqs, [[t] for t in step], run.decode(seqs, step))


@pytest.mark.parametrize("B", [1, 12])
def test_multi_step_graphs_equal_single_steps(run, B):
    import torch
    qw, eng = run.qw, run.eng
    seqs, n, res = list(range(B)), 9, []
    for multi in (True, False):
        qw.qw_kv_reset(eng.kv, -1, eng.stream)
        g = run.prefill(seqs, [_tokens(10 + b, 300 + b) for b in seqs], debug=False, reserve_extra=n + 1)
        first = torch.tensor(g["next"], dtype=torch.int32, device="cuda")
        out = torch.full((n, B), -7, dtype=torch.int32, device="cuda")
        if multi:
            qw.qw_decode_steps(eng.model, eng.kv, seqs, n, first.data_ptr(), out.data_ptr(), eng.stream)
        else:
            for i in range(n):
                qw.qw_decode_step(eng.model, eng.kv, seqs, (first if i == 0 else out[i - 1]).data_ptr(), 0, out[i].data_ptr(), eng.stream)
        assert qw.qw_sync_status(eng.model, eng.stream) == 0
        assert qw.qw_last_launch_count(eng.model) > 0
        res.append((out.cpu().numpy(), run.decode(seqs, out[n - 1].cpu().numpy(), debug=False)["logits"]))
    np.testing.assert_array_equal(res[0][0], res[1][0])
    np.testing.assert_array_equal(res[0][1], res[1][1])


def test_generate_and_eos(run):
    qw, eng = run.qw, run.eng
    seqs, lens, n = [0, 1, 2], [6, 11, 3], 20
    prompt = np.concatenate([np.asarray(_tokens(k, 400 + k), np.int32) for k in lens])
    out = np.zeros((3, n + 1), np.int32)
    for s, k in zip(seqs, lens):
        qw.qw_kv_reserve(eng.kv, s, k + n, eng.stream)
    qw.qw_generate(eng.model, eng.kv, seqs, lens, prompt, n, out, eng.stream)
    assert qw.qw_sync_status(eng.model, eng.stream) == 0
    eos = int(out[1, 4])
    first = [int(np.flatnonzero(np.append(r, eos) == eos)[0]) for r in out]
    qw.qw_kv_reset(eng.kv, -1, eng.stream)
    for s, k in zip(seqs, lens):
        qw.qw_kv_reserve(eng.kv, s, k + n, eng.stream)
    cut, cnt = np.zeros((3, n + 1), np.int32), np.zeros(3, np.int32)
    qw.qw_generate_eos(eng.model, eng.kv, seqs, lens, prompt, n, eos, cut, cnt, eng.stream)
    for b in range(3):
        k = min(first[b], n) + 1
        assert cnt[b] == k
        np.testing.assert_array_equal(cut[b, :k], out[b, :k])
        if first[b] < n:
            assert qw.qw_kv_length(eng.kv, seqs[b]) == lens[b] + first[b]


def test_evict_keeps_positions_and_goes_on(run, model):
    """Two sequences brought back to 48 tokens whenever they pass 64; one is truncated on the way."""
    qw, eng = run.qw, run.eng
    c = Check(run, model)
    seqs, keep, recent = [4, 9], 48, 16
    prompts = [_tokens(60, 500), _tokens(33, 501)]
    g = run.prefill(seqs, prompts, reserve_extra=60)
    c.after(seqs, prompts, g)
    evicted = 0
    for i in range(24):
        step = g["next"].tolist()
        g = run.decode(seqs, step)
        c.after(seqs, [[t] for t in step], g)
        for s in seqs:
            n = c.len[s]
            if n <= 64:
                continue
            before, sc = _held(run, s, n), c.scores(s).copy()
            qw.qw_kv_evict(eng.kv, s, keep, recent, eng.stream)
            assert qw.qw_sync_status(eng.model, eng.stream) == 0
            assert qw.qw_kv_length(eng.kv, s) == keep
            after, sc2 = _held(run, s, keep), c.scores(s)
            for l in range(S.n_layers):
                for h in range(S.n_kv_heads):
                    order = np.lexsort((np.arange(n - recent), -sc[l, h, :n - recent].astype(np.float64)))[:keep - recent]
                    idx = np.concatenate([np.sort(order), np.arange(n - recent, n)])
                    np.testing.assert_array_equal(sc2[l, h, :keep], sc[l, h, idx])
                    assert np.all(sc2[l, h, keep:] == 0)
                    c.score[s][l, h, :keep], c.score[s][l, h, keep:] = c.score[s][l, h, idx], 0
                    for w in range(2):  # the rows themselves, but for codes that became subnormal
                        e = after[l][1][w][:, h]
                        err = np.abs(after[l][0][w][:, h] - before[l][0][w][idx, h])
                        assert np.all(err <= 2.0 ** (e[:, None] - 10.0))
            c.shift[s] = c.shift.get(s, 0) + n - keep
            c.len[s] = keep
            evicted += 1
        if i == 12:  # drop the last 3 tokens of one sequence
            qw.qw_kv_truncate(eng.kv, seqs[0], c.len[seqs[0]] - 3, eng.stream)
            c.len[seqs[0]] -= 3
            assert np.all(c.scores(seqs[0])[..., c.len[seqs[0]]:] == 0)
    assert evicted == 1  # 60 + 5 tokens; then 48 + 19 - 3 = 64, within the budget, and 33 + 24 = 57
    qw.qw_kv_evict(eng.kv, seqs[0], 400, 0, eng.stream)  # within the budget: nothing happens
    assert qw.qw_kv_length(eng.kv, seqs[0]) == c.len[seqs[0]]


def test_refusals(qw, run):
    q, eng = qw.qw, run.eng
    g = run.prefill([0], [_tokens(20, 600)], debug=False)
    del g
    for call in (lambda: q.qw_kv_fill_synthetic(eng.kv, 5, 4, 1, eng.stream),
                 lambda: q.qw_kv_evict(eng.kv, 99, 4, 1, eng.stream), lambda: q.qw_kv_evict(eng.kv, 0, 0, 0, eng.stream),
                 lambda: q.qw_kv_evict(eng.kv, 0, 4, 5, eng.stream), lambda: q.qw_kv_evict(eng.kv, 0, 4, -1, eng.stream)):
        with pytest.raises(q.QwError):
            call()
    assert q.qw_kv8_pool_bytes(eng.model, 0, 1) == 0
    need = q.qw_kv8_pool_bytes(eng.model, 1, 1)
    for ptr, n, seqs in ((eng.pool.data_ptr() + 16, need, 1), (0, need, 1), (eng.pool.data_ptr(), need - 1, 1), (eng.pool.data_ptr(), need, 0)):
        with pytest.raises(q.QwError):
            q.qw_kv8_alloc(eng.model, ptr, n, seqs, False, eng.stream)
    f16 = ctypes.c_void_p()
    import torch
    pool = torch.empty(q.qw_kv_pool_bytes(eng.model, 2, 1), dtype=torch.uint8, device="cuda")
    assert q.load().qw_kv_alloc(eng.model, pool.data_ptr(), pool.numel(), 1, eng.stream.cuda_stream, ctypes.byref(f16)) == 0
    assert q.load().qw_kv_evict(f16, 0, 4, 1, eng.stream.cuda_stream) == -7
    p = ctypes.c_void_p()
    assert q.load().qw_kv8_scores(f16, ctypes.byref(p), None) == -7
    q.qw_free_kv(f16)
    # positions go on after an eviction, so they still count against the context
    q.qw_kv_reserve(eng.kv, 1, 500, eng.stream)
    run.prefill([1], [_tokens(250, 601)], debug=False, reserve=False)
    run.prefill([1], [_tokens(250, 602)], debug=False, reserve=False)
    q.qw_kv_evict(eng.kv, 1, 100, 10, eng.stream)
    assert q.qw_kv_length(eng.kv, 1) == 100
    with pytest.raises(q.QwError):
        run.prefill([1], [_tokens(13, 603)], debug=False, reserve=False)
    run.prefill([1], [_tokens(12, 604)], debug=False, reserve=False)
    with pytest.raises(q.QwError):
        run.decode([1], [3], debug=False)
