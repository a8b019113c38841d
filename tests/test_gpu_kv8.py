"""GPU parity of the 8-bit paged cache's operators (qw_kv8_append, _read, _attn, _evict) with the
fp64 oracle.

Append, read and evict are exact: every value they hold follows from fp16 values by exact or
once-rounded steps that the oracle repeats. Attention: see _check_attn for its tolerances."""

import numpy as np
import pytest

from oracle import kv8

pytestmark = pytest.mark.gpu

F16, BF16, F32 = "f16", "bf16", "f32"


def _dt(name):
    import torch
    return {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}[name]


class Case:
    """A pool of shuffled pages with garbage in every unused byte, its oracle, and device copies of
    the batch's description."""

    def __init__(self, qw, ends, n_kv, hd, seed=0, spare=6, max_pages=None):
        import torch
        self.torch, self.qw = torch, qw.qw
        self.rng = np.random.default_rng(seed)
        self.n_kv, self.hd, self.B = n_kv, hd, len(ends)
        need = [(e + 15) // 16 for e in ends]
        self.maxp = max_pages or max(1, max(need))
        self.n_pages = sum(need) + spare
        perm = self.rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((self.B, self.maxp), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        self.orc = kv8.Cache(self.n_pages, n_kv, hd)
        self.blk = qw.qw.qw_kv8_block_bytes(hd)
        raw = self.rng.integers(0, 256, (self.n_pages, n_kv, self.blk)).astype(np.uint8)
        raw[..., ::7] = 0x7F  # NaN codes
        raw[..., 32 * hd:] = 0xFF  # scales that are NaN
        self.blocks = torch.from_numpy(raw).cuda()
        self.dtable = torch.from_numpy(self.table).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.view = qw.qw.qw_kv8_view(self.blocks.data_ptr(), self.n_pages, n_kv, hd, self.dtable.data_ptr(), self.maxp)

    def i32(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def rows(self, T, heads, dtype, pad=0, scale=1.0, extra=0):
        """[T + extra, heads * hd + pad] of `dtype`, and its [T, heads, hd] in fp64."""
        x = self.rng.normal(0, scale, (T + extra, heads * self.hd + pad)).astype(np.float32)
        x[:, 5::37] *= 6
        t = self.torch.from_numpy(x).cuda().to(_dt(dtype))
        return t, t[:T].double().cpu().numpy()[:, :heads * self.hd].reshape(T, heads, self.hd)

    def append(self, starts, lens, dtype=F16, pad=0, scale=0.5, oracle=True):
        starts, lens = np.asarray(starts), np.asarray(lens)
        cu = np.concatenate([[0], np.cumsum(lens)])
        T = int(cu[-1])
        k, kf = self.rows(T, self.n_kv, dtype, pad, 1.0)
        v, vf = self.rows(T, self.n_kv, dtype, pad, scale)
        ds, dc = self.i32(starts), self.i32(cu)
        self.qw.qw_kv8_append(self.view, self.B, T, max(1, int(lens.max())), ds.data_ptr(), dc.data_ptr(), k.data_ptr(),
                              k.stride(0), v.data_ptr(), v.stride(0), getattr(self.qw, "QW_" + dtype.upper()), self.status.data_ptr())
        if oracle:
            for b in range(self.B):
                self.orc.append(self.table[b], int(starts[b]),
                                [x[cu[b]:cu[b + 1]].astype(np.float16).astype(np.float64) for x in (kf, vf)])
        self.last = (k, v, ds, dc, T, int(lens.max()))

    def check_cache(self, ends):
        got = kv8.Cache.from_blocks(self.blocks.cpu().numpy(), self.hd)
        for b, e in enumerate(ends):
            pages = self.table[b, :(e + 15) // 16]
            for w in range(2):
                np.testing.assert_array_equal(got.e[w][pages], self.orc.e[w][pages])
                np.testing.assert_array_equal(got.x[w][pages], self.orc.x[w][pages])

    def bits(self):
        return int(self.status.item())

    def attn(self, starts, lens, G, dtype=F16, pad=0, score=None, lse=True, qscale=1.5, stream=None, bound=0):
        torch = self.torch
        starts, lens = np.asarray(starts), np.asarray(lens)
        cu = np.concatenate([[0], np.cumsum(lens)])
        T, Hq = int(cu[-1]), self.n_kv * G
        q, qf = self.rows(T, Hq, dtype, pad, qscale)
        mk, ml = int((starts + lens).max()) + bound, int(lens.max()) + bound
        mk = min(mk, self.maxp * 16)
        out = torch.full((T + 3, Hq * self.hd + pad), 7.0, dtype=_dt(dtype), device="cuda")
        z = torch.full((T + 3, Hq), 7.0, device="cuda") if lse else None
        sc = so = None
        if score is not None:
            sc = torch.from_numpy(score).cuda()
            so = torch.full_like(sc, -3.0)
        nb = self.qw.qw_kv8_attn_ws_bytes(self.view, self.B, T, ml, mk, Hq, score is not None)
        ws = torch.full((nb,), 0xAB, dtype=torch.uint8, device="cuda")
        ds, dc = self.i32(starts), self.i32(cu)
        scale = self.hd ** -0.5
        call = lambda: self.qw.qw_kv8_attn(  # noqa: E731
            self.view, self.B, T, ml, mk, ds.data_ptr(), dc.data_ptr(), q.data_ptr(), q.stride(0), Hq,
            getattr(self.qw, "QW_" + dtype.upper()), scale, out.data_ptr(), out.stride(0), z.data_ptr() if lse else 0,
            sc.data_ptr() if score is not None else 0, so.data_ptr() if score is not None else 0,
            sc.shape[2] if score is not None else 0, ws.data_ptr(), nb, self.status.data_ptr(), stream)
        call()
        r = dict(out=out, lse=z, score=so, q=qf, cu=cu, starts=starts, lens=lens, call=call, dtype=dtype, G=G, scale=scale,
                 score_in=score, keep=(q, ws, ds, dc, sc))
        return r

    def check_attn(self, r):
        """Errors: the logit t of a key is off by at most d = (hd + 8) 2^-24 scale |q||k| (fp32 sums
        in any order, the log2 factor and the exponential's 2^-22), a weight by 2 d and, for the PV
        product, its fp16 rounding 2^-11; the normaliser by 2 d; the output's own rounding half an eps.
        Weights below the fp16 normals are off by at most 2^-25 against a largest weight of 2^8."""
        torch = self.torch
        torch.cuda.synchronize()
        eps = torch.finfo(_dt(r["dtype"])).eps / 2
        T, Hq, hd = int(r["cu"][-1]), self.n_kv * r["G"], self.hd
        out = r["out"].double().cpu().numpy()
        assert np.all(out[T:] == 7.0) and np.all(out[:, Hq * hd:] == 7.0)  # untouched
        got = out[:T, :Hq * hd].reshape(T, Hq, hd)
        lse = r["lse"].double().cpu().numpy() if r["lse"] is not None else None
        for b in range(self.B):
            a, z, s = r["cu"][b], r["cu"][b + 1], int(r["starts"][b])
            n = z - a
            if n:
                q = r["q"][a:z]
                want, wl, w, mag = self.orc.attention(self.table[b], s, q, r["scale"])
                k = np.abs(self.orc.rows(0, self.table[b], s + n))
                v = np.abs(self.orc.rows(1, self.table[b], s + n))
                kq = np.stack([(np.abs(q[:, h]) @ k[:, h // r["G"]].T).max(1) for h in range(Hq)], 1)  # [n, Hq]
                d = (hd + 8) * 2.0 ** -24 * r["scale"] * kq + 2.0 ** -22
                tol = mag * (2.0 ** -11 + 4 * d[..., None]) + np.abs(want) * eps + 2.0 ** -25 + (s + n) * 2.0 ** -33 * v.max(initial=0)
                err = np.abs(got[a:z] - want)
                assert np.all(err <= tol), (b, float((err / tol).max()))
                if lse is not None:
                    assert np.all(np.abs(lse[a:z] - wl) <= 2 * d + np.abs(wl) * 2.0 ** -22)
            if r["score"] is not None:
                sc = r["score"][b].double().cpu().numpy()
                assert np.all(sc[:, (s + n) if n else 0:] == -3.0)
                if n:
                    add = w.reshape(self.n_kv, r["G"], n, s + n).sum((1, 2))
                    base = r["score_in"][b][:, :s + n].astype(np.float64)
                    dd = d.max()
                    # weights off by 3 d each (d in the logit, 2 d in the normaliser's log), fp32 sums of n G terms
                    tol = add * (4 * dd + n * r["G"] * 2.0 ** -24) + (base + add) * 2.0 ** -23 + 1e-30
                    err = np.abs(sc[:, :s + n] - (base + add))
                    assert np.all(err <= tol), (b, float((err / tol).max()))
        if lse is not None:
            assert np.all(lse[T:] == 7.0)


def _scores(c, ends, seed=0):
    return np.random.default_rng(seed).random((c.B, c.n_kv, max(ends) + 3)).astype(np.float32)


# ---- append and read -----------------------------------------------------------------------

APPENDS = [  # head_dim, n_kv, type, [(starts, lens), ...] of calls in a row
    (128, 2, F16, [([0, 0, 0], [1, 16, 17]), ([1, 16, 17], [1, 1, 20])]),
    (128, 1, BF16, [([0], [5]), ([5], [1]), ([6], [10]), ([16], [1])]),
    (64, 3, F16, [([0, 0], [40, 3]), ([40, 3], [0, 33])]),
    (64, 8, F32, [([0, 0, 0, 0], [0, 31, 16, 100]), ([0, 31, 16, 100], [2, 2, 2, 2])]),
    (128, 8, F32, [([0], [200]), ([37], [9])]),  # a second call inside the sequence: the rest is dropped
]


@pytest.mark.parametrize("hd,n_kv,dtype,calls", APPENDS)
def test_append_matches_the_oracle_bit_for_bit(qw, hd, n_kv, dtype, calls):
    ends = np.max([np.add(s, n) for s, n in calls], 0)
    c = Case(qw, ends.tolist(), n_kv, hd, seed=hd + n_kv)
    for i, (s, n) in enumerate(calls):
        c.append(s, n, dtype, pad=8 * i, scale=0.2 * 30 ** i)  # later tokens are larger: exponents grow
    last = np.add(*calls[-1])
    c.check_cache(last)
    assert c.bits() == 0


@pytest.mark.parametrize("hd,dtype", [(128, F16), (64, BF16), (128, F32)])
def test_read_returns_the_held_values(qw, hd, dtype):
    import torch
    c = Case(qw, [50, 17, 33], 2, hd, seed=3)
    c.append([0, 0, 0], [50, 17, 33])
    starts, lens = np.array([0, 16, 15]), np.array([50, 1, 0])
    cu = np.concatenate([[0], np.cumsum(lens)])
    out = [torch.full((60, 2 * hd + 8), 9.0, dtype=_dt(dtype), device="cuda") for _ in range(2)]
    ds, dc = c.i32(starts), c.i32(cu)
    c.qw.qw_kv8_read(c.view, 3, 51, 50, ds.data_ptr(), dc.data_ptr(), out[0].data_ptr(), out[0].stride(0), out[1].data_ptr(),
                     out[1].stride(0), getattr(c.qw, "QW_" + dtype.upper()), c.status.data_ptr())
    for w in range(2):
        got = out[w].cpu()
        assert bool((got[51:] == 9).all()) and bool((got[:, 2 * hd:] == 9).all())
        for b in range(3):
            want = c.orc.rows(w, c.table[b], int(starts[b] + lens[b]))[int(starts[b]):]
            want = torch.from_numpy(want).to(_dt(dtype)).reshape(lens[b], 2 * hd)
            assert torch.equal(got[cu[b]:cu[b + 1], :2 * hd], want)
    assert c.bits() == 0


def test_read_of_bad_entries_gives_zeros(qw):
    """A start past the table and a page outside the pool: zeros and the status bit, the rest as ever."""
    import torch
    c = Case(qw, [40, 40, 40], 2, 64, seed=19)
    c.append([0, 0, 0], [40, 40, 40])
    bad = c.table.copy()
    bad[1, 1] = c.n_pages
    c.dtable.copy_(torch.from_numpy(bad))
    out = torch.full((2, 63, 128), 7.0, dtype=torch.float16, device="cuda")
    ds, dc = c.i32([3, 0, 20]), c.i32([0, 20, 40, 60])
    for start in (3, 10 ** 6):
        ds[0] = start
        c.status.zero_()
        c.qw.qw_kv8_read(c.view, 3, 60, 20, ds.data_ptr(), dc.data_ptr(), out[0].data_ptr(), 128, out[1].data_ptr(), 128,
                         c.qw.QW_F16, c.status.data_ptr())
        assert c.bits() == c.qw.QW_KV8_BAD_POS
        for w in range(2):
            got = out[w].double().cpu().numpy().reshape(63, 2, 64)
            want = np.concatenate([c.orc.rows(w, c.table[0], 23)[3:], c.orc.rows(w, c.table[1], 20), c.orc.rows(w, c.table[2], 40)[20:]])
            want[36:40] = 0  # page 1 of entry 1
            if start != 3:
                want[:20] = 0
            np.testing.assert_array_equal(got[:60], want)
            assert np.all(got[60:] == 7.0)


def test_append_flags_what_fp16_cannot_hold_and_bad_pages(qw):
    import torch
    c = Case(qw, [20, 20], 1, 128, seed=5)
    c.append([0, 0], [20, 20], F32)
    k, v, ds, dc, T, ml = c.last
    k[3, 7], k[4, 8], v[25, 1] = float("nan"), 1e6, float("-inf")
    c.qw.qw_kv8_append(c.view, 2, T, ml, ds.data_ptr(), dc.data_ptr(), k.data_ptr(), 128, v.data_ptr(), 128, c.qw.QW_F32, c.status.data_ptr())
    assert c.bits() == c.qw.QW_KV8_RANGE
    kk = k.cpu().numpy().astype(np.float64).reshape(T, 1, 128)
    vv = v.cpu().numpy().astype(np.float64).reshape(T, 1, 128)
    for x in (kk, vv):
        x[~(np.abs(x) <= 65504)] = 0
    for b in range(2):
        c.orc.append(c.table[b], 0, [x[20 * b:20 * b + 20].astype(np.float16).astype(np.float64) for x in (kk, vv)])
    c.check_cache([20, 20])
    before = c.blocks.clone()
    bad = c.table.copy()
    bad[0, 1], bad[1, 0] = c.n_pages, -1
    c.dtable.copy_(torch.from_numpy(bad))
    c.status.zero_()
    c.append([0, 0], [20, 20], oracle=False)
    assert c.bits() == c.qw.QW_KV8_BAD_POS
    changed = (before != c.blocks).flatten(1).any(1).cpu().numpy()
    assert set(np.flatnonzero(changed)) <= {c.table[0, 0], c.table[1, 1]}
    # lengths that break their bounds: nothing is written
    before = c.blocks.clone()
    c.dtable.copy_(torch.from_numpy(c.table))
    for starts, cu, T, ml in (([-1, 0], [0, 5, 5], 5, 5), ([0, 20], [0, 0, 13], 13, 13), ([0, 0], [0, 9, 9], 9, 8),
                              ([0, 0], [0, 0, 9], 8, 16), ([0, 0], [0, 0, -4], 8, 16), ([2147483640, 0], [0, 9, 9], 9, 9)):
        c.status.zero_()
        ds, dc = c.i32(starts), c.i32(cu)
        c.qw.qw_kv8_append(c.view, 2, T, ml, ds.data_ptr(), dc.data_ptr(), k.data_ptr(), 128, v.data_ptr(), 128, c.qw.QW_F32,
                           c.status.data_ptr())
        assert c.bits() == c.qw.QW_KV8_BAD_POS
        assert torch.equal(before, c.blocks)


# ---- attention -----------------------------------------------------------------------------

ATTN = [  # head_dim, n_kv, group, type, starts, lens
    (128, 2, 2, F16, [0], [1]),
    (128, 2, 2, F16, [15, 16, 31], [1, 1, 1]),
    (128, 1, 1, BF16, [100, 0, 47], [1, 1, 0]),
    (128, 8, 2, F16, [1000, 3, 517, 64], [1, 1, 1, 1]),
    (64, 2, 7, BF16, [130, 70], [1, 1]),
    (64, 1, 16, F16, [300], [1]),
    (64, 4, 3, F16, [33, 0, 8], [5, 2, 4]),        # a few queries of every entry
    (128, 1, 8, BF16, [250, 2], [2, 2]),
    (128, 2, 2, F16, [0, 0], [70, 129]),            # prompts
    (128, 1, 4, BF16, [200, 13, 0], [90, 1, 33]),   # chunks over a prefix
    (64, 2, 5, F16, [500, 77], [64, 200]),
    (64, 1, 1, BF16, [0, 1], [300, 257]),
    (128, 1, 16, F16, [40], [65]),
    (128, 1, 3, F16, [3000], [40]),
]


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("hd,n_kv,G,dtype,starts,lens", ATTN)
def test_attention(qw, hd, n_kv, G, dtype, starts, lens, score):
    ends = np.add(starts, lens)
    c = Case(qw, ends.tolist(), n_kv, hd, seed=hd + 7 * G + len(starts))
    c.append([0] * len(ends), ends)
    sc = _scores(c, ends) if score else None
    r = c.attn(starts, lens, G, dtype, pad=16, score=sc, lse=not score or G % 2 == 0)
    c.check_attn(r)
    again = r["out"].clone()
    r["call"]()
    assert c.torch.equal(again, r["out"]) and c.bits() == 0


def test_attention_with_loose_bounds(qw):
    """max_len and max_keys larger than any entry, more table columns than pages."""
    for lens in ([1, 1], [1, 30], [60, 150]):
        c = Case(qw, [200, 411], 2, 128, seed=8, max_pages=90)
        c.append([0, 0], [200, 411])
        starts = [200 - lens[0], 411 - lens[1]]
        c.check_attn(c.attn(starts, lens, 2, bound=500, score=np.zeros((2, 2, 1440), np.float32)))
        assert c.bits() == 0


@pytest.mark.parametrize("hd,G,dtype", [(64, 7, BF16), (128, 2, F16)])
def test_scores_of_a_ragged_batch(qw, hd, G, dtype):
    """Entries of many, one and no rows: each finds its own query tiles."""
    starts, lens = [0, 50, 77, 3, 200, 16], [130, 0, 1, 257, 64, 0]
    ends = np.add(starts, lens)
    c = Case(qw, ends.tolist(), 2, hd, seed=31 + hd)
    c.append([0] * len(ends), ends)
    c.check_attn(c.attn(starts, lens, G, dtype, pad=16, score=_scores(c, ends)))
    assert c.bits() == 0


@pytest.mark.parametrize("n_kv,G,n,dtype,score", [(1, 16, 1, F16, True), (2, 12, 1, BF16, True), (2, 2, 6, F16, True),
                                                  (1, 8, 1, F16, True), (3, 5, 3, BF16, False)])
def test_few_rows_over_long_caches(qw, n_kv, G, n, dtype, score):
    """Up to 16 rows a KV head whose keys many CTAs share, with and without scores."""
    starts = [2900, 1500, 31]
    c = Case(qw, [x + n for x in starts], n_kv, 128, seed=53 + G)
    c.append([0] * 3, [x + n for x in starts])
    r = c.attn(starts, [n] * 3, G, dtype, pad=8, score=_scores(c, [x + n for x in starts]) if score else None)
    c.check_attn(r)
    again = r["out"].clone()
    r["call"]()
    assert c.torch.equal(again, r["out"]) and c.bits() == 0


@pytest.mark.parametrize("lens", [[1, 1], [5, 3], [90, 70]])
def test_query_rows_that_are_not_numbers_stay_alone(qw, lens):
    """A NaN or an infinity in one query row: every other row keeps its bits."""
    import torch
    starts, G = [200, 410], 2
    ends = np.add(starts, lens)
    c = Case(qw, ends.tolist(), 2, 64, seed=61)
    c.append([0, 0], ends)
    r = c.attn(starts, lens, G, F16)
    c.check_attn(r)
    q, want = r["keep"][0], r["out"].clone()
    T = sum(lens)
    for row, head, x in ((0, 1, float("nan")), (T - 1, 2, float("inf"))):
        q[row, head * 64 + 7] = x
        r["out"].fill_(7.0)
        r["call"]()
        same = torch.ones(T, 4, dtype=torch.bool, device="cuda")
        same[0, 1] = False
        same[row, head] = False
        got = r["out"][:T, :256].reshape(T, 4, 64)
        assert torch.equal(got[same], want[:T, :256].reshape(T, 4, 64)[same])
        assert bool(got[0, 1].isnan().all())
    assert c.bits() == 0


@pytest.mark.parametrize("lens", [[1, 1, 1], [40, 9, 100]])
def test_entries_share_a_prefix(qw, lens):
    """Three entries over the same first pages, each with its own last ones."""
    own = [(300 + n + 15) // 16 * 16 for n in lens]
    c = Case(qw, own, 2, 128, seed=67)
    c.table[:, :18] = c.table[0, :18]
    c.dtable.copy_(c.torch.from_numpy(c.table))
    c.append([0, 288, 288], [288, 12, 12])       # the prefix once; positions 288 .. 299 of the other two
    c.append([288, 300, 300], [12 + lens[0], lens[1], lens[2]])
    r = c.attn([300] * 3, lens, 2, score=_scores(c, own))
    c.check_attn(r)
    assert c.bits() == 0


@pytest.mark.parametrize("lens", [[1, 1], [100, 33]])
def test_blocks_past_four_gib(qw, lens):
    """The same pages at the start of a pool and behind its first 2^32 bytes give the same bits."""
    import torch
    ends = [500, 700]
    starts = [e - n for e, n in zip(ends, lens)]
    res = []
    for far in (False, True):
        c = Case(qw, ends, 8, 128, seed=71)
        if far:
            page = 8 * c.blk
            off = 2 ** 32 // page + 3
            big = torch.empty((off + c.n_pages) * page, dtype=torch.uint8, device="cuda")
            big[off * page:] = c.blocks.reshape(-1)
            c.blocks = big
            c.dtable.copy_(torch.from_numpy(np.where(c.table >= 0, c.table + off, -1).astype(np.int32)))
            c.view = c.qw.qw_kv8_view(big.data_ptr(), off + c.n_pages, 8, 128, c.dtable.data_ptr(), c.maxp)
        c.append([0, 0], ends, oracle=False)
        r = c.attn(starts, lens, 2, score=_scores(c, ends))
        kept, new, so = _evict(c, ends, 200, 20, _scores(c, ends), True, None)
        tail = c.blocks.reshape(-1)[-c.n_pages * 8 * c.blk:].clone()
        res.append((r["out"], r["lse"], r["score"], torch.from_numpy(kept), torch.from_numpy(so), tail))
        assert c.bits() == 0
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_calls_of_two_threads(qw):
    """Decode calls of different sizes from two host threads, each on its own stream."""
    import threading
    cases = []
    for seed, G, n in ((41, 1, 700), (42, 8, 900)):
        c = Case(qw, [n, n + 31], 2, 128, seed=seed)
        c.append([0, 0], [n, n + 31])
        r = c.attn([n - 2, n + 29], [2, 2], G)
        c.check_attn(r)
        cases.append((c, r, r["out"].clone()))
    c.torch.cuda.synchronize()
    wrong = []

    def work(c, r, want):
        with c.torch.cuda.stream(c.torch.cuda.Stream()):
            for _ in range(50):
                r["out"].fill_(7.0)  # as the rows behind the last entry are
                r["call"]()
                if not c.torch.equal(r["out"], want):
                    wrong.append(1)

    threads = [threading.Thread(target=work, args=x) for x in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and all(x[0].bits() == 0 for x in cases)


@pytest.mark.parametrize("lens", [[1, 1], [40, 80]])
def test_attention_over_scales_far_apart(qw, lens):
    """Pages whose V differ by 2^30 and K rows that decide the softmax: a page of tiny values that
    gets all the weight next to a page of huge ones that gets none, and the reverse."""
    hd = 128
    c = Case(qw, [160, 160], 1, hd, seed=9)
    T = 320
    k = c.rng.normal(0, 1, (T, 1, hd)).astype(np.float16)
    v = c.rng.normal(0, 1, (T, 1, hd)).astype(np.float16)
    for t in range(T):
        v[t] *= [np.float16(2.0 ** -14), np.float16(1.0), np.float16(4096.0)][t // 16 % 3]
        k[t] *= [np.float16(1), np.float16(0.1), np.float16(8)][(t // 16 + t // 160) % 3]
    dk, dv = c.torch.from_numpy(k).cuda(), c.torch.from_numpy(v).cuda()
    ds, dc = c.i32([0, 0]), c.i32([0, 160, 320])
    c.qw.qw_kv8_append(c.view, 2, T, 160, ds.data_ptr(), dc.data_ptr(), dk.data_ptr(), hd, dv.data_ptr(), hd, c.qw.QW_F16, c.status.data_ptr())
    for b in range(2):
        c.orc.append(c.table[b], 0, [x[160 * b:160 * b + 160].astype(np.float64) for x in (k, v)])
    c.check_cache([160, 160])
    for dtype in (F16, BF16):
        c.check_attn(c.attn([160 - n for n in lens], lens, 4, dtype))


def test_attention_reports_bad_pages_and_lengths(qw):
    import torch
    for lens in ([1, 1], [50, 60]):
        c = Case(qw, [100, 100], 2, 128, seed=10)
        c.append([0, 0], [100, 100])
        bad = c.table.copy()
        bad[0, 2] = c.n_pages + 5
        c.dtable.copy_(torch.from_numpy(bad))
        starts = [100 - n for n in lens]
        r = c.attn(starts, lens, 2, score=np.zeros((2, 2, 112), np.float32))
        assert c.bits() == c.qw.QW_KV8_BAD_POS
        c.status.zero_()
        c.dtable.copy_(torch.from_numpy(c.table))
        r2 = c.attn([5000, starts[1]], lens, 2)  # beyond max_pages
        assert c.bits() == c.qw.QW_KV8_BAD_POS
        out = r2["out"].cpu()
        assert bool((out[:lens[0], :512] == 0).all())
        del r
        # the other entry is as ever
        c.status.zero_()
        r2["starts"] = np.array([0, starts[1]])
        a, z = r2["cu"][1], r2["cu"][2]
        want = c.orc.attention(c.table[1], starts[1], r2["q"][a:z], r2["scale"])[0]
        assert np.abs(out[a:z, :512].double().numpy().reshape(want.shape) - want).max() < 0.02


def test_attention_captured_and_replayed_with_new_lengths(qw):
    """One captured append + attention + scores, replayed as the sequences grow on the device."""
    import torch
    c = Case(qw, [64, 64], 2, 128, seed=11)
    c.append([0, 0], [20, 33])
    lens = np.array([20, 33])
    k, v, q = (torch.zeros((2, n * 128), dtype=torch.float16, device="cuda") for n in (2, 2, 4))
    start, cu = c.i32(lens), c.i32([0, 1, 2])
    out = torch.zeros((2, 512), dtype=torch.float16, device="cuda")
    sc = torch.zeros((2, 2, 64), device="cuda")
    nb = c.qw.qw_kv8_attn_ws_bytes(c.view, 2, 2, 1, 64, 4, True)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.qw.qw_kv8_append(c.view, 2, 2, 1, start.data_ptr(), cu.data_ptr(), k.data_ptr(), 256, v.data_ptr(), 256, c.qw.QW_F16, c.status.data_ptr())
        c.qw.qw_kv8_attn(c.view, 2, 2, 1, 64, start.data_ptr(), cu.data_ptr(), q.data_ptr(), 512, 4, c.qw.QW_F16, 128 ** -0.5,
                         out.data_ptr(), 512, 0, sc.data_ptr(), sc.data_ptr(), 64, ws.data_ptr(), nb, c.status.data_ptr())
        start.add_(1)
    want_sc = np.zeros((2, 2, 64))
    for step in range(30):
        xk, xv, xq = (c.rng.normal(0, 1, t.shape).astype(np.float16) for t in (k, v, q))
        for t, x in ((k, xk), (v, xv), (q, xq)):
            t.copy_(torch.from_numpy(x))
        g.replay()
        torch.cuda.synchronize()
        for b in range(2):
            s = int(lens[b]) + step
            c.orc.append(c.table[b], s, [x[b].astype(np.float64).reshape(1, 2, 128) for x in (xk, xv)])
            want, _, w, mag = c.orc.attention(c.table[b], s, xq[b].astype(np.float64).reshape(1, 4, 128), 128 ** -0.5)
            want_sc[b, :, :s + 1] += w.reshape(2, 2, s + 1).sum(1)
            got = out[b].double().cpu().numpy().reshape(1, 4, 128)
            assert np.all(np.abs(got - want) <= mag * 2.0 ** -10 + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)
    np.testing.assert_allclose(sc.cpu().numpy(), want_sc, rtol=2e-5, atol=1e-6)
    c.check_cache((lens + 30).tolist())
    assert c.bits() == 0


def test_captured_behind_copies_and_other_streams(qw):
    """Calls captured right after a copy, after a join with another captured stream, and after each
    other: every one sees what came before it in the graph."""
    import torch
    c = Case(qw, [300, 40], 2, 128, seed=15)
    c.append([0, 0], [300, 40])
    k, v, ds, dc, T, ml = c.last
    lens = np.array([300, 40])
    q, qf = c.rows(2, 4, F16)
    src = torch.zeros_like(q)
    start, cu = c.i32(lens - 1), c.i32([0, 1, 2])
    hk, hv = torch.zeros_like(k), torch.zeros_like(v)
    out = torch.zeros((2, 512), dtype=torch.float16, device="cuda")
    nb = c.qw.qw_kv8_attn_ws_bytes(c.view, 2, 2, 1, 304, 4, False)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hk.copy_(k)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            hv.copy_(v)
            src.copy_(q)
        main.wait_stream(side)
        c.qw.qw_kv8_append(c.view, 2, T, ml, ds.data_ptr(), dc.data_ptr(), hk.data_ptr(), 256, hv.data_ptr(), 256, c.qw.QW_F16, c.status.data_ptr())
        c.qw.qw_kv8_attn(c.view, 2, 2, 1, 304, start.data_ptr(), cu.data_ptr(), src.data_ptr(), 512, 4, c.qw.QW_F16, 128 ** -0.5,
                         out.data_ptr(), 512, 0, 0, 0, 0, ws.data_ptr(), nb, c.status.data_ptr())
        again = out.clone()
    for seed in range(3):
        new = [torch.randn(x.shape, device="cuda").half() for x in (k, v, q)]
        for x, y in zip((k, v, q), new):
            x.copy_(y)
        c.blocks.fill_(0x7F)
        g.replay()
        torch.cuda.synchronize()
        at = 0
        for b in range(2):
            x = [y[at:at + lens[b]].double().cpu().numpy().reshape(-1, 2, 128) for y in new[:2]]
            at += int(lens[b])
            c.orc.append(c.table[b], 0, x)
            want = c.orc.attention(c.table[b], int(lens[b]) - 1, new[2][b].double().cpu().numpy().reshape(1, 4, 128), 128 ** -0.5)
            got = again[b].double().cpu().numpy().reshape(1, 4, 128)
            assert np.all(np.abs(got - want[0]) <= want[3] * 2.0 ** -10 + np.abs(want[0]) * 2.0 ** -11 + 2.0 ** -24)
        c.check_cache(lens.tolist())
    assert c.bits() == 0


def test_two_streams_with_their_own_workspaces(qw):
    import torch
    c = Case(qw, [900, 700], 2, 128, seed=12)
    c.append([0, 0], [900, 700])
    torch.cuda.synchronize()
    runs = []
    for i in range(6):
        st = torch.cuda.Stream()
        n = [1, 1] if i % 2 else [40, 65]
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            runs.append(c.attn([900 - n[0], 700 - n[1]], n, 2, stream=st, score=np.zeros((2, 2, 912), np.float32)))
    for r in runs:
        c.check_attn(r)
    assert c.bits() == 0


# ---- eviction ------------------------------------------------------------------------------

def _evict(c, lens, keep, recent, score, in_place, dst=None):
    torch = c.torch
    sc = torch.from_numpy(score).cuda()
    so = sc if in_place else torch.full_like(sc, -5.0)
    kept = torch.full((c.B, c.n_kv, keep), -9, dtype=torch.int32, device="cuda")
    new = torch.zeros(c.B, dtype=torch.int32, device="cuda")
    dl = c.i32(lens)
    dd = None
    if dst is not None:
        dd = torch.from_numpy(dst).cuda()
    c.qw.qw_kv8_evict(c.view, c.B, min(max(1, int(max(lens))), sc.shape[2], c.maxp * 16), dl.data_ptr(), keep, recent, dd.data_ptr() if dd is not None else 0,
                      sc.data_ptr(), so.data_ptr(), sc.shape[2], kept.data_ptr(), new.data_ptr(), c.status.data_ptr())
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new.cpu().numpy(), so.cpu().numpy()


EVICT = [  # head_dim, n_kv, lens, keep, recent
    (128, 2, [200, 64, 65, 1, 0], 64, 16),
    (64, 1, [500], 1, 0),
    (64, 3, [333, 47], 33, 33),
    (128, 1, [1500, 40], 700, 0),
    (64, 2, [2100], 17, 3),
    (128, 8, [4100], 1000, 250),
    (128, 2, [9000, 30, 6500], 1000, 250),             # a cluster a head
    (64, 1, [50001], 3000, 100),                       # slices beyond a CTA's shared memory
    (64, 1, [33 + i % 40 for i in range(160)], 40, 5),  # more short entries than SMs
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("hd,n_kv,lens,keep,recent", EVICT)
def test_evict(qw, hd, n_kv, lens, keep, recent, in_place):
    spare = sum((min(n, keep) + 15) // 16 for n in lens) + 2
    c = Case(qw, lens, n_kv, hd, seed=sum(lens), spare=spare)
    c.append([0] * len(lens), lens)
    sc = c.rng.random((c.B, n_kv, max(lens) + 5)).astype(np.float32) ** 3
    sc[sc < 0.05] = 0
    sc = np.where(c.rng.random(sc.shape) < 0.3, np.round(sc * 8) / 8, sc).astype(np.float32)  # ties
    sc[..., 3::50] *= -1
    sc[..., 11::97] = np.nan
    sc[..., 12::97] = np.inf
    dst = None
    if not in_place:
        dst = np.full_like(c.table, -1)
        at = 0
        for b, n in enumerate(lens):
            m = (min(n, keep) + 15) // 16
            dst[b, :m] = c.free[at:at + m]
            at += m
    kept, new, so = _evict(c, lens, keep, recent, sc, in_place, dst)
    assert c.bits() == 0
    to = c.table if in_place else dst
    for b, n in enumerate(lens):
        m = min(n, keep)
        own = c.table[b]
        want_k, want_s = c.orc.evict(own, own if in_place else dst[b], n, keep, recent, sc[b])
        np.testing.assert_array_equal(kept[b], want_k)
        np.testing.assert_array_equal(so[b, :, :n], want_s if n > keep or not in_place else sc[b, :, :n])
        np.testing.assert_array_equal(so[b, :, n:], sc[b, :, n:] if in_place else np.full_like(so[b, :, n:], -5.0))
    np.testing.assert_array_equal(new, np.minimum(lens, keep))
    c.table = to
    c.check_cache([min(n, keep) for n in lens])


@pytest.mark.parametrize("rows_in_place", [False, True])
@pytest.mark.parametrize("lens,keep,recent", [([200, 30], 64, 16), ([1500, 900], 700, 100), ([7000, 10], 600, 0)])
def test_evict_rows_and_scores_apart(qw, lens, keep, recent, rows_in_place):
    """Rows in place with the scores going elsewhere, and the reverse."""
    import torch
    c = Case(qw, lens, 2, 64, seed=83 + keep, spare=2 * ((keep + 15) // 16))
    c.append([0, 0], lens)
    sc = c.rng.random((2, 2, max(lens) + 5)).astype(np.float32)
    dst = np.full_like(c.table, -1)
    for b, n in enumerate(lens):
        m = (min(n, keep) + 15) // 16
        dst[b, :m] = c.free[b * ((keep + 15) // 16):][:m]
    dsc = torch.from_numpy(sc).cuda()
    so = torch.full_like(dsc, -5.0) if rows_in_place else dsc
    kept = torch.full((2, 2, keep), -9, dtype=torch.int32, device="cuda")
    new, dl, dd = c.i32([0, 0]), c.i32(lens), torch.from_numpy(dst).cuda()
    c.qw.qw_kv8_evict(c.view, 2, max(lens), dl.data_ptr(), keep, recent, 0 if rows_in_place else dd.data_ptr(), dsc.data_ptr(),
                      so.data_ptr(), sc.shape[2], kept.data_ptr(), new.data_ptr(), c.status.data_ptr())
    assert c.bits() == 0 and new.tolist() == [min(n, keep) for n in lens]
    to = c.table if rows_in_place else dst
    got_s, kept = so.cpu().numpy(), kept.cpu().numpy()
    for b, n in enumerate(lens):
        own = c.table[b]
        want_k, want_s = c.orc.evict(own, own if rows_in_place else dst[b], n, keep, recent, sc[b])
        np.testing.assert_array_equal(kept[b], want_k)
        np.testing.assert_array_equal(got_s[b, :, :n], want_s)
    c.table = to
    c.check_cache([min(n, keep) for n in lens])


def test_evict_leaves_bad_entries_alone(qw):
    import torch
    c = Case(qw, [100, 100], 1, 128, seed=13)
    c.append([0, 0], [100, 100])
    before = c.blocks.clone()
    bad = c.table.copy()
    bad[1, 6] = -7
    c.dtable.copy_(torch.from_numpy(bad))
    sc = c.rng.random((2, 1, 100)).astype(np.float32)
    kept, new, so = _evict(c, [3000, 100], 20, 4, sc, True)  # a length beyond the table; a bad page
    assert c.bits() == c.qw.QW_KV8_BAD_POS
    assert torch.equal(before, c.blocks) and np.all(kept == -1) and np.array_equal(new, [3000, 100])
    np.testing.assert_array_equal(so, sc)


def test_generation_under_a_budget(qw):
    """The operators as a serving loop runs them: a prompt in chunks with its scores, then steps that
    append, attend, accumulate and evict in place whenever the cache passes its budget."""
    import torch
    hd, n_kv, G, keep, recent = 128, 2, 2, 48, 16
    c = Case(qw, [96, 96], n_kv, hd, seed=14)
    score = np.zeros((2, n_kv, 96))
    lens = np.array([0, 0])
    dev_score = torch.zeros((2, n_kv, 96), device="cuda")

    def step(n):
        nonlocal lens
        n = np.asarray(n)
        c.append(lens, n)
        cu = np.concatenate([[0], np.cumsum(n)])
        T = int(cu[-1])
        q, qf = c.rows(T, n_kv * G, F16)
        out = torch.empty((T, n_kv * G * hd), dtype=torch.float16, device="cuda")
        nb = c.qw.qw_kv8_attn_ws_bytes(c.view, 2, T, int(n.max()), 96, n_kv * G, True)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        ds, dc = c.i32(lens), c.i32(cu)
        c.qw.qw_kv8_attn(c.view, 2, T, int(n.max()), 96, ds.data_ptr(), dc.data_ptr(), q.data_ptr(), n_kv * G * hd, n_kv * G,
                         c.qw.QW_F16, hd ** -0.5, out.data_ptr(), n_kv * G * hd, 0, dev_score.data_ptr(), dev_score.data_ptr(),
                         96, ws.data_ptr(), nb, c.status.data_ptr())
        got = out.double().cpu().numpy().reshape(T, n_kv * G, hd)
        for b in range(2):
            want, _, w, mag = c.orc.attention(c.table[b], int(lens[b]), qf[cu[b]:cu[b + 1]], hd ** -0.5)
            assert np.all(np.abs(got[cu[b]:cu[b + 1]] - want) <= mag * 2.0 ** -10 + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)
            score[b, :, :lens[b] + n[b]] += w.reshape(n_kv, G, n[b], -1).sum((1, 2))
        lens = lens + n
        np.testing.assert_allclose(dev_score.cpu().numpy(), score, rtol=2e-5, atol=1e-6)
        if lens.max() > keep + 16:
            # the library's own scores decide, so that equal selections do not hang on roundings
            host = dev_score.cpu().numpy()
            kept = torch.empty((2, n_kv, keep), dtype=torch.int32, device="cuda")
            new = torch.empty(2, dtype=torch.int32, device="cuda")
            dl = c.i32(lens)
            c.qw.qw_kv8_evict(c.view, 2, 96, dl.data_ptr(), keep, recent, 0, dev_score.data_ptr(), dev_score.data_ptr(), 96,
                              kept.data_ptr(), new.data_ptr(), c.status.data_ptr())
            for b in range(2):
                own = c.table[b]
                wk, _ = c.orc.evict(own, own, int(lens[b]), keep, recent, host[b])
                np.testing.assert_array_equal(kept[b].cpu().numpy(), wk)
                m = min(int(lens[b]), keep)
                moved = np.zeros_like(score[b])
                for h in range(n_kv):
                    moved[h, :m] = score[b, h, wk[h, :m]]
                score[b] = moved
            lens = new.cpu().numpy().astype(np.int64)
            c.check_cache(lens.tolist())

    step([30, 21])
    step([20, 44])
    for _ in range(40):
        step([1, 1])
    assert c.bits() == 0
