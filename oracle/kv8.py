"""fp64 NumPy restatement of the 8-bit paged KV cache: e4m3 codes with a power-of-two scale for each
page of 16 tokens, KV head and tensor; append, attention over it, and eviction by score."""

import numpy as np

PAGE = 16
E_MIN = -32


def e4m3_values():
    """The 256 values of the format: bias 7, subnormals, no infinities, 0x7f / 0xff NaN."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b & 128, -v, v)


def e4m3_round(y):
    """Nearest e4m3 value (even on ties) of |y| <= 448."""
    y = np.asarray(y, np.float64)
    k = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = 2.0 ** (k - 3)
    return np.rint(y / step) * step


def exponent(amax):
    """Smallest e >= -32 with amax <= 448 * 2^e."""
    e = E_MIN
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def chunk_position(hd, tensor, token, i):
    if tensor == 0:
        return i ^ (4 * (token % 2)) if hd == 128 else i
    return i ^ (2 * (token // 4)) if hd == 128 else i ^ (token // 4)


class Cache:
    """Held values [n_pages, n_kv, 16, hd] and exponents [n_pages, n_kv] of K (0) and V (1)."""

    def __init__(self, n_pages, n_kv, hd):
        self.hd, self.n_kv = hd, n_kv
        self.x = [np.zeros((n_pages, n_kv, PAGE, hd)) for _ in range(2)]
        self.e = [np.full((n_pages, n_kv), E_MIN) for _ in range(2)]

    @staticmethod
    def from_blocks(raw, hd):
        """raw: uint8 [n_pages, n_kv, 32 hd + 32]."""
        c = Cache(raw.shape[0], raw.shape[1], hd)
        lut = e4m3_values()
        scale = np.ascontiguousarray(raw[..., 32 * hd:]).view(np.float32)[..., :2].astype(np.float64)
        for w in range(2):
            codes = raw[..., 16 * hd * w:16 * hd * (w + 1)].reshape(raw.shape[0], raw.shape[1], PAGE, hd // 16, 16)
            for t in range(PAGE):
                for i in range(hd // 16):
                    c.x[w][:, :, t, 16 * i:16 * i + 16] = lut[codes[:, :, t, chunk_position(hd, w, t, i)]]
            with np.errstate(invalid="ignore", divide="ignore"):
                c.x[w] *= scale[..., w][..., None, None]
                c.e[w] = np.log2(scale[..., w])
        return c

    def _store(self, w, page, h, rows, floor=None):
        e = exponent(np.abs(rows).max(initial=0.0))
        if floor is not None:
            e = max(e, floor)
        self.x[w][page, h] = e4m3_round(rows * 2.0 ** -e) * 2.0 ** e
        self.e[w][page, h] = e

    def append(self, table, start, new):
        """new: (K, V), each [n, n_kv, hd] fp16-valued, at positions start .. start + n - 1."""
        n = len(new[0])
        for pi in range(start // PAGE, (start + n + PAGE - 1) // PAGE if n else 0):
            page = table[pi]
            had = max(0, start - pi * PAGE)
            a, z = max(start, pi * PAGE), min(start + n, (pi + 1) * PAGE)
            for w in range(2):
                for h in range(self.n_kv):
                    rows = np.zeros((PAGE, self.hd))
                    rows[a - pi * PAGE:z - pi * PAGE] = new[w][a - start:z - start, h]
                    e_new = exponent(np.abs(rows).max())
                    floor = e_new
                    if had:
                        rows[:had] = self.x[w][page, h, :had]
                        floor = max(e_new, int(self.e[w][page, h]))
                    self.x[w][page, h] = e4m3_round(rows * 2.0 ** -floor) * 2.0 ** floor
                    self.e[w][page, h] = floor

    def rows(self, w, table, n):
        """[n, n_kv, hd] held values of positions 0 .. n - 1."""
        pages = table[:(n + PAGE - 1) // PAGE]
        return self.x[w][pages].transpose(0, 2, 1, 3).reshape(-1, self.n_kv, self.hd)[:n]

    def attention(self, table, start, q, scale):
        """q: [n, n_heads, hd] at positions start ...; out, lse, weights [n_heads, n, start + n] and
        sum_j p_j |v_j| (the scale of the output's rounding errors)."""
        n, Hq, _ = q.shape
        G = Hq // self.n_kv
        k, v = self.rows(0, table, start + n), self.rows(1, table, start + n)
        out, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, Hq))
        wts = np.zeros((Hq, n, start + n))
        hidden = np.arange(start + n)[None, :] > start + np.arange(n)[:, None]
        for h in range(Hq):
            s = q[:, h] @ k[:, h // G].T * scale
            s[hidden] = -np.inf
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(1, keepdims=True)
            lse[:, h] = (m + np.log(z))[:, 0]
            wts[h] = p / z
            out[:, h] = wts[h] @ v[:, h // G]
            mag[:, h] = wts[h] @ np.abs(v[:, h // G])
        return out, lse, wts, mag

    def evict(self, table, dst, L, keep, recent, score):
        """score: [n_kv, >= L]; rows move to the pages of dst. Returns kept [n_kv, keep] and scores."""
        n = min(L, keep)
        kept = np.full((self.n_kv, keep), -1, np.int64)
        new = np.zeros((self.n_kv, L), np.float32)
        rows = [self.rows(w, table, L).copy() for w in range(2)]
        for h in range(self.n_kv):
            idx = np.arange(L)
            if L > keep:
                s = np.where(np.isnan(score[h, :L - recent]), np.inf, score[h, :L - recent]).astype(np.float64)
                first = np.where(np.isnan(score[h, :L - recent]), 0, 1)
                order = np.lexsort((np.arange(L - recent), first, -s))[:keep - recent]
                idx = np.concatenate([np.sort(order), np.arange(L - recent, L)])
            kept[h, :n] = idx
            new[h, :n] = score[h, idx]
            for w in range(2):
                # within the budget and in place: the pages stay as they are
                for d in range((n + PAGE - 1) // PAGE if L > keep or dst is not table else 0):
                    r = np.zeros((PAGE, self.hd))
                    part = rows[w][idx[d * PAGE:min(n, (d + 1) * PAGE)], h]
                    r[:len(part)] = part
                    self._store(w, dst[d], h, r)
        return kept, new
