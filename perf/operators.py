"""Measured cases of the 8-bit paged KV cache operators: append, attention and eviction.

The cache holds K and V as e4m3 codes in pages of 16 tokens with one power-of-two scale per
page, KV head and tensor. Definitions (x: the fp16 rounding of the given value):

- append: a page's exponent is the smallest e with max|x| <= 448 2^e over its tokens (-32 for a
  page of zeros), never below the exponent that tokens already in the page have; a code is
  e4m3(x 2^-e), round to nearest even, and tokens already in the page are re-coded from their
  held values when the exponent grew. A cached value is code * 2^e.
- attention: the query at position p (start + i) sees the cached tokens 0..p; query head h reads
  KV head h // group. out = softmax(scale q k) v, lse its natural log-sum-exp, and the score of
  a cached token is what it had plus the attention weights of the call's queries, summed over
  the queries and the heads of the group.
- eviction: a sequence longer than `keep` keeps its last `recent` tokens and, of the others, the
  keep - recent with the largest scores (the lowest position on ties) for each KV head, in
  ascending order; rows move to the head of the sequence (pages coded as by append) and the
  scores move with them.

`own` picks the library's calls (qw_kv8_*); otherwise the plain torch forms run.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
E_MIN = -32


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's new tokens of a batch of 64 over caches of 1024 prompt tokens plus steps
        {"name": "append step 64", "op": "append", "dtype": "f16", "B": 64, "n_kv": 8, "hd": 128,
         "start_lo": 1024, "start_hi": 1152, "len_lo": 1, "len_hi": 1, "ragged": 1},
        # the prompts of a 16 x 512 prefill written into an empty cache
        {"name": "append prefill 16x512", "op": "append", "dtype": "f16", "B": 16, "n_kv": 8, "hd": 128,
         "start_lo": 0, "start_hi": 0, "len_lo": 512, "len_hi": 512, "ragged": 2},
        # chunks of several prompts that continue pages begun by earlier chunks
        {"name": "append ragged 7", "op": "append", "dtype": "bf16", "B": 7, "n_kv": 4, "hd": 64,
         "start_lo": 3, "start_hi": 1000, "len_lo": 1, "len_hi": 700, "ragged": 3},
        # batch 1: a 5-token prompt plus 64 steps, where latency counts
        {"name": "decode 1x69", "op": "attn", "dtype": "f16", "B": 1, "n_kv": 8, "group": 2, "hd": 128,
         "start_lo": 68, "start_hi": 68, "len_lo": 1, "len_hi": 1, "score": False, "ragged": 4},
        # the batch-64 decode workload
        {"name": "decode 64x1100", "op": "attn", "dtype": "f16", "B": 64, "n_kv": 8, "group": 2, "hd": 128,
         "start_lo": 1024, "start_hi": 1151, "len_lo": 1, "len_hi": 1, "score": False, "ragged": 5},
        # the ragged long-context decode workload
        {"name": "decode 8x1k-32k", "op": "attn", "dtype": "f16", "B": 8, "n_kv": 8, "group": 2, "hd": 128,
         "start_lo": 1024, "start_hi": 32767, "len_lo": 1, "len_hi": 1, "score": False, "ragged": 6},
        # decode that keeps each token's accumulated weight for a later eviction
        {"name": "decode scores 8x4k", "op": "attn", "dtype": "bf16", "B": 8, "n_kv": 8, "group": 4, "hd": 128,
         "start_lo": 2000, "start_hi": 6000, "len_lo": 1, "len_hi": 1, "score": True, "ragged": 7},
        # the attention of a 16 x 512 prefill
        {"name": "prefill 16x512", "op": "attn", "dtype": "f16", "B": 16, "n_kv": 8, "group": 2, "hd": 128,
         "start_lo": 0, "start_hi": 0, "len_lo": 512, "len_hi": 512, "score": False, "ragged": 8},
        # a prompt's last chunk over its cached prefix, with the scores that eviction reads
        {"name": "chunk scores 2x400", "op": "attn", "dtype": "bf16", "B": 2, "n_kv": 4, "group": 7, "hd": 64,
         "start_lo": 5000, "start_hi": 9000, "len_lo": 300, "len_hi": 500, "score": True, "ragged": 9},
        # one short sequence brought back under its budget
        {"name": "evict 1x200", "op": "evict", "dtype": "f16", "B": 1, "n_kv": 8, "hd": 128,
         "len_lo": 200, "len_hi": 200, "keep": 128, "recent": 32, "ragged": 10},
        # a batch of long ragged caches cut to 1000 tokens each
        {"name": "evict 8x1k-32k", "op": "evict", "dtype": "f16", "B": 8, "n_kv": 8, "hd": 128,
         "len_lo": 1024, "len_hi": 32768, "keep": 1000, "recent": 250, "ragged": 11},
        # every layer of one 4096-token sequence halved, the 28 layers as batch entries
        {"name": "evict 28 layers 4k", "op": "evict", "dtype": "f16", "B": 28, "n_kv": 8, "hd": 128,
         "len_lo": 4096, "len_hi": 4096, "keep": 2048, "recent": 512, "ragged": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.8e15


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["append", "attn", "attn", "evict"])
        c = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "B": _log_int(rng, 1, 64), "n_kv": rng.choice([1, 2, 4, 8]),
             "hd": rng.choice([64, 128]), "ragged": rng.randrange(1 << 30)}
        if op == "append":
            n = _log_int(rng, 1, 600)
            s = rng.choice([0, _log_int(rng, 1, 2000)])
            c.update(start_lo=s // 2, start_hi=s, len_lo=max(1, n // 2), len_hi=n, dtype=rng.choice(["f16", "bf16", "f32"]))
        elif op == "attn":
            decode = rng.random() < 0.6
            n = 1 if decode else _log_int(rng, 2, 520)
            s = _log_int(rng, 1, 32000 if decode else 9000)
            c.update(group=rng.choice([1, 2, 3, 4, 7, 8]), start_lo=s // 2, start_hi=s, len_lo=max(1, n // 2), len_hi=n,
                     score=rng.random() < 0.4)
        else:
            n = _log_int(rng, 40, 32000)
            k = rng.randrange(max(2, n // 16), n)
            c.update(len_lo=n // 2, len_hi=n, keep=k, recent=rng.randrange(0, k + 1), dtype="f16")
        if _cost(c) <= top[op] and c["B"] * c["len_hi"] <= 300000:
            return c


def _shape(case):
    """Lengths and starts: part of the case, the same for every seed."""
    r = np.random.default_rng(case["ragged"])
    B = case["B"]
    lens = r.integers(case["len_lo"], case["len_hi"] + 1, B)
    starts = r.integers(case["start_lo"], case["start_hi"] + 1, B) if "start_lo" in case else np.zeros(B, np.int64)
    lens[r.integers(B)] = case["len_hi"]
    return starts.astype(np.int64), lens.astype(np.int64)


def work(case):
    starts, lens = _shape(case)
    H, hd = case["n_kv"], case["hd"]
    es = 4 if case["dtype"] == "f32" else 2
    row = 2 * H * hd  # one token's K and V elements (and their code bytes)
    if case["op"] == "append":
        # the new rows, the tokens already in the first page, and the pages' values read back
        old = int((starts % PAGE).sum())
        T = int(lens.sum())
        return {"bytes": T * row * es + (2 * old + T) * row + (old + T) * row * (1 + es), "flops": 2 * (T + old) * row}
    if case["op"] == "attn":
        G = case["group"]
        keys = int((starts + lens).sum())
        pairs = int((lens * starts + lens * (lens + 1) // 2).sum())  # visible (query, key) pairs of one head
        T = int(lens.sum())
        return {"bytes": keys * row + 2 * T * H * G * hd * es + 4 * T * H * G + (8 * keys * H if case["score"] else 0),
                "flops": 4 * pairs * H * G * hd}
    keep = np.minimum(lens, case["keep"])
    # the scores in and out, the kept rows' codes moved, their positions, and the values read back
    return {"bytes": int(8 * lens.sum() * H + keep.sum() * (2 * row + 4 * H + row * (1 + es))),
            "flops": int(2 * keep.sum() * row + 4 * lens.sum() * H)}


# ---- inputs -----------------------------------------------------------------------------------

def _exponent(amax):
    """Smallest e with amax <= 448 2^e = 1.75 2^(e + 8); E_MIN for zero."""
    f, x = torch.frexp(amax)  # amax = f 2^x, f in [0.5, 1)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp_min(E_MIN)


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x):
    """e4m3 codes of fp32 values, as bytes."""
    return x.to(E4M3).view(torch.uint8)


def _values(c):
    return c.view(E4M3).float()


def _pack(ck, cv, ek, ev):
    """The library's page blocks [pages, heads, 32 hd + 32] of codes [pages, heads, 16, hd] and exponents."""
    P, H, _, hd = ck.shape
    t, i = torch.arange(PAGE, device=ck.device)[:, None], torch.arange(hd // 16, device=ck.device)[None, :]
    at_k, at_v = (i ^ (4 * (t % 2)), i ^ (2 * (t // 4))) if hd == 128 else (i + 0 * t, i ^ (t // 4))
    k = ck.view(P, H, PAGE, hd // 16, 16)[:, :, t, at_k].reshape(P, H, -1)
    v = cv.view(P, H, PAGE, hd // 16, 16)[:, :, t, at_v].reshape(P, H, -1)
    tail = torch.zeros((P, H, 8), dtype=torch.float32, device=ck.device)
    tail[..., 0], tail[..., 1] = _pow2(ek), _pow2(ev)
    return torch.cat([k, v, tail.view(torch.uint8).view(P, H, 32)], -1).contiguous()


def _kv_values(gen, shape, dev):
    """K with a few strong channels, as a per-head key norm leaves it, and V."""
    k = torch.randn(shape, generator=gen, device=dev)
    k *= 1 + 5 * (torch.arange(shape[-1], device=dev) % 37 == 5)
    return k, torch.randn(shape, generator=gen, device=dev) * 0.5


def _make_cache(gen, n_pages, H, hd, dev):
    k, v = _kv_values(gen, (n_pages, H, PAGE, hd), dev)
    k, v = k.half().float(), v.half().float()
    ek, ev = _exponent(k.abs().amax((2, 3))), _exponent(v.abs().amax((2, 3)))
    ck, cv = _codes(k * _pow2(-ek)[..., None, None]), _codes(v * _pow2(-ev)[..., None, None])
    return {"ck": ck, "cv": cv, "ek": ek, "ev": ev, "blocks": _pack(ck, cv, ek, ev)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + case["ragged"] % 1000)
    starts, lens = _shape(case)
    B, H, hd, op = case["B"], case["n_kv"], case["hd"], case["op"]
    ends = starts + lens
    maxp = int((ends.max() + PAGE - 1) // PAGE)
    need = (ends + PAGE - 1) // PAGE
    n_pages = int(need.sum())
    extra = (np.minimum(lens, case["keep"]) + PAGE - 1) // PAGE if op == "evict" else np.zeros(B, np.int64)
    total = n_pages + int(extra.sum()) + 3  # some pages of the pool are free
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((B, maxp), -1, np.int32)
    first = np.concatenate([[0], np.cumsum(need)])
    for b in range(B):
        table[b, :need[b]] = perm[first[b]:first[b + 1]]
    st = {"case": case, "maxp": maxp, "n_pages": total, "max_len": int(lens.max()), "max_keys": int(ends.max()),
          "T": int(lens.sum()), **_make_cache(gen, total, H, hd, dev)}
    st["table"] = torch.from_numpy(table).to(dev)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    st["start"], st["len"], st["cu"] = i32(starts), i32(lens), i32(np.concatenate([[0], np.cumsum(lens)]))
    st["ent"] = torch.repeat_interleave(torch.arange(B, device=dev), st["len"].long())
    st["idx"] = torch.arange(st["T"], device=dev) - st["cu"].long()[st["ent"]]
    T = st["T"]
    if op == "append":
        k, v = _kv_values(gen, (T, H, hd), dev)
        st["k"], st["v"] = k.to(DT[case["dtype"]]), v.to(DT[case["dtype"]])
        # read back from the start of the first page touched
        s0, n0 = starts - starts % PAGE, lens + starts % PAGE
        st["rstart"], st["rcu"], st["rmax"] = i32(s0), i32(np.concatenate([[0], np.cumsum(n0)])), int(n0.max())
        st["rT"] = int(n0.sum())
        rl = torch.from_numpy(n0).to(dev)
        st["rent"] = torch.repeat_interleave(torch.arange(B, device=dev), rl)
        st["ridx"] = torch.arange(st["rT"], device=dev) - st["rcu"].long()[st["rent"]]
        # every page touched, one row each: (entry, page of the entry)
        np_ = (ends - 1) // PAGE - starts // PAGE + 1
        st["tent"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.from_numpy(np_).to(dev))
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(np_)])).to(dev)
        st["tpage"] = torch.arange(int(np_.sum()), device=dev) - off[st["tent"]] + st["start"].long()[st["tent"]] // PAGE
    elif op == "attn":
        q = 1.5 * torch.randn((T, H * case["group"], hd), generator=gen, device=dev)
        st["q"] = q.to(DT[case["dtype"]])
        if case["score"]:
            st["score"] = torch.rand((B, H, st["max_keys"]), generator=gen, device=dev) ** 4 * 10
    else:
        dst = np.full((B, maxp), -1, np.int32)
        first = n_pages + np.concatenate([[0], np.cumsum(extra)])
        for b in range(B):
            dst[b, :extra[b]] = perm[first[b]:first[b + 1]]
        st["dst"] = torch.from_numpy(dst).to(dev)
        # heavy-tailed accumulated weights, some equal and some zero
        u = torch.rand((B, H, st["max_keys"]), generator=gen, device=dev)
        s = torch.where(u < 0.1, torch.zeros_like(u), 0.05 / (1.0001 - u))
        st["score"] = torch.where(u < 0.4, (s * 64).round() / 64, s)
        new = np.minimum(lens, case["keep"])
        st["rcu"], st["rT"], st["rmax"] = i32(np.concatenate([[0], np.cumsum(new)])), int(new.sum()), int(new.max())
        st["zero"] = torch.zeros(B, dtype=torch.int32, device=dev)
        st["rent"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.from_numpy(new).to(dev))
        st["ridx"] = torch.arange(st["rT"], device=dev) - st["rcu"].long()[st["rent"]]
    return st


# ---- plain forms --------------------------------------------------------------------------------

def _pages(st, table):
    return table.long().clamp_min(0)


def _dequant(c, e):
    return _values(c) * _pow2(e)[..., None, None]


def _encode(x):
    """Codes and exponents of pages x [..., 16, hd] (values exact in fp32)."""
    e = _exponent(x.abs().amax((-2, -1)))
    return _codes(x * _pow2(-e)[..., None, None]), e


def _plain_append(st):
    case = st["case"]
    H, hd = case["n_kv"], case["hd"]
    pages = st["table"].long()[st["tent"], st["tpage"]]
    pos = st["tpage"][:, None] * PAGE + torch.arange(PAGE, device=pages.device)  # [touched, 16]
    start, n = st["start"].long()[st["tent"]][:, None], st["len"].long()[st["tent"]][:, None]
    new = (pos >= start) & (pos < start + n)
    had = pos < start
    row = (st["cu"].long()[st["tent"]][:, None] + pos - start).clamp(0, st["T"] - 1)
    for c, e, src in (("ck", "ek", "k"), ("cv", "ev", "v")):
        x = st[src].to(torch.float16).float()[row].transpose(1, 2)  # [touched, H, 16, hd]
        x = torch.where(new[:, None, :, None], x, torch.zeros_like(x))
        e_new = _exponent(x.abs().amax((2, 3)))
        held = had.any(1)[:, None]
        e_old = st[e][pages]
        e_all = torch.where(held, torch.maximum(e_new, e_old), e_new)
        old = torch.where(had[:, None, :, None], _dequant(st[c][pages], e_old), torch.zeros_like(x))
        st[c][pages] = _codes((x + old) * _pow2(-e_all)[..., None, None])
        st[e][pages] = e_all
    pos = st["rstart"].long()[st["rent"]] + st["ridx"]
    page, slot = st["table"].long()[st["rent"], pos // PAGE], pos % PAGE
    dt = DT[case["dtype"]]
    return tuple((_values(st[c][page, :, slot]) * _pow2(st[e][page])[..., None]).to(dt) for c, e in (("ck", "ek"), ("cv", "ev")))


def _plain_attn(st):
    case = st["case"]
    B, H, G, hd = case["B"], case["n_kv"], case["group"], case["hd"]
    K, N, T = st["maxp"] * PAGE, st["max_len"], st["T"]
    pages = _pages(st, st["table"])
    k, v = (_dequant(st[c][pages], st[e][pages]).transpose(1, 2).reshape(B, H, K, hd) for c, e in (("ck", "ek"), ("cv", "ev")))
    q = torch.zeros((B, N, H * G, hd), device=k.device)
    q[st["ent"], st["idx"]] = st["q"].float()
    q = q.view(B, N, H, G, hd).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, hd)
    s = torch.matmul(q, k.transpose(2, 3)) * hd ** -0.5  # [B, H, G N, K]
    pos = torch.arange(K, device=k.device)
    qpos = st["start"].long()[:, None] + torch.arange(N, device=k.device)
    real = torch.arange(N, device=k.device) < st["len"].long()[:, None]
    seen = (pos[None, None, :] <= qpos[:, :, None]) & real[:, :, None]  # [B, N, K]
    s = s.view(B, H, G, N, K).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    p = p / z.clamp_min(1e-30)
    o = torch.matmul(p.view(B, H, G * N, K), v).view(B, H, G, N, hd).permute(0, 3, 1, 2, 4)
    lse = (m + torch.log(z.clamp_min(1e-30)))[..., 0].permute(0, 3, 1, 2)
    out = (o[st["ent"], st["idx"]].to(DT[case["dtype"]]).reshape(T, H * G, hd), lse[st["ent"], st["idx"]].reshape(T, H * G))
    if case["score"]:
        return out + (st["score"] + p.sum((2, 3))[..., :st["max_keys"]],)
    return out


def _plain_evict(st):
    case = st["case"]
    B, H, hd, keep, recent = case["B"], case["n_kv"], case["hd"], case["keep"], case["recent"]
    L = st["max_keys"]
    n = st["len"].long()[:, None, None]
    pos = torch.arange(L, device=n.device)
    s = st["score"]
    key = torch.where(pos >= n - recent, math.inf, s)  # the recent tokens come first
    key = torch.where(pos < n, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :min(keep, L)]
    kept = torch.where(order < n, order, L).sort(-1).values
    valid = kept < L
    kept = torch.where(n > keep, kept, torch.arange(kept.shape[-1], device=n.device))
    valid = torch.where(n > keep, valid, kept < n)
    W = (min(keep, L) + PAGE - 1) // PAGE
    pad = W * PAGE - kept.shape[-1]
    src = torch.nn.functional.pad(torch.where(valid, kept, 0), (0, pad))
    ok = torch.nn.functional.pad(valid, (0, pad))
    b, h = torch.arange(B, device=n.device)[:, None, None], torch.arange(H, device=n.device)[None, :, None]
    page = _pages(st, st["table"])[b, src // PAGE]
    vals = []
    dst = st["dst"].long()[:, :W]
    has = dst >= 0
    for c, e in (("ck", "ek"), ("cv", "ev")):
        x = _values(st[c][page, h, src % PAGE]) * _pow2(st[e][page, h])[..., None]
        x = torch.where(ok[..., None], x, torch.zeros_like(x)).view(B, H, W, PAGE, hd).transpose(1, 2)
        code, ex = _encode(x)
        st[c][dst[has]], st[e][dst[has]] = code[has], ex[has]
        r = (_values(code) * _pow2(ex)[..., None, None]).transpose(2, 3).reshape(B, W * PAGE, H, hd)
        vals.append(r[st["rent"], st["ridx"]].to(DT[case["dtype"]]))
    new = torch.zeros_like(s)
    new[..., :kept.shape[-1]] = torch.where(valid, s.gather(-1, torch.where(valid, kept, 0)), 0.0)
    out = torch.full((B, H, keep), -1, dtype=torch.int32, device=n.device)
    out[..., :kept.shape[-1]] = torch.where(valid, kept, -1).int()
    return out, new, vals[0], vals[1]


# ---- the library's calls --------------------------------------------------------------------------

def _lib(st):
    if "qw" not in st:
        from decode_qwen3_decoder_gb300 import qw
        case, dev = st["case"], st["blocks"].device
        H, hd, dt = case["n_kv"], case["hd"], DT[case["dtype"]]
        st["qw"], st["ty"] = qw, {"f16": qw.QW_F16, "bf16": qw.QW_BF16, "f32": qw.QW_F32}[case["dtype"]]
        st["view"] = qw.qw_kv8_view(st["blocks"].data_ptr(), st["n_pages"], H, hd, st["table"].data_ptr(), st["maxp"])
        st["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if case["op"] == "attn":
            Hq = H * case["group"]
            st["out"] = torch.empty((st["T"], Hq, hd), dtype=dt, device=dev)
            st["lse"] = torch.empty((st["T"], Hq), device=dev)
            n = qw.qw_kv8_attn_ws_bytes(st["view"], case["B"], st["T"], st["max_len"], st["max_keys"], Hq, case["score"])
            st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
            # positions past a sequence keep what they had
            st["score_out"] = st["score"].clone() if case["score"] else None
        else:
            st["rk"], st["rv"] = (torch.empty((st["rT"], H, hd), dtype=dt, device=dev) for _ in range(2))
        if case["op"] == "evict":
            st["dview"] = qw.qw_kv8_view(st["blocks"].data_ptr(), st["n_pages"], H, hd, st["dst"].data_ptr(), st["maxp"])
            st["kept"] = torch.empty((case["B"], H, case["keep"]), dtype=torch.int32, device=dev)
            st["new_len"] = torch.empty(case["B"], dtype=torch.int32, device=dev)
            st["score_out"] = torch.zeros_like(st["score"])
    return st["qw"]


def _own_append(st):
    qw, case = _lib(st), st["case"]
    ld = case["n_kv"] * case["hd"]
    qw.qw_kv8_append(st["view"], case["B"], st["T"], st["max_len"], st["start"].data_ptr(), st["cu"].data_ptr(),
                     st["k"].data_ptr(), ld, st["v"].data_ptr(), ld, st["ty"], st["status"].data_ptr())
    qw.qw_kv8_read(st["view"], case["B"], st["rT"], st["rmax"], st["rstart"].data_ptr(), st["rcu"].data_ptr(),
                   st["rk"].data_ptr(), ld, st["rv"].data_ptr(), ld, st["ty"], st["status"].data_ptr())
    return st["rk"], st["rv"]


def _own_attn(st):
    qw, case = _lib(st), st["case"]
    Hq, hd = case["n_kv"] * case["group"], case["hd"]
    sc = case["score"]
    qw.qw_kv8_attn(st["view"], case["B"], st["T"], st["max_len"], st["max_keys"], st["start"].data_ptr(), st["cu"].data_ptr(),
                   st["q"].data_ptr(), Hq * hd, Hq, st["ty"], hd ** -0.5, st["out"].data_ptr(), Hq * hd,
                   st["lse"].data_ptr(), st["score"].data_ptr() if sc else 0, st["score_out"].data_ptr() if sc else 0,
                   st["max_keys"] if sc else 0, st["ws"].data_ptr(), st["ws"].numel(), st["status"].data_ptr())
    return (st["out"], st["lse"], st["score_out"]) if sc else (st["out"], st["lse"])


def _own_evict(st):
    qw, case = _lib(st), st["case"]
    ld = case["n_kv"] * case["hd"]
    qw.qw_kv8_evict(st["view"], case["B"], st["max_len"], st["len"].data_ptr(), case["keep"], case["recent"],
                    st["dst"].data_ptr(), st["score"].data_ptr(), st["score_out"].data_ptr(), st["max_keys"],
                    st["kept"].data_ptr(), st["new_len"].data_ptr(), st["status"].data_ptr())
    qw.qw_kv8_read(st["dview"], case["B"], st["rT"], st["rmax"], st["zero"].data_ptr(), st["rcu"].data_ptr(),
                   st["rk"].data_ptr(), ld, st["rv"].data_ptr(), ld, st["ty"], st["status"].data_ptr())
    return st["kept"], st["score_out"], st["rk"], st["rv"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "evict": _own_evict}[op](state)
    return {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}[op](state)


# ---- the definitions in 64 bits ---------------------------------------------------------------------

def _code64(x, floor=None):
    """Held values of one page's rows x [n, H, hd] and its exponent per head, in 64 bits: e from log2,
    e4m3 from its spacing (2^-9 below 2^-6, else 2^(k - 3) in [2^k, 2^(k + 1)))."""
    a = x.abs().amax((0, 2))
    e = torch.where(a > 0, torch.ceil(torch.log2(a / 448)), torch.full_like(a, float(E_MIN)))
    e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((a > 0) & (a <= 448 * torch.exp2(e - 1)), e - 1, e).clamp_min(float(E_MIN))
    if floor is not None:
        e = torch.maximum(e, floor)
    sc = torch.exp2(e)[None, :, None]
    y = x / sc
    k = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(k - 3)
    return torch.round(y / step) * step * sc, e


def exact(case, seed):
    st = prepare(case, seed)
    starts, lens = _shape(case)
    B, H, hd = case["B"], case["n_kv"], case["hd"]
    table = st["table"].long()
    dt = torch.float64
    held = {c: _values(st[c]).to(dt) * torch.exp2(st[e].to(dt))[..., None, None] for c, e in (("ck", "ek"), ("cv", "ev"))}
    rows = lambda c, b, n: held[c][table[b, :(n + PAGE - 1) // PAGE]].transpose(1, 2).reshape(-1, H, hd)[:n]  # noqa: E731
    if case["op"] == "append":
        out = []
        cu = np.concatenate([[0], np.cumsum(lens)])
        for c, e, src in (("ck", "ek", "k"), ("cv", "ev", "v")):
            got = []
            for b in range(B):
                s, n = int(starts[b]), int(lens[b])
                x = st[src][cu[b]:cu[b + 1]].to(torch.float16).to(dt)
                old = rows(c, b, s)[s - s % PAGE:]
                x = torch.cat([old, x])
                for i in range(0, x.shape[0], PAGE):
                    floor = st[e][table[b, s // PAGE]].to(dt) if i == 0 and s % PAGE else None
                    got.append(_code64(x[i:i + PAGE], floor)[0])
            out.append(torch.cat(got))
        return tuple(out)
    if case["op"] == "attn":
        G, cu = case["group"], np.concatenate([[0], np.cumsum(lens)])
        out = torch.zeros((st["T"], H * G, hd), dtype=dt, device=table.device)
        lse = torch.zeros((st["T"], H * G), dtype=dt, device=table.device)
        score = st["score"].to(dt) if case["score"] else None
        for b in range(B):
            s, n = int(starts[b]), int(lens[b])
            k, v = rows("ck", b, s + n), rows("cv", b, s + n)
            hidden = torch.arange(s + n, device=k.device)[None, :] > s + torch.arange(n, device=k.device)[:, None]
            for h in range(H * G):
                a = st["q"][cu[b]:cu[b + 1], h].to(dt) @ k[:, h // G].T / math.sqrt(hd)
                a[hidden] = -math.inf
                lse[cu[b]:cu[b + 1], h] = torch.logsumexp(a, 1)
                a = torch.softmax(a, 1)
                out[cu[b]:cu[b + 1], h] = a @ v[:, h // G]
                if score is not None:
                    score[b, h // G, :s + n] += a.sum(0)
        return (out, lse, score) if case["score"] else (out, lse)
    keep, recent = case["keep"], case["recent"]
    kept = np.full((B, H, keep), -1, np.int64)
    score = st["score"].to(dt).cpu().numpy()
    moved = np.zeros_like(score)
    vals = {"ck": [], "cv": []}
    for b in range(B):
        n = int(lens[b])
        m = min(n, keep)
        for h in range(H):
            order = np.arange(n)
            if n > keep:
                order = np.lexsort((np.arange(n - recent), -score[b, h, :n - recent]))[:keep - recent]
                order = np.concatenate([np.sort(order), np.arange(n - recent, n)])
            kept[b, h, :m] = order
            moved[b, h, :m] = score[b, h, order]
        idx = torch.from_numpy(kept[b, :, :m]).to(table.device).T  # [m, H]
        for c in vals:
            x = rows(c, b, n).gather(0, idx[:, :, None].expand(m, H, hd))
            vals[c] += [_code64(x[i:i + PAGE])[0] for i in range(0, m, PAGE)]
    return (torch.from_numpy(kept.astype(np.int32)), torch.from_numpy(moved), torch.cat(vals["ck"]), torch.cat(vals["cv"]))
