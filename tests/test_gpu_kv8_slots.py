"""Attention of up to 16 rows a KV head whose (entry, head, page) items are fewer than the kernel's
CTAs: whatever the workspace held before, a call's results hold only what the call computed."""

import numpy as np
import pytest

from test_gpu_kv8 import BF16, F16, Case, _scores

pytestmark = pytest.mark.gpu


def _fill(ws, what):
    """NaN in every word; a partial that would outweigh any other (maximum 50, sum and values 50); zeros."""
    import torch
    if what == "nan":
        ws.fill_(0xFF)
    else:
        ws[:ws.numel() // 4 * 4].view(torch.float32).fill_({"large": 50.0, "zero": 0.0}[what])


FEW = [  # head_dim, n_kv, group, type, starts, lens, bound on the keys (table columns x 16)
    (128, 1, 2, F16, [519], [1], 0),          # 33 items
    (128, 1, 1, BF16, [999], [1], 0),
    (128, 8, 2, F16, [512], [1], 0),          # 264 items
    (128, 8, 2, F16, [69], [1], 4096),        # a short entry under a loose bound
    (128, 2, 8, F16, [33, 64], [1, 1], 1024),
    (64, 1, 16, BF16, [20], [1], 2048),       # 16 rows
    (64, 4, 3, F16, [530, 3, 0], [2, 5, 0], 0),
    (128, 1, 4, F16, [0], [4], 4096),         # one page, one item
    (128, 2, 2, F16, [100, 0], [6, 1], 640),
]


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("hd,n_kv,G,dtype,starts,lens,bound", FEW)
def test_workspace_contents_do_not_matter(qw, hd, n_kv, G, dtype, starts, lens, bound, score):
    ends = np.add(starts, lens)
    c = Case(qw, ends.tolist(), n_kv, hd, seed=hd + 5 * G + n_kv, max_pages=bound // 16 or None)
    c.append([0] * len(ends), ends)
    r = c.attn(starts, lens, G, dtype, pad=8, score=_scores(c, [max(int(ends.max()), bound)] * c.B) if score else None, bound=bound)
    c.check_attn(r)
    outs = [t for t in (r["out"], r["lse"], r["score"]) if t is not None]
    first = [t.clone() for t in outs]
    for what in ("nan", "large", "zero"):
        _fill(r["keep"][1], what)
        r["call"]()
        c.check_attn(r)
        assert all(c.torch.equal(a, b) for a, b in zip(first, outs)), what
    assert c.bits() == 0


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("n_kv", [1, 2, 4, 8])
def test_one_workspace_while_a_sequence_grows(qw, n_kv, score):
    """Steps of one sequence under a bound of 4096 keys that hand their workspace on."""
    c = Case(qw, [700], n_kv, 128, seed=90 + n_kv, max_pages=256)
    c.append([0], [700])
    ws = None
    for n in (700, 16, 17, 40, 100, 129, 300, 33, 513, 600, 700):
        r = c.attn([n - 1], [1], 2, score=_scores(c, [4096]) if score else None, bound=4096)
        mine = r["keep"][1]
        if ws is not None:
            mine.copy_(ws)
            r["call"]()
        c.check_attn(r)
        ws = mine.clone()
    assert c.bits() == 0


def test_scores_under_a_bound_of_more_keys_than_a_launch_has_blocks(qw):
    """Short entries under a bound of 65536 blocks of 1024 keys and some: scores as ever, the rest untouched."""
    import torch
    mk = (1 << 26) + 1024
    c = Case(qw, [200, 33], 1, 64, seed=77, max_pages=mk // 16)
    c.append([0, 0], [200, 33])
    sc = c.rng.random((2, 1, 300)).astype(np.float32)
    so = torch.zeros((2, 1, mk), device="cuda")
    so[:, :, :300] = torch.from_numpy(sc).cuda()
    q, qf = c.rows(2, 2, F16)
    out = torch.empty((2, 128), dtype=torch.float16, device="cuda")
    nb = c.qw.qw_kv8_attn_ws_bytes(c.view, 2, 2, 1, mk, 2, True)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    ds, dc = c.i32([199, 32]), c.i32([0, 1, 2])
    c.qw.qw_kv8_attn(c.view, 2, 2, 1, mk, ds.data_ptr(), dc.data_ptr(), q.data_ptr(), 128, 2, c.qw.QW_F16, 0.125, out.data_ptr(), 128, 0,
                     so.data_ptr(), so.data_ptr(), mk, ws.data_ptr(), nb, c.status.data_ptr())
    assert c.bits() == 0
    for b, n in enumerate((200, 33)):
        want, _, w, mag = c.orc.attention(c.table[b], n - 1, qf[b:b + 1], 0.125)
        got = out[b].double().cpu().numpy().reshape(1, 2, 64)
        assert np.all(np.abs(got - want) <= mag * 2.0 ** -10 + np.abs(want) * 2.0 ** -11 + 2.0 ** -24)
        base = sc[b, 0].astype(np.float64)
        base[:n] += w.reshape(2, n).sum(0)
        np.testing.assert_allclose(so[b, 0, :300].double().cpu().numpy(), base, rtol=2e-5, atol=1e-6)
    assert not bool(so[:, :, 300:].any())
