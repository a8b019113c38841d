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
