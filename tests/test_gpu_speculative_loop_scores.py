"""The speculative loop under capped scores, slopes and a window: what it says, and what it leaves in
the caches, is what one token a step says under the same scores.

The loops are those of test_gpu_speculative_loop.py.  The decode attention knows no such scores, so
one token a step is attended to as a chunk of one drafted token a sequence."""
import numpy as np
import pytest
import torch

import test_gpu_speculative_loop as loop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


class Scores:
    """The package with its attentions under the given scores."""

    def __init__(self, **kw):
        import paged_kv_cache_166_gb300 as m
        self.m, self.kw, self.calls = m, kw, 0

    def __getattr__(self, name):
        return getattr(self.m, name)

    def paged_decode_attention(self, q, kc, vc, tables, ctx, scale, out):
        starts = torch.arange(len(ctx) + 1, dtype=torch.int32, device="cuda")
        self.m.paged_tree_attention(q, kc, vc, tables, ctx, starts, scale, out, **self.kw)

    def paged_tree_attention(self, *args, **kw):
        self.calls += 1
        return self.m.paged_tree_attention(*args, **kw, **self.kw)


@pytest.mark.parametrize("kw", [dict(cap=5.0), dict(cap=1e6), dict(window=9), dict(window=1),
                                dict(cap=30.0, window=20, slopes=True)])
def test_the_loop_under_other_scores(kw, monkeypatch):
    prompts = [[5, 9, 200, 31, 7], [5, 9, 200, 31, 7, 8, 120], list(range(40, 75))]
    model, steps = loop.Model(seed=3), 40
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.exp2(-torch.arange(1.0, model.Hq + 1, device="cuda"))
    scores = Scores(**kw)
    monkeypatch.setattr(loop, "pkv", lambda: scores)
    want, rows = loop.greedy(model, prompts, steps)
    got, got_rows, accepted = loop.speculate(model, prompts, steps, want, np.random.default_rng(3))
    assert scores.calls > 0 and max(accepted) >= 3
    for w, g, p, a, b in zip(want, got, prompts, rows, got_rows):
        n = len(p) + steps
        assert g[:n] == w[:n]
        for x, y in zip(a, b):
            k = min(len(x), len(y), n)
            x, y = x[:k].double(), y[:k].double()
            # as in the loop without: two ways of one kernel round the second layer's inputs
            assert float((x - y).norm() / x.norm()) < 2.0 ** -7
