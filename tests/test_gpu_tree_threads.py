"""Host threads that call the attention of drafted tokens, or the logit adjustment, on one stream:
each gets the results it gets alone.

Calls of the attention share a workspace per stream and hand pieces of units, and where they
belong, from one launch to the next through it, so the launches of two calls must not be queued
crosswise."""
import threading

import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case, i32, osp, pkv

pytestmark = pytest.mark.gpu
ROUNDS = 400


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


class Attention:
    def __init__(self, **kw):
        c = self.c = Case(**kw)
        self.args = (c.q, c.kc, c.vc, i32(c.tables), i32(c.lens), i32(c.starts), c.scale)
        self.kw = {}
        if c.seen is not None:
            self.kw = dict(tree_mask=i32(np.concatenate([osp.words(s, c.W) for s in c.seen])),
                           depths=i32(c.depths))
        self.out = c.out

    def reset(self):
        self.out = self.c.out = torch.full_like(self.c.out, 7.0)

    def run(self):
        for _ in range(ROUNDS):
            pkv().paged_tree_attention(*self.args, self.out[:self.c.T], **self.kw)


class Logits:
    def __init__(self, S, rows, V, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.x = torch.randn((S * rows, V), generator=g, device="cuda").half()
        self.kw = dict(row_start=i32(np.arange(S + 1) * rows),
                       repetition=torch.full((S,), 1.3, device="cuda"),
                       allowed=torch.randint(-2 ** 31, 2 ** 31 - 1, (S * rows, -(-V // 32)), generator=g,
                                             device="cuda", dtype=torch.int32))
        self.history = torch.randint(0, V, (S, 300), generator=g, device="cuda", dtype=torch.int32)
        self.lens = i32([300] * S)
        self.reset()

    def reset(self):
        self.out = torch.full_like(self.x, 7.0)

    def run(self):
        for _ in range(ROUNDS):
            pkv().adjust_logits(self.x, self.history, self.lens, out=self.out, **self.kw)


def test_threads_on_one_stream():
    callers = [Attention(lens=[3000, 700], counts=[12, 40], Hkv=2, G=4, seed=1),
               Attention(lens=[9000], counts=[20], Hkv=1, G=6, dtype="f16", D=64, seed=2),
               Attention(lens=[64] * 90, counts=[3] * 90, kind="chain", seed=3),
               Logits(4, 3, 5000, 4), Logits(1, 1, 32001, 5)]
    want = []
    for c in callers:
        c.run()
        want.append(c.out)
        c.reset()
    torch.cuda.synchronize()
    errors = []

    def go(c):
        try:
            c.run()
        except Exception as e:  # noqa: BLE001 (handed to the test's thread)
            errors.append(e)
    threads = [threading.Thread(target=go, args=(c,)) for c in callers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, out in zip(callers, want):
        assert torch.equal(c.out, out)
