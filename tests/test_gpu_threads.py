"""Host threads that call on one stream: each gets the results it gets alone.

Calls of the attention weights share a workspace per stream and hand their scores from one
launch to the next through it, so the launches of two calls must not be queued crosswise.
"""
import threading

import numpy as np
import pytest
import torch

import batches as BT
from paged_kv_cache_166_gb300 import workloads as W

pytestmark = pytest.mark.gpu
ROUNDS = 400


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def pkv():
    import paged_kv_cache_166_gb300 as m
    return m


class Caller:
    def __init__(self, lens, Hkv, seed):
        w = W.Workload(name="t", seed=seed, num_q_heads=4 * Hkv, num_kv_heads=Hkv, head_dim=128,
                       dtype="bf16", block_size=16)
        self.b = BT.decode_batch(w, np.asarray(lens))
        self.tables, self.ctx, _ = self.b.device_index("cuda")
        self.reset()

    def reset(self):
        b = self.b
        self.out = torch.zeros_like(b.q)
        self.sums = torch.zeros((len(b.ctx), b.w.num_kv_heads, b.tables.shape[1] * 16),
                                device="cuda")

    def run(self):
        b = self.b
        for _ in range(ROUNDS):
            pkv().paged_decode_attention_weights(b.q, b.kc, b.vc, self.tables, self.ctx, b.w.scale,
                                                 self.out, self.sums)


def test_two_threads_on_one_stream():
    callers = [Caller((100, 0, 333, 40), 2, 1), Caller((17, 900), 1, 2), Caller((64,) * 9, 4, 3)]
    want = []
    for c in callers:
        c.run()
        want.append((c.out, c.sums))
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
    for c, (out, sums) in zip(callers, want):
        assert torch.equal(c.out, out) and torch.equal(c.sums, sums)
