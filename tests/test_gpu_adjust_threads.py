"""Logit adjustment by host threads on one stream, one of them with requests that have no rows: the
second kernel of a call follows its first one whatever is queued between them."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROUNDS = 600


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def test_a_call_without_rows_between_the_launches_of_another():
    import paged_kv_cache_166_gb300 as pkv
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    T, V = 16, 100003
    x = torch.randn((T, V), generator=g, device="cuda").half()
    allowed = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, -(-V // 32)), generator=g, device="cuda",
                            dtype=torch.int32)
    history = torch.randint(0, V, (T, 2000), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.full((T,), 2000, dtype=torch.int32, device="cuda")
    rep = torch.full((T,), 1.5, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, idle = torch.empty_like(x), torch.full((4, 64), 7.0, device="cuda")
    small = torch.zeros((4, 64), device="cuda")

    def full():
        return pkv.adjust_logits(x, history, lens, repetition=rep, allowed=allowed, out=out)

    want = full().clone()
    bad = torch.zeros(1, dtype=torch.int64, device="cuda")
    done = threading.Event()

    def empty():
        while not done.is_set():
            pkv.adjust_logits(small, history[:1], lens[:1], row_start=none, out=idle)

    t = threading.Thread(target=empty)
    t.start()
    try:
        for _ in range(ROUNDS):
            out.fill_(7.0)
            full()
            bad += (out != want).sum()
        torch.cuda.synchronize()
    finally:
        done.set()
        t.join()
    assert int(bad) == 0
    assert (idle == 7.0).all()
