"""A prompt cut down right after its prefill.

A prompt's tokens have no attention weight until a call adds some: with sums of zero every
token between the ends is equal and the lowest positions stay.  Weights come from the prompt's
last queries, given to the attention with weights as sequences of their own under the prompt's
block table, query i with the context that it sees.
"""
import numpy as np
import pytest
import torch

import test_gpu_evict as E
from oracle import eviction as oev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def select(sums, t, keep, first, recent):
    H = sums.shape[1]
    kept = torch.zeros((1, H, keep), dtype=torch.int32, device="cuda")
    new = torch.zeros((1, H, keep), device="cuda")
    n = E.i32([0])
    E.pkv().paged_evict_select(sums, E.i32([t]), E.i32([keep]), kept, new, n, first, recent)
    assert int(n) == min(keep, t)
    return kept.cpu().numpy()[0], new


@pytest.mark.parametrize("dtype,D,G,kind", [("bf16", 128, 4, ""), ("f16", 128, 8, "fp8"),
                                            ("bf16", 128, 1, "int8"), ("f32", 64, 2, "")])
def test_prompt_eviction_by_its_last_queries(dtype, D, G, kind):
    t, window, keep, first, recent, Hkv = 333, 32, 100, 4, 32, 2
    b = E.batch(G * Hkv, Hkv, D, dtype, (t,), kind=kind, seed=7)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    b.q = torch.randn((window, G * Hkv, D), generator=g, device="cuda").to(b.q.dtype)
    b.tables = np.repeat(b.tables, window, 0)
    b.ctx = np.arange(t - window + 1, t + 1).astype(np.int32)
    rows = torch.zeros((window, Hkv, b.tables.shape[1] * 16), device="cuda")
    E.attend(b, rows)
    E.check_sums(b, torch.zeros_like(rows), rows)
    sums = rows.sum(0, keepdim=True)
    kept, new = select(sums, t, keep, first, recent)
    x = E.BT.np64(sums)[0]
    for h in range(Hkv):
        want = oev.select(x[h], t, keep, first, recent)
        assert np.array_equal(kept[h], want)
        assert np.array_equal(E.BT.np64(new)[0, h], x[h][want])


def test_without_weights_the_lowest_positions_stay():
    kept, _ = select(torch.zeros((1, 2, 400), device="cuda"), 333, 100, 4, 32)
    assert np.array_equal(kept, np.tile(np.r_[0:68, 301:333], (2, 1)))
