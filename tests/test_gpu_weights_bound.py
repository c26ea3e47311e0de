"""Attention weights with a bound on the batch's tokens: the workspace holds the scores of so
many, the results are the same, and a batch of more is reported and writes nothing behind it."""
import numpy as np
import pytest
import torch

import test_gpu_evict as E
from paged_kv_cache_166_gb300 import _native as N

pytestmark = pytest.mark.gpu
LENS = (1, 17, 0, 40, 100, 16, 15, 333)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def workspace(b, kind, max_tokens):
    """A workspace of exactly the bytes needed, and the bytes behind it."""
    m, w = E.pkv(), b.w
    n = m.weights_workspace_bytes(len(b.ctx), b.tables.shape[1], w.block_size, w.num_q_heads,
                                  w.num_kv_heads, w.head_dim, kind or b.q.dtype,
                                  max_tokens=max_tokens)
    x = torch.zeros(n + (1 << 16), dtype=torch.uint8, device="cuda")
    x[n:] = 0xa5
    return x[:n], x[n:]


CASES = [("f32", 64, 2, ""), ("bf16", 128, 1, ""), ("f16", 128, 8, ""), ("bf16", 128, 8, "fp8"),
         ("f16", 256, 2, "int8")]


@pytest.mark.parametrize("dtype,D,G,kind", CASES)
def test_the_bound_leaves_the_results_as_they_are(dtype, D, G, kind):
    b = E.batch(2 * G, 2, D, dtype, LENS, kind=kind, maxb_extra=1000)
    cols = b.tables.shape[1] * 16
    start = torch.rand((len(LENS), 2, cols), device="cuda")
    want = start.clone()
    out = E.attend(b, want)
    for tokens in (sum(LENS), sum(LENS) + 5, 10 ** 9, 1 << 60):
        ws, behind = workspace(b, kind, tokens)
        sums = start.clone()
        got = E.attend(b, sums, workspace=ws, max_tokens=tokens)
        assert torch.equal(got, out) and torch.equal(sums, want)
        assert bool((behind == 0xa5).all())
        assert E.pkv().decode_status(ws) == 0
    sums = start.clone()  # and in the cached workspace
    assert torch.equal(E.attend(b, sums, max_tokens=sum(LENS)), out) and torch.equal(sums, want)


@pytest.mark.parametrize("dtype,D,G,kind", CASES)
def test_too_many_tokens_are_reported_and_add_nothing(dtype, D, G, kind):
    b = E.batch(2 * G, 2, D, dtype, LENS, kind=kind)
    start = torch.rand((len(LENS), 2, b.tables.shape[1] * 16), device="cuda")
    out = E.attend(b)
    for tokens in (0, 100, sum(LENS) - 16 * len(LENS)):
        ws, behind = workspace(b, kind, tokens)
        sums = start.clone()
        got = E.attend(b, sums, workspace=ws, max_tokens=tokens)
        assert torch.equal(got, out) and torch.equal(sums, start)
        assert bool((behind == 0xa5).all())
        assert E.pkv().decode_status(ws) == N.PKV_DEV_TOO_MANY_TOKENS
        # the workspace serves a batch that fits afterwards
        b1 = E.batch(2 * G, 2, D, dtype, (9,) * len(LENS), kind=kind)
        if tokens >= 9 * len(LENS):
            x, y = (torch.zeros((len(LENS), 2, 16), device="cuda") for _ in range(2))
            assert torch.equal(E.attend(b1, x, workspace=ws, max_tokens=tokens), E.attend(b1, y))
            assert torch.equal(x, y) and E.pkv().decode_status(ws) == 0


def test_refusals():
    b = E.batch(4, 2, 128, "bf16", LENS)
    sums = torch.zeros((len(LENS), 2, b.tables.shape[1] * 16), device="cuda")
    with pytest.raises(ValueError):
        E.attend(b, sums, max_tokens=-1)
    ws, _ = workspace(b, "", 50)
    with pytest.raises(ValueError):
        E.attend(b, sums, workspace=ws, max_tokens=500)
    assert np.all(E.BT.np64(sums) == 0)
