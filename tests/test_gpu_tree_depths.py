"""GPU parity of drafted tokens whose positions are given without a mask: depths that repeat,
stay at 0 or lag behind a token's place, under windows.  The bound is that of
test_gpu_tree_attention.py; a key that the window alone hides must not reach a row, whatever it
holds."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def depths_of(kind, counts):
    out = []
    for c in counts:
        j = np.arange(c)
        out.append({"lag": np.where(j < 192, 0, 30 + (j - 192) // 4),  # hidden, far behind the place
                    "repeat": j // 3,
                    "zero": np.zeros(c, dtype=np.int64),
                    "back": (c - 1 - j) // 2}[kind])  # later tokens nearer to the context's end
    return np.concatenate(out)


@pytest.mark.parametrize("window", [1, 10, 100])
@pytest.mark.parametrize("kind", ["lag", "repeat", "zero", "back"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_depths_without_a_mask_under_a_window(D, kind, window):
    c = Case([224, 400, 151], [224, 230, 150], D=D, dtype="f16" if D == 128 else "bf16",
             kind="chain", seed=D + window)
    c.depths = depths_of(kind, c.counts)
    c.kw = dict(window=window)
    c.check()


@pytest.mark.parametrize("window", [5, 40])
def test_depths_without_a_mask_under_a_window_with_slopes_and_a_cap(window):
    c = Case([300, 224], [260, 200], G=4, D=128, dtype="f16", B=8, kind="chain", seed=window)
    c.depths = depths_of("lag", c.counts)
    c.kw = dict(window=window, cap=20.0, slopes=2.0 ** -np.arange(1.0, 9.0))
    c.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [1, 10])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_the_window_alone_hides_does_not_reach_a_row(D, window, bad):
    c = Case([224, 400], [224, 230], D=D, dtype="bf16", kind="chain", seed=3)
    c.depths = depths_of("lag", c.counts)
    c.kw = dict(window=window)
    want, spread, size = c.oracle()
    hidden = np.zeros(c.T, dtype=bool)
    sees = np.zeros(c.T, dtype=bool)
    for s, j in ((0, 5), (0, 100), (1, 191)):
        p = int(c.lens[s] - c.counts[s]) + j
        c.kc[c.tables[s, p // c.B], :, p % c.B] = bad
        c.vc[c.tables[s, p // c.B], :, p % c.B, ::3] = bad
        d = c.depths[c.starts[s]:c.starts[s + 1]]
        later = np.arange(c.counts[s]) >= j
        sees[c.starts[s]:c.starts[s + 1]] |= later & (d - d[j] < window)
        hidden[c.starts[s]:c.starts[s + 1]] |= later & (d - d[j] >= window)
    assert sees.any() and (hidden & ~sees).any()
    c.call()
    got = np64(c.out[:c.T])
    fine = np.abs(got - want) <= c.bound(want, spread, size)
    assert fine[~sees].all()
    assert not np.isfinite(got[sees][..., ::3]).any()
