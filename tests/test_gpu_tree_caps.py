"""GPU parity of capped scores for caps of any size, the smallest and the largest floats among
them.

Bound: that of test_gpu_tree_attention.py with another term for the score.  A score x before the
cap has terms of at most b in absolute sum, and |cap tanh(x / cap)| <= |x| <= b with a derivative
of at most 1: the fp32 products and sums give (D + 8) 2^-24 b as without a cap.  The cap's own
operations give, with e = 2^-24:
* caps above 128: at most 16 e |x|.  x / cap is off by 4 e of itself (two products, two rounded
  factors), which the odd polynomial of |z| <= 1/2 passes on as at most 4 e |x|, its own sums and
  last product 3 e, its cut-off series 0.2 e; above 1/2 the exponential's argument 2 z log2(e) is
  off by 5 e of itself and the exponential by 3 e more, which moves 1 - 2 / (1 + e^2z) by at most
  4 e (2 w d / (1 + w)^2, w = e^2z), reciprocal and sum by 4 e: 8 e cap <= 16 e |x|;
* caps up to 128: at most 8 e cap, by the same count where the sum 1 + e^2z is rounded to e.
"""
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


def check(c):
    want, spread, _ = c.oracle()
    cap = c.kw.pop("cap")
    _, _, size = c.oracle()  # the terms of a score alone
    c.kw["cap"] = cap
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.call(status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    got = np64(c.out[:c.T])
    assert np.isfinite(got).all()
    u, e, n = torch.finfo(c.dt).eps / 2, 2.0 ** -24, int(c.lens.max())
    score = (c.D + 8 + 16) * e * size[..., None] + (8 * e * cap if cap <= 128 else 0.0)
    rel = u + 2 * (score + 2.0 ** -22) + 2 * (n + 8) * e
    bound = rel * spread + u * np.abs(want) + (2.0 ** -25 if c.dt == torch.float16 else 1e-38)
    over = np.abs(got - want) - bound
    worst = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, (worst, got[worst], want[worst])


@pytest.mark.parametrize("cap", [100.0, 128.0, 129.0, 1e3, 1e4, 1e5, 1e6, 1e7, 1e12, 1e30, 2e38,
                                 3.4028234e38])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_caps_far_above_the_scores(D, cap):
    c = Case([600, 40], [9, 40], D=D, dtype="f16", kind="tree", spread=2.0)
    c.kw = dict(cap=cap)
    check(c)


@pytest.mark.parametrize("cap,spread", [(129.0, 20.0), (200.0, 100.0), (1e3, 400.0), (1e4, 4000.0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_caps_beside_large_scores(D, cap, spread):
    """Scores from far below the cap to above it."""
    c = Case([600, 40], [9, 40], D=D, dtype="bf16", kind="chain", spread=spread)
    c.kw = dict(cap=cap)
    check(c)


@pytest.mark.parametrize("cap", [1e-45, 1e-39, 1e-30, 1e-3])
def test_caps_far_below_the_scores(cap):
    """Next to nothing is left of a score; one of exactly 0 stays 0."""
    c = Case([300, 40], [9, 40], D=64, dtype="f16", kind="tree")
    c.q[::2] = 0
    c.kw = dict(cap=float(np.float32(cap)))
    check(c)


@pytest.mark.parametrize("cap", [300.0, 1e6, 1e38])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0 ** -42, 1e-30])
def test_large_caps_beside_any_scale(scale, cap):
    c = Case([300, 20], [5, 20], D=128, dtype="f16")
    c.scale = scale
    c.kw = dict(cap=cap)
    check(c)


@pytest.mark.parametrize("cap", [300.0, 1e5])
def test_large_caps_with_slopes_windows_and_depths(cap):
    c = Case([1300, 513, 64], [20, 33, 64], Hkv=3, G=5, D=256, dtype="f16", B=8, spread=3.0)
    c.kw = dict(window=300, cap=cap, slopes=np.linspace(0.5, 0.01, 15))
    check(c)


def test_a_large_cap_where_contexts_are_cut_and_joined():
    c = Case([9000, 1, 4100], [12, 1, 30], Hkv=2, G=4, D=128, dtype="bf16", kind="tree")
    c.kw = dict(cap=1e6)
    check(c)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_keys_that_are_not_finite_under_a_large_cap(bad):
    """Rows that do not see them are as without; a NaN that is seen stays one, an infinite score
    is capped (here a single element of a key, with queries that are positive there)."""
    c = Case([300, 61], [12, 40], D=128, dtype="bf16", kind="tree", seed=3)
    c.kw = dict(cap=1e4)
    c.q[..., 0] = c.q[..., 0].abs() + 1
    want, spread, size = c.oracle()
    p = 300 - 12 + 5
    c.kc[c.tables[0, p // 16], :, p % 16, 0] = bad
    sees = np.zeros(c.T, dtype=bool)
    sees[:12] = c.seen[0][:, 5]
    assert sees.any() and not sees[:12].all()
    c.call()
    got = np64(c.out[:c.T])
    assert (np.abs(got - want) <= c.bound(want, spread, size))[~sees].all()
    if bad != bad:
        assert np.isnan(got[sees]).all()
    elif bad > 0:  # a score of 1e4: its value alone
        v = np64(c.vc[c.tables[0, p // 16], :, p % 16])  # [Hkv, D]
        assert np.allclose(got[sees], np.repeat(v, c.G, axis=0)[None], rtol=2.0 ** -7, atol=1e-30)
    else:  # -1e4: as if the key were not there
        c.seen[0][:, 5] = False
        c.kc[c.tables[0, p // 16], :, p % 16, 0] = 0
        want, spread, size = c.oracle()
        assert (np.abs(got - want) <= c.bound(want, spread, size))[sees].all()
