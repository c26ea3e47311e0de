"""GPU: the accepted path's rows moved to the front, bit for bit as the oracle moves them."""
import numpy as np
import pytest
import torch

from oracle import speculative as osp

pytestmark = pytest.mark.gpu
V_POS = np.array([0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15])


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def pkv():
    import paged_kv_cache_166_gb300 as m
    return m


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def move_row(src, dst, a, b):
    dst[b[0], :, b[1]] = src[a[0], :, a[1]]


def move_byte(src, dst, a, b):
    dst[b[0], :, :, V_POS[b[1]]] = src[a[0], :, :, V_POS[a[1]]]


class Case:
    def __init__(self, counts, lens=None, layers=2, Hkv=2, D=64, B=16, dtype=torch.float16, seed=0,
                 whole=False):
        rng = np.random.default_rng(seed)
        counts = np.asarray(counts)
        base = rng.integers(0, 70, len(counts)) if lens is None else np.asarray(lens)
        self.lens = base + counts
        nb = -(-self.lens // B)
        NB = int(nb.sum()) + 2
        order = rng.permutation(NB)
        self.tables = np.full((len(counts), max(1, int(nb.max()))), -9, dtype=np.int64)
        at = 0
        for s, n in enumerate(nb):
            self.tables[s, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum(counts)])
        self.n = np.array([c if whole else rng.integers(0, c + 1) for c in counts])
        P = max(1, int(self.n.max()))
        self.path = np.full((len(counts), P), -1)
        for s, c in enumerate(counts):
            self.path[s, :self.n[s]] = np.sort(rng.permutation(c)[:self.n[s]])
        self.q8 = dtype in (torch.uint8, torch.int8)
        kshape, vshape = (NB, Hkv, B, D), (NB, Hkv, D, B) if self.q8 else (NB, Hkv, B, D)
        bits = lambda sh: torch.as_tensor(rng.integers(0, 256, sh + (dtype.itemsize,), dtype=np.uint8),  # noqa: E731
                                          device="cuda").view(dtype)[..., 0].contiguous()
        self.kc = [bits(kshape) for _ in range(layers)]
        self.vc = [bits(vshape) for _ in range(layers)]

    def call(self, **kw):
        pkv().paged_tree_commit(kw.pop("kc", self.kc), kw.pop("vc", self.vc), i32(self.tables),
                                i32(self.lens), i32(self.starts), i32(self.path), i32(self.n), **kw)

    def raw(self, t):
        return t.contiguous().view(torch.uint8).view(*t.shape, -1).cpu().numpy()

    def check(self):
        want = []
        for caches, move in ((self.kc, move_row), (self.vc, move_byte if self.q8 else move_row)):
            for c in caches:
                x = self.raw(c)
                B = c.shape[3] if move is move_byte else c.shape[2]
                y = x.copy()
                for s in range(len(self.lens)):
                    base = int(self.lens[s]) - int(self.starts[s + 1] - self.starts[s])
                    for j in range(int(self.n[s])):
                        a, b = base + int(self.path[s, j]), base + j
                        move(x, y, (int(self.tables[s, a // B]), a % B),
                             (int(self.tables[s, b // B]), b % B))
                want.append(y)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.call(status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        for c, w in zip(self.kc + self.vc, want):
            assert np.array_equal(self.raw(c), w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16, torch.uint8, torch.int8])
@pytest.mark.parametrize("D", [16, 64, 128])
def test_types(dtype, D):
    Case([1, 5, 17, 40, 3], D=D, dtype=dtype).check()


@pytest.mark.parametrize("B", [1, 5, 8, 16, 32])
def test_block_sizes(B):
    Case([7, 30, 1, 64], B=B, seed=B).check()


@pytest.mark.parametrize("layers", [1, 3, 80, 128])
def test_layers(layers):
    Case([6, 12], layers=layers, Hkv=1, D=16, seed=layers).check()


def test_long_paths():
    Case([300, 150, 64, 65], Hkv=3, D=80, whole=False, seed=7).check()
    Case([300, 150], Hkv=1, D=16, whole=True).check()  # everything accepted: nothing moves


def test_no_path_and_many_sequences():
    Case([0, 4, 0], seed=1).check()
    Case(np.arange(500) % 9, Hkv=2, D=16, B=8, seed=2).check()
    c = Case([3, 4])
    before = [c.raw(x) for x in c.kc]
    c.n[:] = 0
    c.call()
    assert all(np.array_equal(c.raw(a), b) for a, b in zip(c.kc, before))


def test_all_paths_of_a_small_tree():
    """Every ascending choice of six drafted tokens."""
    for bits in range(1, 64):
        c = Case([6], lens=[13], layers=1, Hkv=1, D=16, B=8)
        path = [i for i in range(6) if bits >> i & 1]
        c.path, c.n = np.array([path]), np.array([len(path)])
        c.check()


def test_layers_in_one_tensor():
    c = Case([9, 20], layers=4)
    k, v = torch.stack(c.kc), torch.stack(c.vc)
    c.call(kc=k, vc=v)
    c.check()
    for one, many in ((k, c.kc), (v, c.vc)):
        assert np.array_equal(c.raw(one), c.raw(torch.stack(many)))


def test_what_does_not_fit_is_reported():
    from paged_kv_cache_166_gb300 import _native as N
    for field, at, value, bit in (("n", 0, 9, N.PKV_DEV_BAD_POSITION), ("n", 1, -1, N.PKV_DEV_BAD_POSITION),
                                  ("path", (0, 2), 1, N.PKV_DEV_BAD_POSITION),
                                  ("path", (0, 2), 8, N.PKV_DEV_BAD_POSITION),
                                  ("path", (0, 0), -1, N.PKV_DEV_BAD_POSITION),
                                  ("lens", 1, 3, N.PKV_DEV_BAD_CONTEXT_LEN),
                                  ("lens", 1, 10 ** 6, N.PKV_DEV_BAD_CONTEXT_LEN),
                                  ("lens", 1, -1, N.PKV_DEV_BAD_CONTEXT_LEN)):
        c = Case([8, 6], lens=[20, 30])
        c.path, c.n = np.array([[1, 3, 5], [2, 3, 5]]), np.array([3, 3])
        getattr(c, field)[at] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.call(status=status)
        torch.cuda.synchronize()
        assert int(status) == bit, (field, value)
    c = Case([8], lens=[20])
    c.path, c.n = np.array([[4, 5]]), np.array([2])
    c.tables[0, 1] = 10 ** 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.call(status=status)
    assert int(status) == N.PKV_DEV_BAD_BLOCK_ID
    Case([8], lens=[20]).check()


def test_refusals():
    m = pkv()
    c = Case([4, 5])
    with pytest.raises(ValueError):
        c.call(kc=c.kc[:1])
    with pytest.raises(ValueError):
        c.call(kc=[c.kc[0], c.kc[1][:-1]])
    with pytest.raises(ValueError):
        c.call(kc=[], vc=[])
    with pytest.raises(ValueError):
        c.call(kc=[x.transpose(2, 3) for x in c.kc])
    with pytest.raises(ValueError):
        c.call(kc=torch.stack(c.kc)[:, :, :, :, ::2])
    with pytest.raises(ValueError):
        c.call(status=torch.zeros(1, device="cuda"))
    with pytest.raises(m.PkvError):
        c.call(kc=c.kc * 65, vc=c.vc * 65)
    for kc, vc in ((c.kc[:1] * 2, c.vc), (c.kc, c.vc[:1] * 2), (c.kc, [c.vc[1], c.kc[0]])):
        with pytest.raises(m.PkvError, match="share a cache"):
            c.call(kc=kc, vc=vc)
    c.n = c.n[:1]
    with pytest.raises(ValueError):
        c.call()


def test_graph_and_stream():
    c = Case([12, 30], lens=[50, 7], layers=5, whole=False, seed=4)
    a, b = [x.clone() for x in c.kc], [x.clone() for x in c.vc]
    args = [i32(x) for x in (c.tables, c.lens, c.starts, c.path, c.n)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv().paged_tree_commit(a, b, *args)
    g.replay()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    k2, v2 = [x.clone() for x in c.kc], [x.clone() for x in c.vc]
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        pkv().paged_tree_commit(k2, v2, *args)
    st.synchronize()
    c.check()
    for x, y, z in zip(c.kc + c.vc, a + b, k2 + v2):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(x.view(torch.int16), z.view(torch.int16))


def test_oracle_commit_is_the_same_moves():
    c = Case([9], lens=[20], layers=1)
    x = c.raw(c.kc[0])
    y = x.copy()
    osp.commit(y, c.tables, c.lens, c.starts, c.path, c.n, move_row)
    c.call()
    assert np.array_equal(c.raw(c.kc[0]), y)


def test_caches_past_2_to_the_31_elements():
    NB, Hkv, B, D = 140000, 8, 16, 128
    kc = torch.zeros((NB, Hkv, B, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    kc[NB - 1, :, 9], vc[NB - 1, :, 9] = 3.0, 4.0
    pkv().paged_tree_commit([kc], [vc], i32([[NB - 1]]), i32([12]), i32([0, 8]), i32([[5]]), i32([1]))
    assert (kc[NB - 1, :, 4] == 3).all() and (vc[NB - 1, :, 4] == 4).all()
    assert int(torch.count_nonzero(kc)) == 2 * Hkv * D
