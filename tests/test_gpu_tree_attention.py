"""GPU parity of the attention of drafted tokens against the fp64 oracle.

Bound of an element, with u the type's half step (eps / 2), A = sum_p w_p |V_p| and n the keys:
* the probabilities are rounded to the type, u each, the same for both halves of a sum: u A;
* a score x, of terms of at most b in absolute sum (scale |q| . |k|, the cap, the bias), is off
  by at most (D + 8) 2^-24 b (fp32 products and sums, then its few further operations), its
  exponential by that and 2^-22 more, numerator and denominator alike: twice that times A;
* sums over n keys in fp32: (n + 8) 2^-24 A, numerator and denominator;
* probabilities of f16 below 2^-32 of the largest are lost: n 2^-32 A (covered by the line above);
* one rounding of the result: u |out|, and half the type's smallest step (2^-25 in f16).
"""
import numpy as np
import pytest
import torch

from oracle import speculative as osp

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def pkv():
    import paged_kv_cache_166_gb300 as m
    return m


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def parents_of(rng, c):
    return np.array([rng.integers(-1, i) if i else -1 for i in range(c)], dtype=np.int64)


class Case:
    def __init__(self, lens, counts, Hkv=2, G=2, D=128, B=16, dtype="bf16", kind="tree", seed=0,
                 spread=1.0, extra=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = DT[dtype]
        lens, counts = np.asarray(lens), np.asarray(counts)
        nb = -(-lens // B)
        NB = int(nb.sum()) + 3
        order = rng.permutation(NB)
        tables = np.full((len(lens), max(1, int(nb.max())) + extra), NB + 7, dtype=np.int64)
        at = 0
        for s, n in enumerate(nb):
            tables[s, :n] = order[at:at + n]
            at += n
        T = int(counts.sum())
        self.__dict__.update(lens=lens, counts=counts, tables=tables, NB=NB, B=B, Hkv=Hkv, G=G, D=D,
                             dt=dt, T=T)
        self.q = (torch.randn((T, Hkv * G, D), generator=g, device="cuda") * spread).to(dt)
        self.kc, self.vc = (torch.randn((NB, Hkv, B, D), generator=g, device="cuda").to(dt)
                            for _ in range(2))
        self.starts = np.concatenate([[0], np.cumsum(counts)])
        self.seen = self.mask = self.depths = None
        if kind != "chain":
            both = [osp.tree_masks(parents_of(rng, c)) for c in counts]
            self.seen = [s for s, _ in both]
            if kind == "random":  # any bits: rows may see nothing, not even themselves
                self.seen = [rng.random(s.shape) < 0.3 for s in self.seen]
            self.depths = np.concatenate([d for _, d in both]) if T else np.zeros(0, int)
            self.W = max(1, -(-int(counts.max()) // 32))
        self.scale = 1.0 / np.sqrt(D)
        self.out = torch.full((T + 3, Hkv * G, D), 7.0, dtype=dt, device="cuda")
        self.kw = {}

    def call(self, **more):
        kw = dict(self.kw)
        if self.seen is not None:
            words = np.concatenate([osp.words(s, self.W) for s in self.seen])
            # bits past a sequence's drafted tokens mean nothing
            for s, c in enumerate(self.counts):
                rows = words[self.starts[s]:self.starts[s + 1]].view(np.uint32)
                for w in range(self.W):
                    dead = min(32, max(0, 32 * (w + 1) - c))
                    if dead == 32:
                        rows[:, w] = 0xffffffff
                    elif dead:
                        rows[:, w] |= np.uint32((0xffffffff << (32 - dead)) & 0xffffffff)
            kw["tree_mask"] = i32(words)
        no_depths = kw.pop("no_depths", False)
        if self.depths is not None and not no_depths:
            kw["depths"] = i32(self.depths)
        if kw.get("slopes") is not None:
            kw["slopes"] = torch.tensor(kw["slopes"], dtype=torch.float32, device="cuda")
        kw.update(more)
        return pkv().paged_tree_attention(self.q, self.kc, self.vc, i32(self.tables), i32(self.lens),
                                          i32(self.starts), self.scale, self.out[:self.T], **kw)

    def oracle(self):
        depths = None if self.kw.get("no_depths") else self.depths
        used = np.unique(np.concatenate([t[:-(-n // self.B)] for t, n in zip(self.tables, self.lens)]))
        back = np.zeros(self.NB + 8, dtype=np.int64)
        back[used] = np.arange(len(used))
        at = torch.as_tensor(used, device="cuda")
        return osp.tree_attention(np64(self.q), np64(self.kc[at]), np64(self.vc[at]),
                                  back[np.minimum(self.tables, self.NB + 7)], self.lens, self.starts,
                                  self.scale, self.seen, depths, self.kw.get("cap", 0.0),
                                  self.kw.get("slopes"), self.kw.get("window", 0))

    def bound(self, want, spread, size):
        u = torch.finfo(self.dt).eps / 2
        n = int(self.lens.max()) if len(self.lens) else 0
        rel = u + 2 * ((self.D + 8) * 2.0 ** -24 * size[..., None] + 2.0 ** -22) + 2 * (n + 8) * 2.0 ** -24
        return rel * spread + u * np.abs(want) + (2.0 ** -25 if self.dt == torch.float16 else 1e-38)

    def check(self, **more):
        want, spread, size = self.oracle()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.call(status=status, **more)
        torch.cuda.synchronize()
        assert int(status) == 0
        got = np64(self.out[:self.T])
        assert np.isfinite(got).all()
        over = np.abs(got - want) - self.bound(want, spread, size)
        worst = np.unravel_index(over.argmax(), over.shape) if over.size else None
        assert not over.size or over.max() <= 0, (worst, got[worst], want[worst])
        assert (self.out[self.T:] == 7.0).all()


@pytest.mark.parametrize("kind", ["chain", "tree", "random"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_short_contexts(kind, D, dtype):
    Case([1, 5, 17, 128, 129, 300], [1, 5, 4, 9, 33, 7], D=D, dtype=dtype, kind=kind).check()


@pytest.mark.parametrize("G", list(range(1, 17)))
def test_heads_of_a_group(G):
    Case([40, 257, 90], [17, 40, 3], Hkv=1 + G % 3, G=G, D=64, dtype="f16", seed=G).check()


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_block_sizes_and_ragged_ends(B, D):
    lens = [31, 32, 33, 127, 128, 129, 255, 256, 257, 2]
    Case(lens, [1, 2, 33, 5, 64, 65, 1, 3, 100, 2], B=B, D=D, dtype="bf16", seed=B, extra=2).check()


@pytest.mark.parametrize("D,dtype,kind", [(64, "bf16", "tree"), (128, "f16", "tree"),
                                          (128, "bf16", "chain"), (256, "f16", "random")])
def test_long_contexts_are_cut_and_joined(D, dtype, kind):
    """Three sequences over all SMs: pieces of a unit are joined."""
    Case([9000, 1, 4100], [12, 1, 30], Hkv=2, G=4, D=D, dtype=dtype, kind=kind).check()


def test_many_short_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 700)
    counts = np.minimum(lens, rng.integers(0, 6, 700))
    Case(lens, counts, Hkv=2, G=2, D=64, dtype="f16").check()


def test_a_long_chunk_of_many_tiles():
    Case([1500, 1000], [1100, 700], Hkv=2, G=3, D=64, dtype="f16", kind="chain").check()


def test_scores_that_grow_along_the_context():
    """The running maximum moves often: keys get larger with their position."""
    c = Case([2000, 700], [8, 20], G=4, D=128, dtype="bf16", spread=2.0)
    for s in range(2):
        for p in range(0, int(c.lens[s]), 16):
            c.kc[c.tables[s, p // 16]] *= (1 + p / 400)
    c.check()


def test_one_drafted_token_is_decode_attention():
    c = Case([700, 33, 1, 2000], [1, 1, 1, 1], Hkv=4, G=8, D=128, dtype="bf16", kind="chain")
    c.check()
    ref = torch.empty_like(c.q)
    pkv().paged_decode_attention(c.q, c.kc, c.vc, i32(c.tables), i32(c.lens), c.scale, ref)
    # two kernels within the bound's main terms of the same value: 2 (u A + u |out|)
    _, spread, _ = c.oracle()
    gap = np.abs(np64(c.out[:c.T]) - np64(ref))
    assert (gap <= 2.1 * 2.0 ** -8 * (spread + np.abs(np64(ref)))).all()


@pytest.mark.parametrize("cap", [5.0, 30.0])
@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_capped_scores(cap, kind, D):
    c = Case([600, 40], [9, 40], D=D, dtype="f16", kind=kind, spread=4.0)
    c.kw = dict(cap=cap)
    c.check()


@pytest.mark.parametrize("kind,no_depths", [("chain", False), ("tree", False), ("tree", True)])
@pytest.mark.parametrize("D", [64, 256])
def test_bias_by_distance(kind, no_depths, D):
    c = Case([600, 70, 131], [9, 40, 5], G=4, D=D, dtype="bf16", kind=kind)
    c.kw = dict(slopes=2.0 ** -np.arange(1.0, 9.0), no_depths=no_depths)
    c.check()


@pytest.mark.parametrize("window", [1, 2, 5, 100, 128, 129, 10000, (1 << 31) - 1])
@pytest.mark.parametrize("kind,no_depths", [("chain", False), ("tree", False), ("random", True)])
def test_windows(window, kind, no_depths):
    c = Case([600, 40, 300], [9, 40, 150], G=2, D=128, dtype="f16", kind=kind, seed=window % 97)
    c.kw = dict(window=window, no_depths=no_depths)
    c.check()


def test_everything_at_once():
    c = Case([1300, 513, 64], [20, 33, 64], Hkv=3, G=5, D=256, dtype="f16", B=8, spread=3.0)
    c.kw = dict(window=300, cap=20.0, slopes=np.linspace(0.5, 0.01, 15))
    c.check()


def test_zero_and_negative_scales():
    for scale in (0.0, -0.1):
        c = Case([300, 20], [5, 20], dtype="f16")
        c.scale = scale
        c.check()


@pytest.mark.parametrize("kind", ["chain", "tree", "random"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 256])
def test_what_is_not_seen_does_not_reach_a_row(kind, bad, D):
    """A drafted token whose K and V are not finite: rows that do not see it are as if it were
    0; rows past the context and before the window may hold anything too."""
    c = Case([300, 61], [12, 40], D=D, dtype="bf16", kind=kind, seed=2)
    window = 100
    c.kw = dict(window=window)
    want, spread, size = c.oracle()
    slots = []
    for s, j in ((0, 5), (1, 13), (1, 39)):
        p = int(c.lens[s] - c.counts[s]) + j
        slots.append((int(c.tables[s, p // c.B]), p % c.B))
    sees = np.zeros(c.T, dtype=bool)
    for s, j in ((0, 5), (1, 13), (1, 39)):
        m = np.tri(c.counts[s], dtype=bool) if c.seen is None else c.seen[s]
        sees[c.starts[s]:c.starts[s + 1]] |= m[:, j]
    assert sees.any() and not sees.all()
    for b, i in slots:
        c.kc[b, :, i] = bad
        c.vc[b, :, i, ::3] = bad
    last = c.tables[0, (c.lens[0] - 1) // c.B]  # slots past the context
    c.kc[last, :, c.lens[0] % c.B:] = bad
    c.vc[last, :, c.lens[0] % c.B:] = bad
    first = max(0, int(c.lens[0] - c.counts[0]) - window + 1)  # before every row's window
    for p in range(first):
        c.kc[c.tables[0, p // c.B], :, p % c.B] = bad
        c.vc[c.tables[0, p // c.B], :, p % c.B] = bad
    c.call()
    got = np64(c.out[:c.T])
    fine = np.abs(got - want) <= c.bound(want, spread, size)
    assert fine[~sees].all()
    # a row that sees a NaN or infinite key or value is not finite where the formula is not
    assert not np.isfinite(got[sees][..., ::3]).any()


@pytest.mark.parametrize("kw", [dict(cap=20.0), dict(cap=20.0, slopes=[1.0, 0.5, 0.1, 2.0]),
                                dict(slopes=[1.0, 0.5, 0.1, -2.0])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 256])
def test_what_is_not_seen_does_not_reach_its_neighbours(kw, bad, D):
    """Keys that are not finite between keys that are, under a cap and slopes: rows that do not
    see them are as without; a NaN that is seen stays one (an infinite score is capped)."""
    c = Case([300, 61], [12, 40], D=D, dtype="f16", kind="tree", seed=3)
    c.kw = dict(kw)
    want, spread, size = c.oracle()
    c.kc[c.tables[0, (300 - 12 + 5) // c.B], :, (300 - 12 + 5) % c.B] = bad
    last = c.tables[0, (c.lens[0] - 1) // c.B]  # slots past the context
    c.kc[last, :, c.lens[0] % c.B:] = bad
    sees = np.zeros(c.T, dtype=bool)
    sees[:12] = c.seen[0][:, 5]
    assert sees.any() and not sees[:12].all()
    c.call()
    got = np64(c.out[:c.T])
    fine = np.abs(got - want) <= c.bound(want, spread, size)
    assert fine[~sees].all()
    if bad != bad:
        assert np.isnan(got[sees]).all()


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30, 2.0 ** -42])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_slopes_beside_any_scale(scale, kind):
    c = Case([300, 40], [9, 40], D=128, dtype="f16", kind=kind, seed=5)
    c.scale = scale
    c.kw = dict(slopes=[1.0, 0.0, 0.03125, -0.25])
    c.check()


def test_depths_far_from_a_token_s_place():
    """Depths that leave gaps, under slopes: distances are taken of them, not of places."""
    c = Case([700, 40], [150, 40], D=128, dtype="bf16", kind="tree", seed=6)
    c.depths = c.depths * 1000003 % 40009 + 100
    c.kw = dict(slopes=[1e-4, 3e-5, 1e-3, 2e-4])
    c.check()


def test_value_alone_not_finite():
    """Finite keys, an infinite value: exactly its columns are infinite, in exactly its rows."""
    c = Case([300], [12], D=128, dtype="f16", seed=4)
    want, spread, size = c.oracle()
    p = int(c.lens[0] - c.counts[0]) + 3
    c.vc[c.tables[0, p // 16], :, p % 16, 7] = float("inf")
    c.call()
    got = np64(c.out[:c.T])
    sees = c.seen[0][:, 3]
    assert np.isposinf(got[sees][..., 7]).all()
    got[sees, :, 7] = want[sees, :, 7]
    assert (np.abs(got - want) <= c.bound(want, spread, size)).all()


def test_a_context_value_not_finite_reaches_all_and_only_its_sequence():
    c = Case([300, 300], [12, 12], D=128, dtype="bf16", seed=4)
    want, spread, size = c.oracle()
    c.vc[c.tables[0, 3], :, 5, 7] = float("inf")
    c.call()
    got = np64(c.out[:c.T])
    assert np.isposinf(got[:12, :, 7]).all()
    got[:12, :, 7] = want[:12, :, 7]
    assert (np.abs(got - want) <= c.bound(want, spread, size)).all()


def test_bad_lengths_and_blocks_are_reported():
    m = pkv()
    from paged_kv_cache_166_gb300 import _native as N
    c = Case([100, 64, 30], [4, 5, 3], D=64, dtype="f16", kind="chain")
    for field, s, value, bit in (("lens", 1, -4, N.PKV_DEV_BAD_CONTEXT_LEN),
                                 ("lens", 1, 10 ** 6, N.PKV_DEV_BAD_CONTEXT_LEN),
                                 ("lens", 1, 2, N.PKV_DEV_BAD_CONTEXT_LEN),
                                 ("tables", (1, 1), -1, N.PKV_DEV_BAD_BLOCK_ID),
                                 ("tables", (1, 1), c.NB, N.PKV_DEV_BAD_BLOCK_ID)):
        keep = getattr(c, field).copy()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        getattr(c, field)[s] = value
        c.call(status=status)
        torch.cuda.synchronize()
        assert int(status) & bit, (field, value)
        setattr(c, field, keep)
    starts = c.starts.copy()
    for bad in ([0, 4, 2, 12], [0, 4, 9, 500], [-3, 4, 9, 12]):
        c.starts = np.array(bad)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.call(status=status)
        torch.cuda.synchronize()
        assert int(status) & N.PKV_DEV_BAD_CONTEXT_LEN, bad
    c.starts = starts
    t = Case([100], [40], D=64, dtype="f16")
    t.depths[3] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.call(status=status)
    assert int(status) == N.PKV_DEV_BAD_POSITION
    status.zero_()
    t.depths[3] = 1
    t.call(status=status, tree_mask=torch.full((40, 1), -1, dtype=torch.int32, device="cuda"))
    assert int(status) == N.PKV_DEV_BAD_CONTEXT_LEN  # 40 tokens, 32 bits
    c.check()  # the device is as well as before
    assert m.tree_workspace_bytes(64) > 0


def test_refusals():
    m = pkv()
    c = Case([100, 64], [4, 5], D=64, dtype="f16")
    with pytest.raises(ValueError):
        c.call(tree_mask=torch.zeros((3, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        c.call(tree_mask=torch.zeros((9, 1), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.call(depths=torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        c.call(depths=torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError):
        c.call(slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        c.call(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        c.call(window=1 << 32)
    for kw in (dict(window=-1), dict(cap=-2.0), dict(cap=float("nan"))):
        with pytest.raises(m.PkvError):
            c.call(**kw)
    with pytest.raises(ValueError):
        m.paged_tree_attention(c.q, c.kc, c.vc, i32(c.tables), i32(c.lens), i32(c.starts), 0.1, c.q)
    with pytest.raises(TypeError):
        m.paged_tree_attention(c.q, c.kc, c.vc, i32(c.tables), i32(c.lens), i32(c.starts), 0.1,
                               c.q.float())
    with pytest.raises(ValueError):
        m.paged_tree_attention(c.q, c.kc, c.vc, i32(c.tables), i32(c.lens), i32(c.starts[:2]), 0.1,
                               torch.empty_like(c.q))
    empty = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    m.paged_tree_attention(empty, c.kc, c.vc, i32(c.tables), i32(c.lens), i32([0, 0, 0]), 0.1,
                           torch.empty_like(empty))


def test_the_same_bits_every_time_and_on_other_blocks():
    c = Case([3000, 700, 45], [12, 40, 3], Hkv=2, G=4, D=128, dtype="bf16")
    a = c.call().clone()
    for _ in range(3):
        assert torch.equal(c.call(), a)
    perm = torch.randperm(c.NB, device="cuda")
    kc, vc = torch.empty_like(c.kc), torch.empty_like(c.vc)
    kc[perm], vc[perm] = c.kc, c.vc
    where = np.append(perm.cpu().numpy(), [0] * 8)
    c.kc, c.vc, c.tables = kc, vc, where[np.minimum(c.tables, c.NB)]
    assert torch.equal(c.call(), a)


def test_streams_graphs_and_workspaces():
    """Two streams at once, a captured graph replayed beside eager calls, a workspace of the
    caller's own filled with anything."""
    m = pkv()
    cases = [Case([3000, 700], [12, 40], Hkv=2, G=4, D=128, dtype="bf16", seed=s) for s in range(2)]
    want = [c.call().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                c.out.fill_(7.0)
                c.call()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out[:c.T], w)
    c = cases[0]
    args = (c.q, c.kc, c.vc, i32(c.tables), i32(c.lens), i32(c.starts), c.scale, c.out[:c.T])
    kw = dict(tree_mask=i32(np.concatenate([osp.words(s, c.W) for s in c.seen])), depths=i32(c.depths))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.paged_tree_attention(*args, **kw)
        graphs.append(g)
    for g in graphs:
        c.out.fill_(7.0)
        cases[1].call()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out[:c.T], want[0])
    ws = torch.full((m.tree_workspace_bytes(128),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.call(workspace=ws), want[0])


def test_a_pool_past_2_to_the_31_elements():
    """Blocks whose elements lie past 32 bits."""
    NB, Hkv, B, D = 140000, 8, 16, 128
    kc = torch.zeros((NB, Hkv, B, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    c = Case([200, 90], [6, 9], Hkv=Hkv, G=8, D=D, dtype="bf16")
    far = NB - c.NB + np.arange(c.NB)
    kc[NB - c.NB:], vc[NB - c.NB:] = c.kc, c.vc
    want = c.call().clone()
    c.kc, c.vc, c.tables = kc, vc, np.append(far, [0] * 8)[np.minimum(c.tables, c.NB)]
    assert torch.equal(c.call(), want)
