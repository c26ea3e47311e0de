"""Host side of the speculative step (no GPU): the oracle against the decode oracle along a
tree's paths, trees' masks, sequences cut down, and every refusal."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_166_gb300 as pkv
from oracle import paged_attention
from oracle import rotary as orot
from oracle import speculative as osp
from oracle.block_manager import BlockManager, InvalidOperation
from paged_kv_cache_166_gb300 import _native as N

P = 1 << 20  # an aligned address that no refused call reads


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def random_parents(rng, c):
    return np.array([rng.integers(-1, i) if i else -1 for i in range(c)], dtype=np.int32)


def test_a_tree_is_decode_along_each_path():
    """The drafted tokens that a token sees are a chain: attention over the context and that
    chain alone, laid out as a cache of its own, is the same."""
    rng = np.random.default_rng(0)
    Hq, Hkv, D, B, base, c = 4, 2, 8, 4, 6, 7
    parents = random_parents(rng, c)
    seen, depth = osp.tree_masks(parents)
    kc, vc = rng.standard_normal((2, 8, Hkv, B, D))
    table = rng.permutation(8)[None, :4]
    q = rng.standard_normal((c, Hq, D))
    out, _, _ = osp.tree_attention(q, kc, vc, table, [base + c], [0, c], 0.3, [seen], depth)
    for i in range(c):
        keys = list(range(base)) + [base + j for j in range(c) if seen[i, j]]
        assert len(keys) == base + depth[i] + 1
        k2, v2 = np.zeros((2, 4, Hkv, B, D))
        for n, p in enumerate(keys):
            k2[n // B, :, n % B] = kc[table[0, p // B], :, p % B]
            v2[n // B, :, n % B] = vc[table[0, p // B], :, p % B]
        want = paged_attention.paged_attention(q[i:i + 1], k2, v2, np.arange(4)[None], [len(keys)], 0.3)
        assert np.allclose(out[i], want[0], rtol=0, atol=1e-12)


def test_cap_bias_and_window_on_a_case_by_hand():
    kc = np.zeros((1, 1, 4, 2))
    kc[0, 0, :, 0] = [1, 2, 3, 4]
    vc = np.zeros((1, 1, 4, 2))
    vc[0, 0, :, 0] = [1, 10, 100, 1000]
    q = np.array([[[2.0, 0.0]]])
    out, _, _ = osp.tree_attention(q, kc, vc, [[0]], [4], [0, 1], 0.5, None, None, cap=3.0,
                                   slopes=[0.25], window=3)
    x = 3 * np.tanh(np.array([2, 3, 4]) / 3) + 0.25 * np.array([-2, -1, 0])
    w = np.exp(x) / np.exp(x).sum()
    assert np.allclose(out[0, 0], [w @ [10, 100, 1000], 0], atol=1e-9)
    hidden, _, _ = osp.tree_attention(q, kc, vc, [[0]], [4], [0, 1], 0.5, [np.zeros((1, 1), bool)],
                                      None, window=1)
    assert (hidden == 0).all()  # nothing seen


def test_norm_rotate_without_norm_is_the_rotation():
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((5, 3, 16)), rng.integers(0, 99, 5), orot.frequencies(8)
    for inter in (False, True):
        one = osp.norm_rotate(x, None, None, pos[None], [0] * 4, f, inter)
        assert np.allclose(one, orot.rotate(x, pos, f, inter))
    y = osp.norm_rotate(x, np.full(16, 2.0), 0.0, pos[None], [0] * 4, f)
    assert np.allclose((y * y).mean(-1), 4.0)  # a turn keeps the length


@pytest.mark.parametrize("counts", [[1], [0, 5, 0], [33, 1, 64], [3, 100]])
def test_tree_masks_against_the_oracle(counts):
    rng = np.random.default_rng(2)
    trees = [random_parents(rng, c) for c in counts]
    starts = np.concatenate([[0], np.cumsum(counts)])
    mask, depths = pkv.tree_masks(i32(np.concatenate(trees)), i32(starts))
    W = max(1, -(-max(counts) // 32))
    assert mask.shape == (sum(counts), W)
    for t, a, b in zip(trees, starts, starts[1:]):
        seen, depth = osp.tree_masks(t)
        assert np.array_equal(mask[a:b].numpy(), osp.words(seen, W))
        assert np.array_equal(depths[a:b].numpy(), depth)
    wider, _ = pkv.tree_masks(i32(np.concatenate(trees)), i32(starts), words=W + 2)
    assert np.array_equal(wider[:, :W], mask) and not wider[:, W:].any()


def test_tree_masks_refusals():
    ok = i32([0, 2])
    for parents in ([0, 0], [-1, 1], [-2, 0], [-1, 5]):
        with pytest.raises(pkv.PkvError):
            pkv.tree_masks(i32(parents), ok)
    with pytest.raises(pkv.PkvError):
        pkv.tree_masks(i32([-1] * 40), i32([0, 40]), words=1)
    with pytest.raises(ValueError):
        pkv.tree_masks(i32([-1, 0]), i32([0, 1]))
    with pytest.raises(ValueError):
        pkv.tree_masks(i32([-1, 0]), i32([1, 2]))
    with pytest.raises(TypeError):
        pkv.tree_masks(torch.tensor([-1, 0]), ok)
    with pytest.raises(pkv.PkvError):
        pkv.tree_masks(i32([-1, 0]), i32([0, 3, 2]))
    m, d = pkv.tree_masks(i32([]), i32([0, 0]))
    assert m.shape == (0, 1) and d.shape == (0,)


def test_truncate_against_the_oracle():
    rng = np.random.default_rng(3)
    for trial in range(40):
        B = int(rng.choice([1, 4, 16]))
        a, o = pkv.BlockAllocator(40, B), BlockManager(40, B)
        seqs = []
        for _ in range(60):
            op = rng.integers(0, 5)
            if op == 0 or not seqs:
                seqs.append((a.create(), o.create()))
            elif op == 1:
                x, y = seqs[rng.integers(len(seqs))]
                seqs.append((a.fork(x), o.fork(y)))
            elif op == 2:
                x, y = seqs[rng.integers(len(seqs))]
                n = int(rng.integers(0, 2 * B + 2))
                if o.blocks_needed(y, n) <= o.num_free():
                    s1, c1 = a.append(x, n)
                    s2, c2 = o.append(y, n)
                    assert list(s1) == s2 and [tuple(c) for c in c1] == c2
            else:
                pick = rng.permutation(len(seqs))[:rng.integers(1, 4)]
                ids = [seqs[i] for i in pick]
                lens = [int(rng.integers(0, o.lengths[y] + 1)) for _, y in ids]
                a.truncate([x for x, _ in ids], lens)
                o.truncate([y for _, y in ids], lens)
            for x, y in seqs:
                assert a.length(x) == o.lengths[y] and a.table(x) == o.tables[y]
            assert a.num_free() == o.num_free()


def test_truncate_refusals_change_nothing():
    a = pkv.BlockAllocator(8, 4)
    s, t = a.create(), a.create()
    a.append(s, 9)
    a.append(t, 5)
    before = a.table(s), a.table(t), a.num_free()
    for seqs, lens in (([s, t], [3, 6]), ([s, s], [3, 3]), ([s], [-1]), ([s, 7], [1, 1])):
        with pytest.raises(pkv.PkvError):
            a.truncate(seqs, lens)
        assert (a.table(s), a.table(t), a.num_free()) == before
    with pytest.raises(ValueError):
        a.truncate([s], [1, 2])
    a.truncate([], [])
    a.truncate([s, t], [9, 0])
    assert a.length(s) == 9 and a.table(t) == []
    a.swap_out(s)
    with pytest.raises(pkv.PkvError):
        a.truncate([s], [2])
    o = BlockManager(8, 4)
    with pytest.raises(InvalidOperation):
        o.truncate([o.create()], [1])


def refused(fn, base, cases):
    for kw, code in cases:
        assert set(kw) <= set(base), kw
        assert fn(*{**base, **kw}.values()) == code, kw


A, D_, U = N.PKV_ERR_INVALID_ARG, N.PKV_ERR_DTYPE, N.PKV_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def test_tree_attention_refusals():
    base = dict(q=P, kc=P, vc=P, bt=P, maxb=4, ctx=P, qs=P, mask=P, words=1, depths=P, slopes=P,
                cap=0.0, window=0, S=2, T=4, Hq=8, Hkv=2, D=128, B=16, NB=8, scale=0.1, out=P,
                status=P, ws=P, wsb=1 << 30, dt=N.PKV_BF16, stream=None)
    refused(N.lib().pkv_tree_attention, base, [
        (dict(dt=N.PKV_F32), D_), (dict(dt=N.PKV_FP8_E4M3), D_), (dict(dt=9), D_),
        (dict(S=-1), U), (dict(S=2049), U), (dict(Hq=7), A), (dict(Hq=0), A), (dict(Hkv=0), A),
        (dict(Hq=34), U), (dict(D=96), U), (dict(D=32), U), (dict(B=4), U), (dict(B=12), U),
        (dict(maxb=0), A), (dict(NB=0), A), (dict(maxb=1 << 27), U), (dict(NB=1 << 27), U),
        (dict(T=-1), A), (dict(T=1 << 30), U), (dict(scale=NAN), A), (dict(scale=INF), A),
        (dict(cap=-1.0), A), (dict(cap=NAN), A), (dict(cap=INF), A), (dict(window=-1), A),
        (dict(words=0), A), (dict(words=-3), A),
        (dict(q=None), A), (dict(kc=None), A), (dict(vc=None), A), (dict(bt=None), A),
        (dict(ctx=None), A), (dict(qs=None), A), (dict(out=None), A), (dict(ws=None), A),
        (dict(q=P + 8), A), (dict(kc=P + 8), A), (dict(out=P + 2), A), (dict(mask=P + 2), A),
        (dict(depths=P + 1), A), (dict(slopes=P + 2), A), (dict(status=P + 2), A),
        (dict(ws=P + 128), A)])
    for kw in (dict(S=0), dict(T=0)):  # nothing to do, and nothing looked at
        assert N.lib().pkv_tree_attention(*{**base, **kw, "q": None}.values()) == N.PKV_OK
    n = ctypes.c_size_t()
    assert N.lib().pkv_tree_workspace_size(96, ctypes.byref(n)) == U
    assert N.lib().pkv_tree_workspace_size(128, None) == A


def test_norm_rotary_refusals():
    ax = (ctypes.c_int32 * 64)(*([0, 1] * 32))
    bad = (ctypes.c_int32 * 64)(*([0, 2] * 32))
    base = dict(codes=0, q=P, qst=1024, k=P, kst=256, v=P, vst=256, qw=P, kw=P, wdt=N.PKV_BF16,
                per_head=0, eps=1e-6, pos=P, axes=ax, A=2, table=P, maxp=100, rot=128, inter=0,
                slots=P, T=3, kc=P, vc=P, ks=None, vs=None, NB=8, Hq=8, Hkv=2, B=16, D=128, qo=P,
                qost=1024, status=P, dt=N.PKV_BF16, stream=None)
    refused(N.lib().pkv_norm_rotary_write, base, [
        (dict(codes=7), D_), (dict(dt=5), D_), (dict(wdt=N.PKV_F16), D_), (dict(wdt=7), D_),
        (dict(eps=NAN), A), (dict(eps=INF), A), (dict(eps=-1.0), A), (dict(A=0), U), (dict(A=5), U),
        (dict(axes=None), A), (dict(axes=bad), A), (dict(qw=P + 1), A), (dict(kw=P + 1), A),
        (dict(rot=0), A), (dict(rot=3), A), (dict(rot=130), A), (dict(D=320, rot=64), U),
        (dict(T=-1), A), (dict(NB=0), A), (dict(maxp=0), A), (dict(qst=1000), A), (dict(kst=100), A),
        (dict(vst=0), A), (dict(qost=8), A), (dict(q=None), A), (dict(pos=None), A),
        (dict(slots=None), A), (dict(table=P + 4), A), (dict(kc=P + 8), A), (dict(status=P + 1), A),
        (dict(codes=N.PKV_INT8), A), (dict(codes=N.PKV_FP8_E4M3, B=8), U),
        (dict(inter=1, q=P + 2), A), (dict(D=12, rot=4), A)])
    none = dict(base, T=0, q=None, k=None)
    assert N.lib().pkv_norm_rotary_write(*none.values()) == N.PKV_OK


def test_commit_refusals():
    one, two = (ctypes.c_void_p * 2)(P, P + 64), (ctypes.c_void_p * 2)(P + 128, P + 192)
    same, other = (ctypes.c_void_p * 2)(P, P), (ctypes.c_void_p * 2)(P + 128, P)
    off = (ctypes.c_void_p * 2)(P, P + 8)
    gone = (ctypes.c_void_p * 2)(P, None)
    base = dict(kc=one, vc=two, L=2, bt=P, maxb=4, ctx=P, qs=P, path=P, cols=3, lens=P, S=2, NB=8,
                Hkv=2, B=16, D=128, status=P, dt=N.PKV_BF16, stream=None)
    refused(N.lib().pkv_tree_commit, base, [
        (dict(dt=9), D_), (dict(L=0), U), (dict(L=129), U), (dict(S=-1), A), (dict(cols=-1), A),
        (dict(maxb=0), A), (dict(NB=0), A), (dict(Hkv=0), A), (dict(B=0), A), (dict(D=0), A),
        (dict(dt=N.PKV_INT8, B=8), U), (dict(D=4), A), (dict(D=8192), A), (dict(Hkv=70000), U),
        (dict(maxb=1 << 28), U), (dict(NB=1 << 28), U), (dict(kc=None), A), (dict(vc=None), A),
        (dict(kc=off), A), (dict(vc=off), A), (dict(kc=gone), A), (dict(bt=None), A),
        (dict(kc=same), A), (dict(vc=same), A), (dict(vc=other), A), (dict(vc=same, S=0), A),
        (dict(ctx=None), A), (dict(qs=None), A), (dict(path=None), A), (dict(lens=None), A),
        (dict(path=P + 2), A), (dict(status=P + 1), A)])
    for kw in (dict(S=0), dict(cols=0)):
        assert N.lib().pkv_tree_commit(*{**base, **kw, "bt": None}.values()) == N.PKV_OK


def test_adjust_refusals():
    base = dict(x=P, st=1000, out=P, ost=1000, T=4, V=1000, rows=P, S=2, hist=P, L=10, lens=P,
                prompts=P, rep=P, freq=P, pres=P, path=P, cols=3, bt=P, bv=P, bcols=4, ok=P,
                words=32, dt=N.PKV_BF16, stream=None)
    refused(N.lib().pkv_adjust_logits, base, [
        (dict(dt=3), D_), (dict(T=-1), A), (dict(S=-1), A), (dict(V=0), A), (dict(L=-1), A),
        (dict(cols=-1), A), (dict(bcols=-1), A), (dict(words=-1), A), (dict(words=31), A),
        (dict(V=(1 << 30) + 1), U), (dict(S=65536), U), (dict(L=1 << 24), U), (dict(cols=1 << 24), U),
        (dict(rows=None), A), (dict(st=999), A), (dict(ost=999), A), (dict(ost=1001), A),
        (dict(bt=None), A), (dict(bv=None), A), (dict(x=None), A), (dict(out=None), A),
        (dict(hist=None), A), (dict(lens=None), A), (dict(x=P + 1), A), (dict(hist=P + 2), A),
        (dict(rep=P + 1), A), (dict(ok=P + 2), A), (dict(path=P + 1), A)])
    for kw in (dict(T=0), dict(S=0)):
        assert N.lib().pkv_adjust_logits(*{**base, **kw, "x": None}.values()) == N.PKV_OK


def test_host_tensors_are_refused():
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_tree_attention(h(2, 4, 64), h(8, 4, 16, 64), h(8, 4, 16, 64), z(1, 2), z(1), z(2),
                                 0.1, h(2, 4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_norm_rotary_write(h(2, 4, 64), h(2, 4, 64), h(2, 4, 64), None, None, 1e-6, z(2),
                                    torch.zeros(9, 64), z(2), h(8, 4, 16, 64), h(8, 4, 16, 64),
                                    h(2, 4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_tree_commit([h(8, 4, 16, 64)], [h(8, 4, 16, 64)], z(1, 2), z(1), z(2), z(1, 2), z(1))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.adjust_logits(h(2, 50), z(2, 5), z(2))
