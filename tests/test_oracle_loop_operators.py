"""Pins of the oracle's rotary, eviction and beam functions, the library's host side of them
(frequencies, the block manager's eviction and reordering) and the refusals of the new
entry points.  No GPU needed.

* Rotary: a hand-worked pair, invariance of q . k under a common shift of positions, the
  layouts as permutations of one another, the scalings' end points.
* Eviction: hand-worked rows with ties, NaN and both kept ends.
* Beam: hand-worked candidates, ties, dead beams.
* pkv_rotary_frequencies against the oracle; pkv_seq_evict and pkv_seq_reorder against
  the oracle's block manager on seeded random operations.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import beam as obeam
from oracle import eviction as oev
from oracle import paged_attention as opa
from oracle import rotary as orot
from oracle.block_manager import BlockManager, InvalidOperation, OutOfBlocks as OracleOOB

pkv = pytest.importorskip("paged_kv_cache_166_gb300")
from paged_kv_cache_166_gb300 import _native as N  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# --- rotary ------------------------------------------------------------------------
def test_rotary_of_a_hand_worked_pair():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1.0, 2.0, 3.0, 5.0]
    f = np.array([math.pi / 2])  # a quarter turn a position
    assert np.allclose(orot.rotate(x, [1], f, interleaved=True)[0, 0], [-2, 1, 3, 5])
    assert np.allclose(orot.rotate(x, [2], f, interleaved=False)[0, 0], [-1, -2, 3, 5])


def test_rotary_keeps_products_under_a_common_shift():
    g = np.random.default_rng(0)
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    f = orot.frequencies(12)
    dots = [float((orot.rotate(q, [p + 7], f) * orot.rotate(k, [p], f)).sum())
            for p in (0, 5, 1000)]
    assert np.ptp(dots) < 1e-11


def test_rotary_layouts_are_permutations():
    x = np.random.default_rng(1).standard_normal((3, 2, 10))
    f = orot.frequencies(8)
    perm = [0, 4, 1, 5, 2, 6, 3, 7, 8, 9]  # half layout -> interleaved
    a = orot.rotate(x, [3, 0, 9], f)[..., perm]
    assert np.allclose(a, orot.rotate(x[..., perm], [3, 0, 9], f, interleaved=True))


def test_rotary_scalings():
    plain = orot.frequencies(64)
    assert plain[0] == 1.0 and np.isclose(plain[-1], 10000.0 ** (-62 / 64))
    assert np.allclose(orot.frequencies(64, scaling="linear", factor=4.0), plain / 4)
    ntk = orot.frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], plain[-1] / 4)
    bands = orot.frequencies(64, scaling="bands", factor=8.0, original_length=4096)
    assert bands[0] == plain[0] and np.isclose(bands[-1], plain[-1] / 8)
    assert np.all(np.diff(bands) < 0)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands"])
@pytest.mark.parametrize("rot", [2, 32, 128, 256])
def test_library_frequencies(scaling, rot):
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, original_length=8192, low_turns=1.0,
              high_turns=4.0)
    got = pkv.rotary_frequencies(rot, **kw).numpy()
    want = orot.frequencies(rot, **kw)
    # two libm's pow and a few products: 8 units in the last place
    assert got.shape == want.shape and np.all(np.abs(got - want) <= 8 * 2.0 ** -52 * want)


def test_library_frequencies_refusals():
    lib = N.lib()
    out = (ctypes.c_double * 8)()
    bad = [(3, 10000.0, 0, 1.0, 0, 1.0, 4.0), (0, 10000.0, 0, 1.0, 0, 1.0, 4.0),
           (258, 10000.0, 0, 1.0, 0, 1.0, 4.0), (16, 1.0, 0, 1.0, 0, 1.0, 4.0),
           (16, float("nan"), 0, 1.0, 0, 1.0, 4.0), (16, 10000.0, 4, 1.0, 0, 1.0, 4.0),
           (16, 10000.0, 1, 0.5, 0, 1.0, 4.0), (16, 10000.0, 3, 2.0, 0, 1.0, 4.0),
           (16, 10000.0, 3, 2.0, 4096, 4.0, 4.0)]
    for a in bad:
        assert lib.pkv_rotary_frequencies(*a, out) == N.PKV_ERR_INVALID_ARG, a
    assert lib.pkv_rotary_frequencies(16, 10000.0, 0, 1.0, 0, 1.0, 4.0, None) == N.PKV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(16, scaling="other")


# --- eviction ----------------------------------------------------------------------
def test_select_of_hand_worked_rows():
    s = np.array([5.0, 1.0, 3.0, 3.0, np.nan, 3.0, 0.0, 9.0])
    assert oev.select(s, 8, 3).tolist() == [0, 2, 7]           # ties: the lower position
    assert oev.select(s, 8, 4, first=2, recent=1).tolist() == [0, 1, 2, 7]
    assert oev.select(s, 8, 2, first=2, recent=2).tolist() == [6, 7]  # the last come first
    assert oev.select(s, 8, 7).tolist() == [0, 1, 2, 3, 5, 6, 7]      # NaN goes first
    assert oev.select(s, 3, 9).tolist() == [0, 1, 2]
    assert oev.select(s, 0, 4).tolist() == [] and oev.select(s, 8, 0, 1, 1).tolist() == []


def test_attention_weights_agree_with_the_oracle_attention():
    g = np.random.default_rng(2)
    q, kc, vc = (g.standard_normal(s) for s in ((1, 4, 8), (3, 2, 16, 8), (3, 2, 16, 8)))
    table, t, scale = np.array([[2, 0, 1]]), 37, 0.25
    keys, vals = (np.stack([opa.gather_sequence(c, table[0], t, h) for h in range(2)])
                  for c in (kc, vc))
    w = oev.attention_weights(q[0], keys, scale)
    assert np.allclose(w.sum(-1), 2.0)  # two query heads a group, each of weight 1
    one = oev.attention_weights(q[0, :1], keys[:1], scale)
    out = opa.paged_attention(q, kc, vc, table, [t], scale)
    assert np.allclose(one[0] @ vals[0], out[0, 0])


def test_gather_moves_rows_and_nothing_else():
    kc, vc = (np.arange(4 * 4 * 2, dtype=np.float64).reshape(4, 1, 4, 2) + 100 * i for i in (0, 1))
    k0 = kc.copy()
    oev.gather(kc, vc, [0, 1], [1, 4, 6], [3], 0)
    assert np.array_equal(kc[3, 0, :3], k0[[0, 1, 1], 0, [1, 0, 2]])
    assert np.array_equal(kc[3, 0, 3], k0[3, 0, 3]) and np.array_equal(kc[:3], k0[:3])


# --- beam --------------------------------------------------------------------------
def test_beam_of_hand_worked_candidates():
    logits = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.6, 0.3]]))
    s, b, t = obeam.select(logits, np.log([0.4, 0.6]), 4)  # 0.36, 0.2, 0.18, 0.12
    assert np.allclose(np.exp(s), [0.36, 0.2, 0.18, 0.12])
    assert b.tolist() == [1, 0, 1, 0] and t.tolist() == [1, 0, 2, 1]


def test_beam_ties_and_dead_beams():
    s, b, t = obeam.select(np.zeros((2, 3)), [0.0, 0.0], 5)
    assert (b.tolist(), t.tolist()) == ([0, 0, 0, 1, 1], [0, 1, 2, 0, 1])
    s, b, t = obeam.select([[0.0, np.nan, 1.0], [9.0, 9.0, 9.0]], [0.0, -np.inf], 5)
    assert (b.tolist(), t.tolist()) == ([0, 0, 0, 1, 1], [2, 0, 1, 0, 1])
    assert np.isneginf(s[2:]).all() and np.isfinite(s[:2]).all()


# --- block manager -----------------------------------------------------------------
@pytest.mark.parametrize("seed", range(6))
def test_evict_and_reorder_bit_exact(seed):
    r = np.random.default_rng(300 + seed)
    B, nb = int(r.choice([1, 4, 16])), int(r.integers(24, 96))
    order = r.permutation(nb).astype(np.int32)
    c, o = pkv.BlockAllocator(nb, B, order), BlockManager(nb, B, order)
    live = []
    for _ in range(400):
        op = r.integers(0, 10)
        if op < 2 or len(live) < 2:
            live.append(c.create())
            assert o.create() == live[-1]
        elif op < 5:
            s, n = live[r.integers(len(live))], int(r.integers(0, 3 * B + 2))
            try:
                want = o.append(s, n)
            except OracleOOB:
                with pytest.raises(N.OutOfBlocks):
                    c.append(s, n)
            else:
                got = c.append(s, n)
                assert list(got[0]) == want[0] and got[1] == want[1]
        elif op < 6:
            parent = live[r.integers(len(live))]
            live.append(c.fork(parent))
            assert o.fork(parent) == live[-1]
        elif op < 7:
            s = live.pop(r.integers(len(live)))
            c.free(s), o.free(s)
        elif op < 8:
            seqs = [int(x) for x in r.permutation(live)[:int(r.integers(0, 4))]]
            lens = [int(x) for x in r.integers(0, 4 * B, len(seqs))]
            try:
                want = o.evict(seqs, lens)
            except OracleOOB:
                with pytest.raises(N.OutOfBlocks):
                    c.evict(seqs, lens, 4)
            else:
                got = c.evict(seqs, lens, 4)
                assert got.tolist() == [t + [0] * (4 - len(t)) for t in want]
        else:
            seqs = [int(x) for x in r.permutation(live)[:int(r.integers(0, len(live) + 1))]]
            parents = [int(x) for x in r.integers(0, max(1, len(seqs)), len(seqs))]
            c.reorder(seqs, parents), o.reorder(seqs, parents)
        assert c.num_free() == o.num_free()
        assert [c.refcount(b) for b in range(nb)] == o.refcount
        for s in live:
            assert c.table(s) == o.tables[s] and c.length(s) == o.lengths[s]


def test_evict_and_reorder_refusals_leave_the_state():
    a = pkv.BlockAllocator(6, 4)
    s, t = a.create(), a.create()
    a.append(s, 16)
    with pytest.raises(N.OutOfBlocks):
        a.evict([s], [12], 3)  # three fresh blocks beside the four held, two free
    assert a.length(s) == 16 and a.num_free() == 2
    for seqs, lens, mb in (([s], [-1], 4), ([99], [1], 4), ([s, s], [1, 1], 4), ([s], [8], 1)):
        with pytest.raises(N.PkvError):
            a.evict(seqs, lens, mb)
    with pytest.raises(ValueError):
        a.evict([s, t], [1], 4)
    assert N.lib().pkv_seq_evict(a._h, None, 1, None, 1, None) == N.PKV_ERR_INVALID_ARG
    assert a.evict([], [], 4).shape == (0, 4)
    for seqs, parents in (([s, s], [0, 0]), ([s, 7], [0, 0]), ([s, t], [0, 2]), ([s, t], [-1, 0])):
        with pytest.raises(N.PkvError):
            a.reorder(seqs, parents)
    with pytest.raises(ValueError):
        a.reorder([s, t], [0])
    assert a.length(s) == 16 and a.length(t) == 0 and a.num_free() == 2
    out = a.swap_out(s)
    with pytest.raises(N.PkvError):
        a.evict([s], [4], 4)
    with pytest.raises(N.PkvError):
        a.reorder([s], [0])
    assert len(out) == 4
    with pytest.raises(InvalidOperation):
        BlockManager(4, 4).reorder([0], [0])


def test_evict_takes_every_new_block_before_it_gives_any_back():
    """One gather moves all the rows: no new block is an old block of the list."""
    a = pkv.BlockAllocator(12, 4)
    seqs = [a.create() for _ in range(2)]
    for s in seqs:
        a.append(s, 16)
    old = {b for s in seqs for b in a.table(s)}
    new = a.evict(seqs, [8, 5], 2)
    assert not old & set(new.ravel().tolist()) and len(set(new.ravel().tolist())) == 4
    assert [a.length(s) for s in seqs] == [8, 5] and a.num_free() == 8


# --- refusals of the device entry points (checked before anything is launched) -------
P = 4096  # any 256-byte aligned address: a refused call reads nothing


def _rotary_args(**kw):
    a = dict(q=P, qs=1024, k=P, ks=256, v=P, vs=256, pos=P, table=P, maxp=64, rot=64, inter=0,
             slots=P, T=2, kc=P, vc=P, NB=4, Hq=8, Hkv=2, B=16, D=128, qo=P, qos=1024, st=None,
             dt=N.PKV_BF16, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), N.PKV_ERR_DTYPE), (dict(dt=N.PKV_INT8), N.PKV_ERR_DTYPE),
    (dict(T=-1), N.PKV_ERR_INVALID_ARG), (dict(NB=0), N.PKV_ERR_INVALID_ARG),
    (dict(rot=3), N.PKV_ERR_INVALID_ARG), (dict(rot=130), N.PKV_ERR_INVALID_ARG),
    (dict(rot=0), N.PKV_ERR_INVALID_ARG), (dict(maxp=0), N.PKV_ERR_INVALID_ARG),
    (dict(D=512, rot=64, qs=4096, ks=1024, vs=1024, qos=4096), N.PKV_ERR_UNSUPPORTED),
    (dict(Hq=65536, qs=1 << 23, qos=1 << 23), N.PKV_ERR_UNSUPPORTED),
    (dict(Hkv=1 << 24, ks=1 << 31, vs=1 << 31), N.PKV_ERR_UNSUPPORTED),
    (dict(D=4, rot=4), N.PKV_ERR_INVALID_ARG), (dict(qs=1023), N.PKV_ERR_INVALID_ARG),
    (dict(vs=8), N.PKV_ERR_INVALID_ARG), (dict(qos=0), N.PKV_ERR_INVALID_ARG),
    (dict(q=None), N.PKV_ERR_INVALID_ARG), (dict(table=None), N.PKV_ERR_INVALID_ARG),
    (dict(kc=P + 8), N.PKV_ERR_INVALID_ARG), (dict(q=P + 1), N.PKV_ERR_INVALID_ARG),
    (dict(table=P + 4), N.PKV_ERR_INVALID_ARG), (dict(st=P + 2), N.PKV_ERR_INVALID_ARG),
    (dict(inter=1, q=P + 2), N.PKV_ERR_INVALID_ARG),
    (dict(inter=1, ks=257), N.PKV_ERR_INVALID_ARG),
    (dict(NB=1 << 28), N.PKV_ERR_INVALID_ARG)])
def test_rotary_write_refusals(kw, code):
    assert N.lib().pkv_rotary_write(*_rotary_args(**kw)) == code
    assert N.lib().pkv_last_error_string()


def test_rotary_write_8bit_refusals_and_empty_call():
    a = _rotary_args()
    scaled = a[:15] + [P, P] + a[15:]
    small = list(scaled)
    small[20] = 32  # block_size
    for fn in (N.lib().pkv_rotary_write_fp8, N.lib().pkv_rotary_write_int8):
        assert fn(*small) == N.PKV_ERR_UNSUPPORTED
        assert fn(*(a[:15] + [None, P] + a[15:])) == N.PKV_ERR_INVALID_ARG
    assert N.lib().pkv_rotary_write(*_rotary_args(T=0, q=None)) == N.PKV_OK


def test_weights_refusals():
    lib = N.lib()

    def args(**kw):
        a = dict(q=P, kc=P, vc=P, bt=P, maxb=4, ctx=P, S=2, Hq=8, Hkv=2, D=128, B=16, NB=8,
                 scale=0.1, out=P, sums=P, cols=64, ws=P, wsb=1 << 30, warps=8, dt=N.PKV_BF16,
                 stream=None)
        a.update(kw)
        return list(a.values())
    n = ctypes.c_size_t()
    assert lib.pkv_decode_weights_workspace_size(2, 4, 16, 8, 2, 128, N.PKV_BF16, 8,
                                                 ctypes.byref(n)) == N.PKV_OK
    base = ctypes.c_size_t()
    lib.pkv_decode_workspace_size(8, 2, 128, N.PKV_BF16, 8, ctypes.byref(base))
    # the decode workspace, 3 schedule words, 2 x 8 lse, 2 x 8 x 64 scores
    assert n.value == base.value + 256 + 256 + 2 * 8 * 64 * 4
    for kw, code in ((dict(wsb=n.value - 1), N.PKV_ERR_INVALID_ARG),
                     (dict(cols=0), N.PKV_ERR_INVALID_ARG),
                     (dict(sums=None), N.PKV_ERR_INVALID_ARG),
                     (dict(sums=P + 2), N.PKV_ERR_INVALID_ARG), (dict(Hq=6), N.PKV_ERR_UNSUPPORTED),
                     (dict(D=96), N.PKV_ERR_UNSUPPORTED), (dict(dt=N.PKV_FP8_E4M3), N.PKV_ERR_DTYPE),
                     (dict(S=4096), N.PKV_ERR_UNSUPPORTED), (dict(ws=P + 8), N.PKV_ERR_INVALID_ARG)):
        assert lib.pkv_decode_attention_weights(*args(**kw)) == code, kw
    assert lib.pkv_decode_weights_workspace_size(2, 0, 16, 8, 2, 128, N.PKV_BF16, 8,
                                                 ctypes.byref(n)) == N.PKV_ERR_INVALID_ARG


def test_evict_refusals():
    lib = N.lib()

    def sel(**kw):
        a = dict(sums=P, cols=64, ctx=P, keep=P, S=2, H=2, first=0, recent=0, kept=P, kc=8,
                 new=P + 256, nc=8, lens=P + 512, st=None, stream=None)
        a.update(kw)
        return list(a.values())
    for kw in (dict(S=-1), dict(H=0), dict(cols=0), dict(kc=0), dict(nc=0), dict(first=-1),
               dict(recent=-1), dict(sums=None), dict(new=P), dict(lens=P), dict(kept=P + 2)):
        assert lib.pkv_evict_select(*sel(**kw)) == N.PKV_ERR_INVALID_ARG, kw
    assert lib.pkv_evict_select(*sel(S=1 << 20, H=1 << 10)) == N.PKV_ERR_UNSUPPORTED
    for kw in (dict(cols=(1 << 30) + 1), dict(kc=(1 << 31) - 1), dict(nc=(1 << 31) - 1)):
        assert lib.pkv_evict_select(*sel(**kw)) == N.PKV_ERR_UNSUPPORTED, kw
    assert lib.pkv_evict_select(*sel(S=0, sums=None)) == N.PKV_OK

    def gat(**kw):
        a = dict(kc=P, vc=P, bt=P, maxb=4, kept=P, cols=8, lens=P, nt=P + 256, newb=1, S=2, NB=8,
                 H=2, B=16, D=128, st=None, dt=N.PKV_BF16, stream=None)
        a.update(kw)
        return list(a.values())
    for kw, code in ((dict(dt=7), N.PKV_ERR_DTYPE), (dict(D=4), N.PKV_ERR_INVALID_ARG),
                     (dict(D=4096), N.PKV_ERR_INVALID_ARG), (dict(S=70000), N.PKV_ERR_UNSUPPORTED),
                     (dict(nt=P), N.PKV_ERR_INVALID_ARG), (dict(kc=P + 4), N.PKV_ERR_INVALID_ARG),
                     (dict(newb=0), N.PKV_ERR_INVALID_ARG), (dict(lens=None), N.PKV_ERR_INVALID_ARG),
                     (dict(dt=N.PKV_INT8, B=8), N.PKV_ERR_UNSUPPORTED),
                     (dict(cols=(1 << 31) - 1), N.PKV_ERR_UNSUPPORTED),
                     (dict(maxb=1 << 28), N.PKV_ERR_INVALID_ARG)):
        assert lib.pkv_evict_gather(*gat(**kw)) == code, kw


def test_beam_refusals():
    lib = N.lib()

    def args(**kw):
        a = dict(logits=P, ss=400, bs=100, scores_in=P, S=2, K=4, V=100, N=8, scores=P + 256,
                 beams=P + 512, tokens=P + 768, ws=P, wsb=1 << 30, dt=N.PKV_F32, stream=None)
        a.update(kw)
        return list(a.values())
    for kw, code in ((dict(dt=N.PKV_INT8), N.PKV_ERR_DTYPE), (dict(S=-1), N.PKV_ERR_INVALID_ARG),
                     (dict(K=0), N.PKV_ERR_INVALID_ARG), (dict(V=0), N.PKV_ERR_INVALID_ARG),
                     (dict(N=0), N.PKV_ERR_INVALID_ARG), (dict(K=65), N.PKV_ERR_UNSUPPORTED),
                     (dict(N=129), N.PKV_ERR_UNSUPPORTED), (dict(V=1, N=5), N.PKV_ERR_INVALID_ARG),
                     (dict(S=20000), N.PKV_ERR_UNSUPPORTED),
                     (dict(V=(1 << 31) - 8192), N.PKV_ERR_UNSUPPORTED),
                     (dict(ss=-1), N.PKV_ERR_INVALID_ARG), (dict(bs=-4), N.PKV_ERR_INVALID_ARG),
                     (dict(logits=None), N.PKV_ERR_INVALID_ARG),
                     (dict(logits=P + 2), N.PKV_ERR_INVALID_ARG),
                     (dict(tokens=P + 2), N.PKV_ERR_INVALID_ARG),
                     (dict(scores=P), N.PKV_ERR_INVALID_ARG),
                     (dict(beams=P + 768), N.PKV_ERR_INVALID_ARG),
                     (dict(ws=None), N.PKV_ERR_INVALID_ARG),
                     (dict(ws=P + 128), N.PKV_ERR_INVALID_ARG)):
        assert lib.pkv_beam_select(*args(**kw)) == code, kw
    assert lib.pkv_beam_select(*args(S=0, logits=None)) == N.PKV_OK
    n = ctypes.c_size_t()
    assert lib.pkv_beam_workspace_size(1, 65, 100, 4, N.PKV_F32, ctypes.byref(n)) \
        == N.PKV_ERR_UNSUPPORTED
    assert lib.pkv_beam_workspace_size(1, 4, 100, 4, N.PKV_F32, None) == N.PKV_ERR_INVALID_ARG


def test_python_refusals_of_host_tensors():
    z = torch.zeros
    i32 = torch.int32
    q, kv = z(2, 4, 64), z(2, 2, 64)
    cache = z(4, 2, 16, 64)
    calls = [
        lambda: pkv.paged_rotary_write(q, kv, kv, z(2, dtype=i32), z(8, 64), z(2, dtype=i32),
                                       cache, cache, q),
        lambda: pkv.paged_decode_attention_weights(q, cache, cache, z(2, 2, dtype=i32),
                                                   z(2, dtype=i32), 0.1, q, z(2, 2, 32)),
        lambda: pkv.paged_evict_select(z(2, 2, 32), z(2, dtype=i32), z(2, dtype=i32),
                                       z(2, 2, 8, dtype=i32), z(2, 2, 8), z(2, dtype=i32)),
        lambda: pkv.paged_evict_gather(cache, cache, z(2, 2, dtype=i32), z(2, 2, 8, dtype=i32),
                                       z(2, dtype=i32), z(2, 1, dtype=i32)),
        lambda: pkv.beam_select(z(1, 2, 10), z(1, 2), z(1, 2), z(1, 2, dtype=i32),
                                z(1, 2, dtype=i32)),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
