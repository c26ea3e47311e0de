"""The operators together, as a decode loop uses them, against fp64 models of the loop.

* A budgeted loop: rotary write of every new token, attention with weights, eviction to
  the budget every few steps through the block manager, positions counted on from the
  original ones.  The model keeps the library's choice of tokens (compared with the
  oracle's choice from the library's own sums) and holds every K and V row in fp64.
* A beam search: beams forked from one prompt, rotary write with copy-on-write copies,
  attention, logits from the attention output, selection, reordering of the tables; the
  model keeps a whole K and V history for every beam and never shares anything.
"""
import numpy as np
import pytest
import torch

from oracle import beam as obeam
from oracle import eviction as oev
from oracle import rotary as orot

pytestmark = pytest.mark.gpu


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
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def attention(q, k, v, scale):
    """q [Hq, D], k and v [Hkv, t, D] -> [Hq, D]."""
    G = q.shape[0] // k.shape[0]
    out = np.zeros_like(q)
    for h in range(q.shape[0]):
        x = scale * (k[h // G] @ q[h])
        w = np.exp(x - x.max())
        out[h] = (w @ v[h // G]) / w.sum()
    return out


def row_error(got, want):
    return (np.abs(got - want).max(-1) / np.linalg.norm(want, axis=-1)).max()


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 2e-2)])
def test_budgeted_decode_loop(dtype, tol):
    # tolerance: the model turns and stores exact values; a stored bf16 row is off by 2^-8
    # of its elements (K and V) and q likewise, scores by a few 2^-8 of their size
    m = pkv()
    Hq, Hkv, D, B, NB, MAXB, S = 8, 2, 64, 16, 64, 8, 3
    budget, first, recent = 40, 4, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    alloc = m.BlockAllocator(NB, B, np.random.default_rng(1).permutation(NB).astype(np.int32))
    kc, vc = torch.zeros((NB, Hkv, B, D), dtype=dtype, device="cuda"), None
    vc = torch.zeros_like(kc)
    freq = m.rotary_frequencies(D)
    table = m.rotary_table(512, freq)
    scale = D ** -0.5
    seqs = [alloc.create() for _ in range(S)]
    prompts = [37, 5, 64]
    sums = torch.zeros((S, Hkv, MAXB * B), device="cuda")
    hist = [[np.zeros((Hkv, 0, D)), np.zeros((Hkv, 0, D))] for _ in range(S)]

    def write(tokens, pos, slots, owner):
        q, k, v = rnd(tokens, Hq, D), rnd(tokens, Hkv, D), rnd(tokens, Hkv, D)
        q0, k0, v0 = np64(q), np64(k), np64(v)
        m.paged_rotary_write(q, k, v, i32(pos), table, i32(slots), kc, vc, q)
        kt = orot.rotate(k0, pos, freq.numpy())
        for i, s in enumerate(owner):
            hist[s] = [np.concatenate([h, x[i][:, None]], 1) for h, x in zip(hist[s], (kt, v0))]
        return q, orot.rotate(q0, pos, freq.numpy())

    pos = np.zeros(S, dtype=np.int64)
    for s in range(S):
        slots, _ = alloc.append(seqs[s], prompts[s])
        write(prompts[s], np.arange(prompts[s]), slots, [s] * prompts[s])
        pos[s] = prompts[s]
    evictions = 0
    for step in range(30):
        slots, cows = alloc.append_one_each(seqs)
        assert not cows
        q, q64 = write(S, pos, slots, range(S))
        pos += 1
        tables, ctx = alloc.export_tables(seqs, MAXB)
        out = torch.empty_like(q)
        before = sums.clone()
        m.paged_decode_attention_weights(q, kc, vc, i32(tables), i32(ctx), scale, out, sums)
        got = np64(out)
        added = np64(sums) - np64(before)
        for s in range(S):
            assert hist[s][0].shape[1] == ctx[s]
            assert row_error(got[s], attention(q64[s], *hist[s], scale)) < tol
            w = oev.attention_weights(q64[s], hist[s][0], scale)
            assert np.abs(added[s, :, :ctx[s]] - w).max() < tol
        if step % 7 != 6:
            continue
        # cut every sequence down to the budget; its rows move into fresh blocks
        kept = torch.zeros((S, Hkv, budget), dtype=torch.int32, device="cuda")
        new_sums = torch.zeros_like(sums)
        new_lens = i32(np.zeros(S))
        m.paged_evict_select(sums, i32(ctx), i32([budget] * S), kept, new_sums, new_lens,
                             first=first, recent=recent)
        new = alloc.evict(seqs, [budget] * S, -(-budget // B))
        m.paged_evict_gather(kc, vc, i32(tables), kept, new_lens, i32(new))
        x, k = np64(sums), kept.cpu().numpy()
        for s in range(S):
            n = min(budget, int(ctx[s]))
            assert int(new_lens[s]) == n == alloc.length(seqs[s])
            evictions += n < ctx[s]
            rows = [oev.select(x[s, h], int(ctx[s]), budget, first, recent) for h in range(Hkv)]
            for h in range(Hkv):
                assert np.array_equal(k[s, h, :n], rows[h])
            hist[s] = [np.stack([c[h][rows[h]] for h in range(Hkv)]) for c in hist[s]]
        sums = new_sums
    assert evictions >= 6


def test_beam_search_over_the_paged_cache():
    m = pkv()
    dtype = torch.float32
    Hq, Hkv, D, B, NB, MAXB, K, V = 4, 2, 64, 16, 64, 8, 4, 700
    R = 2  # requests
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    emb, head = rnd(V, Hq + 2 * Hkv, D), rnd(Hq * D, V) * 0.2
    emb64, head64 = np64(emb), np64(head)
    freq = m.rotary_frequencies(D, scaling="linear", factor=2.0)
    table = m.rotary_table(256, freq)
    scale = D ** -0.5
    alloc = m.BlockAllocator(NB, B)
    kc = torch.zeros((NB, Hkv, B, D), dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    prompts = [np.random.default_rng(r).integers(0, V, n) for r, n in enumerate((21, 16))]

    def rows64(tokens, pos):
        e = emb64[tokens]
        turn = lambda x: orot.rotate(x, pos, freq.numpy())  # noqa: E731
        return turn(e[:, :Hq]), turn(e[:, Hq:Hq + Hkv]), e[:, Hq + Hkv:]

    def write(tokens, pos, slots):
        x = emb[torch.from_numpy(np.asarray(tokens)).cuda()]
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]  # slices of one projection
        out = torch.empty((len(tokens), Hq, D), device="cuda")
        return m.paged_rotary_write(q, k, v, i32(pos), table, i32(slots), kc, vc, out)

    beams = []
    hist = []
    for p in prompts:
        s = alloc.create()
        slots, _ = alloc.append(s, len(p) - 1)
        write(p[:-1], np.arange(len(p) - 1), slots)
        beams.append([s] + [alloc.fork(s) for _ in range(K - 1)])
        _, k, v = rows64(p[:-1], np.arange(len(p) - 1))
        hist.append([(k, v, [])] * K)
    seqs = [s for b in beams for s in b]
    tokens = np.repeat([p[-1] for p in prompts], K)
    pos = np.repeat([len(p) - 1 for p in prompts], K)
    bs = torch.full((R, K), -float("inf"), device="cuda")
    bs[:, 0] = 0.0
    scores = torch.empty_like(bs)
    who, what = (torch.empty((R, K), dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(20):
        slots, cows = alloc.append_one_each(seqs)
        if cows:
            m.paged_copy_blocks(kc, vc, i32(cows))
        q = write(tokens, pos, slots)
        tables, ctx = alloc.export_tables(seqs, MAXB)
        out = torch.empty_like(q)
        m.paged_decode_attention(q, kc, vc, i32(tables), i32(ctx), scale, out)
        logits = (out.view(R * K, -1) @ head).view(R, K, V)
        m.beam_select(logits, bs, scores, who, what)
        # the model: every beam's own history, the selection of the library's logits
        q64, k64, v64 = rows64(tokens, pos)
        w_h, t_h = who.cpu().numpy(), what.cpu().numpy()
        for r in range(R):
            grown = []
            for b in range(K):
                k, v, toks = hist[r][b]
                i = r * K + b
                k, v = np.concatenate([k, k64[i:i + 1]]), np.concatenate([v, v64[i:i + 1]])
                grown.append((k, v, toks + [int(tokens[i])]))
                a = attention(q64[i], k.transpose(1, 0, 2), v.transpose(1, 0, 2), scale)
                assert row_error(np64(out[i]), a) < 1e-4
            ws, wb, wt = obeam.select(np64(logits[r]), bs[r].cpu().numpy(), K)
            assert np.allclose(np64(scores[r]), ws, rtol=0, atol=1e-4)
            assert np.array_equal(w_h[r], wb) and np.array_equal(t_h[r], wt)
            hist[r] = [grown[b] for b in w_h[r]]
        for r in range(R):
            alloc.reorder(beams[r], w_h[r].tolist())
        tokens, pos = t_h.reshape(-1).astype(np.int64), pos + 1
        bs.copy_(scores)
    for r in range(R):
        for s in beams[r]:
            assert alloc.length(s) == len(prompts[r]) - 1 + 20
            alloc.free(s)
    assert alloc.num_free() == NB
