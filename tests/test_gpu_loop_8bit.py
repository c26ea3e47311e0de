"""The budgeted decode loop over fp8 and int8 caches: rotary write, attention with weights,
eviction through the block manager, step after step.

The model takes the library's turned q, its codes and its choice of tokens, each after
comparing them (q with the turned q, a code's value with the turned k or the v, the choice
with the oracle's from the library's own sums), and holds every row in fp64; after an
eviction the rows in the new blocks have to be the model's, bit for bit.

Tolerances.  q: half a step of f16 beside the fp32 arithmetic (2^-11 and 3 2^-24 (|x1| + |x2|)).
A code's value: half a step of E4M3 (2^-4 of the value, half of 2^-9 scales near zero), or half
a scale for int8, beside that arithmetic; the draws stay within the codes' range.  Weights: a
score is off by at most D 2^-23 scale sum |q k|, here below 6e-4, a weight by twice that, and a
group's four by 5e-3.  out: probabilities rounded to f16 and out itself (2^-11 each of values
of at most a few times the row's norm): 2e-2 of the norm.
"""
import numpy as np
import pytest
import torch

from oracle import eviction as oev
from oracle import fp8 as ofp8
from oracle import int8 as oint8
from oracle import rotary as orot
from test_gpu_loop import attention, i32, np64, pkv, row_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_budgeted_decode_loop_8bit(kind):
    m = pkv()
    Hq, Hkv, D, B, NB, MAXB, S = 8, 2, 128, 16, 64, 8, 3
    budget, first, recent = 40, 4, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    alloc = m.BlockAllocator(NB, B, np.random.default_rng(1).permutation(NB).astype(np.int32))
    ct = torch.uint8 if kind == "fp8" else torch.int8
    kc = torch.zeros((NB, Hkv, B, D), dtype=ct, device="cuda")
    vc = torch.zeros((NB, Hkv, D, B), dtype=ct, device="cuda")
    ks, vs = (torch.tensor(x, device="cuda") for x in ([0.06, 0.08], [0.07, 0.05]))
    ks_h, vs_h = ks.cpu().numpy(), vs.cpu().numpy()
    o, gather = (ofp8, ofp8.gather_fp8) if kind == "fp8" else (oint8, oint8.gather_int8)
    write_op = getattr(m, "paged_rotary_write_" + kind)
    weigh = getattr(m, "paged_decode_attention_weights_" + kind)
    freq = m.rotary_frequencies(D)
    table = m.rotary_table(512, freq)
    scale = D ** -0.5
    seqs = [alloc.create() for _ in range(S)]
    prompts = [37, 5, 64]
    sums = torch.zeros((S, Hkv, MAXB * B), device="cuda")
    hist = [[np.zeros((Hkv, 0, D)), np.zeros((Hkv, 0, D))] for _ in range(S)]

    def rows(table_row, t):
        """K and V [Hkv, t, D] of a sequence, as the cache holds them."""
        kv = [gather(kc.cpu().numpy(), vc.cpu().numpy(), ks_h, vs_h, table_row, t, h)
              for h in range(Hkv)]
        return np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv])

    def near(got, want, s):
        step = np.maximum(np.abs(want) * 2.0 ** -4, s * 2.0 ** -10) if kind == "fp8" else s / 2
        assert np.all(np.abs(got - want) <= step + 6 * 2.0 ** -24 * 8)

    def write(tokens, pos, slots, owner):
        q, k, v = rnd(tokens, Hq, D), rnd(tokens, Hkv, D), rnd(tokens, Hkv, D)
        q64 = orot.rotate(np64(q), pos, freq.numpy())
        k64, v64 = orot.rotate(np64(k), pos, freq.numpy()), np64(v)
        write_op(q, k, v, i32(pos), table, i32(slots), kc, vc, ks, vs, q)
        assert np.all(np.abs(np64(q) - q64) <= 2.0 ** -11 * np.abs(q64) + 2.0 ** -18)
        codes_k, codes_v = kc.cpu().numpy(), vc.cpu().numpy()
        for i, s in enumerate(owner):
            blk, off = divmod(int(slots[i]), B)
            kk = o.decode(codes_k[blk, :, off]) * ks_h[:, None].astype(np.float64)
            vv = o.decode(codes_v[blk, :, :, ofp8.V_POS[off]]) * vs_h[:, None].astype(np.float64)
            near(kk, k64[i], ks_h[:, None])
            near(vv, v64[i], vs_h[:, None])
            hist[s] = [np.concatenate([h, x[:, None]], 1) for h, x in zip(hist[s], (kk, vv))]
        return q

    pos = np.zeros(S, dtype=np.int64)
    for s in range(S):
        slots, _ = alloc.append(seqs[s], prompts[s])
        write(prompts[s], np.arange(prompts[s]), slots, [s] * prompts[s])
        pos[s] = prompts[s]
    evictions = 0
    for step in range(30):
        slots, cows = alloc.append_one_each(seqs)
        assert not cows
        q = write(S, pos, slots, range(S))
        pos += 1
        tables, ctx = alloc.export_tables(seqs, MAXB)
        out = torch.empty_like(q)
        before = sums.clone()
        weigh(q, kc, vc, ks, vs, i32(tables), i32(ctx), scale, out, sums)
        got, added = np64(out), np64(sums) - np64(before)
        for s in range(S):
            assert hist[s][0].shape[1] == ctx[s]
            assert row_error(got[s], attention(np64(q)[s], *hist[s], scale)) < 2e-2
            w = oev.attention_weights(np64(q)[s], hist[s][0], scale)
            assert np.abs(added[s, :, :ctx[s]] - w).max() < 5e-3
            assert not added[s, :, ctx[s]:].any()
        if step % 7 != 6:
            continue
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
            keep = [oev.select(x[s, h], int(ctx[s]), budget, first, recent) for h in range(Hkv)]
            for h in range(Hkv):
                assert np.array_equal(k[s, h, :n], keep[h])
            hist[s] = [np.stack([c[h][keep[h]] for h in range(Hkv)]) for c in hist[s]]
            for a, b in zip(rows(new[s], n), hist[s]):
                assert np.array_equal(a, b)
        sums = new_sums
    assert evictions >= 6
