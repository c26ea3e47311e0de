"""GPU parity of the attention weights and of eviction by them.

Weights: out carries the bits of pkv_decode_attention; the sums are held to the fp64
weights within a bound of the fp32 arithmetic.  A score is a sum of head_dim exact
products accumulated in fp32 (at most 2^-23 of the running magnitudes a step: the tensor
cores truncate), so it is off by A = D 2^-23 scale sum|q k| at most; the log-sum-exp by A
and by its own sum (at most (t / 16 + 64) roundings); a weight is its exponential.
Eviction is exact: positions, sums and rows are compared for equality.
"""

import numpy as np
import pytest
import torch

import batches as BT
from oracle import eviction as oev
from oracle import fp8 as ofp8
from oracle import int8 as oint8
from oracle import paged_attention as opa
from paged_kv_cache_166_gb300 import workloads as W

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
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


# --- weights -------------------------------------------------------------------------
def batch(Hq, Hkv, D, dtype, lens, B=16, seed=3, kind="", **kw):
    """A decode batch; kind "fp8"/"int8": its caches as codes with scales too."""
    w = W.Workload(name="t", seed=seed, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                   dtype=dtype, block_size=B)
    b = BT.decode_batch(w, np.asarray(lens), **kw)
    if kind:
        fill = W.fill_fp8_codes_ if kind == "fp8" else W.fill_int8_codes_
        sc = W.fp8_scales if kind == "fp8" else W.int8_scales
        ct = torch.uint8 if kind == "fp8" else torch.int8
        b.ks_h, b.vs_h = sc(Hkv, seed), sc(Hkv, seed + 1)
        b.ks, b.vs = (torch.from_numpy(x).cuda() for x in (b.ks_h, b.vs_h))
        b.kc = fill(torch.empty((b.NB, Hkv, 16, D), dtype=ct, device="cuda"), b.ks_h, seed, 21)
        b.vc = fill(torch.empty((b.NB, Hkv, D, 16), dtype=ct, device="cuda"), b.vs_h, seed, 22)
    b.kind = kind
    return b


def attend(b, sums=None, num_warps=0, **kw):
    tables, ctx, _ = b.device_index("cuda")
    out = torch.full_like(b.q, float("nan"))
    m = pkv()
    sc = (b.ks, b.vs) if b.kind else ()
    tail = "_" + b.kind if b.kind else ""
    if sums is None:
        fn = getattr(m, "paged_decode_attention" + tail)
        return fn(b.q, b.kc, b.vc, *sc, tables, ctx, b.w.scale, out, num_warps=num_warps)
    fn = getattr(m, "paged_decode_attention_weights" + tail)
    return fn(b.q, b.kc, b.vc, *sc, tables, ctx, b.w.scale, out, sums, num_warps=num_warps, **kw)


def keys_of(b, s):
    t = int(b.ctx[s])
    if not b.kind:
        kc = BT.np64(b.kc)
        return np.stack([opa.gather_sequence(kc, b.tables[s], t, g)
                         for g in range(b.w.num_kv_heads)])
    gather = ofp8.gather_fp8 if b.kind == "fp8" else oint8.gather_int8
    return np.stack([gather(b.kc.cpu().numpy(), b.vc.cpu().numpy(), b.ks_h, b.vs_h, b.tables[s],
                            t, g)[0] for g in range(b.w.num_kv_heads)])


def check_sums(b, before, after, seqs=None):
    before, after, q = BT.np64(before), BT.np64(after), BT.np64(b.q)
    G = b.w.num_q_heads // b.w.num_kv_heads
    cols = before.shape[2]
    for s in range(len(b.ctx)) if seqs is None else seqs:
        t = int(b.ctx[s])
        n = min(t, cols)
        assert np.array_equal(after[s, :, n:], before[s, :, n:])
        if t == 0:
            continue
        keys = keys_of(b, s)
        want = oev.attention_weights(q[s], keys, b.w.scale)[:, :n]
        for g in range(b.w.num_kv_heads):
            qg = np.abs(q[s, g * G:(g + 1) * G])
            A = b.w.head_dim * 2.0 ** -23 * b.w.scale * (np.abs(keys[g]) @ qg.T).max()
            if b.kind:  # q's conversion to f16: half a subnormal step where |q| < 2^-14
                A += b.w.head_dim * 2.0 ** -25 * b.w.scale * np.abs(keys[g]).max()
            # exponent and lse in log2 units: a rounding of up to |x| each
            A += 4 * 2.0 ** -24 * b.w.scale * (np.abs(keys[g]) @ qg.T).max()
            rel = 2 * A + (t / 16 + 64 + 2 * G) * 2.0 ** -24
            bound = want[g] * rel + np.abs(before[s, g, :n] + want[g]) * 2.0 ** -24
            assert np.all(np.abs(after[s, g, :n] - before[s, g, :n] - want[g]) <= bound + 1e-38)


LENS = (1, 17, 0, 40, 100, 16, 15, 333)


@pytest.mark.parametrize("dtype,D,B", [("f32", 32, 16), ("f32", 64, 16), ("f32", 128, 16),
                                       ("f16", 64, 16), ("bf16", 128, 16), ("f16", 256, 16),
                                       ("bf16", 128, 8), ("f16", 128, 32), ("bf16", 64, 32)])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_weights(dtype, D, B, G):
    b = batch(2 * G, 2, D, dtype, LENS, B=B)
    cols = b.tables.shape[1] * B
    sums = torch.rand((len(LENS), 2, cols), device="cuda")
    before = sums.clone()
    out = attend(b, sums)
    assert torch.equal(out, attend(b))
    check_sums(b, before, sums)


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 8), ("f16", 128, 1), ("bf16", 256, 4),
                                       ("f16", 256, 2)])
def test_weights_8bit(kind, dtype, D, G):
    b = batch(2 * G, 2, D, dtype, LENS, kind=kind)
    sums = torch.rand((len(LENS), 2, b.tables.shape[1] * 16), device="cuda")
    before = sums.clone()
    out = attend(b, sums)
    assert torch.equal(out, attend(b))
    check_sums(b, before, sums)


@pytest.mark.parametrize("num_warps", [1, 3, 64, 5000])
def test_weights_any_split(num_warps):
    """Contexts cut into many pieces, or none."""
    b = batch(8, 2, 128, "bf16", (1500, 3, 77))
    sums = torch.zeros((3, 2, b.tables.shape[1] * 16), device="cuda")
    out = attend(b, sums, num_warps=num_warps)
    assert torch.equal(out, attend(b, num_warps=num_warps))
    check_sums(b, torch.zeros_like(sums), sums)


def test_weights_accumulate_and_repeat_bit_for_bit():
    b = batch(16, 4, 128, "bf16", (700, 20, 1, 333))
    shape = (4, 4, b.tables.shape[1] * 16)
    runs = []
    for _ in range(2):
        sums = torch.zeros(shape, device="cuda")
        for _ in range(3):
            attend(b, sums)
        runs.append(sums)
    assert torch.equal(*runs)
    # each step adds weights of sum G per KV head
    total = runs[0].sum(-1)
    assert torch.allclose(total, torch.full_like(total, 12.0), rtol=1e-4)


def test_weights_ignore_what_lies_past_the_context():
    """NaN in every unused slot and in the sums' unused columns, entries past the tables."""
    b = batch(8, 2, 64, "f16", (5, 31, 16), maxb_extra=3)
    used = np.zeros((b.NB, 16), dtype=bool)
    for s in range(3):
        for p in range(int(b.ctx[s])):
            used[b.tables[s, p // 16], p % 16] = True
    mask = torch.from_numpy(~used).cuda().view(b.NB, 1, 16, 1)
    b.kc.masked_fill_(mask, float("nan"))
    b.vc.masked_fill_(mask, float("nan"))
    sums = torch.full((3, 2, b.tables.shape[1] * 16), float("nan"), device="cuda")
    for s in range(3):
        sums[s, :, :int(b.ctx[s])] = 0.5
    before = sums.clone()
    out = attend(b, sums)
    assert torch.isfinite(out).all()
    for s in range(3):
        n = int(b.ctx[s])
        assert torch.isfinite(sums[s, :, :n]).all() and torch.isnan(sums[s, :, n:]).all()
    z = torch.nan_to_num(before), torch.nan_to_num(sums)
    b.kc = torch.nan_to_num(b.kc)
    check_sums(b, *z)


def test_weights_fewer_columns_than_the_table_holds():
    b = batch(4, 2, 128, "bf16", (40, 100))
    m = pkv()
    sums = torch.zeros((2, 2, 100), device="cuda")
    ws = torch.zeros(m.weights_workspace_bytes(2, b.tables.shape[1], 16, 4, 2, 128, b.q.dtype),
                     dtype=torch.uint8, device="cuda")
    attend(b, sums, workspace=ws)
    assert m.decode_status(ws) == 0
    check_sums(b, torch.zeros_like(sums), sums)
    short = torch.zeros((2, 2, 64), device="cuda")
    attend(b, short, workspace=ws)
    assert m.decode_status(ws) == 1  # a context longer than the sums' columns
    assert torch.equal(short, sums[:, :, :64])


def test_weights_peaked_scores():
    """Scores hundreds apart: weights down to nothing, none of them NaN."""
    b = batch(8, 1, 128, "bf16", (600,))
    b.q *= 60
    sums = torch.zeros((1, 1, b.tables.shape[1] * 16), device="cuda")
    attend(b, sums)
    check_sums(b, torch.zeros_like(sums), sums)
    assert abs(float(sums.sum()) - 8) < 1e-2


def test_weights_long_context_and_full_batch():
    b = batch(64, 8, 128, "bf16", (70001, 1, 33000))
    sums = torch.zeros((3, 8, b.tables.shape[1] * 16), device="cuda")
    out = attend(b, sums)
    assert torch.equal(out, attend(b))
    check_sums(b, torch.zeros_like(sums), sums, seqs=[1, 2])


def test_weights_graphs_do_not_share_a_workspace():
    """Two captured graphs replayed on two streams at once, and an eager call between."""
    bs = [batch(32, 4, 128, "bf16", (2000, 64, 999), seed=s) for s in (4, 5)]
    refs = []
    for b in bs:
        r = torch.zeros((3, 4, b.tables.shape[1] * 16), device="cuda")
        attend(b, r)
        refs.append(r)
    args, graphs = [], []
    for b in bs:
        tables, ctx, _ = b.device_index("cuda")
        sums, out = torch.zeros_like(refs[len(args)]), torch.empty_like(b.q)
        args.append((tables, ctx, sums, out))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv().paged_decode_attention_weights(b.q, b.kc, b.vc, tables, ctx, b.w.scale, out, sums)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in bs]
    for a in args:
        a[2].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for b, a, r in zip(bs, args, refs):
        want = torch.zeros_like(r)
        for _ in range(5):
            want += r
        assert torch.equal(a[2], want)


def test_weights_on_two_streams_at_once():
    bs = [batch(32, 4, 128, "bf16", (3000, 64, 999), seed=s) for s in (7, 8)]
    refs, sums, idx = [], [], []
    for b in bs:
        r = torch.zeros((3, 4, b.tables.shape[1] * 16), device="cuda")
        attend(b, r)
        refs.append(r)
        sums.append(torch.zeros_like(r))
        idx.append(b.device_index("cuda"))
    outs = [torch.empty_like(b.q) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(4):
        for b, st, s, (tables, ctx, _), out in zip(bs, streams, sums, idx, outs):
            with torch.cuda.stream(st):
                pkv().paged_decode_attention_weights(b.q, b.kc, b.vc, tables, ctx, b.w.scale, out, s)
    torch.cuda.synchronize()
    for s, r in zip(sums, refs):
        want = torch.zeros_like(r)
        for _ in range(4):
            want += r
        assert torch.equal(s, want)


def test_weights_beyond_32_bit_offsets():
    """2^31 scores and more: 2048 blocks shared by long tables; all sequences alike, so every
    row of sums is the first one's, the pieces' order of summing aside."""
    S, G, D, nb = 260, 8, 64, 65536
    t = nb * 16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kc, vc = (torch.randn((2048, 1, 16, D), generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    q = torch.randn((1, G, D), generator=g, device="cuda").to(torch.bfloat16).expand(S, G, D)
    tables = (torch.arange(nb, dtype=torch.int32, device="cuda") % 2048).expand(S, nb)
    sums = torch.zeros((S, 1, t), device="cuda")
    q = q.contiguous()
    pkv().paged_decode_attention_weights(q, kc, vc, tables.contiguous(),
                                         torch.full((S,), t, dtype=torch.int32, device="cuda"),
                                         0.125, torch.empty_like(q), sums)
    x = 0.125 * q[0].double() @ kc[:, 0].reshape(-1, D).double().T  # [G, 2048 * 16]
    w = (torch.softmax(x, 1).sum(0) / (t // (2048 * 16))).float()
    A = D * 2.0 ** -23 * 0.125 * (kc.abs().reshape(-1, D).double()
                                  @ q[0].abs().double().T).max().item()
    rel = 2 * A + (t / 16 + 64 + 2 * G) * 2.0 ** -24 + 2.0 ** -23
    for s in (0, 1, 130, S - 1):
        got = sums[s, 0].view(-1, 2048 * 16)
        assert bool(((got - w).abs() <= rel * w).all()), s
    torch.cuda.synchronize()
    del sums
    pkv().ops._WORKSPACES.clear()
    torch.cuda.empty_cache()


def test_empty_batches():
    m, i = pkv(), dict(dtype=torch.int32, device="cuda")
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.float16, device="cuda")
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    none, table = torch.zeros(0, **i), torch.zeros((0, 2), **i)
    m.paged_decode_attention_weights(q, kc, kc.clone(), table, none, 0.1, torch.empty_like(q),
                                     torch.zeros((0, 2, 32), device="cuda"))
    kept, sums = torch.zeros((0, 2, 8), **i), torch.zeros((0, 2, 8), device="cuda")
    m.paged_evict_select(torch.zeros((0, 2, 32), device="cuda"), none, none, kept, sums,
                         torch.zeros(0, **i))
    m.paged_evict_gather(kc, kc.clone(), table, kept, none, torch.zeros((0, 1), **i))
    # contexts that are all empty: zero rows, untouched sums
    q = torch.ones((2, 4, 64), dtype=torch.float16, device="cuda")
    sums = torch.full((2, 2, 32), 3.0, device="cuda")
    out = m.paged_decode_attention_weights(q, kc, kc.clone(), torch.zeros((2, 2), **i),
                                           torch.zeros(2, **i), 0.1, torch.empty_like(q), sums)
    torch.cuda.synchronize()
    assert not out.any() and bool((sums == 3.0).all())


# --- select --------------------------------------------------------------------------
def select(sums, ctx, keep, cols=None, first=0, recent=0, status=None, ncols=None):
    S, H, W_ = sums.shape
    cols = cols or max(1, int(max(keep)))
    kept = torch.full((S, H, cols), -7, dtype=torch.int32, device="cuda")
    new = torch.full((S, H, ncols or cols), -3.0, device="cuda")
    lens = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    pkv().paged_evict_select(sums, i32(ctx), i32(keep), kept, new, lens, first=first,
                             recent=recent, status=status)
    torch.cuda.synchronize()
    return kept, new, lens


def check_select(sums, ctx, keep, first=0, recent=0, **kw):
    kept, new, lens = select(sums, ctx, keep, first=first, recent=recent, **kw)
    k, n, x = kept.cpu().numpy(), new.cpu().numpy(), sums.cpu().numpy()
    for s in range(sums.shape[0]):
        m = max(0, min(int(keep[s]), int(ctx[s])))
        assert int(lens[s]) == m
        for h in range(sums.shape[1]):
            want = fast_select(x[s, h], int(ctx[s]), int(keep[s]), first, recent)
            assert np.array_equal(k[s, h, :m], want), (s, h)
            assert np.array_equal(n[s, h, :m], x[s, h][want], equal_nan=True)
            assert np.all(k[s, h, m:] == -7) and np.all(n[s, h, m:] == -3.0)


def fast_select(x, t, keep, first, recent):
    """oracle.eviction.select with a stable sort, for long rows."""
    n = max(0, min(keep, t))
    r = min(recent, n)
    f = min(first, n - r)
    v = np.where(np.isnan(x[f:t - r]), -np.inf, x[f:t - r]).astype(np.float64)
    best = np.argsort(-v, kind="stable")[:n - r - f] + f
    return np.sort(np.concatenate([np.arange(f), best, np.arange(t - r, t)]))


def test_fast_select_is_the_oracle():
    g = np.random.default_rng(0)
    for _ in range(200):
        x = g.integers(0, 5, 40).astype(np.float64)
        x[g.random(40) < 0.1] = np.nan
        a = (int(g.integers(0, 41)), int(g.integers(0, 45)), int(g.integers(0, 9)),
             int(g.integers(0, 9)))
        assert np.array_equal(oev.select(x, *a), fast_select(x, *a)), a


@pytest.mark.parametrize("cols,first,recent", [(1, 0, 0), (33, 4, 5), (500, 0, 0), (2048, 4, 64),
                                               (2049, 0, 32), (16384, 4, 0), (16385, 1, 7),
                                               (40000, 4, 128), (131072, 4, 256),
                                               (131073, 0, 9), (300000, 4, 128)])
def test_select_sizes(cols, first, recent):
    g = np.random.default_rng(cols)
    S, H = (6, 3) if cols <= 2049 else (5, 2)
    sums = torch.from_numpy(np.exp(2 * g.standard_normal((S, H, cols))).astype(np.float32)).cuda()
    sums[torch.from_numpy(g.random((S, H, cols)) < 0.1).cuda()] = 0.0
    ctx = [cols, 0, 1, max(1, cols // 2), max(1, cols - 3)] + [cols] * (S - 5)
    keep = [max(1, cols // 3), 5, 4, max(1, cols // 2), 1] + [cols] * (S - 5)
    check_select(sums, ctx, keep, first, recent, cols=cols)


@pytest.mark.parametrize("cols", [700, 5000, 70000, 140001])
def test_select_ties_and_strange_values(cols):
    g = np.random.default_rng(cols)
    rows = [np.zeros(cols), np.full(cols, 2.5), g.integers(0, 3, cols),  # few values
            np.where(g.random(cols) < 0.5, 0.0, -0.0), g.standard_normal(cols),
            np.where(g.random(cols) < 0.7, np.nan, 1.0), np.full(cols, -np.inf),
            np.where(g.random(cols) < 0.3, np.inf, g.standard_normal(cols)),
            np.full(cols, 1e-42), np.arange(cols), -np.arange(cols)]
    sums = torch.from_numpy(np.stack(rows).astype(np.float32)[:, None]).cuda()
    n = len(rows)
    for keep in (1, cols // 2, cols - 1):
        check_select(sums, [cols] * n, [keep] * n)
        check_select(sums, [cols - 1] * n, [keep] * n, 2, 3)


def test_select_budgets_smaller_than_the_ends():
    sums = torch.rand((4, 2, 100), device="cuda")
    check_select(sums, [100, 50, 3, 100], [6, 2, 9, 0], first=4, recent=5, cols=16)
    check_select(sums, [100, 50, 3, 100], [-3, 2, 9, 100], first=200, recent=1, cols=100)


def test_select_reports_what_it_clamps():
    sums = torch.rand((3, 1, 64), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new, lens = select(sums, [70, -2, 10], [64, 3, 4], cols=64, status=st)
    assert int(st) == 1 and lens.tolist() == [64, 0, 4]
    st.zero_()
    kept, new, lens = select(sums, [64, 64, 64], [9, 8, 3], cols=8, status=st)
    assert int(st) == 1 and lens.tolist() == [8, 8, 3]
    st.zero_()
    kept, new, lens = select(sums, [64, 64, 64], [9, 8, 3], cols=9, ncols=8, status=st)
    assert int(st) == 1 and lens.tolist() == [8, 8, 3]
    st.zero_()
    select(sums, [5, 6, 7], [99, 99, 99], cols=8, status=st)
    assert int(st) == 0  # a budget above the context is no fault


def test_select_row_beyond_32_bit_offsets():
    """Rows past 2^31 sums."""
    H, cols = 3, 1 << 30
    sums = torch.zeros((1, H, cols), device="cuda")
    at = [5, 1 << 20, cols - 2]
    sums[0, :, at] = torch.tensor([[1.0, 3.0, 2.0]] * 3, device="cuda")
    kept, new, lens = select(sums, [cols], [3], cols=3)
    for h in range(H):
        assert kept[0, h].tolist() == at and new[0, h].tolist() == [1.0, 3.0, 2.0]
    del sums
    torch.cuda.empty_cache()


# --- gather --------------------------------------------------------------------------
def pools(kind, NB, H, B, D, seed):
    g = np.random.default_rng(seed)
    if kind in ("fp8", "int8"):
        dt = torch.uint8 if kind == "fp8" else torch.int8
        k = torch.from_numpy(g.integers(0, 127, (NB, H, B, D)).astype(np.uint8)).cuda().to(dt)
        v = torch.from_numpy(g.integers(0, 127, (NB, H, D, B)).astype(np.uint8)).cuda().to(dt)
        return k, v
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]
    k, v = (torch.from_numpy(g.standard_normal((NB, H, B, D)).astype(np.float32)).cuda().to(dt)
            for _ in range(2))
    return k, v


@pytest.mark.parametrize("kind,B,D", [("bf16", 16, 128), ("f16", 8, 64), ("bf16", 32, 256),
                                      ("f32", 16, 32), ("f32", 16, 128), ("f16", 16, 96),
                                      ("f32", 16, 1024), ("bf16", 24, 128), ("f16", 1, 64),
                                      ("fp8", 16, 128), ("int8", 16, 256),
                                      ("int8", 16, 48)])
def test_gather(kind, B, D):
    g = np.random.default_rng(D + B)
    S, H = 4, 3
    lens, n = [200, 1, 77, 16], [70, 1, 0, 16]
    nb = [-(-t // B) for t in lens]
    mb = [-(-t // B) for t in n]
    NB = sum(nb) + sum(mb) + 4
    order = g.permutation(NB)
    tables, new = np.full((S, max(nb)), -1), np.full((S, max(mb)), -1)  # padding never read
    at = 0
    for s in range(S):
        tables[s, :nb[s]] = order[at:at + nb[s]]
        at += nb[s]
        new[s, :mb[s]] = order[at:at + mb[s]]
        at += mb[s]
    K = 80
    kept = np.full((S, H, K), -1)
    for s in range(S):
        for h in range(H):
            kept[s, h, :n[s]] = np.sort(g.permutation(lens[s])[:n[s]])
    k, v = pools(kind, NB, H, B, D, 1)
    kw, vw = (x.float().cpu().numpy().copy() for x in (k, v))
    k0, v0 = kw.copy(), vw.copy()
    vpos = ofp8.V_POS if kind in ("fp8", "int8") else None
    for s in range(S):
        for h in range(H):
            for j in range(n[s]):
                p = kept[s, h, j]
                src, dst = tables[s, p // B], new[s, j // B]
                kw[dst, h, j % B] = k0[src, h, p % B]
                if vpos is None:
                    vw[dst, h, j % B] = v0[src, h, p % B]
                else:
                    vw[dst, h, :, vpos[j % B]] = v0[src, h, :, vpos[p % B]]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv().paged_evict_gather(k, v, i32(tables), i32(kept), i32(n), i32(new), status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert np.array_equal(k.float().cpu().numpy(), kw) and np.array_equal(v.float().cpu().numpy(), vw)


@pytest.mark.parametrize("D", [16, 48, 64, 128, 256, 512])
def test_gather_v8_leaves_the_slots_of_bad_places(D):
    """A whole tile one of whose tokens cannot be moved: its slot keeps its bytes."""
    k, v = pools("int8", 12, 2, 16, D, 5)
    k0, v0 = k.cpu().numpy(), v.cpu().numpy()
    n = 40
    kept = np.tile(np.arange(n) * 2, (1, 2, 1))
    kept[0, :, 5] = 4000
    kept[0, 1, 33] = -2
    pkv().paged_evict_gather(k, v, i32([[1, 9, 2, 7, 0]]), i32(kept), i32([n]), i32([[4, 11, 5]]))
    torch.cuda.synchronize()
    want = v0.copy()
    for h in range(2):
        for j in range(n):
            p = kept[0, h, j]
            if 0 <= p < 80:
                src, dst = [1, 9, 2, 7, 0][p // 16], [4, 11, 5][j // 16]
                want[dst, h, :, ofp8.V_POS[j % 16]] = v0[src, h, :, ofp8.V_POS[p % 16]]
    assert np.array_equal(v.cpu().numpy(), want)


@pytest.mark.parametrize("kind,NB", [("bf16", 140000), ("int8", 140000)])
def test_gather_beyond_32_bit_offsets(kind, NB):
    H, B, D = 8, 16, 128
    dt = torch.bfloat16 if kind == "bf16" else torch.int8
    k = torch.zeros((NB, H, B, D), dtype=dt, device="cuda")
    v = torch.zeros((NB, H, B, D) if kind == "bf16" else (NB, H, D, B), dtype=dt, device="cuda")
    src, dst = NB - 1, NB - 3
    k[src], v[src] = torch.randint(1, 100, k[src].shape, device="cuda").to(dt), 5
    kept = i32(np.tile([3, 7, 9], (1, H, 1)))
    pkv().paged_evict_gather(k, v, i32([[src]]), kept, i32([3]), i32([[dst]]))
    torch.cuda.synchronize()
    assert torch.equal(k[dst, :, :3], k[src][:, [3, 7, 9]]) and not k[dst, :, 3:].any()
    if kind == "bf16":
        assert bool((v[dst, :, :3] == 5).all()) and not v[dst, :, 3:].any()
    else:
        at = torch.tensor(ofp8.V_POS[:3].copy(), device="cuda")
        assert bool((v[dst][:, :, at] == 5).all()) and int(v[dst].sum()) == 5 * 3 * H * D
    assert not k[:NB - 3].any() and not v[:NB - 3].any()
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_gather_skips_and_reports_bad_places(kind):
    NB, H, B, D = 8, 1, 16, 128
    k, v = pools(kind, NB, H, B, D, 2)
    k0, v0 = k.clone(), v.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = np.array([[[0, 1, 40, -1, 20]]])  # 40: past the table's blocks
    pkv().paged_evict_gather(k, v, i32([[2, 99]]), i32(kept), i32([5]), i32([[5]]), status=st)
    torch.cuda.synchronize()
    assert int(st) == 2  # positions 40 and -1, and 20 in a block that is not there
    assert torch.equal(k[5, 0, :2], k0[2, 0, :2]) and torch.equal(k[5, 0, 2:], k0[5, 0, 2:])
    k[5], v[5] = k0[5], v0[5]
    assert torch.equal(k, k0)
    if kind == "bf16":
        assert torch.equal(v, v0)
    k, v = k0.clone(), v0.clone()
    st.zero_()
    pkv().paged_evict_gather(k, v, i32([[2]]), i32([[[0, 1]]]), i32([2]), i32([[-1]]), status=st)
    torch.cuda.synchronize()
    assert int(st) == 2 and torch.equal(k, k0) and torch.equal(v, v0)


def test_select_and_gather_in_a_graph():
    g = np.random.default_rng(1)
    b = batch(8, 2, 128, "bf16", (200, 40), pool_blocks=24)
    sums = torch.rand((2, 2, 208), device="cuda")
    tables, ctx, _ = b.device_index("cuda")
    spare = sorted(set(range(b.NB)) - set(b.tables[0, :13].tolist()) - set(b.tables[1, :3].tolist()))
    new = i32(np.array(spare[:4]).reshape(2, 2))
    keep = i32([20, 30])
    kept = torch.zeros((2, 2, 32), dtype=torch.int32, device="cuda")
    ns, nl = torch.zeros((2, 2, 32), device="cuda"), i32([0, 0])

    def step():
        pkv().paged_evict_select(sums, ctx, keep, kept, ns, nl, first=1, recent=2)
        pkv().paged_evict_gather(b.kc, b.vc, tables, kept, nl, new)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (kept, ns, nl, b.kc, b.vc)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    sums.copy_(torch.from_numpy(g.random((2, 2, 208)).astype(np.float32)))
    graph.replay()
    torch.cuda.synchronize()
    other = [t.clone() for t in (kept, ns, nl, b.kc, b.vc)]
    assert not torch.equal(other[0], want[0])
    step()
    torch.cuda.synchronize()
    for t, w in zip((kept, ns, nl, b.kc, b.vc), other):
        assert torch.equal(t, w)


def test_python_refusals():
    m, z = pkv(), torch.zeros
    dev = dict(device="cuda")
    i = dict(dtype=torch.int32, device="cuda")
    sums, ctx, keep = z(2, 3, 64, **dev), z(2, **i), z(2, **i)
    kept, new, lens = z(2, 3, 8, **i), z(2, 3, 8, **dev), z(2, **i)
    for kw, err in ((dict(kept=kept.long()), TypeError), (dict(new_sums=new.double()), TypeError),
                    (dict(kept=kept[:, :2].contiguous()), ValueError),
                    (dict(keep_lens=keep[:1]), ValueError), (dict(first=-1), m.PkvError),
                    (dict(weight_sums=sums[..., ::2]), ValueError),
                    (dict(new_sums=sums), m.PkvError), (dict(new_lens=ctx), m.PkvError)):
        a = dict(weight_sums=sums, context_lens=ctx, keep_lens=keep, kept=kept, new_sums=new,
                 new_lens=lens)
        a.update(kw)
        with pytest.raises(err):
            m.paged_evict_select(**a)
    kc = z(4, 3, 16, 64, dtype=torch.float16, **dev)
    t, nt = z(2, 4, **i), z(2, 1, **i)
    for kw, err in ((dict(v_cache=kc.float()), ValueError), (dict(kept=kept[:, :1]), ValueError),
                    (dict(new_tables=nt[:1]), ValueError), (dict(new_tables=t), m.PkvError),
                    (dict(k_cache=kc.to(torch.int8), v_cache=kc.to(torch.int8)), ValueError)):
        a = dict(k_cache=kc, v_cache=kc.clone(), block_tables=t, kept=kept, new_lens=lens,
                 new_tables=nt)
        a.update(kw)
        with pytest.raises(err):
            m.paged_evict_gather(**a)
    q = z(2, 6, 64, dtype=torch.float16, **dev)
    for kw, err in ((dict(weight_sums=sums.double()), ValueError),
                    (dict(weight_sums=sums[:, :2].contiguous()), ValueError),
                    (dict(workspace=z(256, dtype=torch.uint8, **dev)), ValueError)):
        a = dict(q=q, k_cache=kc, v_cache=kc.clone(), block_tables=t, context_lens=ctx, scale=0.1,
                 out=torch.empty_like(q), weight_sums=sums)
        a.update(kw)
        with pytest.raises(err):
            m.paged_decode_attention_weights(**a)
