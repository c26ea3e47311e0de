"""GPU parity of beam search's selection.

Scores: lse is a sum of fp32 exponentials 2^(d log2 e) (the exponent's rounding is 2^-24 |d|
log2 e, so 2^-20.4 of a term where it counts, |d| < 17; the function 2^-22), 16 of a thread's
terms added in fp32 (16 roundings, 2^-20), rescaled when its maximum grows (2^-22 each), the
rest carried or in 64-bit integers: below 2^-18 relative, so 2^-18 absolute in the log; the score is
rounded to fp32 once.  Beams
and tokens: equal to the oracle's where candidates of different beams lie further apart
than that; within a beam the order is exact whatever the distance.
"""
import numpy as np
import pytest
import torch

from oracle import beam as obeam

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def pkv():
    import paged_kv_cache_166_gb300 as m
    return m


def run(logits, bs, N, **kw):
    S = logits.shape[0]
    scores = torch.full((S, N), float("nan"), device="cuda")
    beams, tokens = (torch.full((S, N), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pkv().beam_select(logits, bs, scores, beams, tokens, **kw)
    torch.cuda.synchronize()
    return scores, beams, tokens


def check(logits, bs, N, out=None):
    scores, beams, tokens = (t.cpu().numpy() for t in (out or run(logits, bs, N)))
    x, b = logits.double().cpu().numpy(), bs.cpu().numpy()
    for s in range(x.shape[0]):
        cand = obeam.candidate_scores(x[s], b[s])
        ws, wb, wt = obeam.select(x[s], b[s], N)
        live = np.isfinite(ws)
        assert np.array_equal(np.isneginf(scores[s]), ~live)
        bound = TOL + 2.0 ** -23 * np.abs(ws[live])
        assert np.all(np.abs(scores[s][live] - ws[live]) <= bound)
        # no candidate twice, and every one as good as the oracle's in its place
        assert len(set(zip(beams[s].tolist(), tokens[s].tolist()))) == N
        assert np.all(np.abs(cand[beams[s], tokens[s]][live] - ws[live]) <= 2 * bound)
        # where the oracle's neighbours of other beams are further away, exactly its own
        gap = np.full(N, np.inf)
        order = np.sort(cand[np.isfinite(cand)])[::-1]
        for j in np.nonzero(live)[0]:
            others = cand[np.arange(len(cand)) != wb[j]]
            near = np.abs(others[np.isfinite(others)] - ws[j])
            gap[j] = near.min() if near.size else np.inf
        clear = gap > 4 * TOL + 2.0 ** -21 * np.abs(np.where(live, ws, 0.0))
        if clear[live].all():
            assert np.array_equal(beams[s], wb) and np.array_equal(tokens[s], wt)
        assert order.size or not live.any()


def make(S, K, V, dtype, seed=0, scale=2.5, banned=0.02):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((S, K, V), generator=g, device="cuda") * scale
    x[torch.rand((S, K, V), generator=g, device="cuda") < banned] = -float("inf")
    bs = -10 * torch.rand((S, K), generator=g, device="cuda")
    return x.to(DT[dtype]), bs


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S,K,V,N", [(1, 1, 1, 1), (1, 2, 3, 6), (1, 1, 700001, 128), (3, 3, 4097, 5), (2, 4, 100, 8), (3, 4, 2047, 8),
                                     (1, 4, 2049, 4), (2, 3, 8191, 7), (5, 8, 8193, 16),
                                     (1, 64, 1000, 128), (2, 16, 32000, 32), (40, 2, 20011, 4),
                                     (1, 1, 200003, 1)])
def test_sizes(dtype, S, K, V, N):
    x, bs = make(S, K, V, dtype, seed=V)
    check(x, bs, N)


def test_many_rows_take_large_chunks():
    x, bs = make(70, 8, 9000, "bf16", seed=3)
    check(x, bs, 16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,N", [(5000, 128), (40000, 16)])
def test_sorted_and_clustered_logits(dtype, V, N):
    """The best candidates next to each other, in one thread's or one chunk's hands."""
    up = torch.linspace(-8, 8, V, device="cuda")
    x = torch.stack([up, up.flip(0), torch.where(up > 7.9, up, -up.abs()),
                     (up * 4).round() / 4])[None].to(DT[dtype])
    bs = torch.tensor([[-1.0, -1.25, -0.4, -2.0]], device="cuda")
    check(x, bs, N)


def test_equal_logits_go_by_beam_and_token():
    for V, N in ((10, 25), (5000, 8), (9001, 40)):
        x = torch.zeros((2, 3, V), device="cuda")
        s, b, t = run(x, torch.zeros((2, 3), device="cuda"), N)
        for r in range(2):
            assert b[r].tolist() == [j // V for j in range(N)]
            assert t[r].tolist() == [j % V for j in range(N)]
        assert torch.allclose(s, torch.full_like(s, -float(np.log(V))), atol=2e-6)


def test_one_beam_is_an_exact_top_n():
    """A 16-bit row has many equal logits: lower tokens first."""
    x, bs = make(3, 1, 65537, "bf16", seed=1)
    s, b, t = run(x, bs, 128)
    v, i = torch.sort(x[:, 0].float(), dim=-1, descending=True, stable=True)
    assert torch.equal(t.long(), i[:, :128]) and int(b.abs().sum()) == 0


def test_first_step_one_live_beam():
    x, bs = make(2, 4, 3000, "f32", seed=2, banned=0.0)
    bs[:, 1:] = -float("inf")
    x[:, 1:] = float("nan")  # logits of dead beams are not looked at
    check(x, bs, 8)
    s, b, t = run(x, bs, 8)
    assert int(b.sum()) == 0


def test_dead_beams_banned_tokens_and_strange_values():
    inf, nan = float("inf"), float("nan")
    x = torch.full((7, 2, 40), -inf, device="cuda")
    x[0, 0, [3, 30]] = torch.tensor([1.0, 2.0], device="cuda")    # two tokens allowed
    x[1] = nan                                                     # nothing but NaN
    x[2, 0] = torch.arange(40.0, device="cuda")
    x[2, 1, 7] = inf                                               # no finite maximum
    x[3] = 0.0
    x[4, 0] = 0.0
    x[4, 1, 39] = -300.0
    x[5] = 3e38
    x[6, :, ::3] = nan
    x[6, :, 1::3] = torch.randn((2, 13), device="cuda")
    bs = torch.tensor([[0.0, -1.0], [0.0, 0.0], [0.0, 0.0], [nan, inf], [-inf, -2.0], [0.0, -1e30],
                       [0.0, 0.0]], device="cuda")
    for N in (1, 2, 5, 80):
        check(x, bs, N)
    for dt in (torch.float16, torch.bfloat16):
        check(x.to(dt), bs, 5)


def test_logits_whose_maximum_grows_to_huge_values():
    """A part's sums rescaled from tile to tile, across magnitudes that overflow times log2 e."""
    V = 30000
    x = torch.randn((4, 2, V), device="cuda")
    x[3, 0] += 1048575.0  # steps of 1/16, around the border of the two ways
    x[3, 1, 12000:] += 1048570.0
    x[0, 0, 9000:] += 60
    x[0, 0, 25000:] += 60
    x[1, 0, :] = -3.3e38
    x[1, 0, 12000:] = -1e30
    x[1, 0, 24000:] = torch.randn(6000, device="cuda")
    x[2, 0, 12000:] = 3e38
    x[2, 0, 29999] = 3.2e38
    bs = torch.zeros((4, 2), device="cuda")
    check(x, bs, 8)
    check(x.repeat(30, 4, 1), bs.repeat(30, 4), 8)
    bs[:, 1] = -100.0  # other beams' candidates are far away: the order is exact
    check(x, bs, 8)
    many = x.repeat(30, 4, 1)  # enough rows for parts of several tiles
    check(many, bs.repeat(30, 4) - 0.25 * torch.arange(8, device="cuda"), 8)


def test_every_candidate():
    x, bs = make(2, 4, 32, "f32", seed=9, banned=0.3)
    check(x, bs, 128)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("V,offset", [(5003, 1), (5003, 3), (20000, 5), (9, 2)])
def test_strides_and_alignment(dtype, V, offset):
    """Rows at any element's alignment, padded vocabularies, beams and requests in any order."""
    x, bs = make(3, 4, V, dtype, seed=V + offset)
    N = 8
    want = run(x, bs, N)
    pad = torch.full((3, 4, V + 13), 50.0, dtype=x.dtype, device="cuda")
    flat = torch.full((3 * 4 * (V + 13) + 16,), 50.0, dtype=x.dtype, device="cuda")
    view = flat[offset:offset + pad.numel()].view(3, 4, V + 13)[..., :V]
    view.copy_(x)
    turned = torch.full((4, 3, V + 5), 50.0, dtype=x.dtype, device="cuda").transpose(0, 1)[..., :V]
    turned.copy_(x)
    for y in (view, turned):
        assert y.stride(2) == 1 and not y.is_contiguous()
        for a, b in zip(run(y, bs, N), want):
            assert torch.equal(a, b)


def test_shared_logits_row():
    """Every beam reading one row (stride 0)."""
    row = torch.randn(4001, device="cuda")
    x = row.expand(2, 3, 4001)
    bs = torch.tensor([[-1.0, -2.0, -3.0], [0.0, 0.0, 0.0]], device="cuda")
    check(x, bs, 6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_rows_tie_whatever_their_alignment(dtype):
    """Three beams with the same logits and score, rows of an odd width: by beam, then token."""
    V = 20011
    row, _ = make(1, 1, V, dtype, seed=12)
    x = row.expand(2, 3, V).contiguous()
    s, b, t = run(x, torch.full((2, 3), -1.5, device="cuda"), 12)
    assert torch.equal(s[:, 0::3], s[:, 1::3]) and torch.equal(s[:, 0::3], s[:, 2::3])
    v, i = torch.sort(row[0, 0].float(), descending=True, stable=True)
    if len(set(v[:4].tolist())) == 4:
        assert b[0].tolist() == [0, 1, 2] * 4 and t[0].tolist() == i[:4].repeat_interleave(3).tolist()


def test_offsets_past_32_bits():
    S, K, V = 3, 2, 4096
    big = torch.zeros((1 << 31) + 3 * V, dtype=torch.float16, device="cuda")
    x = big.as_strided((S, K, V), (1 << 30, V, 1))
    src, bs = make(S, K, V, "f16", seed=4)
    x.copy_(src)
    for a, b in zip(run(x, bs, 4), run(src, bs, 4)):
        assert torch.equal(a, b)


def test_one_workspace_for_calls_of_any_sizes():
    x, bs = make(6, 4, 30000, "f32", seed=6)
    want = run(x, bs, 8)
    m = pkv()
    n = m.beam_workspace_bytes(6, 4, 30000, 8, torch.float32)
    for fill in (0, 255):  # the tickets start at zero, the rest at anything
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        ws[:512 << 10] = 0
        for _ in range(3):
            for a, b in zip(run(x, bs, 8, workspace=ws), want):
                assert torch.equal(a, b)
    # a smaller batch in the same workspace, then the large one again
    y, ys = make(2, 2, 500, "bf16", seed=7)
    check(y, ys, 3, run(y, ys, 3, workspace=ws))
    for a, b in zip(run(x, bs, 8, workspace=ws), want):
        assert torch.equal(a, b)
    assert int(ws[:512 << 10].sum()) == 0


def test_two_graphs_and_eager_calls():
    m = pkv()
    data = [make(8, 4, 40000, "f16", seed=s) for s in (1, 2)]
    want = [run(x, bs, 8) for x, bs in data]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    graphs = []
    for (x, bs), o in zip(data, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.beam_select(x, bs, *o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        run(*data[0], 8)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    m = pkv()
    data = [make(16, 4, 50000, "f32", seed=s) for s in (3, 4)]
    want = [run(x, bs, 8) for x, bs in data]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(10):
        for (x, bs), o, s in zip(data, outs, streams):
            with torch.cuda.stream(s):
                m.beam_select(x, bs, *o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("K,N,V", [(64, 128, 20000), (16, 128, 60000), (8, 64, 33000)])
def test_many_candidates_are_merged_by_row(K, N, V):
    x, bs = make(2, K, V, "bf16", seed=N + V)
    check(x, bs, N)


def test_python_refusals():
    m = pkv()
    x, bs = make(2, 3, 50, "f32")
    sc = torch.empty((2, 4), device="cuda")
    be, to = (torch.empty((2, 4), dtype=torch.int32, device="cuda") for _ in range(2))

    def call(**kw):
        a = dict(logits=x, beam_scores=bs, scores=sc, beams=be, tokens=to)
        a.update(kw)
        m.beam_select(**a)
    for kw, err in ((dict(logits=x.double()), TypeError), (dict(logits=x.cpu()), ValueError),
                    (dict(logits=x.transpose(1, 2)), ValueError), (dict(beams=be.long()), TypeError),
                    (dict(beam_scores=bs.double()), TypeError), (dict(tokens=to[:, :2]), ValueError),
                    (dict(logits=x[..., ::2]), ValueError),
                    (dict(beam_scores=bs[:, :2].contiguous()), ValueError),
                    (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), ValueError)):
        with pytest.raises(err):
            call(**kw)
    three = torch.zeros((2, 3), device="cuda")
    i3 = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="beam_scores"):
        m.beam_select(x, three, three, i3, i3.clone())
    for S, K, V, N in ((1, 65, 100, 4), (1, 4, 100, 129), (1, 2, 3, 7), (2000, 40, 100, 4),
                       (1, 1, (1 << 31) - 8192, 1)):
        with pytest.raises(m.PkvError):
            m.beam_workspace_bytes(S, K, V, N, torch.float32)
    empty = torch.empty((0, 3, 50), device="cuda")
    m.beam_select(empty, bs[:0], sc[:0], be[:0], to[:0])
