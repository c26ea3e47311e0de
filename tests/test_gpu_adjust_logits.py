"""GPU parity of penalties, biases and masks on logits.

Bound: up to five fp32 operations (quotient or product by the repetition, frequency times count
and its difference, presence, bias), each off by u = 2^-24 of its result, whose parts are at most
m = |x| max(r, 1 / r) + |frequency| n + |presence| + |bias| in size: 5 u m; then half a step of the
type.  Logits that nothing touches keep their bits; banned ones are -infinity.
"""
import numpy as np
import pytest
import torch

from oracle import speculative as osp

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


def f32(a):
    return torch.tensor(np.asarray(a, dtype=np.float32), device="cuda")


class Case:
    def __init__(self, counts, V, L, dtype="f32", seed=0, path=0, bias=0, masked=False, prompt=True,
                 penalties="rfp", pad=0, apart=False, tail=0, common=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        S, T = len(counts), int(sum(counts)) + tail
        self.__dict__.update(S=S, T=T, V=V, apart=apart)
        self.starts = np.concatenate([[0], np.cumsum(counts)])
        full = (torch.randn((T, V + pad), generator=g, device="cuda") * 3).to(DT[dtype])
        self.logits = full[:, pad // 2:pad // 2 + V]
        self.out = torch.full((T, V + pad), 9.0, dtype=DT[dtype], device="cuda")[:, :V] if apart else None
        top = max(2, V // 50) if common else V
        self.history = rng.integers(-1, top, (S, L))
        self.history[:, ::3] = rng.integers(0, V, self.history[:, ::3].shape)
        if L > 4:
            self.history[0, :4] = [-5, V, V + 100, V - 1]
        self.lens = rng.integers(0, L + 1, S)
        self.lens[0] = L
        self.prompts = rng.integers(0, L + 1, S) if prompt else None
        self.rep = rng.uniform(0.8, 1.5, S).astype(np.float32) if "r" in penalties else None
        self.freq = rng.uniform(-0.5, 1.0, S).astype(np.float32) if "f" in penalties else None
        self.pres = rng.uniform(-0.5, 1.0, S).astype(np.float32) if "p" in penalties else None
        self.path = rng.integers(-1, top, (T, path)) if path else None
        self.bt = self.bv = self.ok = None
        if bias:
            self.bt = rng.integers(-1, V, (S, bias))
            self.bt[:, -1] = self.bt[:, 0]  # the same token twice
            self.bv = rng.standard_normal((S, bias)).astype(np.float32) * 3
        if masked:
            W = -(-V // 32)
            p = rng.choice([0.02, 0.5, 0.98, 0.0, 1.0], (T, 1))
            self.ok = rng.random((T, W * 32)) < p

    def args(self):
        opt = lambda f, x: None if x is None else f(x)  # noqa: E731
        allowed = None
        if self.ok is not None:
            allowed = i32(np.packbits(self.ok, axis=1, bitorder="little").view(np.int32))
        return dict(history=i32(self.history), history_lens=i32(self.lens),
                    prompt_lens=opt(i32, self.prompts), row_start=i32(self.starts),
                    repetition=opt(f32, self.rep), frequency=opt(f32, self.freq),
                    presence=opt(f32, self.pres), path=opt(i32, self.path),
                    bias_tokens=opt(i32, self.bt), bias_values=opt(f32, self.bv), allowed=allowed,
                    out=self.out)

    def oracle(self):
        rows = np.full(self.T, -1)
        for s in range(self.S):
            rows[self.starts[s]:self.starts[s + 1]] = s
        ok = None if self.ok is None else self.ok[:, :self.V]
        a = (self.history, self.lens, self.prompts, rows, self.rep, self.freq, self.pres, self.path,
             self.bt, self.bv)
        x = np64(self.logits)
        want = osp.adjust_logits(x, *a, ok)
        # the size of the terms: every part with its absolute value
        size = np.abs(x) * 1.5 + np.zeros_like(x)
        mags = osp.adjust_logits(np.zeros_like(x), self.history, self.lens, self.prompts, rows, None,
                                 None if self.freq is None else -np.abs(self.freq),
                                 None if self.pres is None else -np.abs(self.pres), self.path, self.bt,
                                 None if self.bv is None else np.abs(self.bv))
        return want, size + mags, rows

    def check(self):
        want, size, rows = self.oracle()
        before = self.logits.clone()
        got = pkv().adjust_logits(self.logits, **self.args())
        torch.cuda.synchronize()
        assert got is (self.out if self.apart else self.logits)
        if self.apart:
            assert torch.equal(self.logits, before)
        y, u = np64(got), torch.finfo(got.dtype).eps / 2
        live = rows >= 0
        keep = np64(before) if not self.apart else np.full_like(y, 9.0)
        assert np.array_equal(y[~live], keep[~live])
        y, want, size, x = y[live], want[live], size[live], np64(before)[live]
        assert np.array_equal(np.isneginf(y), np.isneginf(want))
        fine = np.isfinite(want)
        tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134
        bound = 5 * 2.0 ** -24 * size + u * (np.abs(want) + 5 * 2.0 ** -24 * size) + tiny
        assert (np.abs(y[fine] - want[fine]) <= bound[fine]).all()
        same = fine & (want == x)
        assert np.array_equal(y[same], x[same])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 7, 33, 1000, 8191, 8193, 32000, 50257])
def test_vocabularies(dtype, V):
    Case([1, 3, 1], V, 200, dtype, path=4, bias=5, masked=True).check()
    Case([1, 3, 1], V, 200, dtype, path=4, bias=5, masked=False).check()


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("bias", [0, 1, 300])
@pytest.mark.parametrize("path", [0, 1, 9])
def test_parts(masked, apart, bias, path):
    Case([2, 0, 5, 1], 9001, 700, "bf16", path=path, bias=bias, masked=masked, apart=apart).check()


@pytest.mark.parametrize("penalties", ["", "r", "f", "p", "rf"])
@pytest.mark.parametrize("prompt", [False, True])
def test_penalties_one_by_one(penalties, prompt):
    Case([1] * 5, 4000, 333, "f32", penalties=penalties, prompt=prompt).check()


@pytest.mark.parametrize("pad", [1, 3, 8, 16])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("apart", [False, True])
def test_rows_at_any_alignment(pad, dtype, apart):
    """Odd strides, rows that start anywhere, out at another alignment than logits."""
    Case([3, 2], 10001, 300, dtype, pad=pad, masked=True, bias=3, apart=apart).check()
    Case([3, 2], 10001, 300, dtype, pad=pad, masked=False, bias=3, apart=apart).check()


@pytest.mark.parametrize("L", [0, 1, 2, 3, 5, 4097, 40000])
def test_history_lengths(L):
    Case([1, 1], 5000, L, "f32").check()


def test_long_histories_count_right():
    """One token 100,000 times: counts are whole numbers."""
    c = Case([1], 20000, 100000, "f32", penalties="fp", prompt=False)
    c.history[0] = 777
    c.lens[0] = 100000
    c.check()


def test_rows_behind_the_last_request():
    Case([2, 3], 6000, 100, "f16", tail=3, masked=True, bias=2).check()
    Case([2, 3], 6000, 100, "f16", tail=3, masked=True, bias=2, apart=True).check()


def test_many_requests_and_many_rows():
    Case([1] * 300, 3001, 50, "bf16", masked=True).check()
    Case([150], 9000, 500, "bf16", path=5, bias=4).check()
    Case([150], 40000, 500, "bf16", path=5, masked=True).check()


def test_without_row_start():
    c = Case([1, 1, 1], 2000, 80, "f32", bias=3)
    want, _, _ = c.oracle()
    a = c.args()
    a["row_start"] = None
    y = pkv().adjust_logits(c.logits, **a)
    assert np.allclose(np64(y), want, rtol=1e-5, atol=1e-5)


def test_infinities_and_nan():
    """A banned logit is -infinity whatever it was; the others follow the formula."""
    c = Case([2], 300, 60, "f32", masked=True)
    c.ok[:] = True
    c.ok[:, 5] = False
    c.history[0, :6] = [5, 6, 7, 8, 9, 10]
    c.lens[0], c.prompts[0] = 6, 0
    c.logits[:, 5] = float("nan")
    c.logits[:, 6] = float("nan")
    c.logits[:, 7] = float("inf")
    c.logits[:, 8] = -float("inf")
    c.logits[:, 200] = float("nan")
    y = pkv().adjust_logits(c.logits, **c.args())
    assert torch.isneginf(y[:, 5]).all() and torch.isnan(y[:, 6]).all()
    assert torch.isposinf(y[:, 7]).all() and torch.isneginf(y[:, 8]).all()
    assert torch.isnan(y[:, 200]).all()


def test_lengths_out_of_range_are_clamped():
    c = Case([1, 1], 500, 20, "f32", penalties="f")
    c.lens[:] = [1000, -3]
    c.prompts[:] = [-5, 10]
    want, _, _ = c.oracle()
    y = pkv().adjust_logits(c.logits, **c.args())
    assert np.allclose(np64(y), want, rtol=1e-5, atol=1e-5)


def test_the_same_bits_streams_and_graphs():
    c = Case([4, 4], 30000, 900, "bf16", path=4, bias=20, masked=True, apart=True)
    a = c.args()
    want = pkv().adjust_logits(c.logits, **a).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv().adjust_logits(c.logits, **a)
    for _ in range(3):
        c.out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
    st = torch.cuda.Stream()
    c.out.fill_(9.0)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        pkv().adjust_logits(c.logits, **a)
    st.synchronize()
    assert torch.equal(c.out, want)


def test_refusals():
    m = pkv()
    c = Case([2, 1], 100, 20, "f32", path=2, bias=2, masked=True)
    good = c.args()
    for kw in (dict(row_start=i32([0, 2])), dict(history_lens=i32([1])), dict(prompt_lens=i32([1])),
               dict(repetition=f32([1])), dict(path=i32(np.zeros((2, 2)))),
               dict(bias_values=None), dict(bias_tokens=None), dict(bias_values=f32([[1, 2]])),
               dict(allowed=i32(np.zeros((2, 4)))), dict(frequency=torch.ones(2)),
               dict(out=torch.empty((3, 99), device="cuda")), dict(out=c.logits.half()),
               dict(history=i32(np.zeros((2, 3, 4))))):
        with pytest.raises(ValueError):
            m.adjust_logits(c.logits, **{**good, **kw})
    for kw in (dict(row_start=i32([0, 2, 3]).long()), dict(presence=i32([1, 2]))):
        with pytest.raises(TypeError):
            m.adjust_logits(c.logits, **{**good, **kw})
    with pytest.raises(m.PkvError):
        m.adjust_logits(c.logits, **{**good, "allowed": i32(np.zeros((3, 3)))})
    with pytest.raises(m.PkvError):
        m.adjust_logits(c.logits, **{**good, "row_start": None})
    with pytest.raises(ValueError):
        m.adjust_logits(c.logits.t(), **good)


def test_before_beams_are_selected():
    """A banned or penalised token next to the selection that reads the logits."""
    m = pkv()
    c = Case([3], 4000, 50, "f32", masked=True)
    c.ok[:, :] = False
    c.ok[:, 10:20] = True
    y = m.adjust_logits(c.logits, **c.args())
    scores = torch.empty((1, 4), device="cuda")
    beams, tokens = (torch.empty((1, 4), dtype=torch.int32, device="cuda") for _ in range(2))
    m.beam_select(y[None], torch.zeros((1, 3), device="cuda"), scores, beams, tokens)
    p = torch.log_softmax(y.double(), -1).flatten()
    best = torch.sort(p, descending=True, stable=True).indices[:4]
    assert torch.equal(beams[0].long(), best // 4000) and torch.equal(tokens[0].long(), best % 4000)
    assert ((tokens >= 10) & (tokens < 20)).all()


def test_logits_past_2_to_the_31_elements():
    T, V = 70000, 32000
    x = torch.zeros((T, V), dtype=torch.float16, device="cuda")
    h = torch.full((1, 8), 31999, dtype=torch.int32, device="cuda")
    m = pkv()
    m.adjust_logits(x, h, i32([8]), row_start=i32([0, T]), frequency=f32([0.5]))
    assert (x[:, 31999] == -4).all() and int(torch.count_nonzero(x)) == T
