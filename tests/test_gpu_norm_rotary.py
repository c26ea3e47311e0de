"""GPU parity of the norm, rotation and cache write in one pass.

Bound of an element (u = 2^-24): the sum of D squares is off by at most (D + 1) u relative, the
mean (1 / D and the product with it) and eps by u each, half of which reaches the root; the
root's Newton step adds 2 u, the two products of the norm u each: a normed value is off by
((D + 1) / 2 + 6) u relative.  Turning
it: cos and sin are off by u (relative to 1), each product and the sum by u: 3 u (|y1| + |y2|)
beside the values' own error.  One rounding to the type adds half a step.  A norm that is not
asked for leaves the rotation's part.  8-bit codes lie between the codes of the bound's ends.
"""
import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import int8 as oint8
from oracle import rotary as orot
from oracle import speculative as osp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
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


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, dtype, B=16, kind="", inter=False, fused=False, seed=0,
                 A=1, weight="same", per_head=False, eps=1e-6, span=3000, offset=0, scale=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        h = np.random.default_rng(seed)
        dt = DT[dtype]
        self.__dict__.update(T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, B=B, kind=kind, inter=inter, dt=dt,
                             eps=eps, A=A)
        n = Hq + 2 * Hkv
        if fused:
            width = n * D + (offset + 7) // 8 * 8 + 8
            x = (torch.randn((T, width), generator=g, device="cuda") * scale).to(dt)
            x = x[:, offset:offset + n * D].unflatten(1, (n, D))
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = ((torch.randn((T, m, D), generator=g, device="cuda") * scale).to(dt)
                                      for m in (Hq, Hkv, Hkv))
        wt = torch.float32 if weight == "f32" else dt
        self.qw = self.kw = None
        if eps is not None and weight is not None:
            self.qw, self.kw = (torch.randn(((m, D) if per_head else (D,)), generator=g,
                                            device="cuda").to(wt) for m in (Hq, Hkv))
        NB = -(-T // B) + 3
        self.NB = NB
        slots = h.permutation(NB * B)[:T].astype(np.int64)
        if T > 3:
            slots[1], slots[2] = -1, NB * B + 5  # padding, and outside the pool
        self.slots = slots
        self.pos = h.integers(0, span, (A, T))
        self.axes = [int(x) for x in h.integers(0, A, rot // 2)]
        self.freq = pkv().rotary_frequencies(rot)
        self.table = pkv().rotary_table(span, self.freq)
        self.ks = self.vs = None
        if kind:
            self.ks, self.vs = ((torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.01)
                                for _ in range(2))
            ct = torch.uint8 if kind == "fp8" else torch.int8
            self.kc = torch.full((NB, Hkv, B, D), 3, dtype=ct, device="cuda")
            self.vc = torch.full((NB, Hkv, D, B), 3, dtype=ct, device="cuda")
        else:
            self.kc = torch.full((NB, Hkv, B, D), 7.0, dtype=dt, device="cuda")
            self.vc = torch.full((NB, Hkv, B, D), 7.0, dtype=dt, device="cuda")
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")

    def call(self, **kw):
        m = pkv()
        fn = getattr(m, "paged_norm_rotary_write" + ("_" + self.kind if self.kind else ""))
        scales = (self.ks, self.vs) if self.kind else ()
        args = dict(interleaved=self.inter, axes=self.axes if self.A > 1 else None)
        args.update(kw)
        pos = i32(self.pos if self.A > 1 else self.pos[0])
        return fn(self.q, self.k, self.v, self.qw, self.kw, self.eps, pos, self.table,
                  i32(self.slots), self.kc, self.vc, *scales, self.q_out, **args)

    def turned(self, x, w):
        """(value, bound before the last rounding) in fp64."""
        x = np64(x)
        wn = None if w is None else np64(w)
        y = osp.norm_rotate(x, wn, self.eps, np.zeros_like(self.pos), self.axes, self.freq.numpy(),
                            self.inter)  # the norm alone
        z = osp.norm_rotate(x, wn, self.eps, self.pos, self.axes, self.freq.numpy(), self.inter)
        rel = 0 if self.eps is None else ((self.D + 1) / 2 + 6) * U
        half, both = self.rot // 2, np.zeros_like(y)
        one, two = ((slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.inter
                    else (slice(0, half), slice(half, self.rot)))
        both[..., one] = both[..., two] = np.abs(y[..., one]) + np.abs(y[..., two])
        both[..., self.rot:] = np.abs(y[..., self.rot:])
        turn = np.zeros(self.D)
        turn[:self.rot] = 3 * U
        return z, (rel + turn) * both * (1 + 1e-3) + 1e-44

    def check(self):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kc0, vc0 = self.kc.clone(), self.vc.clone()
        r = self.call(status=status)
        assert r is self.q_out and int(status) == 0
        u = torch.finfo(self.dt).eps / 2
        tiny = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[self.dt]
        z, b = self.turned(self.q, self.qw)
        assert (np.abs(np64(self.q_out) - z) <= b + u * (np.abs(z) + b) + tiny).all()
        z, b = self.turned(self.k, self.kw)
        live = (self.slots >= 0) & (self.slots < self.NB * self.B)
        at, off = self.slots[live] // self.B, self.slots[live] % self.B
        kc, vc = self.kc.cpu().numpy() if self.kind else np64(self.kc), None
        k = kc[at, :, off]
        if not self.kind:
            assert (np.abs(k - z[live]) <= (b + u * (np.abs(z) + b) + tiny)[live]).all()
            v = np64(self.vc)[at, :, off]
            assert np.array_equal(v, np64(self.v)[live])
        else:
            quant = ofp8.quantize if self.kind == "fp8" else oint8.quantize
            value = ofp8.decode if self.kind == "fp8" else (lambda c: c.astype(np.float64))
            s = np64(self.ks)[None, :, None]
            lo, hi = quant(z[live] - b[live], s), quant(z[live] + b[live], s)
            assert (value(lo) <= value(k)).all() and (value(k) <= value(hi)).all()
            vc = self.vc.cpu().numpy()
            v = vc[at, :, :, V_POS[off]]
            assert np.array_equal(v, quant(np64(self.v)[live].astype(np.float32),
                                           np64(self.vs)[None, :, None]))
        # the other slots are as they were
        rest = np.ones(self.NB * self.B, dtype=bool)
        rest[self.slots[live]] = False
        rest = np.nonzero(rest)[0]
        rb, ro = (torch.as_tensor(x, device="cuda") for x in (rest // self.B, rest % self.B))
        assert torch.equal(self.kc[rb, :, ro], kc0[rb, :, ro])
        if self.kind:
            vp = torch.as_tensor(V_POS, device="cuda")[ro]
            assert torch.equal(self.vc[rb, :, :, vp], vc0[rb, :, :, vp])
        else:
            assert torch.equal(self.vc[rb, :, ro], vc0[rb, :, ro])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (128, 64), (256, 32), (128, 20),
                                   (96, 2), (80, 80), (8, 4), (256, 254)])
def test_shapes(dtype, inter, D, rot):
    if D * DT[dtype].itemsize % 16:
        pytest.skip("rows of whole 16 bytes")
    Case(37, 6, 2, D, rot, dtype, inter=inter, seed=D + rot).check()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter,D,rot", [(False, 128, 128), (True, 128, 64), (False, 64, 20),
                                         (True, 256, 256)])
def test_8_bit_caches(kind, dtype, inter, D, rot):
    Case(53, 4, 3, D, rot, dtype, kind=kind, inter=inter, fused=True).check()


@pytest.mark.parametrize("A", [2, 3, 4])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,kind", [("f32", ""), ("bf16", ""), ("f16", "fp8")])
def test_axes(A, inter, dtype, kind):
    Case(41, 4, 2, 128, 96, dtype, A=A, inter=inter, kind=kind).check()


@pytest.mark.parametrize("weight", ["same", "f32", None])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_weights(weight, per_head, dtype):
    Case(19, 5, 2, 128, 128, dtype, weight=weight, per_head=per_head).check()


@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_one_projection(offset, dtype):
    Case(33, 4, 2, 64, 64, dtype, fused=True, offset=offset).check()


@pytest.mark.parametrize("offset", [1, 3])
def test_8_bit_slices(offset):
    Case(33, 4, 2, 128, 128, "bf16", kind="int8", fused=True, offset=offset).check()


@pytest.mark.parametrize("T", [1, 2, 700, 3001])
def test_token_counts(T):
    Case(T, 8, 2, 128, 128, "bf16", fused=True, A=3).check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot,A", [(64, 64, 1), (128, 64, 2), (256, 256, 1), (96, 32, 4), (8, 8, 1)])
@pytest.mark.parametrize("weight,per_head", [("same", False), ("f32", True), (None, False)])
def test_many_tokens(dtype, inter, D, rot, A, weight, per_head):
    """Several tokens through each SM."""
    if D * DT[dtype].itemsize % 16:
        pytest.skip("rows of whole 16 bytes")
    Case(1300, 6, 2, D, rot, dtype, inter=inter, A=A, weight=weight, per_head=per_head).check()


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter,A", [(False, 3), (True, 1)])
def test_many_tokens_8_bit(kind, dtype, inter, A):
    Case(1500, 4, 3, 128, 64, dtype, kind=kind, inter=inter, fused=True, A=A).check()


def test_many_tokens_of_large_rows():
    Case(700, 128, 8, 256, 256, "bf16").check()
    Case(700, 32, 8, 128, 128, "f32").check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("inter,D,rot,A", [(False, 128, 128, 1), (False, 128, 48, 3),
                                           (True, 64, 64, 1), (True, 256, 128, 2),
                                           (False, 256, 256, 4), (True, 96, 40, 1),
                                           (False, 64, 16, 1)])
@pytest.mark.parametrize("weight,eps", [(None, 1e-6), ("f32", 1e-5), ("own", 0.0), (None, None)])
def test_a_prompt(dtype, inter, D, rot, A, weight, eps):
    """More tokens than CTAs, several of them through each."""
    Case(2501, 7, 3, D, rot, dtype, inter=inter, A=A, weight=weight, eps=eps, fused=True,
         seed=D + rot).check()


def test_a_prompt_of_many_heads():
    Case(1000, 80, 32, 128, 128, "bf16").check()
    Case(1000, 88, 32, 128, 128, "bf16").check()


def test_a_prompt_in_place_and_out_of_range():
    from paged_kv_cache_166_gb300 import _native as N
    c = Case(2000, 4, 2, 128, 128, "f16", A=2, fused=True)
    c.call()
    want, kc = c.q_out.clone(), c.kc.clone()
    c.kc.fill_(7.0)
    c.q_out = c.q
    q = c.q.clone()
    assert torch.equal(c.call(), want) and torch.equal(c.kc, kc)
    c.q.copy_(q)
    c.pos[0, 1900], c.pos[1, 3] = -1, 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.call(status=status).clone()
    assert int(status) == N.PKV_DEV_BAD_POSITION
    c.q.copy_(q)
    c.pos[0, 1900], c.pos[1, 3] = 0, 2999
    status.zero_()
    assert torch.equal(c.call(status=status), got) and int(status) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps", [None, 1e-5])
def test_a_tokens_bits_do_not_depend_on_how_many_come(dtype, inter, eps):
    """The same tokens in one call and by few at a time, and out of tensors at odd places."""
    c = Case(1000, 6, 2, 128, 64, dtype, inter=inter, eps=eps, A=2)
    c.call()
    q, kc, vc = c.q_out.clone(), c.kc.clone(), c.vc.clone()
    whole = c.q, c.k, c.v, c.q_out, c.pos, c.slots
    c.kc.fill_(7.0)
    c.vc.fill_(7.0)
    c.q_out.zero_()
    for a in range(0, 1000, 300):
        c.q, c.k, c.v, c.q_out = (x[a:a + 300] for x in whole[:4])
        c.pos, c.slots = whole[4][:, a:a + 300], whole[5][a:a + 300]
        c.call()
    assert torch.equal(whole[3], q) and torch.equal(c.kc, kc) and torch.equal(c.vc, vc)
    c.q, c.k, c.v, c.q_out, c.pos, c.slots = whole
    odd = torch.zeros((1000, 6 * 128 + 2), dtype=c.dt, device="cuda")[:, 2:].unflatten(1, (6, 128))
    odd.copy_(c.q)
    c.q = odd
    c.kc.fill_(7.0)
    c.q_out.zero_()
    c.call()
    assert torch.equal(c.q_out, q) and torch.equal(c.kc, kc)


@pytest.mark.parametrize("B", [1, 5, 8, 32])
def test_block_sizes(B):
    Case(70, 4, 2, 64, 64, "f16", B=B).check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_without_norm_it_is_the_rotary_write(dtype, inter):
    """The same bits as paged_rotary_write."""
    c = Case(45, 6, 2, 128, 64, dtype, inter=inter, eps=None)
    c.check()
    q, kc, vc = c.q_out.clone(), c.kc.clone(), c.vc.clone()
    c.kc.fill_(7.0)
    c.vc.fill_(7.0)
    pkv().paged_rotary_write(c.q, c.k, c.v, i32(c.pos[0]), c.table, i32(c.slots), c.kc, c.vc,
                             c.q_out, interleaved=inter)
    assert torch.equal(q, c.q_out) and torch.equal(kc, c.kc) and torch.equal(vc, c.vc)


def test_passing_bits_without_norm():
    c = Case(9, 2, 1, 64, 32, "bf16", eps=None)
    c.q[..., 40] = float("nan")
    c.v[0, 0, 3] = float("nan")
    c.call()
    assert torch.equal(c.q_out[..., 32:].view(torch.int16), c.q[..., 32:].view(torch.int16))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_bits_do_not_depend_on_alignment(dtype, inter):
    """The same tokens in tensors of their own and in slices at odd places."""
    c = Case(30, 4, 2, 128, 128, dtype, inter=inter)
    c.call()
    q, kc = c.q_out.clone(), c.kc.clone()
    n, off = 8, 2 if inter else 1
    x = torch.zeros((30, n * 128 + 6), dtype=c.dt, device="cuda")
    s = x[:, off:off + n * 128].unflatten(1, (n, 128))
    s[:, :4], s[:, 4:6], s[:, 6:] = c.q, c.k, c.v
    c.q, c.k, c.v = s[:, :4], s[:, 4:6], s[:, 6:]
    c.kc.fill_(7.0)
    c.call()
    assert torch.equal(q, c.q_out) and torch.equal(kc, c.kc)


def test_q_out_may_be_q():
    c = Case(20, 4, 2, 128, 128, "f16", fused=True)
    c.call()
    want = c.q_out.clone()
    c.q_out = c.q
    assert torch.equal(c.call(), want)


def test_large_and_small_values():
    """Squares summed in fp32: bf16 values up to 2^40, and a head of zeros."""
    c = Case(12, 3, 2, 128, 128, "bf16", scale=2.0 ** 40)
    c.check()
    c = Case(12, 3, 2, 128, 128, "bf16")
    c.q[3, 1] = 0
    c.k[5] = 0
    c.check()
    assert (c.q_out[3, 1] == 0).all()


def test_positions_out_of_range():
    from paged_kv_cache_166_gb300 import _native as N
    c = Case(12, 3, 2, 64, 64, "f16", A=3)
    c.pos[1, 4], c.pos[2, 5] = -3, 10 ** 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.call(status=status)
    assert int(status) == N.PKV_DEV_BAD_POSITION
    got = c.q_out.clone()
    c.pos[1, 4], c.pos[2, 5] = 0, 2999
    status.zero_()
    c.call(status=status)
    assert int(status) == 0 and torch.equal(got, c.q_out)


def test_refusals():
    c = Case(6, 2, 1, 64, 64, "f16")
    m = pkv()
    with pytest.raises(ValueError):
        c.call(axes=[0] * 32)          # positions [T] with axes
    c.eps = None
    with pytest.raises(ValueError):
        c.call()                       # weights without a norm
    c.eps = -1.0
    with pytest.raises(ValueError):
        c.call()
    c.eps = 1e-6
    keep = c.qw
    for w in (keep[:32], keep.double(), keep.cpu(), keep.float(), keep[None].repeat(2, 1)):
        c.qw = w
        with pytest.raises((ValueError, TypeError)):
            c.call()
    c.qw = keep
    c.pos = c.pos.repeat(2, axis=0)
    c.A = 2
    for axes in ([0] * 31, [0] * 31 + [2], [0] * 31 + [-1]):
        with pytest.raises((ValueError, m.PkvError)):
            c.call(axes=axes)
    c.call(axes=[0, 1] * 16)


def test_graph_and_stream():
    c = Case(64, 8, 2, 128, 128, "bf16", A=3)
    c.call()
    want = c.q_out.clone(), c.kc.clone()
    pos, slots = i32(c.pos), i32(c.slots)
    run = lambda: pkv().paged_norm_rotary_write(c.q, c.k, c.v, c.qw, c.kw, c.eps, pos, c.table,  # noqa: E731
                                                slots, c.kc, c.vc, c.q_out, axes=c.axes)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    c.q_out.zero_()
    c.kc.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, want[0]) and torch.equal(c.kc, want[1])
    c.q_out.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    st.synchronize()
    assert torch.equal(c.q_out, want[0])


def test_no_tokens():
    c = Case(4, 2, 1, 64, 64, "f16")
    kc = c.kc.clone()
    e = lambda x: x[:0]  # noqa: E731
    pkv().paged_norm_rotary_write(e(c.q), e(c.k), e(c.v), c.qw, c.kw, 1e-6, i32([]), c.table, i32([]),
                                  c.kc, c.vc, e(c.q_out))
    assert torch.equal(kc, c.kc)
