"""GPU parity of the rotary table and of the cache write that turns q and k.

Bounds (fp32 arithmetic, each operation rounded once, u = 2^-24): cos and sin are off by
u each (rounded once from 64 bits, relative to 1), a product by u more, the sum by u, so
a turned element by at most 3 u (|x1| + |x2|) times the magnitude; one rounding to the
type adds half a step of the value.  8-bit codes are the quantisation of a value within
that bound: the code lies between the codes of its two ends.
"""
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import int8 as oint8
from oracle import rotary as orot

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
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


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, dtype, B=16, kind="", inter=False, fused=False,
                 scaling="none", seed=0, span=4096, offset=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        h = np.random.default_rng(seed)
        dt = DT[dtype]
        self.__dict__.update(T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, B=B, kind=kind, inter=inter, dt=dt)
        n = Hq + 2 * Hkv
        if fused:  # slices of one projection, `offset` elements into a row of n * D + pad
            width = n * D + (offset + 7) // 8 * 8 + 8
            x = torch.randn((T, width), generator=g, device="cuda").to(dt)
            x = x[:, offset:offset + n * D].unflatten(1, (n, D))
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = (torch.randn((T, m, D), generator=g, device="cuda").to(dt)
                                      for m in (Hq, Hkv, Hkv))
        NB = -(-T // B) + 3
        self.NB = NB
        slots = h.permutation(NB * B)[:T].astype(np.int64)
        if T > 3:
            slots[1], slots[2] = -1, NB * B + 5  # padding, and outside the pool
        self.slots = slots
        self.pos = h.integers(0, span, T)
        self.freq = pkv().rotary_frequencies(rot, 10000.0, scaling, 4.0, 512, 1.0, 4.0)
        self.span = span
        self.table = pkv().rotary_table(span, self.freq)
        if kind:
            self.ks, self.vs = ((torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.01)
                                for _ in range(2))
            ct = torch.uint8 if kind == "fp8" else torch.int8
            self.kc = torch.full((NB, Hkv, B, D), 3, dtype=ct, device="cuda")
            self.vc = torch.full((NB, Hkv, D, B), 3, dtype=ct, device="cuda")
        else:
            self.kc = torch.full((NB, Hkv, B, D), 7.0, dtype=dt, device="cuda")
            self.vc = torch.full((NB, Hkv, B, D), 7.0, dtype=dt, device="cuda")

    def run(self, q_out=None, status=None):
        out = torch.full((self.T, self.Hq, self.D), float("nan"), dtype=self.dt, device="cuda") \
            if q_out is None else q_out
        a = (self.q, self.k, self.v, i32(self.pos), self.table, i32(self.slots), self.kc, self.vc)
        m = pkv()
        if self.kind == "fp8":
            m.paged_rotary_write_fp8(*a, self.ks, self.vs, out, self.inter, status)
        elif self.kind == "int8":
            m.paged_rotary_write_int8(*a, self.ks, self.vs, out, self.inter, status)
        else:
            m.paged_rotary_write(*a, out, self.inter, status)
        torch.cuda.synchronize()
        return out

    def bound(self, x):
        """Absolute bound of the fp32 arithmetic, per element of x [T, H, D]."""
        x = np.abs(np64(x))
        out = np.zeros_like(x)
        r = self.rot
        one, two = ((slice(0, r, 2), slice(1, r, 2)) if self.inter
                    else (slice(0, r // 2), slice(r // 2, r)))
        s = 3 * U * (x[..., one] + x[..., two])
        out[..., one], out[..., two] = s, s
        return out

    def check(self, out):
        eps = torch.finfo(self.dt).eps / 2
        tiny = torch.finfo(self.dt).smallest_normal * eps  # half a step of the subnormals
        turn = lambda x: orot.rotate(np64(x), self.pos, self.freq.numpy(), self.inter)  # noqa: E731
        want, b = turn(self.q), self.bound(self.q)
        assert np.all(np.abs(np64(out) - want) <= (1 + eps) * b + eps * np.abs(want) + tiny)
        k, kb, v = turn(self.k), self.bound(self.k), np64(self.v)
        written = np.zeros((self.NB, self.B), dtype=bool)
        kc, vc = (c.cpu().numpy() if self.kind else np64(c) for c in (self.kc, self.vc))
        for i, s in enumerate(self.slots):
            if s < 0 or s >= self.NB * self.B:
                continue
            blk, off = divmod(int(s), self.B)
            written[blk, off] = True
            if not self.kind:
                assert np.all(np.abs(kc[blk, :, off] - k[i])
                              <= (1 + eps) * kb[i] + eps * np.abs(k[i]) + tiny)
                assert np.array_equal(vc[blk, :, off], v[i])
                continue
            o = ofp8 if self.kind == "fp8" else oint8
            ks, vs = (t.cpu().numpy()[:, None] for t in (self.ks, self.vs))
            got = o.decode(kc[blk, :, off])
            # the bound, and one fp32 rounding each for the value and the oracle's quotient
            d = kb[i] + 2 * U * np.abs(k[i])
            lo, hi = (o.decode(o.quantize(k[i] + sgn * d, ks)) for sgn in (-1, 1))
            assert np.all((got >= lo) & (got <= hi))
            vpos = ofp8.V_POS[off]
            assert np.array_equal(o.decode(vc[blk, :, :, vpos]), o.decode(o.quantize(v[i], vs)))
        # nothing else was touched
        fill = 3 if self.kind else 7.0
        mask = ~written
        assert np.all(kc.transpose(0, 2, 1, 3)[mask] == fill)
        if self.kind:
            back = vc[:, :, :, ofp8.V_POS]  # token order
            assert np.all(back.transpose(0, 3, 1, 2)[mask] == fill)
        else:
            assert np.all(vc.transpose(0, 2, 1, 3)[mask] == fill)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands"])
def test_table(scaling):
    f = pkv().rotary_frequencies(64, 10000.0, scaling, 8.0, 4096)
    P = 131072
    t = np64(pkv().rotary_table(P, f, magnitude=1.25))
    p = np.array([0, 1, 2, 511, 4095, 65537, P - 1])
    ang = p[:, None] * f.numpy()
    want = 1.25 * np.concatenate([np.cos(ang), np.sin(ang)], 1)
    # one rounding to fp32 of a 64-bit value, and the oracle's own 64-bit angle (2^-52 * 131072)
    assert np.all(np.abs(t[p] - want) <= 1.25 * (U + 2.0 ** -34))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,D,rot,B", [
    ("bf16", 128, 128, 16), ("f16", 128, 64, 8), ("bf16", 64, 64, 32), ("f16", 256, 256, 16),
    ("f32", 64, 64, 16), ("f32", 128, 32, 16),
    # rotary parts that 16-byte pieces do not divide
    ("bf16", 128, 20, 16), ("f16", 64, 2, 16), ("f32", 32, 6, 16), ("bf16", 256, 250, 16)])
def test_write_shapes(inter, dtype, D, rot, B):
    for T, Hq, Hkv in ((1, 8, 8), (37, 6, 2), (130, 8, 1)):
        c = Case(T, Hq, Hkv, D, rot, dtype, B=B, inter=inter, seed=T + D + rot)
        c.check(c.run())


@pytest.mark.parametrize("B", [1, 5, 24])
def test_block_sizes_that_are_no_power_of_two(B):
    for inter in (False, True):
        c = Case(50, 4, 2, 128, 128, "bf16", B=B, inter=inter, seed=B)
        c.check(c.run())


@pytest.mark.parametrize("dtype,D", [("f32", 4), ("bf16", 8), ("f16", 24), ("f32", 36)])
def test_small_and_odd_heads(dtype, D):
    for rot in sorted({2, max(2, D // 4 * 2), D}):
        for inter in (False, True):
            c = Case(21, 3, 1, D, rot, dtype, inter=inter, seed=D + rot)
            c.check(c.run())


def test_no_tokens():
    c = Case(4, 4, 2, 64, 64, "f16")
    c.T = 0
    c.q, c.k, c.v, c.pos, c.slots = c.q[:0], c.k[:0], c.v[:0], c.pos[:0], c.slots[:0]
    assert c.run().shape == (0, 4, 64)
    assert bool((c.kc == 7.0).all())


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,D,rot", [("bf16", 128, 128), ("f16", 256, 64), ("f32", 128, 96),
                                         ("bf16", 128, 36)])
def test_write_8bit(kind, inter, dtype, D, rot):
    for T, Hq, Hkv in ((1, 4, 4), (67, 8, 2)):
        c = Case(T, Hq, Hkv, D, rot, dtype, kind=kind, inter=inter, seed=T + rot)
        c.check(c.run())


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_codes_are_those_of_the_cache_write(kind, dtype):
    """Every 16-bit pattern (fp32: magnitudes over the whole range, and quotients next to the
    codes' borders) as V, over scales up to the extreme: the bytes paged_kv_write leaves."""
    m, Hkv, D = pkv(), 8, 128
    scales = torch.tensor([0.01, 1.0, 3.0, 448.0, 1e-30, 1e30, 2.0 ** -70, 1.7e-5], device="cuda")
    if dtype == "f32":
        g = torch.Generator(device="cuda")
        g.manual_seed(0)
        x = torch.randint(-2 ** 31, 2 ** 31, (128, Hkv, D), generator=g, device="cuda",
                          dtype=torch.int64).to(torch.int32).view(torch.float32)
        # k / 32 times the scale: ties of the codes among them, and their neighbours
        k = torch.randint(-1024 * 32, 1024 * 32, (384, Hkv, D), generator=g, device="cuda") / 32.0
        y = k * scales[:, None]
        y = torch.nextafter(y, y + torch.randint(-1, 2, y.shape, generator=g, device="cuda") * y.abs())
        v = torch.cat([x, y])
    else:
        v = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
        v = v.view(DT[dtype]).view(512, 1, D).expand(512, Hkv, D).contiguous()
    T = v.shape[0]
    k = torch.zeros_like(v)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    ct = torch.uint8 if kind == "fp8" else torch.int8
    caches = [[torch.zeros((T // 16, Hkv) + s, dtype=ct, device="cuda") for s in ((16, D), (D, 16))]
              for _ in range(2)]
    freq = m.rotary_frequencies(D)
    table, pos = m.rotary_table(4, freq), torch.zeros(T, dtype=torch.int32, device="cuda")
    getattr(m, "paged_rotary_write_" + kind)(k, k, v, pos, table, slots, *caches[0], scales, scales,
                                             torch.empty_like(k))
    getattr(m, "paged_kv_write_" + kind)(k, v, slots, *caches[1], scales, scales)
    torch.cuda.synchronize()
    assert torch.equal(caches[0][1].view(torch.uint8), caches[1][1].view(torch.uint8))


@pytest.mark.parametrize("kind", ["", "fp8", "int8"])
@pytest.mark.parametrize("T,first", [(16, 0), (64, 0), (83, 5), (40, 15), (33, 16), (7, 9)])
def test_prompt_order(kind, T, first):
    """Consecutive tokens in consecutive slots of permuted blocks, starting anywhere in one."""
    c = Case(T, 4, 2, 128, 128, "bf16", kind=kind, seed=T)
    order = np.random.default_rng(T).permutation(c.NB)
    p = np.arange(T) + first
    c.slots = order[p // 16] * 16 + p % 16
    c.check(c.run())


@pytest.mark.parametrize("kind", ["", "fp8"])
@pytest.mark.parametrize("offset", [0, 8, 3, 2])
def test_write_strided(kind, offset):
    """Slices of a fused projection, aligned to 16 bytes or not."""
    for inter in (False, True):
        if inter and offset % 2:
            continue
        c = Case(45, 8, 2, 128, 64, "bf16", kind=kind, inter=inter, fused=True, offset=offset)
        assert not c.q.is_contiguous()
        c.check(c.run())


def test_interleaved_refuses_odd_alignment():
    c = Case(5, 8, 2, 128, 64, "bf16", inter=True, fused=True, offset=3)
    with pytest.raises(pkv().PkvError, match="interleaved"):
        c.run()


def test_in_place_equals_out_of_place():
    for fused in (False, True):
        a, b = (Case(70, 8, 2, 128, 96, "f16", fused=fused, seed=5) for _ in range(2))
        want = a.run()
        got = b.run(q_out=b.q)
        assert torch.equal(got, want) and torch.equal(a.kc, b.kc) and torch.equal(a.vc, b.vc)


def test_plain_angle_zero_and_passing_elements_keep_their_bits():
    c = Case(9, 4, 2, 128, 64, "bf16", seed=1)
    c.pos[:] = 0
    c.q[0, 0, 64:68] = torch.tensor([float("nan"), float("inf"), -0.0, 1.0], device="cuda")
    out = c.run()
    assert torch.equal(out.view(torch.int16), c.q.view(torch.int16))


def test_bad_positions_are_clamped_and_reported():
    c = Case(6, 4, 2, 64, 64, "f32", span=100)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.run(status=st)
    assert int(st) == 0
    c.pos = np.array([5, 100, -1, 99, 1 << 30, 0])
    c.run(status=st)
    assert int(st) == 16
    c.pos = np.clip(c.pos, 0, 99)
    want = Case(6, 4, 2, 64, 64, "f32", span=100)
    want.pos = c.pos
    assert torch.equal(c.run(), want.run())


def test_far_positions():
    c = Case(33, 4, 2, 128, 128, "f32", span=1 << 20, seed=3)
    c.pos[:4] = (1 << 20) - 1 - np.arange(4)
    out = c.run()
    # the oracle's own angle: 2^20 * 2^-53 relative to 1
    want = orot.rotate(np64(c.q), c.pos, c.freq.numpy())
    assert np.all(np.abs(np64(out) - want) <= c.bound(c.q) * (1 + 2.0 ** -6) + U * np.abs(want))


def test_write_equals_rotation_then_kv_write():
    """The joined write leaves the bits of turning first and paged_kv_write after."""
    c = Case(50, 8, 4, 128, 128, "bf16", seed=8)
    c.run()
    d = Case(50, 8, 4, 128, 128, "bf16", seed=8)
    scratch = torch.empty_like(d.k)
    # k turned as if it were q (its cache rows are thrown away)
    pkv().paged_rotary_write(d.k, d.k, d.v, i32(d.pos), d.table, i32(np.full(50, -1)),
                             d.kc.clone(), d.vc.clone(), scratch)
    pkv().paged_kv_write(scratch, d.v, i32(d.slots), d.kc, d.vc)
    torch.cuda.synchronize()
    assert torch.equal(c.kc, d.kc) and torch.equal(c.vc, d.vc)


def test_many_tokens_of_a_row_past_32_bit_offsets():
    """Token offsets above 2^31 elements of a strided projection."""
    T, D, width = 2, 128, (1 << 31) + 1024
    x = torch.zeros(width + 3 * D, dtype=torch.float16, device="cuda")
    q = x.as_strided((T, 1, D), (width, D, 1))
    k = x.as_strided((T, 1, D), (width, D, 1), D)
    v = x.as_strided((T, 1, D), (width, D, 1), 2 * D)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    for t in (q, k, v):
        t.copy_(torch.randn((T, 1, D), generator=g, device="cuda").half())
    c = Case(2, 1, 1, D, D, "f16")
    c.q, c.k, c.v = q, k, v
    c.check(c.run())


def test_two_streams_and_a_captured_graph():
    cases = [Case(40, 8, 2, 128, 128, "bf16", seed=s) for s in (1, 2)]
    want = [Case(40, 8, 2, 128, 128, "bf16", seed=s) for s in (1, 2)]
    refs = [w.run() for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.empty_like(r) for r in refs]
    idx = [(i32(c.pos), i32(c.slots)) for c in cases]
    torch.cuda.synchronize()
    for c, s, o, (p, sl) in zip(cases, streams, outs, idx):
        with torch.cuda.stream(s):
            pkv().paged_rotary_write(c.q, c.k, c.v, p, c.table, sl, c.kc, c.vc, o)
    torch.cuda.synchronize()
    for c, w, o, r in zip(cases, want, outs, refs):
        assert torch.equal(o, r) and torch.equal(c.kc, w.kc) and torch.equal(c.vc, w.vc)
    c, (p, sl) = cases[0], idx[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv().paged_rotary_write(c.q, c.k, c.v, p, c.table, sl, c.kc, c.vc, outs[0])
    outs[0].zero_()
    c.kc.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], refs[0]) and torch.equal(c.kc, want[0].kc)


def test_python_refusals():
    c = Case(4, 4, 2, 64, 64, "f16")
    m, p, s = pkv(), i32(c.pos), i32(c.slots)
    out = torch.empty_like(c.q)

    def call(**kw):
        a = dict(q=c.q, k=c.k, v=c.v, positions=p, table=c.table, slot_mapping=s, k_cache=c.kc,
                 v_cache=c.vc, q_out=out)
        a.update(kw)
        m.paged_rotary_write(**a)
    for kw, err in ((dict(positions=p.long()), TypeError), (dict(slot_mapping=s[:3]), ValueError),
                    (dict(q=c.q.float()), TypeError), (dict(k=c.k[:, :1]), ValueError),
                    (dict(q=c.q.cpu()), ValueError), (dict(table=c.table.double()), ValueError),
                    (dict(table=c.table[:, ::2]), ValueError),
                    (dict(q=c.q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(k=c.k[:1].expand(4, 2, 64)), m.PkvError),
                    (dict(status=torch.zeros(1, device="cuda")), ValueError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(ValueError):
        m.rotary_table(0, c.freq)
    with pytest.raises(ValueError):
        m.rotary_table(8, c.freq.float())
    assert math.isfinite(float(out.float().nan_to_num().sum()))
