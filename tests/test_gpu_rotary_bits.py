"""Rotary arithmetic bit for bit: products and sums of fp32, each rounded once.

The formula is computed by torch operations of one rounding each, from the library's own
table, so its results are the ones the library states; whatever path a call takes (16-byte
pieces or small ones, half layout or interleaved) has to give the same bits.
"""
import numpy as np
import pytest
import torch

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


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def turned(x, pos, table, inter):
    """x [T, H, D] turned, in fp32: every product, and every sum, a rounding of its own."""
    y = x.float().clone()
    half = table.shape[1] // 2
    row = table[pos.long()][:, None]
    c, s = row[..., :half], row[..., half:]
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter
                else (slice(0, half), slice(half, 2 * half)))
    a, b = x.float()[..., one], x.float()[..., two]
    ac, bs, bc, asn = a * c, b * s, b * c, a * s
    y[..., one], y[..., two] = ac - bs, bc + asn
    return y


def inputs(dtype, T, Hq, Hkv, D, offset, seed):
    """q, k, v as slices of one projection, `offset` elements off a 16-byte boundary."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = (Hq + 2 * Hkv) * D
    x = torch.zeros((T, n + 16), dtype=DT[dtype], device="cuda")
    x[:, offset:offset + n] = torch.randn((T, n), generator=g, device="cuda").to(DT[dtype])
    h = x[:, offset:offset + n].unflatten(1, (Hq + 2 * Hkv, D))
    return h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:]


T, HQ, HKV = 333, 8, 2


def setup(rot, seed):
    m = pkv()
    table = m.rotary_table(4096, m.rotary_frequencies(rot))
    r = np.random.default_rng(seed)
    pos = torch.from_numpy(r.integers(0, 4096, T).astype(np.int32)).cuda()
    slots = torch.from_numpy(r.permutation(T + 19)[:T].astype(np.int32)).cuda()
    return table, pos, slots, (T + 19) // 16 + 1


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (128, 20)])
def test_every_path_gives_the_formulas_bits(dtype, inter, D, rot):
    table, pos, slots, NB = setup(rot, D + rot)
    for offset in (0, 2) if inter else (0, 1):  # 16-byte pieces, and small ones
        q, k, v = inputs(dtype, T, HQ, HKV, D, offset, 5)
        kc, vc = (torch.zeros((NB, HKV, 16, D), dtype=DT[dtype], device="cuda") for _ in range(2))
        out = torch.empty((T, HQ, D), dtype=DT[dtype], device="cuda")
        pkv().paged_rotary_write(q, k, v, pos, table, slots, kc, vc, out, inter)
        s = slots.long()
        assert torch.equal(bits(out), bits(turned(q, pos, table, inter).to(DT[dtype])))
        assert torch.equal(bits(kc[s // 16, :, s % 16]),
                           bits(turned(k, pos, table, inter).to(DT[dtype])))


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_codes_of_the_turned_k_are_those_of_the_formula(kind, dtype, inter):
    """k's codes: what paged_kv_write leaves of the formula's fp32 values."""
    D, m = 128, pkv()
    table, pos, slots, NB = setup(D, 9)
    ks, vs = (torch.rand(HKV, device="cuda") * 0.02 + 0.01 for _ in range(2))
    ct = torch.uint8 if kind == "fp8" else torch.int8
    caches = [[torch.zeros((NB, HKV) + s, dtype=ct, device="cuda") for s in ((16, D), (D, 16))]
              for _ in range(2)]
    for offset in (0, 2) if inter else (0, 1):
        q, k, v = inputs(dtype, T, HQ, HKV, D, offset, 6)
        out = torch.empty((T, HQ, D), dtype=DT[dtype], device="cuda")
        getattr(m, "paged_rotary_write_" + kind)(q, k, v, pos, table, slots, *caches[0], ks, vs,
                                                 out, inter)
        getattr(m, "paged_kv_write_" + kind)(turned(k, pos, table, inter),
                                             v.float().contiguous(), slots, *caches[1], ks, vs)
        assert torch.equal(bits(caches[0][0]), bits(caches[1][0]))
        assert torch.equal(bits(caches[0][1]), bits(caches[1][1]))
