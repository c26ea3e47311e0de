"""Decode attention whose out lies on inputs of the cache write before it.

The attention starts while the write in front of it still runs.  A program's allocator may
hand it, as out, the memory of a projection that the write reads and nobody needs
afterwards: nothing may be written there, not the zero rows of empty contexts either, before
the write has read it.
"""
import numpy as np
import pytest
import torch

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


T, HQ, HKV, D, B, S, MAXB = 4096, 16, 16, 128, 16, 1024, 4
NB = T // B + MAXB


def tensors(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").half() for h in (HQ, HKV, HKV))
    caches = [torch.zeros((NB, HKV, B, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    tables = torch.zeros((S, MAXB), dtype=torch.int32, device="cuda")
    ctx = torch.zeros(S, dtype=torch.int32, device="cuda")
    ctx[S // 2] = 50
    tables[S // 2] = torch.arange(MAXB, device="cuda", dtype=torch.int32)
    return q, k, v, caches, slots, tables, ctx


@pytest.mark.parametrize("dead", [0, 1, 2])
@pytest.mark.parametrize("weights", [False, True])
def test_out_on_a_dead_projection_of_the_rotary_write(dead, weights):
    m = pkv()
    table = m.rotary_table(T, m.rotary_frequencies(D))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    for seed in range(5):
        q, k, v, caches, slots, tables, ctx = tensors(seed)
        want = [c.clone() for c in caches]
        turned = torch.empty_like(q)
        m.paged_rotary_write(q, k, v, pos, table, slots, *want, turned)
        q_s = turned[:S].clone()
        wanted_out = torch.empty_like(q_s)
        m.paged_decode_attention(q_s, *want, tables, ctx, 0.1, wanted_out)
        torch.cuda.synchronize()
        q_out = torch.empty_like(q)
        out = (q, k, v)[dead][-S:]  # the rows that are read last
        sums = torch.zeros((S, HKV, MAXB * B), device="cuda")
        torch.cuda.synchronize()
        m.paged_rotary_write(q, k, v, pos, table, slots, *caches, q_out)
        if weights:
            m.paged_decode_attention_weights(q_s, *caches, tables, ctx, 0.1, out, sums)
        else:
            m.paged_decode_attention(q_s, *caches, tables, ctx, 0.1, out)
        torch.cuda.synchronize()
        assert torch.equal(q_out, turned)
        assert all(torch.equal(a, b) for a, b in zip(caches, want))
        assert torch.equal(out, wanted_out)


@pytest.mark.parametrize("dead", [1, 2])
def test_out_on_dead_inputs_of_the_cache_write(dead):
    m = pkv()
    for seed in range(5):
        q, k, v, caches, slots, tables, ctx = tensors(10 + seed)
        want = [c.clone() for c in caches]
        m.paged_kv_write(k, v, slots, *want)
        q_s = q[:S].clone()
        wanted_out = torch.empty_like(q_s)
        m.paged_decode_attention(q_s, *want, tables, ctx, 0.1, wanted_out)
        torch.cuda.synchronize()
        out = (q, k, v)[dead][-S:]
        m.paged_kv_write(k, v, slots, *caches)
        m.paged_decode_attention(q_s, *caches, tables, ctx, 0.1, out)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(caches, want))
        assert torch.equal(out, wanted_out)
        empty = torch.from_numpy(np.delete(np.arange(S), S // 2)).cuda()
        assert not out[empty].any()
