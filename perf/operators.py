"""Cases, plain forms and calls of the operators around a decode step of the paged cache.

* rotary: rotary positions of q and k, k and v written into the paged cache
  (``paged_rotary_write``, ``paged_rotary_write_fp8``);
* weights: decode attention that also adds each cached token's attention weight to a
  running sum (``paged_decode_attention_weights`` and its fp8 form);
* evict: the tokens with the largest sums picked for every KV head, their rows moved
  into fresh blocks (``paged_evict_select``, ``paged_evict_gather``);
* beam: one beam-search selection over beams and vocabulary (``beam_select``).

``own`` false: the plain forms, in elementary torch operations.  ``own`` true: the calls a
user makes of the package.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# byte of token t (0..15) inside a 16-byte row of a transposed 8-bit V tile
V_POS = [0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15]


# ---------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a 70B-shaped batch: latency, scaled positions of long contexts
        rotary("rotary_step_70b_bf16", T=256, Hq=64, Hkv=8, D=128, rot=128, dtype="bf16",
               scaling="bands", factor=8.0, span=131072, interleaved=False, fused=False),
        # packed prompt of a 13B-shaped model, part of the head, slices of one projection
        rotary("rotary_prompt_13b_f16", T=8191, Hq=40, Hkv=40, D=128, rot=64, dtype="f16",
               scaling="none", factor=1.0, span=8192, interleaved=True, fused=True),
        # prompt chunk into an fp8 cache, grouped heads
        rotary("rotary_prompt_fp8", T=4099, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
               cache="fp8", scaling="linear", factor=4.0, span=32768, interleaved=False,
               fused=True),
        # the smallest call: four short contexts, fp32
        weights("weights_tiny_f32", S=4, Hq=4, Hkv=4, D=64, dtype="f32", kind="fixed", lo=1,
                hi=100, lens_seed=0),
        # 13B-shaped decode batch, one head a group
        weights("weights_13b_f16", S=64, Hq=40, Hkv=40, D=128, dtype="f16", kind="lognormal",
                lo=1, hi=2048, median=300.0, sigma=1.0, lens_seed=1),
        # 70B-shaped decode batch
        weights("weights_70b_bf16", S=256, Hq=64, Hkv=8, D=128, dtype="bf16", kind="lognormal",
                lo=1, hi=8192, median=1024.0, sigma=1.2, lens_seed=2),
        # few long contexts over an fp8 cache
        weights("weights_long_fp8", S=8, Hq=64, Hkv=8, D=128, dtype="bf16", cache="fp8",
                kind="uniform", lo=32768, hi=131072, lens_seed=4),
        # a 13B-shaped batch cut down to a budget of 256 tokens
        evict("evict_13b_f16", S=64, Hkv=40, D=128, dtype="f16", kind="lognormal", lo=1, hi=2048,
              median=300.0, sigma=1.0, lens_seed=1, keep=256, first=4, recent=32),
        # long contexts cut down to 4096 tokens
        evict("evict_long_bf16", S=8, Hkv=8, D=128, dtype="bf16", kind="uniform", lo=32768,
              hi=131072, lens_seed=4, keep=4096, first=4, recent=256),
        # one request, four beams
        beam("beam_one_f32", S=1, K=4, V=32000, N=8, dtype="f32"),
        # a batch with an odd vocabulary in 16 bits
        beam("beam_odd_f16", S=32, K=4, V=65537, N=8, dtype="f16"),
        # a large batch and vocabulary in 32 bits
        beam("beam_large_f32", S=64, K=8, V=131072, N=16, dtype="f32"),
    ]


def rotary(name=None, **c):
    return _case("rotary", name, dict(cache="same", B=16, base=10000.0), c)


def weights(name=None, **c):
    return _case("weights", name, dict(cache="same", B=16, median=0.0, sigma=0.0), c)


def evict(name=None, **c):
    return _case("evict", name, dict(cache="same", B=16, median=0.0, sigma=0.0), c)


def beam(name=None, **c):
    return _case("beam", name, {}, c)


def _case(op, name, defaults, c):
    out = {"op": op, **defaults, **c}
    if name is not None:
        out["name"] = name
    return out


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotary", "weights", "evict", "beam"])
    if op == "beam":
        K = _log(rng, 1, 16)
        V = _log(rng, 1000, 160000)
        S = _log(rng, 1, max(1, min(64, (1 << 26) // (K * V))))
        return beam(S=S, K=K, V=V, N=rng.choice([K, 2 * K]),
                    dtype=rng.choice(["f32", "f16", "bf16"]))
    Hkv = rng.choice([1, 2, 4, 8, 16, 40])
    G = rng.choice([1, 2, 4, 8]) if Hkv < 40 else 1
    cache = rng.choice(["same", "same", "fp8"])
    if cache == "fp8":
        D, dtype, B = 128, rng.choice(["f16", "bf16"]), 16
    else:
        dtype = rng.choice(["f32", "f16", "bf16"])
        D = rng.choice([64, 128]) if dtype == "f32" else rng.choice([64, 128, 256])
        B = 16 if dtype == "f32" else rng.choice([8, 16, 32])
    if op == "rotary":
        most = max(2, min(16384, (1 << 28) // ((G + 2) * Hkv * D * 4)))
        rot = rng.choice([D, D // 2, D // 4])
        return rotary(T=_log(rng, 1, most), Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, dtype=dtype,
                      cache=cache, B=B, base=rng.choice([10000.0, 500000.0]),
                      scaling=rng.choice(["none", "linear", "ntk", "bands"]),
                      factor=rng.choice([2.0, 4.0, 8.0]), span=_log(rng, 16384, 131072),
                      interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
    hi = _log(rng, 1, 65536)
    row = Hkv * D * 2 * (4 if dtype == "f32" else 2)
    S = _log(rng, 1, max(1, min(256, int(1.2e9) // (row * hi))))
    common = dict(S=S, Hkv=Hkv, D=D, dtype=dtype, cache=cache, B=B, kind="uniform",
                  lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, lens_seed=rng.randrange(1 << 20))
    if op == "weights":
        return weights(Hq=Hkv * G, **common)
    keep = _log(rng, 1, max(1, hi))
    return evict(keep=keep, first=min(4, keep), recent=rng.choice([0, keep // 8, keep // 2]),
                 **common)


def lens_of(case):
    """The batch's context lengths: they belong to the case, not to the seed of its values."""
    g = np.random.default_rng(case["lens_seed"])
    S, lo, hi = case["S"], case["lo"], case["hi"]
    if case["kind"] == "fixed":  # spread evenly over the range
        x = np.linspace(lo, hi, S)
    elif case["kind"] == "lognormal":
        x = g.lognormal(math.log(case["median"]), case["sigma"], S)
    else:
        x = g.integers(lo, hi, S, endpoint=True)
    return np.clip(np.rint(x), lo, hi).astype(np.int64)


def work(case):
    op = case["op"]
    if op == "beam":
        S, K, V, N = case["S"], case["K"], case["V"], case["N"]
        elt = 4 if case["dtype"] == "f32" else 2
        return {"bytes": S * K * V * elt + 4 * S * K + 12 * S * N, "flops": 4.0 * S * K * V}
    elt = 4 if case["dtype"] == "f32" else 2
    celt = 1 if case["cache"] == "fp8" else elt
    Hkv, D = case["Hkv"], case["D"]
    if op == "rotary":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        move = T * D * (2 * Hq * elt + 2 * Hkv * (elt + celt))
        return {"bytes": move + T * (rot * 4 + 8), "flops": 3.0 * T * (Hq + Hkv) * rot}
    lens = lens_of(case)
    tokens = int(lens.sum())
    tables = int((-(-lens // case["B"])).sum()) * 4
    if op == "weights":
        Hq, S = case["Hq"], case["S"]
        b = 2 * tokens * Hkv * D * celt + 8 * tokens * Hkv + 2 * S * Hq * D * elt + tables
        return {"bytes": b, "flops": 4.0 * tokens * Hq * D}
    n = int(np.minimum(lens, case["keep"]).sum())
    b = 4 * tokens * Hkv + 8 * n * Hkv + 4 * n * Hkv * D * celt + tables
    return {"bytes": b, "flops": float(tokens * Hkv)}


# ---------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _filled(shape, dtype, g):
    """A pool of N(0,1) values, drawn in pieces so that it needs no fp32 copy of its size."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for i in range(0, shape[0], 4096):
        t[i:i + 4096] = _randn(t[i:i + 4096].shape, g, dtype)
    return t


def _fp8_pool(shape, scale, g):
    """E4M3 codes of N(0,1) values over their head's scale, as bytes."""
    t = torch.empty(shape, dtype=torch.uint8, device="cuda")
    inv = (1.0 / scale).view((1, -1) + (1,) * (len(shape) - 2))
    for i in range(0, shape[0], 4096):
        x = (_randn(t[i:i + 4096].shape, g) * inv).clamp(-448.0, 448.0)
        t[i:i + 4096] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return t


def _caches(case, NB, g):
    """{kc, vc, ks, vs}: K and V pools; the scales are None unless the cache is 8-bit."""
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    if case["cache"] == "fp8":
        ks, vs = ((torch.rand(Hkv, generator=g, device="cuda") * 3 + 3) / 448.0 for _ in range(2))
        return {"kc": _fp8_pool((NB, Hkv, B, D), ks, g), "vc": _fp8_pool((NB, Hkv, D, B), vs, g),
                "ks": ks, "vs": vs}
    dt = DTYPES[case["dtype"]]
    return {"kc": _filled((NB, Hkv, B, D), dt, g), "vc": _filled((NB, Hkv, B, D), dt, g),
            "ks": None, "vs": None}


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def frequencies(case):
    """Angle per position of each pair of elements, in 64 bits."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    i = np.arange(0, rot, 2, dtype=np.float64)
    if case["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2.0))
    inv = base ** (-i / rot)
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "bands":  # long wavelengths stretched, short ones kept
        turns = 4096.0 * inv / (2 * math.pi)
        t = np.clip((turns - 1.0) / 3.0, 0.0, 1.0)
        inv = inv * ((1 - t) / f + t)
    return inv


def prepare(case, seed):
    g, h = _gen(seed), np.random.default_rng(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "beam":
        S, K, V, N = case["S"], case["K"], case["V"], case["N"]
        x = _randn((S, K, V), g) * 2.5
        x[torch.rand((S, K, V), generator=g, device="cuda") < 0.01] = -math.inf  # banned tokens
        st["logits"] = x.to(DTYPES[case["dtype"]])
        st["beam_scores"] = -8.0 * torch.rand((S, K), generator=g, device="cuda")
        st["scores"] = torch.empty((S, N), dtype=torch.float32, device="cuda")
        st["beams"] = torch.empty((S, N), dtype=torch.int32, device="cuda")
        st["tokens"] = torch.empty((S, N), dtype=torch.int32, device="cuda")
        return st
    B, Hkv, D, dt = case["B"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    if op == "rotary":
        T, Hq = case["T"], case["Hq"]
        NB = -(-T // B) + max(1, T // (10 * B))
        st.update(_caches(case, NB, g))
        x = _randn((T, Hq + 2 * Hkv, D), g, dt)
        parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        st["q"], st["k"], st["v"] = parts if case["fused"] else (p.contiguous() for p in parts)
        # one packed prompt's positions, or for short batches one far position a sequence
        start = 0 if T > 512 else None
        pos = np.arange(T) + start if start is not None else h.integers(0, case["span"], T)
        st["positions"] = _i32(pos % case["span"])
        # consecutive tokens fill whole blocks of a pool in random order
        order = h.permutation(NB)
        st["slots"] = _i32(order[np.arange(T) // B] * B + np.arange(T) % B)
        st["freq"] = torch.from_numpy(frequencies(case)).cuda()
        ang = torch.arange(case["span"], device="cuda", dtype=torch.float64)[:, None] * st["freq"]
        st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        return st
    lens = lens_of(case)
    S, nb = case["S"], -(-lens // B)
    n_new = -(-min(case["keep"], int(lens.max())) // B) if op == "evict" else 0
    NB = int(nb.sum() + S * n_new) + max(1, int(nb.sum()) // 10)
    order = h.permutation(NB)
    tables = np.zeros((S, int(nb.max())), dtype=np.int64)
    at = 0
    for s in range(S):
        tables[s, :nb[s]] = order[at:at + nb[s]]
        at += nb[s]
    st["tables"], st["ctx"] = _i32(tables), _i32(lens)
    st.update(_caches(case, NB, g))
    W = tables.shape[1] * B
    if op == "weights":
        Hq = case["Hq"]
        st["q"] = (_randn((S, Hq, D), g) * 1.5).to(dt)
        st["scale"] = 1.0 / math.sqrt(D)
        st["out"] = torch.empty_like(st["q"])
        # a few steps' weights so far: about 1 / length a head and step
        st["sums"] = torch.rand((S, Hkv, W), generator=g, device="cuda") * \
            (4.0 * (Hq // Hkv) / st["ctx"].float())[:, None, None]
        return st
    # accumulated weights: a long tail, and tokens whose weight was always zero
    sums = torch.exp(2.0 * _randn((S, Hkv, W), g))
    sums[torch.rand((S, Hkv, W), generator=g, device="cuda") < 0.05] = 0.0
    st["sums"] = sums
    K = min(case["keep"], int(lens.max()))
    st["keep"] = _i32(np.full(S, case["keep"]))
    st["new_tables"] = _i32(order[at:at + S * n_new].reshape(S, n_new))
    st["kept"] = torch.zeros((S, Hkv, K), dtype=torch.int32, device="cuda")
    st["new_sums"] = torch.zeros((S, Hkv, n_new * B), dtype=torch.float32, device="cuda")
    st["new_lens"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        return {"rotary": own_rotary, "weights": own_weights, "evict": own_evict,
                "beam": own_beam}[op](state)
    return {"rotary": plain_rotary, "weights": plain_weights, "evict": plain_evict,
            "beam": plain_beam}[op](state)


def _cache_out(st):
    """The caches as the values they hold (8-bit ones as the codes' own type)."""
    if st["ks"] is not None:
        return {"kc": st["kc"].view(torch.float8_e4m3fn), "vc": st["vc"].view(torch.float8_e4m3fn)}
    return {"kc": st["kc"], "vc": st["vc"]}


def own_rotary(st):
    import paged_kv_cache_166_gb300 as pkv
    c = st["case"]
    if st["ks"] is not None:
        pkv.paged_rotary_write_fp8(st["q"], st["k"], st["v"], st["positions"], st["table"],
                                   st["slots"], st["kc"], st["vc"], st["ks"], st["vs"],
                                   st["q_out"], interleaved=c["interleaved"])
    else:
        pkv.paged_rotary_write(st["q"], st["k"], st["v"], st["positions"], st["table"],
                               st["slots"], st["kc"], st["vc"], st["q_out"],
                               interleaved=c["interleaved"])
    return {"q": st["q_out"], **_cache_out(st)}


def own_weights(st):
    import paged_kv_cache_166_gb300 as pkv
    if st["ks"] is not None:
        pkv.paged_decode_attention_weights_fp8(
            st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["ctx"], st["scale"],
            st["out"], st["sums"])
    else:
        pkv.paged_decode_attention_weights(st["q"], st["kc"], st["vc"], st["tables"], st["ctx"],
                                           st["scale"], st["out"], st["sums"])
    return {"out": st["out"], "sums": st["sums"]}


def own_evict(st):
    import paged_kv_cache_166_gb300 as pkv
    c = st["case"]
    pkv.paged_evict_select(st["sums"], st["ctx"], st["keep"], st["kept"], st["new_sums"],
                           st["new_lens"], first=c["first"], recent=c["recent"])
    pkv.paged_evict_gather(st["kc"], st["vc"], st["tables"], st["kept"], st["new_lens"],
                           st["new_tables"])
    return {"kept": st["kept"], "sums": st["new_sums"], "lens": st["new_lens"], **_cache_out(st)}


def own_beam(st):
    import paged_kv_cache_166_gb300 as pkv
    pkv.beam_select(st["logits"], st["beam_scores"], st["scores"], st["beams"], st["tokens"])
    return {"scores": st["scores"], "beams": st["beams"], "tokens": st["tokens"]}


def plain_rotary(st):
    c = st["case"]
    rot, B = c["rot"], c["B"]
    ang = st["positions"].double()[:, None] * st["freq"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turned(x):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    st["q_out"].copy_(turned(st["q"]))
    block, at = (st["slots"] // B).long(), (st["slots"] % B).long()
    k, v = turned(st["k"]), st["v"].float()
    if st["ks"] is None:
        st["kc"][block, :, at] = k.to(st["kc"].dtype)
        st["vc"][block, :, at] = v.to(st["vc"].dtype)
    else:
        vpos = torch.tensor(V_POS, device="cuda")[at]
        code = lambda x, s: (x / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)  # noqa: E731
        st["kc"][block, :, at] = code(k, st["ks"]).view(torch.uint8)
        st["vc"][block, :, :, vpos] = code(v, st["vs"]).view(torch.uint8)
    return {"q": st["q_out"], **_cache_out(st)}


def _gathered(st):
    """K and V of every sequence in fp32, [S, Hkv, L, D], L the padded length."""
    t = st["tables"].long()
    k, v = st["kc"][t], st["vc"][t]  # [S, MAXB, Hkv, ., .]
    if st["ks"] is not None:
        vpos = torch.tensor(V_POS, device="cuda")
        k = k.view(torch.float8_e4m3fn).float() * st["ks"][:, None, None]
        v = v[..., vpos].transpose(-1, -2).contiguous().view(torch.float8_e4m3fn).float()
        v = v * st["vs"][:, None, None]
    k, v = k.transpose(1, 2).flatten(2, 3).float(), v.transpose(1, 2).flatten(2, 3).float()
    return k, v


def plain_weights(st):
    c = st["case"]
    S, Hq, Hkv, D = c["S"], c["Hq"], c["Hkv"], c["D"]
    k, v = _gathered(st)
    L = k.shape[2]
    there = torch.arange(L, device="cuda") < st["ctx"][:, None]  # [S, L]
    q = st["q"].float().view(S, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    x = torch.where(there[:, None, None], x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    e = torch.where(there[:, None, None], torch.exp(x - top), torch.zeros_like(x))
    total = e.sum(-1, keepdim=True)
    w = e / torch.where(total > 0, total, torch.ones_like(total))
    st["out"].copy_(torch.matmul(w, v).view(S, Hq, D))
    st["sums"][:, :, :L] += w.sum(2)
    return {"out": st["out"], "sums": st["sums"]}


def plain_evict(st):
    c = st["case"]
    B, first, recent = c["B"], c["first"], c["recent"]
    S, Hkv, W = st["sums"].shape
    K = st["kept"].shape[2]
    pos = torch.arange(W, device="cuda")
    ctx = st["ctx"].long()
    n = torch.minimum(ctx, st["keep"].long()).clamp(max=K)
    r = n.clamp(max=recent)
    f = torch.minimum(n - r, torch.full_like(n, first))
    forced = (pos < f[:, None]) | ((pos >= (ctx - r)[:, None]) & (pos < ctx[:, None]))
    rank = torch.where(forced, 0, torch.where(pos < ctx[:, None], 1, 2))[:, None].expand(S, Hkv, W)
    key = torch.where(torch.isnan(st["sums"]), torch.full_like(st["sums"], -math.inf), st["sums"])
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, stable=True).indices)
    taken = torch.where(torch.arange(K, device="cuda") < n[:, None, None], order[..., :K], W)
    idx = torch.sort(taken, dim=-1).values  # ascending, the absent ones (W) last
    live = idx < W
    idx = torch.where(live, idx, 0)
    st["kept"].copy_(torch.where(live, idx, st["kept"].long()))
    st["new_sums"][..., :K] = torch.where(live, st["sums"].gather(-1, idx), st["new_sums"][..., :K])
    st["new_lens"].copy_(n)
    head = torch.arange(Hkv, device="cuda")[:, None]
    j = torch.arange(K, device="cuda")
    src = st["tables"].long().gather(1, (idx // B).flatten(1)).view(S, Hkv, K)
    dst = st["new_tables"].long()[:, j // B][:, None].expand(S, Hkv, K)
    a, b = idx % B, (j % B).expand(S, Hkv, K)
    # rows past the kept ones keep what they hold
    st["kc"][dst, head, b] = torch.where(live[..., None], st["kc"][src, head, a],
                                         st["kc"][dst, head, b])
    if st["ks"] is None:
        st["vc"][dst, head, b] = torch.where(live[..., None], st["vc"][src, head, a],
                                             st["vc"][dst, head, b])
    else:
        vpos = torch.tensor(V_POS, device="cuda")
        d = torch.arange(c["D"], device="cuda")
        s4, d4 = (src[..., None], head[..., None], d, vpos[a][..., None]), \
            (dst[..., None], head[..., None], d, vpos[b][..., None])
        st["vc"][d4] = torch.where(live[..., None], st["vc"][s4], st["vc"][d4])
    return {"kept": st["kept"], "sums": st["new_sums"], "lens": st["new_lens"], **_cache_out(st)}


def plain_beam(st):
    S, K, V = st["logits"].shape
    N = st["scores"].shape[1]
    x = st["logits"].double()  # candidates of different beams lie next to each other
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    top = x.amax(-1, keepdim=True)
    fine = torch.isfinite(top)
    e = torch.exp(torch.where(fine, x - top, torch.zeros_like(x)))
    score = st["beam_scores"].double()[..., None] + (x - (top + torch.log(e.sum(-1, keepdim=True))))
    score = torch.where(fine & ~torch.isnan(score), score, torch.full_like(score, -math.inf))
    best = torch.sort(score.view(S, K * V), dim=-1, descending=True, stable=True)
    idx = best.indices[:, :N]
    st["scores"].copy_(best.values[:, :N])
    st["beams"].copy_(idx // V)
    st["tokens"].copy_(idx % V)
    return {"scores": st["scores"], "beams": st["beams"], "tokens": st["tokens"]}


# ---------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "beam":
        S, K, V, N = case["S"], case["K"], case["V"], case["N"]
        scores = torch.empty((S, N), dtype=torch.float64, device="cuda")
        beams, tokens = (torch.empty((S, N), dtype=torch.int64, device="cuda") for _ in range(2))
        for s in range(S):
            x = st["logits"][s].double()
            p = st["beam_scores"][s].double()[:, None] + x - torch.logsumexp(x, -1, keepdim=True)
            value, at = torch.sort(p.flatten(), descending=True, stable=True)
            scores[s], beams[s], tokens[s] = value[:N], at[:N] // V, at[:N] % V
        return {"scores": scores, "beams": beams, "tokens": tokens}
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    fp8 = case["cache"] == "fp8"
    wide = lambda t: (t.view(torch.float8_e4m3fn) if fp8 else t).double()  # noqa: E731
    order = torch.tensor(V_POS, device="cuda")
    if op == "rotary":
        rot, T = case["rot"], case["T"]
        z = torch.polar(torch.ones(T, rot // 2, dtype=torch.float64, device="cuda"),
                        torch.outer(st["positions"].double(), st["freq"]))[:, None]

        def turned(x):
            y = x.double().clone()
            one, two = ((slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"]
                        else (slice(0, rot // 2), slice(rot // 2, rot)))
            w = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * z
            y[..., one], y[..., two] = w.real, w.imag
            return y

        kc, vc = wide(st["kc"]), wide(st["vc"])
        k, v = turned(st["k"]), st["v"].double()
        block, at = (st["slots"] // B).long(), (st["slots"] % B).long()
        if fp8:
            k = (k / st["ks"].double()[:, None]).clamp(-448, 448)
            v = (v / st["vs"].double()[:, None]).clamp(-448, 448)
            vc[block, :, :, order[at]] = v
        else:
            vc[block, :, at] = v
        kc[block, :, at] = k
        return {"q": turned(st["q"]), "kc": kc, "vc": vc}
    lens = lens_of(case)
    if op == "weights":
        Hq = case["Hq"]
        out = torch.zeros((case["S"], Hq, D), dtype=torch.float64, device="cuda")
        sums = st["sums"].double()
        for s in range(case["S"]):
            t, n = st["tables"][s].long(), int(lens[s])
            t = t[:-(-n // B)]
            k, v = wide(st["kc"][t]), wide(st["vc"][t])  # [blocks, Hkv, ., .]
            if fp8:
                k, v = k * st["ks"].double()[:, None, None], v * st["vs"].double()[:, None, None]
                v = v[..., order].transpose(-1, -2)
            k, v = (y.transpose(0, 1).reshape(Hkv, -1, D)[:, :n] for y in (k, v))
            q = st["q"][s].double().view(Hkv, Hq // Hkv, D)
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k) * st["scale"], -1)
            out[s] = torch.einsum("hgn,hnd->hgd", w, v).reshape(Hq, D)
            sums[s, :, :n] += w.sum(1)
        return {"out": out, "sums": sums}
    # evict: row by row, from the definition
    kept, new_sums = st["kept"].clone(), st["new_sums"].double()
    kc, vc = wide(st["kc"]), wide(st["vc"])
    heads = torch.arange(Hkv, device="cuda")[:, None]
    for s in range(case["S"]):
        c = int(lens[s])
        n = min(c, case["keep"])
        r = min(case["recent"], n)
        f = min(case["first"], n - r)
        x = st["sums"][s, :, f:c - r].double()
        best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :n - r - f] + f
        ends = torch.cat([torch.arange(f, device="cuda"), torch.arange(c - r, c, device="cuda")])
        idx = torch.sort(torch.cat([best, ends.expand(Hkv, -1)], 1), dim=1).values
        kept[s, :, :n] = idx.int()
        new_sums[s, :, :n] = st["sums"][s].double().gather(1, idx)
        j = torch.arange(n, device="cuda")
        src, dst = st["tables"][s].long()[idx // B], st["new_tables"][s].long()[j // B]
        kc[dst, heads, j % B] = wide(st["kc"][src, heads, idx % B])
        if fp8:
            d = torch.arange(D, device="cuda")
            vc[dst[:, None], heads[..., None], d, order[j % B][:, None]] = wide(
                st["vc"][src[..., None], heads[..., None], d, order[idx % B][..., None]])
        else:
            vc[dst, heads, j % B] = wide(st["vc"][src, heads, idx % B])
    return {"kept": kept, "sums": new_sums, "lens": _i32(np.minimum(lens, case["keep"])),
            "kc": kc, "vc": vc}
