"""Cases, plain forms and calls of the operators of a speculative step over the paged cache.

* tree: attention of drafted tokens (a tree of them, or a plain chunk) over the cache, its
  scores capped by a tanh, with a bias or a window by distance (``paged_tree_attention``);
* norm: norms of q and k for each head, rotary positions on one or several axes, k and v
  written into the paged cache (``paged_norm_rotary_write``, ``paged_norm_rotary_write_fp8``);
* adjust: penalties for repeated tokens, biases and masks of allowed tokens on logits
  (``adjust_logits``);
* commit: the rows of the accepted path moved together in every layer's cache
  (``paged_tree_commit``).

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
        # the smallest call: two short contexts, a handful of drafted tokens
        tree("tree_tiny_f16", S=2, Hq=4, Hkv=4, D=64, dtype="f16", nodes=5, kind="uniform", lo=6,
             hi=100, seed=0),
        # a 70B-shaped batch verifying small trees
        tree("tree_70b_bf16", S=128, Hq=64, Hkv=8, D=128, dtype="bf16", nodes=8,
             kind="lognormal", lo=8, hi=8192, median=1024.0, sigma=1.2, seed=2),
        # few long contexts, trees that fill a tile of rows
        tree("tree_long_bf16", S=4, Hq=64, Hkv=8, D=128, dtype="bf16", nodes=16, kind="uniform",
             lo=32768, hi=131072, seed=4),
        # capped scores and a sliding window, wide heads
        tree("tree_capped_f16", S=32, Hq=16, Hkv=8, D=256, dtype="f16", nodes=12, cap=50.0,
             window=4096, kind="uniform", lo=1000, hi=16384, seed=5),
        # a prompt's next chunk with a bias by distance, 13B-shaped, causal
        tree("chunk_bias_13b_f16", S=8, Hq=40, Hkv=40, D=128, dtype="f16", nodes=513, chain=True,
             even=True, slopes=True, kind="uniform", lo=513, hi=2048, seed=1),
        # one step of a 70B-shaped batch with four drafted tokens a sequence: latency
        norm("norm_step_70b_bf16", T=256, Hq=64, Hkv=8, D=128, rot=128, dtype="bf16", axes=1,
             span=131072, interleaved=False, fused=True, per_head=False),
        # an image's tokens in a packed prompt: time, height and width
        norm("norm_prompt_axes_f16", T=8191, Hq=40, Hkv=40, D=128, rot=128, dtype="f16", axes=3,
             span=8192, interleaved=False, fused=True, per_head=False),
        # prompt chunk into an fp8 cache, grouped heads, a weight for each head, half turned
        norm("norm_prompt_fp8", T=4099, Hq=32, Hkv=8, D=128, rot=64, dtype="bf16", cache="fp8",
             axes=1, span=32768, interleaved=True, fused=True, per_head=True),
        # one step of four requests, penalties and biases alone
        adjust("adjust_step_f32", S=4, nodes=1, V=32000, dtype="f32", hi=2000, bias=32,
               masked=False, apart=False, seed=3),
        # a batch's drafted tokens under a grammar
        adjust("adjust_verify_bf16", S=32, nodes=8, V=131072, dtype="bf16", hi=8192, bias=8,
               masked=True, apart=False, seed=4),
        # four requests, two layers
        commit("commit_tiny_f16", S=4, Hkv=4, D=64, dtype="f16", layers=2, nodes=8, most=4,
               hi=100, seed=0),
        # a 70B-shaped batch, 32 layers
        commit("commit_70b_bf16", S=64, Hkv=8, D=128, dtype="bf16", layers=32, nodes=48, most=8,
               hi=128, seed=1),
    ]


def tree(name=None, **c):
    return _case("tree", name, dict(B=16, median=0.0, sigma=0.0, cap=0.0, window=0, slopes=False,
                                    chain=False, even=False), c)


def norm(name=None, **c):
    return _case("norm", name, dict(cache="same", B=16, base=10000.0, eps=1e-6), c)


def adjust(name=None, **c):
    return _case("adjust", name, {}, c)


def commit(name=None, **c):
    return _case("commit", name, dict(cache="same", B=16), c)


def _case(op, name, defaults, c):
    out = {"op": op, **defaults, **c}
    if name is not None:
        out["name"] = name
    return out


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "norm", "adjust", "commit"])
    if op == "adjust":
        V, nodes = _log(rng, 1000, 160000), _log(rng, 1, 64)
        S = _log(rng, 1, max(1, min(64, (1 << 25) // (nodes * V))))
        return adjust(S=S, nodes=nodes, V=V, dtype=rng.choice(["f32", "f16", "bf16"]),
                      hi=_log(rng, 1, 16384), bias=rng.choice([0, 8, 300]),
                      masked=rng.random() < 0.5, apart=rng.random() < 0.3,
                      seed=rng.randrange(1 << 20))
    Hkv, G = rng.choice([1, 2, 4, 8, 16, 40]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    if Hkv == 40:
        G = 1
    if op == "tree":
        D, nodes = rng.choice([64, 128, 256]), _log(rng, 1, 512)
        hi = _log(rng, nodes, 65536)
        # the plain form's scores are S * Hq * nodes * hi values, its K and V S * Hkv * hi * D
        most = min(int(3e8) // (Hkv * G * nodes * hi), int(3e8) // (Hkv * hi * D))
        S = _log(rng, 1, max(1, min(128, most)))
        if most < 1:
            hi = max(nodes, min(hi, 4096))
            Hkv = min(Hkv, 8)
        return tree(S=S, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["f16", "bf16"]), nodes=nodes,
                    chain=rng.random() < 0.3, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                    window=rng.choice([0, 0, 100, 1024]), slopes=rng.random() < 0.3,
                    kind="uniform", lo=max(nodes, hi // rng.choice([1, 2, 16])), hi=hi,
                    B=rng.choice([8, 16, 32]), seed=rng.randrange(1 << 20))
    cache = rng.choice(["same", "same", "fp8"])
    if cache == "fp8":
        D, dtype, B = 128, rng.choice(["f16", "bf16"]), 16
    else:
        dtype = rng.choice(["f32", "f16", "bf16"])
        D, B = rng.choice([64, 128, 256]), rng.choice([8, 16, 32])
    if op == "norm":
        most = max(2, min(16384, (1 << 28) // ((G + 2) * Hkv * D * 4)))
        return norm(T=_log(rng, 1, most), Hq=Hkv * G, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2, D // 4]), dtype=dtype, cache=cache, B=B,
                    base=rng.choice([10000.0, 500000.0]), axes=rng.choice([1, 1, 2, 3]),
                    span=_log(rng, 16384, 131072), interleaved=rng.random() < 0.5,
                    fused=rng.random() < 0.5, per_head=rng.random() < 0.3)
    nodes, layers, hi = _log(rng, 1, 64), _log(rng, 1, 32), _log(rng, 64, 1024)
    S = _log(rng, 1, max(1, min(128, int(1e8) // (layers * Hkv * D * hi))))
    return commit(S=S, Hkv=Hkv, D=D, dtype=dtype, cache=cache, layers=layers, nodes=nodes,
                  most=_log(rng, 1, nodes), hi=hi, B=B, seed=rng.randrange(1 << 20))


def lens_of(case):
    """The batch's context lengths, drafted tokens included: they belong to the case, not to
    the seed of its values."""
    g = np.random.default_rng(case["seed"])
    S, lo, hi = case["S"], case["lo"], case["hi"]
    if case["kind"] == "lognormal":
        x = g.lognormal(math.log(case["median"]), case["sigma"], S)
    else:
        x = g.integers(lo, hi, S, endpoint=True)
    return np.clip(np.rint(x), lo, hi).astype(np.int64)


def counts_of(case):
    """Drafted tokens of every sequence."""
    g = np.random.default_rng(case["seed"] + 1)
    if case.get("even"):  # chunks of one size
        return np.full(case["S"], case["nodes"], dtype=np.int64)
    return g.integers(max(1, case["nodes"] // 2), case["nodes"], case["S"], endpoint=True)


def trees_of(case):
    """Each sequence's drafted tokens as a tree: lists of parents (-1: the context's end)."""
    g = np.random.default_rng(case["seed"] + 2)
    out = []
    for c in counts_of(case):
        if case.get("chain"):
            out.append(np.arange(-1, c - 1))
        else:  # mostly recent parents: depths of some ten for a few dozen tokens
            back = 1 + np.minimum(g.geometric(0.4, c) - 1, np.arange(c))
            out.append(np.arange(c) - back)
    return out


def masks_of(parents):
    """(seen [c, c], depths [c]) of one tree: which drafted tokens each one sees."""
    c = len(parents)
    seen, depth = np.zeros((c, c), dtype=bool), np.zeros(c, dtype=np.int64)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
            depth[i] = depth[p] + 1
        seen[i, i] = True
    return seen, depth


def work(case):
    op = case["op"]
    elt = 4 if case["dtype"] == "f32" else 2
    if op == "adjust":
        # what is put: banned logits, and those of tokens seen or biased, read and written
        S, nodes, V = case["S"], case["nodes"], case["V"]
        rows, held = S * nodes, int(history_lens_of(case).sum())
        touched = min(V, case["hi"] // 2 + case["bias"])
        b = 4 * held + 8 * S * case["bias"] + 2 * elt * rows * touched
        if case["masked"]:
            b += rows * V // 8 + rows * (V - touched) // 2 * elt
        if case["apart"]:
            b = 4 * held + 2 * rows * V * elt + (rows * V // 8 if case["masked"] else 0)
        return {"bytes": b, "flops": 4.0 * rows * touched}
    celt = 1 if case.get("cache") == "fp8" else elt
    Hkv, D = case["Hkv"], case["D"]
    if op == "norm":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        move = T * D * (2 * Hq * elt + 2 * Hkv * (elt + celt))
        return {"bytes": move + T * (rot * 4 + 4 + 4 * case["axes"]),
                "flops": T * (Hq + Hkv) * (4.0 * D + 3.0 * rot)}
    if op == "commit":
        path, n = paths_of(case)
        moved = int(((path != np.arange(path.shape[1])) & (np.arange(path.shape[1]) < n[:, None])).sum())
        return {"bytes": 4 * moved * case["layers"] * Hkv * D * celt + 4 * int(n.sum()), "flops": 0}
    lens, counts, S, Hq = lens_of(case), counts_of(case), case["S"], case["Hq"]
    base, window = lens - counts, case["window"]
    first = np.maximum(0, base - window + 1) if window else np.zeros_like(base)
    b = 2 * int((lens - first).sum()) * Hkv * D * elt + 2 * int(counts.sum()) * Hq * D * elt
    b += int((-(-lens // case["B"])).sum()) * 4
    if case["chain"]:
        seen = counts * (counts + 1) // 2
    else:
        b += int(counts.sum()) * 4 * (-(-case["nodes"] // 32))
        seen = np.array([masks_of(p)[0].sum() for p in trees_of(case)])
    pairs = int((counts * (base - first) + seen).sum())
    return {"bytes": b, "flops": 4.0 * pairs * Hq * D}


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
    for x in t.view(-1).split(1 << 26):
        x.copy_(_randn(x.shape, g, dtype))
    return t


def _codes(shape, g):
    """E4M3 codes of N(0,1) values over a scale of about 4 / 448, as bytes."""
    t = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for x in t.view(-1).split(1 << 26):
        y = (_randn(x.shape, g) * 112.0).clamp(-448.0, 448.0)
        x.copy_(y.to(torch.float8_e4m3fn).view(torch.uint8))
    return t


def _caches(case, lead, g):
    """K and V pools [*lead, Hkv, B, D] (8-bit: V tiles transposed)."""
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    if case["cache"] == "fp8":
        return {"kc": _codes((*lead, Hkv, B, D), g), "vc": _codes((*lead, Hkv, D, B), g)}
    dt = DTYPES[case["dtype"]]
    return {"kc": _filled((*lead, Hkv, B, D), dt, g), "vc": _filled((*lead, Hkv, B, D), dt, g)}


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _tables(lens, B, h):
    """Block tables of a pool in random order, and the pool's size."""
    nb = -(-lens // B)
    NB = int(nb.sum()) + max(1, int(nb.sum()) // 10)
    order = h.permutation(NB)
    tables = np.zeros((len(lens), int(nb.max())), dtype=np.int64)
    at = 0
    for s in range(len(lens)):
        tables[s, :nb[s]] = order[at:at + nb[s]]
        at += nb[s]
    return tables, NB


def history_lens_of(case):
    g = np.random.default_rng(case["seed"])
    return g.integers(max(1, case["hi"] // 4), case["hi"], case["S"], endpoint=True)


def paths_of(case):
    """The accepted path of every sequence's tree, [S, most], and its length."""
    g = np.random.default_rng(case["seed"] + 3)
    counts = counts_of(case)
    n = np.minimum(g.integers(1, case["most"], case["S"], endpoint=True), counts)
    path = np.zeros((case["S"], case["most"]), dtype=np.int64)
    for s in range(case["S"]):
        path[s, :n[s]] = np.sort(g.permutation(counts[s])[:n[s]])
    return path, n


def pair_axes(case):
    """The axis of each pair of turning elements: the pairs in as many sections as axes."""
    return [i * case["axes"] // (case["rot"] // 2) for i in range(case["rot"] // 2)]


def prepare(case, seed):
    g, h = _gen(seed), np.random.default_rng(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"case": case, "op": op}
    if op == "adjust":
        S, nodes, V = case["S"], case["nodes"], case["V"]
        T = S * nodes
        st["logits"] = (_randn((T, V), g) * 2.5).to(dt)
        st["out"] = torch.empty_like(st["logits"]) if case["apart"] else st["logits"]
        lens = history_lens_of(case)
        # a text's tokens: few of them often, the rest seldom
        tokens = np.minimum((V - 1) * h.random((S, case["hi"])) ** 4, V - 1).astype(np.int64)
        st["history"], st["lens"] = _i32(tokens), _i32(lens)
        st["prompts"] = _i32((lens * h.random(S)).astype(np.int64))
        st["rows"] = _i32(np.arange(S + 1) * nodes)
        st["repetition"] = 1.0 + 0.3 * torch.rand(S, generator=g, device="cuda")
        st["frequency"] = 0.5 * torch.rand(S, generator=g, device="cuda")
        st["presence"] = 0.5 * torch.rand(S, generator=g, device="cuda")
        st["path"] = None
        if nodes > 1:  # each drafted token's ancestors
            path = h.integers(0, V, (T, 8))
            path[h.random((T, 8)) < 0.4] = -1
            st["path"] = _i32(path)
        n = min(case["bias"], V)
        st["bias_tokens"] = st["bias_values"] = st["allowed"] = None
        if n:
            st["bias_tokens"] = _i32(np.stack([h.choice(V, n, replace=False) for _ in range(S)]))
            st["bias_values"] = _randn((S, n), g) * 4.0
        if case["masked"]:  # few tokens allowed (in a structure), or most (in a text)
            few = torch.rand((T, 1), generator=g, device="cuda") < 0.5
            on = torch.rand((T, -(-V // 32) * 32), generator=g, device="cuda") < \
                torch.where(few, 0.02, 0.98)
            word = on.view(T, -1, 32).long() << torch.arange(32, device="cuda")
            word = word.sum(-1)
            st["allowed"] = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
        return st
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if op == "norm":
        T, Hq, rot, A = case["T"], case["Hq"], case["rot"], case["axes"]
        NB = -(-T // B) + max(1, T // (10 * B))
        st.update(_caches(case, (NB,), g))
        st["ks"] = st["vs"] = None
        if case["cache"] == "fp8":
            st["ks"], st["vs"] = ((torch.rand(Hkv, generator=g, device="cuda") * 3 + 3) / 448.0
                                  for _ in range(2))
        # a projection's output: each head of its own size
        x = _randn((T, Hq + 2 * Hkv, D), g) * torch.exp(_randn((1, Hq + 2 * Hkv, 1), g))
        x = x.to(dt)
        parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        st["q"], st["k"], st["v"] = parts if case["fused"] else (p.contiguous() for p in parts)
        st["qw"], st["kw"] = ((1.0 + 0.2 * _randn(((H, D) if case["per_head"] else (D,)), g)).to(dt)
                              for H in (Hq, Hkv))
        if A == 1:
            pos = h.integers(0, case["span"], T) if T <= 512 else np.arange(T) % case["span"]
        else:  # an image of some hundred columns: row and column beside the token's time
            wide = 100
            pos = np.stack([np.arange(T), np.arange(T) // wide, np.arange(T) % wide][:A])
            pos = pos % case["span"]
        st["positions"], st["axes"] = _i32(pos), pair_axes(case) if A > 1 else None
        order = h.permutation(NB)
        st["slots"] = _i32(order[np.arange(T) // B] * B + np.arange(T) % B)
        inv = case["base"] ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
        st["freq"] = torch.from_numpy(inv).cuda()
        ang = torch.arange(case["span"], device="cuda", dtype=torch.float64)[:, None] * st["freq"]
        st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        return st
    counts = counts_of(case)
    if op == "commit":
        lens = np.random.default_rng(case["seed"]).integers(1, case["hi"], case["S"]) + counts
        tables, NB = _tables(lens, B, h)
        st.update(_caches(case, (case["layers"], NB), g))
        path, n = paths_of(case)
        st["path"], st["lens"] = _i32(path), _i32(n)
    else:
        lens = lens_of(case)
        tables, NB = _tables(lens, B, h)
        st.update(_caches({**case, "cache": "same"}, (NB,), g))
        T, Hq = int(counts.sum()), case["Hq"]
        st["q"] = (_randn((T, Hq, D), g) * 1.5).to(dt)
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(D)
        st["mask"] = st["depths"] = st["slopes"] = None
        if not case["chain"]:
            W = -(-int(counts.max()) // 32)
            both = [masks_of(p) for p in trees_of(case)]
            bits = np.zeros((T, W * 32), dtype=np.uint8)
            at = 0
            for seen, _ in both:
                bits[at:at + len(seen), :len(seen)] = seen
                at += len(seen)
            st["mask"] = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little")
                                          .view(np.int32).copy()).cuda()
            st["depths"] = _i32(np.concatenate([d for _, d in both]))
        if case["slopes"]:  # 2^(-8 (h + 1) / heads)
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda").float() / Hq)
    st["tables"], st["ctx"] = _i32(tables), _i32(lens)
    st["starts"] = _i32(np.concatenate([[0], np.cumsum(counts)]))
    st["most_nodes"] = int(counts.max())
    return st


# ---------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        return {"tree": own_tree, "norm": own_norm, "adjust": own_adjust,
                "commit": own_commit}[op](state)
    return {"tree": plain_tree, "norm": plain_norm, "adjust": plain_adjust,
            "commit": plain_commit}[op](state)


def _cache_out(st):
    """The caches as the values they hold (8-bit ones as the codes' own type)."""
    if st["kc"].dtype == torch.uint8:
        return {"kc": st["kc"].view(torch.float8_e4m3fn), "vc": st["vc"].view(torch.float8_e4m3fn)}
    return {"kc": st["kc"], "vc": st["vc"]}


def own_tree(st):
    import paged_kv_cache_166_gb300 as pkv
    c = st["case"]
    pkv.paged_tree_attention(st["q"], st["kc"], st["vc"], st["tables"], st["ctx"], st["starts"],
                             st["scale"], st["out"], tree_mask=st["mask"], depths=st["depths"],
                             cap=c["cap"], slopes=st["slopes"], window=c["window"])
    return st["out"]


def own_norm(st):
    import paged_kv_cache_166_gb300 as pkv
    c = st["case"]
    if st["ks"] is not None:
        pkv.paged_norm_rotary_write_fp8(st["q"], st["k"], st["v"], st["qw"], st["kw"], c["eps"],
                                        st["positions"], st["table"], st["slots"], st["kc"],
                                        st["vc"], st["ks"], st["vs"], st["q_out"],
                                        interleaved=c["interleaved"], axes=st["axes"])
    else:
        pkv.paged_norm_rotary_write(st["q"], st["k"], st["v"], st["qw"], st["kw"], c["eps"],
                                    st["positions"], st["table"], st["slots"], st["kc"], st["vc"],
                                    st["q_out"], interleaved=c["interleaved"], axes=st["axes"])
    return {"q": st["q_out"], **_cache_out(st)}


def own_adjust(st):
    import paged_kv_cache_166_gb300 as pkv
    pkv.adjust_logits(st["logits"], st["history"], st["lens"], st["prompts"],
                      row_start=st["rows"], repetition=st["repetition"],
                      frequency=st["frequency"], presence=st["presence"], path=st["path"],
                      bias_tokens=st["bias_tokens"], bias_values=st["bias_values"],
                      allowed=st["allowed"], out=st["out"])
    return st["out"]


def own_commit(st):
    import paged_kv_cache_166_gb300 as pkv
    pkv.paged_tree_commit(st["kc"], st["vc"], st["tables"], st["ctx"], st["starts"], st["path"],
                          st["lens"])
    return _cache_out(st)


def plain_tree(st):
    c = st["case"]
    S, Hq, Hkv, D, C = c["S"], c["Hq"], c["Hkv"], c["D"], st["most_nodes"]
    G, t = Hq // Hkv, st["tables"].long()
    k = st["kc"][t].transpose(1, 2).flatten(2, 3).float()  # [S, Hkv, L, D]
    v = st["vc"][t].transpose(1, 2).flatten(2, 3).float()
    L = k.shape[2]
    starts, ctx = st["starts"].long(), st["ctx"].long()
    count = starts[1:] - starts[:-1]
    base = (ctx - count)[:, None]
    i, p = torch.arange(C, device="cuda"), torch.arange(L, device="cuda")
    live = i < count[:, None]  # [S, C]
    row = torch.where(live, starts[:-1, None] + i, 0)
    q = st["q"][row].float().view(S, C, Hkv, G, D).permute(0, 2, 3, 1, 4)
    # positions of queries and keys, and which drafted key each query sees
    depth = i.expand(S, C) if st["depths"] is None else st["depths"].long()[row]
    at = p.expand(S, L)
    j = (p - base).clamp(0, C - 1)  # [S, L]: a drafted key's place in its tree
    if st["depths"] is not None:
        at = torch.where(p < base, at, base + depth.gather(1, j))
    far = (base + depth)[:, :, None] - at[:, None]  # [S, C, L]
    if st["mask"] is None:
        seen = j[:, None] <= i[:, None]
    else:
        word = st["mask"][row].long()  # [S, C, W]
        seen = (word.gather(2, (j // 32)[:, None].expand(S, C, L)) >> (j % 32)[:, None]) & 1 == 1
    seen = (p < base)[:, None] | (seen & (p < ctx[:, None])[:, None])
    if c["window"]:
        seen = seen & (far < c["window"])
    x = torch.matmul(q.reshape(S, Hkv, G * C, D), k.transpose(-1, -2)).view(S, Hkv, G, C, L)
    x = x * st["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if st["slopes"] is not None:
        x = x - st["slopes"].view(Hkv, G, 1, 1) * far[:, None, None].float()
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    w = e / torch.where(total > 0, total, 1.0)
    y = torch.matmul(w.view(S, Hkv, G * C, L), v).view(S, Hkv, G, C, D)
    y = y.permute(0, 3, 1, 2, 4).reshape(S, C, Hq, D)
    st["out"].copy_(y[live])
    return st["out"]


def plain_norm(st):
    c = st["case"]
    rot, B = c["rot"], c["B"]
    pos = st["positions"].double()
    if st["axes"] is not None:  # each pair's own position, [T, rot / 2]
        pos = pos[torch.tensor(st["axes"], device="cuda")].T
    else:
        pos = pos[:, None]
    ang = pos * st["freq"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + c["eps"]) * w.float()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    st["q_out"].copy_(turned(st["q"], st["qw"]))
    block, at = (st["slots"] // B).long(), (st["slots"] % B).long()
    k, v = turned(st["k"], st["kw"]), st["v"].float()
    if st["ks"] is None:
        st["kc"][block, :, at] = k.to(st["kc"].dtype)
        st["vc"][block, :, at] = v.to(st["vc"].dtype)
    else:
        vpos = torch.tensor(V_POS, device="cuda")[at]
        code = lambda x, s: (x / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)  # noqa: E731
        st["kc"][block, :, at] = code(k, st["ks"]).view(torch.uint8)
        st["vc"][block, :, :, vpos] = code(v, st["vs"]).view(torch.uint8)
    return {"q": st["q_out"], **_cache_out(st)}


def plain_adjust(st):
    c = st["case"]
    S, V = c["S"], c["V"]
    T = st["logits"].shape[0]
    request = torch.arange(S, device="cuda").repeat_interleave((st["rows"][1:] - st["rows"][:-1]).long())
    at = torch.arange(st["history"].shape[1], device="cuda")
    held, said = at < st["lens"][:, None], at >= st["prompts"][:, None]
    tok = torch.where(held, st["history"].long(), V)  # column V: of no token
    zero = torch.zeros((S, V + 1), dtype=torch.int32, device="cuda")
    count = zero.scatter_add(1, tok, said.int())[:, :V]  # in what the model has written
    seen = zero.scatter_add(1, tok, torch.ones_like(tok, dtype=torch.int32))[:, :V] > 0
    n, seen = count[request], seen[request]
    if st["path"] is not None:
        p = torch.where(st["path"] >= 0, st["path"].long(), V)
        more = torch.zeros((T, V + 1), dtype=torch.int32, device="cuda")
        n = n + more.scatter_add(1, p, torch.ones_like(p, dtype=torch.int32))[:, :V]
    seen = seen | (n > 0)
    x = st["logits"].float()
    r = st["repetition"][request][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - st["frequency"][request][:, None] * n - st["presence"][request][:, None] * (n > 0)
    if st["bias_tokens"] is not None:
        bias = torch.zeros((S, V), device="cuda").scatter(1, st["bias_tokens"].long(), st["bias_values"])
        x = x + bias[request]
    if st["allowed"] is not None:
        v = torch.arange(V, device="cuda")
        ok = (st["allowed"][:, v // 32] >> (v % 32).int()) & 1 == 1
        x = torch.where(ok, x, -math.inf)
    st["out"].copy_(x)
    return st["out"]


def plain_commit(st):
    c = st["case"]
    B, Hkv = c["B"], c["Hkv"]
    S, P = st["path"].shape
    starts = st["starts"].long()
    base = (st["ctx"].long() - (starts[1:] - starts[:-1]))[:, None]
    j = torch.arange(P, device="cuda")
    live = j < st["lens"][:, None]  # [S, P]
    src, dst = (base + st["path"].long())[live], (base + j)[live]
    seq = torch.arange(S, device="cuda")[:, None].expand(S, P)[live]
    t = st["tables"].long()
    sb, db, so, do = t[seq, src // B], t[seq, dst // B], src % B, dst % B
    kc, vc = st["kc"], st["vc"]
    kc[:, db, :, do] = kc[:, sb, :, so]
    if c["cache"] == "fp8":
        vpos = torch.tensor(V_POS, device="cuda")
        vc[:, db, :, :, vpos[do]] = vc[:, sb, :, :, vpos[so]]
    else:
        vc[:, db, :, do] = vc[:, sb, :, so]
    return _cache_out(st)


# ---------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": exact_tree, "norm": exact_norm, "adjust": exact_adjust,
            "commit": exact_commit}[case["op"]](case, st)


def exact_tree(case, st):
    """Sequence by sequence, from the definition."""
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["B"]
    lens, counts, trees = lens_of(case), counts_of(case), trees_of(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for s in range(case["S"]):
        n, c = int(lens[s]), int(counts[s])
        blocks = st["tables"][s].long()[:-(-n // B)]
        k, v = (y[blocks].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
                for y in (st["kc"], st["vc"]))
        seen, depth = masks_of(trees[s])
        pos = torch.from_numpy(np.concatenate([np.arange(n - c), n - c + depth])).cuda()
        far = (pos[n - c:, None] - pos[None, :]).double()  # [c, n]
        ok = torch.ones((c, n), dtype=torch.bool, device="cuda")
        ok[:, n - c:] = torch.from_numpy(seen).cuda()
        if case["window"]:
            ok &= far < case["window"]
        for g in range(Hkv):
            q = st["q"][at:at + c, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)].double()
            x = torch.einsum("chd,nd->hcn", q, k[g]) * st["scale"]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if st["slopes"] is not None:
                m = st["slopes"][g * (Hq // Hkv):(g + 1) * (Hq // Hkv)].double()
                x = x - m[:, None, None] * far
            w = torch.softmax(x.masked_fill(~ok, -math.inf), -1)
            out[at:at + c, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] = \
                torch.einsum("hcn,nd->chd", w, v[g])
        at += c
    return out


def exact_norm(case, st):
    rot, T, B, fp8 = case["rot"], case["T"], case["B"], case["cache"] == "fp8"
    wide = lambda t: (t.view(torch.float8_e4m3fn) if fp8 else t).double()  # noqa: E731
    pos = st["positions"].double().view(-1, T)
    axis = torch.tensor(pair_axes(case), device="cuda")
    z = torch.polar(torch.ones((T, rot // 2), dtype=torch.float64, device="cuda"),
                    pos.T[:, axis] * st["freq"])[:, None]

    def turned(x, w):
        y = x.double()
        y = y / ((y * y).sum(-1, keepdim=True) / case["D"] + case["eps"]).sqrt() * w.double()
        one, two = ((slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"]
                    else (slice(0, rot // 2), slice(rot // 2, rot)))
        r = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * z
        y[..., one], y[..., two] = r.real, r.imag
        return y

    kc, vc = wide(st["kc"]), wide(st["vc"])
    k, v = turned(st["k"], st["kw"]), st["v"].double()
    block, at = (st["slots"] // B).long(), (st["slots"] % B).long()
    if fp8:
        k = (k / st["ks"].double()[:, None]).clamp(-448, 448)
        vc[block, :, :, torch.tensor(V_POS, device="cuda")[at]] = \
            (v / st["vs"].double()[:, None]).clamp(-448, 448)
    else:
        vc[block, :, at] = v
    kc[block, :, at] = k
    return {"q": turned(st["q"], st["qw"]), "kc": kc, "vc": vc}


def exact_adjust(case, st):
    """Row by row: a list of tokens and how often each came."""
    V, nodes = case["V"], case["nodes"]
    out = st["logits"].double()
    tokens, lens, prompts = (st[x].cpu().numpy() for x in ("history", "lens", "prompts"))
    path = None if st["path"] is None else st["path"].cpu().numpy()
    for t in range(out.shape[0]):
        s = t // nodes
        old, new = tokens[s, :prompts[s]], tokens[s, prompts[s]:lens[s]]
        if path is not None:
            new = np.concatenate([new, path[t][path[t] >= 0]])
        ids = torch.from_numpy(np.union1d(old, new).astype(np.int64)).cuda()
        x, r = out[t, ids], st["repetition"][s].double()
        out[t, ids] = torch.where(x > 0, x / r, x * r)
        ids, n = (torch.from_numpy(a.astype(np.int64)).cuda()
                  for a in np.unique(new, return_counts=True))
        out[t, ids] -= st["frequency"][s].double() * n + st["presence"][s].double()
        if st["bias_tokens"] is not None:
            out[t, st["bias_tokens"][s].long()] += st["bias_values"][s].double()
        if st["allowed"] is not None:
            bits = np.unpackbits(st["allowed"][t].cpu().numpy().view(np.uint8), bitorder="little")
            out[t, torch.from_numpy(bits[:V] == 0).cuda()] = -math.inf
    return out


def exact_commit(case, st):
    fp8, B = case["cache"] == "fp8", case["B"]
    wide = lambda t: (t.view(torch.float8_e4m3fn) if fp8 else t).double()  # noqa: E731
    kc, vc = wide(st["kc"]), wide(st["vc"])
    path, lens = paths_of(case)
    base = st["ctx"].cpu().numpy() - counts_of(case)
    t = st["tables"].cpu().numpy()
    for s in range(case["S"]):
        for j in range(int(lens[s])):  # ascending: a row is read before anything is put there
            a, b = int(base[s] + path[s, j]), int(base[s]) + j
            (x, i), (y, o) = (t[s, a // B], a % B), (t[s, b // B], b % B)
            kc[:, y, :, o] = kc[:, x, :, i].clone()
            if fp8:
                vc[:, y, :, :, V_POS[o]] = vc[:, x, :, :, V_POS[i]].clone()
            else:
                vc[:, y, :, o] = vc[:, x, :, i].clone()
    return {"kc": kc, "vc": vc}
