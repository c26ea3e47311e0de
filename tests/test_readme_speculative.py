"""The README's example of a speculative step stays in step with the binding (no GPU needed).

Both examples of README.md are run one after the other on the host, as a reader would: device set
to the CPU, ops that launch kernels replaced by stand-ins that only bind the call's arguments to
the real op's signature; the block manager and the trees' masks run for real.
"""
import inspect
import os
import re

import torch

from conftest import ROOT


def test_readme_speculative_example_matches_the_binding(monkeypatch):
    from paged_kv_cache_166_gb300 import ops
    text = open(os.path.join(ROOT, "README.md")).read()
    first, = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    second, = re.findall(r"```py\n(.*?)```", text, flags=re.S)
    called, kept = [], []
    names = [n for n in dir(ops) if n.startswith("paged_")] + ["adjust_logits", "rotary_table"]
    for name in names:
        real = getattr(ops, name)

        def stand_in(*args, _real=real, _name=name, **kw):
            bound = inspect.signature(_real).bind(*args, **kw)
            called.append(_name)
            kept.append((_name, bound.arguments))
            return torch.zeros((args[0], 2 * len(args[1]))) if _name == "rotary_table" else None

        monkeypatch.setattr(ops, name, stand_in)
    space = {"__name__": "readme_example"}
    exec(compile(first.replace('dev = "cuda"', 'dev = "cpu"'), "README.md example", "exec"), space)
    del called[:], kept[:]
    exec(compile(second, "README.md speculative example", "exec"), space)
    called = [n for n in called if n != "paged_copy_blocks"]
    assert called == ["rotary_table", "paged_norm_rotary_write", "paged_tree_attention",
                      "adjust_logits", "paged_tree_commit"]
    args = dict(kept)
    write, attend, adjust = (args[n] for n in ("paged_norm_rotary_write", "paged_tree_attention",
                                               "adjust_logits"))
    ctx, starts = attend["context_lens"], attend["query_start"]
    drafted = starts[1:] - starts[:-1]
    # the drafted tokens' positions, and a history that ends in front of them
    first_of = (ctx - drafted).repeat_interleave(drafted)
    assert torch.equal(write["positions"], first_of + attend["depths"])
    assert torch.equal(adjust["history_lens"], ctx - drafted)
    alloc, seqs = space["alloc"], space["seqs"]
    taken = args["paged_tree_commit"]["path_lens"]
    assert [alloc.length(s) for s in seqs] == (ctx - drafted + taken).tolist()
