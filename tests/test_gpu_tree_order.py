"""The attention of drafted tokens behind kernels that write what it reads: lengths, rows' borders,
block tables, masks, depths, slopes and the status word put in place on the GPU by the kernel
directly in front, eagerly and in a captured graph."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case, i32, osp, pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()


def two_steps(D, seed):
    """Inputs of two batches of the same shapes over the same caches: a, b."""
    lens = [[3000, 700, 45, 900], [44, 2900, 1100, 60]]
    counts = [[12, 40, 3, 9], [40, 3, 12, 9]]
    cs = [Case(l, c, Hkv=2, G=4, D=D, dtype="bf16", seed=seed, extra=200) for l, c in zip(lens, counts)]
    NB = min(c.NB for c in cs)
    out = []
    for n, c in enumerate(cs):
        words = np.concatenate([osp.words(s, 2) for s in c.seen])
        tables = np.zeros((4, 200), dtype=np.int64)
        tables[:, :min(200, c.tables.shape[1])] = np.minimum(c.tables, NB - 1)[:, :200]
        out.append(dict(tables=i32(tables), lens=i32(c.lens), starts=i32(c.starts), mask=i32(words),
                        depths=i32(c.depths),
                        slopes=torch.rand(8, device="cuda") if n else torch.zeros(8, device="cuda")))
    return cs[0], out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("captured", [False, True])
def test_what_the_kernel_in_front_wrote(D, captured):
    c, (a, b) = two_steps(D, 7 + D)
    names = list(a)
    flag = torch.zeros((), dtype=torch.bool, device="cuda")
    now = {k: v.clone() for k, v in a.items()}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def attend(out, x):
        pkv().paged_tree_attention(c.q, c.kc, c.vc, x["tables"], x["lens"], x["starts"], c.scale,
                                   out, tree_mask=x["mask"], depths=x["depths"],
                                   slopes=x["slopes"], status=status)

    def step(last):
        """All inputs put in place, `last` by the kernel directly in front of the attention."""
        torch.logical_not(flag, out=flag)
        for k in [n for n in names if n != last] + [last]:
            torch.where(flag, b[k], a[k], out=now[k])
        attend(out, now)

    want = []
    out = torch.empty_like(c.q)
    for x in (a, b):
        out.fill_(7.0)
        attend(out, x)
        torch.cuda.synchronize()
        want.append(out.clone())
    assert int(status) == 0 and not torch.equal(*want)
    if captured:
        graphs = []
        for k in names:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step(k)
            graphs.append(g)
        steps = [g.replay for g in graphs]
    else:
        steps = [lambda k=k: step(k) for k in names]
    which = 0
    for _ in range(30):
        for s in steps:
            which ^= 1
            s()
            got = out.clone()
            assert torch.equal(got, want[which])
    assert int(status) == 0


def test_a_status_word_cleared_directly_in_front():
    """Bits of this call stay, those of an earlier one are gone."""
    c = Case([100, 64, 30], [4, 5, 3], D=64, dtype="f16", kind="chain")
    lens = i32([100, -4, 30])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(50):
        torch.add(zero, zero, out=status)
        pkv().paged_tree_attention(c.q, c.kc, c.vc, i32(c.tables), lens, i32(c.starts), c.scale,
                                   c.out[:c.T], status=status)
        assert int(status) != 0
