"""Tensors of another accelerator, whose devices are numbered as GPUs are, are refused before
anything is launched (stand-ins for them; no GPU needed)."""
import pytest
import torch

from paged_kv_cache_166_gb300 import ops


class Elsewhere:
    """What the checks see of a tensor on device `number` of another accelerator (kind "cuda": a
    GPU's)."""

    def __init__(self, shape, dtype, kind="xpu", number=0):
        self.shape, self.dtype, self.kind, self.number = torch.Size(shape), dtype, kind, number
        self.is_cuda = kind == "cuda"
        self.device = torch.device(kind, number)

    def get_device(self):
        return self.number

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        if i is None:
            return tuple(self.stride(x) for x in range(len(self.shape)))
        n = 1
        for x in self.shape[i + 1:]:
            n *= x
        return n

    def numel(self):
        return self.stride(0) * self.shape[0] if self.shape else 1

    def element_size(self):
        return 4

    def data_ptr(self):
        return 1 << 20


def gpu(*shape, dtype=torch.int32):
    return Elsewhere(shape, dtype, "cuda")


def other(*shape, dtype=torch.int32):
    return Elsewhere(shape, dtype)


def test_another_accelerator_s_tensors():
    with pytest.raises(ValueError, match="CUDA tensors"):
        ops._check_cuda(other(3), other(3))
    with pytest.raises(ValueError, match="CUDA tensors"):
        ops._check_cuda(gpu(3), other(3))
    with pytest.raises(ValueError, match="one device"):
        ops._check_cuda(gpu(3), Elsewhere((3,), torch.int32, "cuda", 1))
    assert ops._check_cuda(gpu(3), gpu(3)) == torch.device("cuda", 0)
    with pytest.raises(ValueError, match="CUDA tensors"):
        ops._check_cuda(torch.zeros(3), torch.zeros(3))


@pytest.fixture
def no_call(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            def call(*args):
                raise AssertionError("the library was called")
            return call
    monkeypatch.setattr(ops.N, "lib", Lib)
    monkeypatch.setattr(ops, "_current", lambda dev: ops._HERE)
    monkeypatch.setattr(ops, "_stream", lambda dev: 0)


@pytest.mark.parametrize("which", ["q", "k", "v", "q_out", "q_weight", "k_weight"])
def test_norm_and_rotary_write(no_call, which):
    h = torch.float16
    kw = dict(q=gpu(4, 8, 64, dtype=h), k=gpu(4, 2, 64, dtype=h), v=gpu(4, 2, 64, dtype=h),
              q_weight=gpu(64, dtype=h), k_weight=gpu(64, dtype=h), q_out=gpu(4, 8, 64, dtype=h))
    same = dict(eps=1e-6, positions=gpu(4), table=gpu(100, 64, dtype=torch.float32),
                slot_mapping=gpu(4), k_cache=gpu(9, 2, 16, 64, dtype=h),
                v_cache=gpu(9, 2, 16, 64, dtype=h))
    with pytest.raises(AssertionError, match="was called"):
        ops.paged_norm_rotary_write(**kw, **same)
    kw[which] = Elsewhere(kw[which].shape, h)
    with pytest.raises(ValueError, match="device"):
        ops.paged_norm_rotary_write(**kw, **same)


@pytest.mark.parametrize("which", ["logits", "out", "allowed", "repetition"])
def test_logit_adjustment(no_call, which):
    f = torch.float32
    kw = dict(logits=gpu(2, 100, dtype=f), out=gpu(2, 100, dtype=f), allowed=gpu(2, 4),
              repetition=gpu(2, dtype=f))
    same = dict(history=gpu(2, 9), history_lens=gpu(2))
    with pytest.raises(AssertionError, match="was called"):
        ops.adjust_logits(**kw, **same)
    kw[which] = Elsewhere(kw[which].shape, kw[which].dtype)
    with pytest.raises(ValueError, match="device"):
        ops.adjust_logits(**kw, **same)
