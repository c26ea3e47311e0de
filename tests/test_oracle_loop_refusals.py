"""Host-side properties of the decode loop's operators (no GPU): frequencies of settings that
fp32 does not hold, and arguments that the library's 32-bit integers do not."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_166_gb300 as pkv
from oracle import rotary as orot
from paged_kv_cache_166_gb300 import _native as N


@pytest.mark.parametrize("kw", [
    dict(base=10000.1), dict(base=500000.3, scaling="linear", factor=1.1),
    dict(scaling="ntk", factor=1.3),
    dict(scaling="bands", factor=2.7, original_length=4000, low_turns=0.9, high_turns=30.1)])
def test_frequencies_of_settings_in_64_bits(kw):
    got, want = pkv.rotary_frequencies(128, **kw).numpy(), orot.frequencies(128, **kw)
    # pow twice (ntk's base is raised to at most -1), a band's weight t of a difference that
    # is at least 2^-3 of its terms or else multiplies little: some 16 units in the last place
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -52 * want)


def test_frequencies_f64_refusals_and_agreement():
    lib = N.lib()
    out, ref = (ctypes.c_double * 8)(), (ctypes.c_double * 8)()
    four = ctypes.c_double * 4
    assert lib.pkv_rotary_frequencies_f64(16, None, 0, 0, out) == N.PKV_ERR_INVALID_ARG
    for bad in ((1.0, 1, 1, 4), (float("nan"), 1, 1, 4), (float("inf"), 1, 1, 4)):
        assert lib.pkv_rotary_frequencies_f64(16, four(*bad), 0, 0, out) == N.PKV_ERR_INVALID_ARG
    assert lib.pkv_rotary_frequencies_f64(16, four(1e4, 0.5, 1, 4), 1, 0, out) == N.PKV_ERR_INVALID_ARG
    assert lib.pkv_rotary_frequencies_f64(16, four(1e4, 2, 4, 4), 3, 9, out) == N.PKV_ERR_INVALID_ARG
    for scaling in range(4):
        assert lib.pkv_rotary_frequencies_f64(16, four(1e4, 2, 1, 4), scaling, 4096, out) == 0
        assert lib.pkv_rotary_frequencies(16, 1e4, scaling, 2.0, 4096, 1.0, 4.0, ref) == 0
        assert list(out) == list(ref)


def test_sizes_that_32_bits_do_not_hold_are_refused():
    """Cut to 32 bits, these would be small valid values."""
    import torch
    x, i = torch.zeros(1, 1, 8), torch.zeros(1, dtype=torch.int32)
    kept = torch.zeros((1, 1, 8), dtype=torch.int32)
    for kw in (dict(first=1 << 32), dict(recent=(1 << 32) + 3), dict(first=-(1 << 40))):
        with pytest.raises(ValueError, match="32 bits"):
            pkv.paged_evict_select(x, i, i.clone(), kept, x.clone(), i.clone(), **kw)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.rotary_frequencies((1 << 32) + 16)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.rotary_frequencies(16, scaling="bands", factor=2.0, original_length=(1 << 32) + 4096)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.rotary_table((1 << 32) + 8, pkv.rotary_frequencies(16))


def test_weights_workspace_of_bounded_tokens():
    import torch
    size = lambda **kw: pkv.weights_workspace_bytes(256, 8192, 16, 64, 8, 128,  # noqa: E731
                                                    torch.bfloat16, num_warps=608, **kw)
    base = size(max_tokens=0) - 256 * 64 * 16 * 4  # no tokens: a step for each sequence's rest
    assert base < 20 << 20
    assert size() - base == 256 * 64 * 131072 * 4
    # 451,896 tokens: their scores and a step of 16 more a sequence
    assert size(max_tokens=451896) - base == (451896 // 16 + 256) * 16 * 64 * 4
    assert size(max_tokens=256 * 131072) == size(max_tokens=1 << 60) == size()
    with pytest.raises(ValueError):
        size(max_tokens=-1)


def test_bounded_weights_refusals():
    lib, P = N.lib(), 1 << 20

    def call(**kw):
        a = dict(codes=0, q=P, kc=P, vc=P, ks=None, vs=None, bt=P, maxb=4, ctx=P, S=2, Hq=8, Hkv=2,
                 D=128, B=16, NB=8, scale=0.1, out=P, sums=P, cols=64, tokens=20, ws=P, wsb=1 << 30,
                 warps=8, dt=N.PKV_BF16, stream=None)
        a.update(kw)
        return lib.pkv_decode_attention_weights_tokens(*a.values())
    n = ctypes.c_size_t()
    assert lib.pkv_decode_weights_workspace_size_tokens(2, 4, 16, 8, 2, 128, N.PKV_BF16, 8, 20,
                                                        ctypes.byref(n)) == N.PKV_OK
    for kw, code in ((dict(wsb=n.value - 1), N.PKV_ERR_INVALID_ARG), (dict(codes=5), N.PKV_ERR_DTYPE),
                     (dict(codes=N.PKV_INT8), N.PKV_ERR_INVALID_ARG),
                     (dict(sums=None), N.PKV_ERR_INVALID_ARG), (dict(cols=0), N.PKV_ERR_INVALID_ARG),
                     (dict(tokens=21 * 16, wsb=n.value), N.PKV_ERR_INVALID_ARG)):
        assert call(**kw) == code, kw
    assert lib.pkv_decode_weights_workspace_size_tokens(2, 4, 16, 8, 2, 128, N.PKV_BF16, 8, 20,
                                                        None) == N.PKV_ERR_INVALID_ARG
