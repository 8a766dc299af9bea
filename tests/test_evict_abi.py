"""What the calls on keys' weights and on eviction refuse, before anything touches CUDA."""
import ctypes

import pytest
import torch

import exact_attention_114_b200 as fa

A = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(8)]   # far apart, never dereferenced
BAD = fa.FA_ERR_INVALID_ARGUMENT


def fwd(dtype=0, q=A[0], lse=A[4], w_in=None, w_out=A[6], Hq=2, Hkv=1, Nq=1, d=64, scale=0.1, causal=0):
    return fa.lib().fa_fwd_weights(dtype, q, A[1], A[2], A[3], lse, w_in, w_out, 1, Hq, Hkv, Nq, 300, d, scale, causal, None)


def keys(dtype=0, k=A[1], lse=A[4], w_in=None, w_out=A[6], d=64, causal=0):
    return fa.lib().fa_key_weights(dtype, A[0], k, lse, w_in, w_out, 1, 2, 1, 5, 300, d, 0.1, causal, None)


@pytest.mark.parametrize("call,kw,status", [
    (fwd, dict(dtype=3), BAD), (fwd, dict(q=None), BAD), (fwd, dict(w_out=None), BAD), (fwd, dict(Hq=3, Hkv=2), BAD),
    (fwd, dict(w_out=ctypes.c_void_p(0x10002)), BAD), (fwd, dict(w_in=ctypes.c_void_p(A[6].value + 4)), BAD),
    (fwd, dict(causal=2), BAD), (fwd, dict(scale=0.0), BAD), (fwd, dict(d=40), fa.FA_ERR_UNSUPPORTED),
    (fwd, dict(lse=ctypes.c_void_p(0x10001)), BAD),
    (keys, dict(lse=None), BAD), (keys, dict(k=None), BAD), (keys, dict(w_out=None), BAD), (keys, dict(dtype=-1), BAD),
    (keys, dict(w_in=ctypes.c_void_p(A[6].value - 1196)), BAD), (keys, dict(d=512), fa.FA_ERR_UNSUPPORTED),
])
def test_weights_refuse(call, kw, status):
    assert call(**kw) == status and fa.last_error_message()


def evict(dtype=0, k=A[0], v=A[1], w=A[2], lens=None, ko=A[3], vo=A[4], wo=A[5], io=A[6], B=1, Hkv=2, Nk=300, d=64, keep=20, recent=5):
    return fa.lib().fa_kv_evict(dtype, k, v, w, lens, ko, vo, wo, io, B, Hkv, Nk, d, keep, recent, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), BAD), (dict(k=None), BAD), (dict(w=None), BAD), (dict(vo=None), BAD), (dict(keep=0), BAD),
    (dict(recent=-1), BAD), (dict(recent=21), BAD), (dict(Nk=0), BAD), (dict(B=0), BAD), (dict(d=50), fa.FA_ERR_UNSUPPORTED),
    (dict(ko=A[0]), BAD), (dict(ko=A[1]), BAD), (dict(vo=A[3]), BAD), (dict(wo=A[2]), BAD), (dict(io=A[5]), BAD),
    (dict(lens=ctypes.c_void_p(A[6].value + 8)), BAD), (dict(lens=ctypes.c_void_p(0x10001)), BAD),
    (dict(keep=1 << 29, d=256), fa.FA_ERR_UNSUPPORTED),
])
def test_evict_refuses(kw, status):
    assert evict(**kw) == status and fa.last_error_message()


def test_binding_refuses():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_kv_evict(x, x, torch.zeros(1, 2, 4), 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_fwd_weights(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_key_weights(x, x, torch.zeros(1, 2, 4))
