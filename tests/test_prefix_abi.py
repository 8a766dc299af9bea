"""What fa_fwd_prefix refuses, before anything touches CUDA."""
import ctypes

import pytest
import torch

import exact_attention_114_b200 as fa

FAKE = ctypes.c_void_p(0x10000)
BAD, UNSUPPORTED = fa.FA_ERR_INVALID_ARGUMENT, fa.FA_ERR_UNSUPPORTED


def call(dtype=0, q=FAKE, kp=FAKE, lens=None, lse=None, B=4, Hq=8, Hkv=2, Nq=1, Np=500, Ns=64, d=128, scale=0.1, causal=1,
         ws=None, n=0):
    return fa.lib().fa_fwd_prefix(dtype, q, kp, FAKE, FAKE, FAKE, lens, FAKE, lse, B, Hq, Hkv, Nq, Np, Ns, d, scale, causal,
                                  ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), BAD), (dict(q=None), BAD), (dict(kp=ctypes.c_void_p(0x10004)), BAD), (dict(lens=ctypes.c_void_p(0x10001)), BAD),
    (dict(lse=ctypes.c_void_p(0x10003)), BAD), (dict(Np=0), BAD), (dict(Ns=0), BAD), (dict(Nq=0), BAD), (dict(B=0), BAD),
    (dict(Hq=7), BAD), (dict(causal=-1), BAD), (dict(scale=float("inf")), BAD), (dict(d=100), UNSUPPORTED), (dict(d=320), UNSUPPORTED),
    (dict(Np=1 << 30, Ns=1 << 20, Hkv=1, B=1), UNSUPPORTED), (dict(ws=ctypes.c_void_p(0x100080), n=1 << 30), BAD),
    (dict(ws=ctypes.c_void_p(0x100000), n=16), fa.FA_ERR_WORKSPACE),
])
def test_refuses(kw, status):
    assert call(**kw) == status and fa.last_error_message()


def test_workspace_sizes():
    assert fa.fa_fwd_prefix_workspace_size(4, 8, 2, 1, 500, 64, 128) > 4 * 8 * 128 * 4
    assert fa.fa_fwd_prefix_workspace_size(1, 8, 2, 17, 500, 64, 128) == 0     # one sequence: one launch of tiles
    assert fa.fa_fwd_prefix_workspace_size(4, 8, 2, 64, 500, 64, 128) == 0     # a sequence's rows fill a tile
    assert fa.fa_fwd_prefix_workspace_size(4, 8, 2, 1, 0, 64, 128) == 0


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Np,d,packs", [
    (8, 32, 8, 5, 128, 128, False), (8, 32, 8, 5, 2048, 128, False), (8, 32, 8, 5, 2049, 128, True), (2, 4, 1, 9, 32768, 128, False),
    (2, 4, 1, 9, 32769, 128, True), (2, 4, 1, 1, 200, 256, False), (64, 32, 8, 1, 300, 256, True), (1, 4, 1, 9, 90000, 128, False),
    (64, 32, 8, 17, 4096, 128, False),
])
def test_short_prefixes_are_read_per_sequence(B, Hq, Hkv, Nq, Np, d, packs):
    """More rows than the split-KV pass takes: up to 2048 tiles of 64 keys over the batch's kv heads (and 32768
    keys) one launch without partials of its own, beyond that the prefix in a pass of its own."""
    assert (fa.fa_fwd_prefix_workspace_size(B, Hq, Hkv, Nq, Np, 100, d) > 0) == packs


def test_binding_refuses():
    x, p = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 9, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_fwd_prefix(x, p, p, x, x)
