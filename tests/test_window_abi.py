"""What the windowed calls refuse, before anything touches CUDA."""
import ctypes

import pytest
import torch

import exact_attention_114_b200 as fa

FAKE = ctypes.c_void_p(0x10000)


def fwd(dtype=0, q=FAKE, lse=None, B=1, Hq=2, Hkv=1, Nq=300, Nk=300, d=64, scale=0.1, window=10, sinks=0):
    return fa.lib().fa_fwd_window(dtype, q, FAKE, FAKE, FAKE, lse, B, Hq, Hkv, Nq, Nk, d, scale, window, sinks, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), fa.FA_ERR_INVALID_ARGUMENT), (dict(q=None), fa.FA_ERR_INVALID_ARGUMENT),
    (dict(q=ctypes.c_void_p(0x10008)), fa.FA_ERR_INVALID_ARGUMENT),
    (dict(lse=ctypes.c_void_p(0x10002)), fa.FA_ERR_INVALID_ARGUMENT),
    (dict(window=0), fa.FA_ERR_INVALID_ARGUMENT), (dict(window=-1), fa.FA_ERR_INVALID_ARGUMENT),
    (dict(sinks=-1), fa.FA_ERR_INVALID_ARGUMENT), (dict(Nq=0), fa.FA_ERR_INVALID_ARGUMENT),
    (dict(Hq=3, Hkv=2), fa.FA_ERR_INVALID_ARGUMENT), (dict(scale=-1.0), fa.FA_ERR_INVALID_ARGUMENT),
    (dict(d=80), fa.FA_ERR_UNSUPPORTED), (dict(d=288), fa.FA_ERR_UNSUPPORTED),
])
def test_forward_refuses(kw, status):
    assert fwd(**kw) == status and fa.last_error_message()


def test_backward_refuses():
    def bwd(ws=None, n=0, window=10, sinks=1, d=64, **over):
        return fa.lib().fa_bwd_window(0, *[FAKE] * 9, 1, 2, 1, 300, 300, d, 0.1, window, sinks, ws, n, None)

    assert bwd(window=0) == fa.FA_ERR_INVALID_ARGUMENT
    assert bwd(sinks=-5) == fa.FA_ERR_INVALID_ARGUMENT
    assert bwd(d=40) == fa.FA_ERR_UNSUPPORTED
    assert bwd(ws=ctypes.c_void_p(0x100010), n=1 << 30) == fa.FA_ERR_INVALID_ARGUMENT
    assert bwd(ws=ctypes.c_void_p(0x100000), n=1024) == fa.FA_ERR_WORKSPACE
    assert fa.fa_bwd_window_workspace_size(1, 2, 1, 300, 300, 64, 0) == 0
    assert fa.fa_bwd_window_workspace_size(1, 2, 1, 300, 300, 64, 10, -1) == 0
    assert fa.fa_bwd_window_workspace_size(1, 2, 1, 300, 300, 64, 10, 4) >= 2 * 2 * 320 * 4 + 2 * 320 * 64 * 4


@pytest.mark.parametrize("shape", [(1, 32, 8, 8192, 8192, 128, 4096, 4), (1, 32, 8, 8192, 8192, 128, 1024, 4),
                                   (1, 8, 1, 1500, 1500, 64, 1400, 4), (1, 2, 1, 2500, 2500, 256, 70, 200),
                                   (2, 8, 8, 1000, 1000, 64, 200, 1), (1, 8, 1, 2048, 2048, 128, 512, 0)], ids=str)
def test_workspace_holds_every_partial(shape):
    """The workspace's partials are the slots that the launch's units use: of a unit shared by n CTAs none for
    n = 1, one for n = 2, n for more, the sinks' units and the others each with their own n."""
    B, Hq, Hkv, Nq, Nk, d, window, sinks = shape
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    rows, kd = B * Hq * (-(-Nq // 64) * 64), 64 if d <= 64 else 128 if d <= 128 else 256
    least = 2 * up(rows * 4) + up(rows * kd * 4)
    split, sink_split = fa.fa_bwd_window_query_split(*shape)
    per_block = B * Hkv * (2 if kd == 256 else 1)
    n_kb, sink_kb = -(-Nk // 128), -(-min(sinks, Nk) // 128)
    slots = lambda n: 0 if n == 1 else 1 if n == 2 else n  # noqa: E731
    n = per_block * (sink_kb * slots(sink_split) + (n_kb - sink_kb) * slots(split))
    want = least if n == 0 else least + up(n * 2 * min(kd, 128) * 128 * 4) + up(per_block * n_kb * 8)
    assert fa.fa_bwd_window_workspace_size(*shape) == want
    assert fa.fa_bwd_window_query_split(1, 3, 2, 8, 8, 64, 1) == (0, 0)


def test_paged_refuses():
    def call(window=10, sinks=0, page=64, Nq=1, d=128, table=FAKE, ws=None, n=0):
        return fa.lib().fa_fwd_paged_window(0, FAKE, FAKE, FAKE, table, FAKE, FAKE, None, 2, 8, 2, Nq, d, page, 100,
                                            20, 0.1, window, sinks, ws, n, None)

    assert call(window=0) == fa.FA_ERR_INVALID_ARGUMENT
    assert call(sinks=-1) == fa.FA_ERR_INVALID_ARGUMENT
    assert call(page=32) == fa.FA_ERR_INVALID_ARGUMENT
    assert call(table=None) == fa.FA_ERR_INVALID_ARGUMENT
    assert call(Nq=8) == fa.FA_ERR_UNSUPPORTED
    assert call(d=256) == fa.FA_ERR_UNSUPPORTED
    need = fa.fa_fwd_paged_window_workspace_size(2, 8, 2, 1, 64, 20, 128, 500, 4)
    assert need > 0 and call(window=500, sinks=4, ws=ctypes.c_void_p(0x100000), n=need - 16) == fa.FA_ERR_WORKSPACE
    assert fa.fa_fwd_paged_window_workspace_size(2, 8, 2, 1, 64, 20, 128, 0, 4) == 0


def test_size_queries_leave_the_last_error():
    assert fwd(window=0) == fa.FA_ERR_INVALID_ARGUMENT
    message = fa.last_error_message()
    assert "window=0" in message
    for B in (1, 0):   # sizes that the calls take, and sizes that they refuse
        fa.fa_bwd_window_workspace_size(B, 2, 1, 300, 300, 64, 10, 4)
        fa.fa_bwd_window_query_split(B, 2, 1, 300, 300, 64, 10, 4)
        fa.fa_fwd_paged_window_workspace_size(B, 8, 2, 1, 64, 20, 128, 500, 4)
        fa.fa_fwd_prefix_workspace_size(B, 8, 2, 1, 500, 64, 128)
        assert fa.last_error_message() == message


def test_binding_refuses():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_fwd_window(x, x, x, 3)
    with pytest.raises(ValueError, match="dtype"):
        fa.fa_fwd_window(x.float(), x.float(), x.float(), 3)


def test_numbers_of_keys_that_do_not_fit_an_int():
    """Far below zero is refused as negative, not taken for its remainder; far above is the largest."""
    size, split = fa.fa_bwd_window_workspace_size, fa.fa_bwd_window_query_split
    shape = (1, 2, 1, 300, 300, 64)
    for n in (-1, -2 ** 31 - 5, -2 ** 32 + 10, -2 ** 40):
        assert size(*shape, n) == 0 and size(*shape, 10, n) == 0 and split(*shape, n) == (0, 0)
        assert fa.fa_fwd_paged_window_workspace_size(2, 8, 2, 1, 64, 20, 128, n, 4) == 0
    for n in (300, 2 ** 31, 2 ** 32 + 10, 2 ** 40):
        assert size(*shape, n, n) == size(*shape, 300, 300) > 0
