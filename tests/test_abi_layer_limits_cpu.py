"""Sizes of the attention that no launch holds, and the largest that one does:
checks of the C ABI that need no GPU (the fake addresses are refused before any
HIP call)."""

import pytest

import bit_nf4_quantized_12_amd as q
from tests import test_abi_layer_cpu as base


@pytest.fixture(scope="module")
def lib():
    return q.load_library()


# (B + 7) H against 2^24 - 256 (forward: workgroups of 256 threads), 2^23 - 256 (backward: 512)
@pytest.mark.parametrize("B,H,Hkv", [(65535, 256, 256), (65535, 256, 1), (256, 65535, 1), (65529, 256, 8), (65528, 256, 8)])
def test_sequences_times_heads(lib, B, H, Hkv):
    a = base._attn(B=B, H=H, Hkv=Hkv, max_q=1, max_k=1)
    assert base._attn_calls(lib, a) == (base.SHAPE, base.SHAPE)


@pytest.mark.parametrize("B,H,fits", [(65535, 128, False), (65527, 128, False), (65526, 128, True), (121, 65535, False),
                                      (120, 65535, True)])
def test_sequences_times_heads_of_the_backward(lib, B, H, fits):
    assert fits == ((B + 7) * H < 2 ** 23 - 256)
    a = base._attn(B=B, H=H, Hkv=1, max_q=1, max_k=1)
    assert (lib.qlora_window_attn_bwd_workspace_bytes(a) > 0) == fits


@pytest.mark.parametrize("longest,window", [(512, 256), (1664, 256), (4096, 4096)])
def test_first_tokens_take_no_workspace_where_no_kernel_of_theirs_runs(lib, longest, window):
    # (longest <= 2 (64 + window) + 1024: key block 0 walks over all its queries itself)
    size = lambda sinks: lib.qlora_window_attn_bwd_workspace_bytes(  # noqa: E731
        base._attn(B=400, Tq=400 * longest, Tk=400 * longest, H=64, Hkv=64, D=128, max_q=longest, max_k=longest,
                   window=window, sinks=sinks))
    assert size(4) == size(0) > 0
    far = dict(B=4, Tq=4 * 9000, Tk=4 * 9000, H=64, Hkv=64, D=128, max_q=9000, max_k=9000, window=window)
    assert (lib.qlora_window_attn_bwd_workspace_bytes(base._attn(**far, sinks=4))
            > lib.qlora_window_attn_bwd_workspace_bytes(base._attn(**far, sinks=0))) == (9000 > 2 * (64 + window) + 1024)
