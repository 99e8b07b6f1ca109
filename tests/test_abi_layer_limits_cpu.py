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
