"""The window backward's workspace follows the device it is asked for on."""
import pytest
import torch


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,N", [(1, 1, 40000), (2, 4, 8192), (1, 16, 3000), (3, 200, 700), (1, 1, 5000)])
def test_parts_of_the_first_tokens(B, Hkv, N):
    """Two parts to a multiprocessor over all key heads, of 16 rows at least, 256 to a head at most, and
    the main kernel's: each dK and dV of the first tokens in fp32."""
    from exact_attention_98_gb300 import fa

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    heads, d = B * Hkv, 64
    slots = max(1, min(256, 2 * sms // heads))
    rows = -(-(-(-N // slots)) // 16) * 16
    slots = -(-N // rows)
    with_tokens, without = (fa.fa_bwd_window_workspace_bytes(B, 2 * Hkv, Hkv, N, d, 100, s) for s in (9, 0))
    assert with_tokens - without == (slots + 1) * heads * 2 * 16 * d * 4
