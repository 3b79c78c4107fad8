"""Gradients over packed sequences on the GPU where the backward walks many tiles
sequence by sequence, dK and dV at offsets past 32 bits, and the binding's calls of the
C functions against the public ones (tests/packed.py has the plain forms and bounds)."""
import ctypes

import numpy as np
import pytest
import torch

from packed import HALF, batch, check_backward, f64, plain_backward, rows, within

LENGTHS = [129 + 37 * i % 400 for i in range(60)]


def tiles(lengths):
    return sum((n + 127) // 128 for n in lengths)


def parts(lengths, rows_, H, Hkv, d):
    """What the workspace says: parts of each item (1: not split)."""
    from exact_attention_98_gb300 import fa

    whole = 256 + 2 * ((rows_ * H * 4 + 255) // 256 * 256) + (rows_ * H * d * 4 + 255) // 256 * 256
    n = (fa.fa_bwd_packed_workspace_bytes(len(lengths), rows_, H, Hkv, d) - whole) // (2 * Hkv * rows_ * d * 4)
    return max(n, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,H,Hkv,split", [
    (LENGTHS, 2, 1, False),
    (LENGTHS, 3, 3, False),
    (LENGTHS, 4, 2, False),
    ([1, 700, 0, 128] + LENGTHS, 4, 4, False),
    ([129 + i % 2 for i in range(77)], 64, 1, True),
])
@pytest.mark.parametrize("causal", [True, False])
def test_many_tiles(lengths, H, Hkv, split, causal, d):
    """More than 152 tiles in sequences of several: key tiles in the order of the sequences."""
    from exact_attention_98_gb300 import fa

    assert tiles(lengths) > 152 and max(lengths) > 128
    cu, n = batch(lengths, 5, 70)
    assert (parts(lengths, n, H, Hkv, d) > 1) == split
    q, k, v, do = rows(n, H, d, 1), rows(n, Hkv, d, 2), rows(n, Hkv, d, 3), rows(n, H, d, 4)
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    o, lse = fa.packed_forward(q, k, v, plan)
    grads = fa.packed_backward(q, k, v, o, lse, do, plan)
    assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
    check_backward(grads, q, k, v, o, lse, do, cu, fa.default_scale(d), causal)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_key_gradients_past_32_bits(d):
    """Every element of dK and dV, summed over a group, at the end of tensors of more than 2^31 elements."""
    from exact_attention_98_gb300 import fa

    H, Hkv, lengths = 256, 2, [300, 77]
    G = H // Hkv
    n = 2 ** 31 // (H * d) + 1000
    cu, n = batch(lengths, n - sum(lengths), 5)
    first = cu[0]
    assert first * H * d > 2 ** 31
    q, k, v, do = (torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv, H))
    for i, t in enumerate((q, k, v, do)):
        t[first:] = rows(n - first, t.shape[1], d, i, "dense")
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
    o, lse = fa.packed_forward(q, k, v, plan)
    _, dk, dv = fa.packed_backward(q, k, v, o, lse, do, plan)
    assert fa.fa_last_device_status() == fa.FA_OK
    q, k, v, o, lse, do, dk, dv = (f64(t[first:]) for t in (q, k, v, o, lse, do, dk, dv))
    for b in range(len(lengths)):
        s = slice(cu[b] - first, cu[b + 1] - first)
        for hk in range(Hkv):
            want, err = [0, 0], [0, 0]
            for h in range(hk * G, hk * G + G):
                g, e = plain_backward(q[s, h], k[s, hk], v[s, hk], o[s, h], lse[s, h], do[s, h],
                                      fa.default_scale(d), True)
                want = [x + y for x, y in zip(want, g[1:])]
                err = [x + y for x, y in zip(err, e[1:])]
            for got, x, e, name in ((dk, want[0], err[0], "dk"), (dv, want[1], err[1], "dv")):
                within(got[s, hk], x, e + HALF * 1.01 * np.abs(x), (name, b, hk))


def described(t):
    from exact_attention_98_gb300 import fa

    return ctypes.byref(fa.Rows(t.data_ptr(), t.stride(0), t.stride(1)))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_direct_calls(d):
    """fa_fwd_packed, fa_bwd_packed and fa_rotate of the binding give what the public calls give."""
    from exact_attention_98_gb300 import fa

    lengths, H, Hkv = [300, 1, 77], 4, 2
    cu, n = batch(lengths)
    q, k, v, do = rows(n, H, d, 1), rows(n, Hkv, d, 2), rows(n, Hkv, d, 3), rows(n, H, d, 4)
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
    table = fa.rope_table(300, d // 2)
    for backward in (False, True):
        want = fa.rotate(q, k, plan.positions, table, True, backward)
        q2, k2 = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        fa.fa_rotate(described(q), described(q2), H, described(k), described(k2), Hkv, plan.positions, n, d, table,
                     300, d // 2, True, backward)
        assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    o, lse = fa.packed_forward(q, k, v, plan)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    fa.fa_fwd_packed(plan.plan, len(lengths), n, described(q), described(k), described(v), described(o2), lse2, H, Hkv,
                     d, fa.default_scale(d))
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    want = fa.packed_backward(q, k, v, o, lse, do, plan)
    got = [torch.zeros_like(t) for t in want]
    ws = torch.empty(fa.fa_bwd_packed_workspace_bytes(len(lengths), n, H, Hkv, d), dtype=torch.uint8, device="cuda")
    fa.fa_bwd_packed(plan.plan, len(lengths), n, described(q), described(k), described(v), described(o), lse,
                     described(do), *map(described, got), H, Hkv, d, fa.default_scale(d), ws)
    assert fa.fa_last_device_status() == fa.FA_OK
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    check_backward(got, q, k, v, o, lse, do, cu, fa.default_scale(d), True)
