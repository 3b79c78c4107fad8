"""Rotation of rows by their positions, and its transpose, against a plain 64-bit
implementation: products and sums in fp32 (2^-24 each of the magnitudes), one
rounding to bf16 (2^-8 of the value)."""
import numpy as np
import pytest
import torch

from packed import batch, f64, rows, within


def plain(x, pos, table, inter, backward):
    """[n, heads, d] -> the rotated rows and their error bounds."""
    rot = table.shape[1]
    out, err = x.copy(), np.zeros_like(x)
    cos, sin = table[pos, : rot // 2][:, None], table[pos, rot // 2:][:, None] * (-1 if backward else 1)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    xa, xb = x[..., a], x[..., b]
    for at, u, w in ((a, xa * cos, -xb * sin), (b, xb * cos, xa * sin)):
        out[..., at] = u + w
        err[..., at] = 2.0 ** -8 * 1.01 * np.abs(u + w) + 2.0 ** -22 * (np.abs(u) + np.abs(w))
    return out, err


def check(n, H, Hkv, d, rot, inter, backward, layout="fused", length=200, seed=0):
    from exact_attention_98_gb300 import fa

    q, k = rows(n, H, d, seed, layout), rows(n, Hkv, d, seed + 1, layout)
    table = fa.rope_table(length, rot)
    pos = torch.randint(0, length, (n,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    got = fa.rotate(q, k, pos, table, interleaved=inter, backward=backward)
    assert fa.fa_last_device_status() == fa.FA_OK
    for x, y in zip((q, k), got):
        ref, err = plain(f64(x), pos.cpu().numpy(), f64(table), inter, backward)
        within(f64(y), ref, err, (rot, inter, backward))
    return q, k, pos, table, got


@pytest.mark.gpu
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 32), (64, 64), (128, 48), (128, 64), (128, 128)])
def test_rotate(d, rot, inter, backward):
    check(77, 5, 2, d, rot, inter, backward, seed=rot)


@pytest.mark.gpu
@pytest.mark.parametrize("n,H,Hkv,layout", [(1, 1, 1, "dense"), (1, 32, 8, "fused"), (33, 4, 4, "heads"),
                                            (3000, 7, 1, "dense"), (5000, 32, 8, "fused")])
def test_sizes_and_layouts(n, H, Hkv, layout):
    check(n, H, Hkv, 128, 64, False, False, layout, seed=n)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_in_place_and_one_tensor(inter):
    from exact_attention_98_gb300 import fa

    q, k, pos, table, (q1, k1) = check(50, 4, 2, 64, 32, inter, False)
    only, none = fa.rotate(q, None, pos, table, interleaved=inter)
    assert none is None and torch.equal(only, q1)
    none, only = fa.rotate(None, k, pos, table, interleaved=inter)
    assert none is None and torch.equal(only, k1)
    assert fa.rotate(q, k, pos, table, interleaved=inter, out=(q, k))[0] is q
    assert torch.equal(q, q1) and torch.equal(k, k1)


@pytest.mark.gpu
def test_same_bits_as_append():
    """The paged cache's append rotates to the same bits."""
    from exact_attention_98_gb300 import fa

    for rot, inter in ((128, False), (64, True)):
        n, H, Hkv, d = 60, 4, 2, 128
        q, k, v = rows(n, H, d, 1), rows(n, Hkv, d, 2), rows(n, Hkv, d, 3)
        table = fa.rope_table(100, rot)
        pages = fa.paged_pages(4, Hkv, 16, d)
        tab = torch.arange(4, dtype=torch.int32, device="cuda")[None]
        lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, n]))
        want_q = fa.paged_append(k, v, pages, tab, lens, cu, q=q, rope=table, interleaved=inter)
        want_k, _ = fa.paged_read(pages, tab, lens, cu, n, d)
        plan = fa.packed_plan(cu, n)
        got_q, got_k = fa.rotate(q, k, plan.positions, table, interleaved=inter)
        assert torch.equal(got_q, want_q) and torch.equal(got_k, want_k)


@pytest.mark.gpu
def test_rows_without_a_position():
    """Padding rows are left as they were; a position past the table is recorded and its row left, too."""
    from exact_attention_98_gb300 import fa

    cu, n = batch([20, 13], 2, 5)
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
    q, k = rows(n, 3, 64, 0), rows(n, 1, 64, 1)
    q[:2], q[cu[-1]:] = float("nan"), float("nan")
    out = tuple(torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k))
    fa.rotate(q, k, plan.positions, fa.rope_table(20, 64), out=out)
    assert fa.fa_last_device_status() == fa.FA_OK
    pad = plan.positions < 0
    assert int(pad.sum()) == 7
    for x in out:
        assert (x[pad] == 7).all() and torch.isfinite(x).all() and not (x[~pad] == 7).all(-1).any()
    before = [x.clone() for x in out]
    fa.rotate(q, k, plan.positions, fa.rope_table(19, 64), out=out)
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
    for x, y in zip(out, before):  # row 19 of the first sequence has no place in the table
        assert torch.equal(x[cu[0] + 19], y[cu[0] + 19])


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    """The transpose against differences of sum(y w): the map is linear, so a step of 1 along each element
    gives its gradient, here as one product with the rotated identity."""
    from exact_attention_98_gb300 import fa

    d, rot = 64, 32
    table = fa.rope_table(50, rot) * 1.25  # a scaled table: not a rotation alone
    pos = torch.full((d,), 37, dtype=torch.int32, device="cuda")
    eye = torch.eye(d, dtype=torch.bfloat16, device="cuda")[:, None]
    columns = fa.rotate(eye, None, pos, table, interleaved=inter)[0][:, 0]  # row j: the image of element j
    back = fa.rotate(eye, None, pos, table, interleaved=inter, backward=True)[0][:, 0]
    assert torch.equal(back, columns.T)
