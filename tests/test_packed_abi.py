"""What the calls on packed sequences refuse on the host (no GPU needed: the
calls return before any CUDA work), their sizes, and the rotation's tables."""
import ctypes
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def fa():
    from exact_attention_98_gb300 import build

    build.build()
    from exact_attention_98_gb300 import fa

    return fa


P = ctypes.c_void_p
A = 0x100000
BIG = 1 << 40


def block(fa, data=A, row=1024, head=128):
    return ctypes.byref(fa.Rows(data, row, head))


def plan(fa, cu=A, n=3, rows=100, causal=1, plan=A, nbytes=BIG):
    return fa.lib.fa_packed_plan(P(cu), n, rows, causal, P(plan), nbytes, None)


def forward(fa, plan=A, n=3, rows=100, lse=A, H=4, Hkv=2, d=128, scale=0.1, ws=0, nbytes=0, **t):
    r = [t.get(x, block(fa)) for x in ("q", "k", "v", "o")]
    return fa.lib.fa_fwd_packed(P(plan), n, rows, *r, P(lse), H, Hkv, d, scale, P(ws), nbytes, None)


def backward(fa, plan=A, n=3, rows=100, lse=A, H=4, Hkv=2, d=128, scale=0.1, ws=A, nbytes=BIG, **t):
    r = [t.get(x, block(fa)) for x in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")]
    return fa.lib.fa_bwd_packed(P(plan), n, rows, *r[:4], P(lse), *r[4:], H, Hkv, d, scale, P(ws), nbytes, None)


def rotate(fa, H=4, Hkv=2, pos=A, rows=100, d=128, rope=A, length=50, rot=128, inter=0, back=0, **t):
    r = [t.get(x, block(fa)) for x in ("q", "q_out", "k", "k_out")]
    return fa.lib.fa_rotate(r[0], r[1], H, r[2], r[3], Hkv, P(pos), rows, d, P(rope), length, rot, inter, back, None)


def test_plan_is_checked(fa):
    bad, un, ws = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE
    need = fa.fa_packed_plan_bytes(3, 100)
    for kw, want in ((dict(n=-1), bad), (dict(rows=-1), bad), (dict(causal=2), bad), (dict(cu=0), bad),
                     (dict(cu=A + 2), bad), (dict(rows=2 ** 30 + 1), un), (dict(n=2 ** 30 + 1), un), (dict(plan=0), ws),
                     (dict(plan=A + 16), ws), (dict(nbytes=need - 1), ws), (dict(rows=0, cu=0, plan=0), fa.FA_OK)):
        assert plan(fa, **kw) == want, kw


def test_plan_bytes(fa):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731

    def want(n, rows):
        tiles = [up(16 * (rows // size + min(n, rows))) for size in (128, 256)]
        return 256 + up(4 * rows) + 2 * tiles[0] + tiles[1]

    for n, rows in ((1, 1), (3, 100), (5, 2), (0, 7), (1000, 1 << 20), (1 << 30, 1 << 30)):
        assert fa.fa_packed_plan_bytes(n, rows) == want(n, rows)
    for n, rows in ((-1, 5), (3, 0), (3, -1), (2 ** 30 + 1, 5)):
        assert fa.fa_packed_plan_bytes(n, rows) == 0


def test_plan_bytes_hold_every_batch(fa):
    """The lists' places for any lengths: a tile that is not full for each sequence with rows."""
    r = np.random.default_rng(0)
    for _ in range(200):
        n, rows = int(r.integers(1, 40)), int(r.integers(1, 3000))
        cuts = np.sort(r.integers(0, rows + 1, n + 1))
        for size in (128, 256):
            assert sum(-(-int(x) // size) for x in np.diff(cuts)) <= rows // size + min(n, rows)


@pytest.mark.parametrize("call", [forward, backward])
def test_attention_is_checked(fa, call):
    bad, un = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw, want in ((dict(n=-1), bad), (dict(rows=-1), bad), (dict(H=-1), bad), (dict(Hkv=-1), bad), (dict(Hkv=3), bad),
                     (dict(Hkv=0), bad), (dict(scale=0.0), bad), (dict(scale=float("nan")), bad),
                     (dict(scale=float("inf")), bad), (dict(d=96), un), (dict(plan=0), bad), (dict(plan=A + 128), bad),
                     (dict(lse=0), bad), (dict(lse=A + 2), bad), (dict(rows=2 ** 30 + 1), un),
                     (dict(rows=2 ** 30, H=2 ** 12, Hkv=2), un)):
        assert call(fa, **kw) == want, kw
    assert call(fa, n=0) == fa.FA_OK
    assert call(fa, rows=0, plan=0) == fa.FA_OK
    assert call(fa, H=0) == fa.FA_OK


ROWS = [
    None,                              # no tensor
    dict(data=0), dict(data=A + 8),
    dict(row=1020), dict(head=132),    # not multiples of 8
    dict(row=-1024), dict(head=-128),
    dict(row=0), dict(head=0),         # one row or head for all
    dict(row=64), dict(head=64),       # rows of d elements overlap
    dict(row=128, head=128),           # a token's heads are the next token's
    dict(row=376, head=128),
    dict(row=128, head=99 * 128),      # a head's last row is the next head's first
    dict(row=1 << 38), dict(head=1 << 38),
]


@pytest.mark.parametrize("rows", ROWS)
def test_rows_are_checked(fa, rows):
    t = None if rows is None else block(fa, **rows)
    for x in ("q", "k", "v", "o"):
        if x in "kv" and rows == dict(row=376, head=128):
            continue  # enough for two heads
        assert forward(fa, **{x: t}) == fa.FA_ERR_INVALID_ARG, x
    for x in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
        if x in ("k", "v", "dk", "dv") and rows == dict(row=376, head=128):
            continue
        assert backward(fa, **{x: t}) == fa.FA_ERR_INVALID_ARG, x
    for x in ("q", "q_out"):
        assert rotate(fa, **{x: t}) == fa.FA_ERR_INVALID_ARG, x


def test_forward_workspace(fa):
    """Optional, where there are few items of long sequences; a short or misaligned one is refused."""
    need = fa.fa_fwd_packed_workspace_bytes(1, 4096, 4, 2, 128)
    assert need >= 2 * 4096 * 4 * (128 * 4 + 4)
    kw = dict(n=1, rows=4096, H=4, Hkv=2)
    for bad in (dict(nbytes=need - 1), dict(nbytes=BIG, ws=A + 64)):
        assert forward(fa, **{**kw, "ws": A, **bad}) == fa.FA_ERR_WORKSPACE, bad
    for a in ((0, 4096, 4, 2, 128), (1, 0, 4, 2, 128), (1, 4096, 0, 2, 128), (1, 4096, 4, 3, 128), (1, 4096, 4, 2, 96),
              (-1, 4096, 4, 2, 128), (1, 1, 1, 1, 64), (100, 4096, 4, 2, 128), (1, 4096, 64, 8, 128),
              (1, 2 ** 30, 1, 1, 64)):
        assert fa.fa_fwd_packed_workspace_bytes(*a) == 0, a


def test_backward_workspace(fa):
    need = fa.fa_bwd_packed_workspace_bytes(3, 100, 4, 2, 128)
    assert need >= 100 * 4 * (2 * 4 + 128 * 4)
    for kw in (dict(ws=0), dict(nbytes=need - 1), dict(ws=A + 64)):
        assert backward(fa, **kw) == fa.FA_ERR_WORKSPACE, kw
    for a in ((0, 100, 4, 2, 128), (3, 0, 4, 2, 128), (3, 100, 0, 2, 128), (3, 100, 4, 3, 128), (3, 100, 4, 2, 96),
              (-1, 100, 4, 2, 128), (1, 2 ** 30, 4, 2, 128)):
        assert fa.fa_bwd_packed_workspace_bytes(*a) == 0, a
    assert backward(fa, n=1, rows=2 ** 29, H=8, Hkv=8) == fa.FA_ERR_UNSUPPORTED


def test_rotate_is_checked(fa):
    bad, un = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw, want in ((dict(rows=-1), bad), (dict(H=-1), bad), (dict(Hkv=-1), bad), (dict(length=-1), bad),
                     (dict(inter=2), bad), (dict(back=-1), bad), (dict(d=96), un), (dict(rot=0), bad), (dict(rot=8), bad),
                     (dict(rot=24), bad), (dict(rot=144), bad), (dict(pos=0), bad), (dict(pos=A + 1), bad),
                     (dict(rope=0), bad), (dict(rope=A + 8), bad), (dict(rows=2 ** 30 + 1), un),
                     (dict(rows=2 ** 30, H=4), un), (dict(H=2 ** 28), un)):
        assert rotate(fa, **kw) == want, kw
    assert rotate(fa, rows=0, pos=0) == fa.FA_OK
    assert rotate(fa, H=0, Hkv=0, pos=0) == fa.FA_OK


def test_binding_refuses_host_tensors(fa):
    cu = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.packed_plan(cu, 4)
    host = fa.PackedPlan(torch.zeros(1024, dtype=torch.uint8), 4, 2, True)
    with pytest.raises(ValueError, match="PackedPlan"):
        fa.packed_forward(x, x, x, cu)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.packed_forward(x, x, x, host)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.packed_backward(x, x, x, x, torch.zeros(4, 2), x, host)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.rotate(x, x, cu, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.rotate(None, None, cu, torch.zeros(4, 64))


def test_rope_table(fa):
    length, rot, base = 40, 32, 10000.0
    rate = [base ** (-2 * i / rot) for i in range(rot // 2)]

    def check(rates, magnitude=1.0, **kw):
        got = fa.rope_table(length, rot, base, device="cpu", magnitude=magnitude, **kw).double().numpy()
        angle = np.arange(length)[:, None] * np.array(rates)
        want = magnitude * np.concatenate([np.cos(angle), np.sin(angle)], 1)
        assert np.abs(got - want).max() <= 2.0 ** -24 * magnitude

    check(rate)
    check([r / 4 for r in rate], scale=4.0)
    check(rate, magnitude=1.25)
    # by parts: few turns over the length trained on are stretched, many are kept
    trained, low, high = 2048, 1.0, 32.0
    mixed = []
    for r in rate:
        turns = trained * r / (2 * math.pi)
        kept = min(1.0, max(0.0, (turns - low) / (high - low)))
        mixed.append(kept * r + (1 - kept) * r / 8)
    assert mixed[0] == rate[0] and mixed[-1] == rate[-1] / 8 and any(r / 8 < m < r for m, r in zip(mixed, rate))
    check(mixed, scale=8.0, trained=trained, turns=(low, high))
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(trained=-1), dict(turns=(3.0, 3.0)), dict(turns=(-1.0, 2.0))):
        with pytest.raises(ValueError):
            fa.rope_table(length, rot, base, device="cpu", **kw)
