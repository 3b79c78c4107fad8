"""What the paged cache's calls refuse on the host (no GPU needed: the calls
return before any CUDA work), and the block sizes."""
import ctypes

import numpy as np
import pytest
import torch

from paged import E2M1, E4M3, nearest, quantise, values


@pytest.fixture(scope="module")
def fa():
    from exact_attention_98_gb300 import build

    build.build()
    from exact_attention_98_gb300 import fa

    return fa


P = ctypes.c_void_p
A = 0x100000


def cache(fa, **kw):
    f = dict(pages=A, page_table=A, seq_lens=A, k_scale=None, v_scale=None, format=0, B=2, Hkv=2, d=128, num_pages=4,
             page_size=64, max_pages=3)
    f.update(kw)
    return fa.PagedCache(*[f[n] for n, _ in fa.PagedCache._fields_])


def append(fa, c=None, k=A, k_row=256, k_head=128, v=A, cu=A, rows=5, q=A, q_row=512, q_out=A, H=4, rope=A, rope_len=9,
           rot=128, inter=0):
    c = cache(fa) if c is None else c
    return fa.lib.fa_paged_append(ctypes.byref(c), P(k), k_row, k_head, P(v), 256, 128, P(cu), rows, P(q), q_row, 128,
                                  P(q_out), H, P(rope), rope_len, rot, inter, None)


def read(fa, c=None, cu=A, rows=5, k=A, v=A):
    c = cache(fa) if c is None else c
    return fa.lib.fa_paged_read(ctypes.byref(c), P(cu), rows, P(k), P(v), None)


def forward(fa, c=None, q=A, q_row=512, o=A, lse=A, cu=A, rows=5, max_new=1, H=4, scale=0.1, window=0, sinks=0, ws=A,
            nbytes=1 << 40):
    c = cache(fa) if c is None else c
    return fa.lib.fa_fwd_paged(ctypes.byref(c), P(q), q_row, 128, P(o), P(lse), P(cu), rows, max_new, H, scale, window,
                               sinks, P(ws), nbytes, None)


def test_block_bytes(fa):
    n = fa.fa_paged_block_bytes
    assert n(0, 64, 128) == 2 * 64 * 256
    assert n(1, 64, 128) == 2 * 64 * (64 + 8)
    assert n(1, 16, 64) == 2 * 16 * (32 + 4)
    for bad in ((2, 64, 128), (-1, 64, 128), (0, 8, 128), (0, 48, 128), (0, 256, 128), (0, 64, 96)):
        assert n(*bad) == 0


@pytest.mark.parametrize("call", [append, read, forward])
def test_cache_is_checked(fa, call):
    bad, un = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw, want in ((dict(B=-1), bad), (dict(Hkv=-1), bad), (dict(num_pages=-1), bad), (dict(max_pages=-2), bad),
                     (dict(num_pages=0), bad), (dict(max_pages=0), bad), (dict(format=2), un), (dict(d=96), un),
                     (dict(page_size=48), un), (dict(page_size=0), un), (dict(pages=0), bad), (dict(page_table=0), bad),
                     (dict(seq_lens=0), bad), (dict(pages=A + 8), bad), (dict(page_table=A + 2), bad),
                     (dict(k_scale=A), bad),  # factors belong to 4-bit caches
                     (dict(num_pages=2 ** 30), un), (dict(max_pages=2 ** 30), un), (dict(format=1, v_scale=A + 1), bad)):
        assert call(fa, cache(fa, **kw)) == want, kw
    assert call(fa, rows=-1) == bad
    assert call(fa, cu=0) == bad
    # nothing to do
    assert call(fa, cache(fa, B=0, pages=0, page_table=0, seq_lens=0)) == fa.FA_OK
    assert call(fa, cache(fa, Hkv=0)) == fa.FA_OK
    assert call(fa, rows=0) == fa.FA_OK


def test_null_cache(fa):
    assert fa.lib.fa_paged_read(None, P(A), 1, P(A), P(A), None) == fa.FA_ERR_INVALID_ARG


def test_append_arguments(fa):
    bad = fa.FA_ERR_INVALID_ARG
    for kw in (dict(k=0), dict(v=0), dict(k=A + 8), dict(k_row=12), dict(k_head=4), dict(k_head=64), dict(k_row=-256),
               dict(q=A + 2), dict(q_row=100), dict(q_out=0), dict(q_out=A + 8), dict(H=0), dict(H=-1), dict(rope=0),
               dict(rope=A + 4), dict(rope_len=-1), dict(rot=-16), dict(rot=8), dict(rot=144), dict(inter=2)):
        assert append(fa, **kw) == bad, kw


def test_forward_arguments(fa):
    bad = fa.FA_ERR_INVALID_ARG
    for kw in (dict(q=0), dict(q=A + 8), dict(q_row=4), dict(o=0), dict(o=A + 8), dict(lse=0), dict(lse=A + 2),
               dict(H=3), dict(H=-2), dict(max_new=0), dict(max_new=-1), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=-1), dict(sinks=-1)):
        assert forward(fa, **kw) == bad, kw
    assert forward(fa, max_new=2 ** 31 - 1) == fa.FA_ERR_UNSUPPORTED
    assert forward(fa, H=0) == fa.FA_OK
    assert forward(fa, ws=0) == fa.FA_ERR_WORKSPACE
    assert forward(fa, ws=A + 16) == fa.FA_ERR_WORKSPACE
    assert fa.fa_fwd_paged_workspace_bytes(96) == 0


def test_read_arguments(fa):
    for kw in (dict(k=0), dict(v=0), dict(k=A + 2), dict(v=A + 8)):
        assert read(fa, **kw) == fa.FA_ERR_INVALID_ARG


def test_binding_refuses(fa):
    """Host tensors, wrong types and shapes raise before any C call."""
    host = torch.zeros(2, 1, 2, 16, 64, dtype=torch.bfloat16)
    ints = torch.zeros(1, 2, dtype=torch.int32)
    row = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.paged_append(row, row, host, ints, ints[0], ints[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.paged_forward(row, host, ints, ints[0], ints[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.paged_read(host, ints, ints[0], ints[0], 1, 64)
    with pytest.raises(ValueError, match="expected q"):
        fa.paged_forward(row[0], host, ints, ints[0], ints[0])
    with pytest.raises(ValueError, match="expected k"):
        fa.paged_append(row[0], row, host, ints, ints[0], ints[0])
    with pytest.raises(ValueError, match="format"):
        fa.paged_pages(1, 1, 16, 64, "int4", device="cpu")
    with pytest.raises(ValueError, match="page_size"):
        fa.paged_pages(1, 1, 24, 64, device="cpu")


def test_pages_and_rotation_table(fa):
    assert fa.paged_pages(3, 2, 16, 64, device="cpu").shape == (3, 2, 2, 16, 64)
    p4 = fa.paged_pages(3, 2, 16, 64, "fp4", device="cpu")
    assert p4.shape == (3, 2, 2, 16 * 36) and p4.dtype == torch.uint8
    assert p4[0, 0].numel() == fa.fa_paged_block_bytes(fa.FA_CACHE_FP4, 16, 64)
    t = fa.rope_table(70000, 64, device="cpu").double().numpy()
    p, i = 69999, 3
    angle = p * 10000.0 ** (-2 * i / 64)
    assert abs(t[p, i] - np.cos(angle)) <= 2.0 ** -24 and abs(t[p, 32 + i] - np.sin(angle)) <= 2.0 ** -24


def test_plain_4_bits():
    """The tests' own 4-bit format: its levels, its ties, and the error of a value (half a gap of codes,
    and the scale's rounding where the block's largest magnitude is cut off)."""
    assert E4M3[-1] == 448.0 and E4M3[1] == 2.0 ** -9 and len(E4M3) == 127
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 100.0])
    assert list(E2M1[nearest(x, E2M1)]) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0]
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)).astype(np.float32)
    code, byte = quantise(x, 0.7)
    v = values(code, byte, 0.7)
    amax = np.abs(x).reshape(50, 4, 16).max(-1).repeat(16, -1)
    # gaps of at most 2 scales; a scale is at most 2^-4 off amax / 6, so the top code 2^-4 of amax
    assert (np.abs(v - x) <= amax * (1 / 6 + 2.0 ** -4) * 1.07).all()
