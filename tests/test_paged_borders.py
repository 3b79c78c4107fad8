"""4-bit rounding right beside its borders: numbers a last place or two away
from where one code, or one scale, turns into the next.

bf16 rows cannot hold such numbers, but K is rotated in fp32 on its way: with
sines of 0 and cosines of the test's choosing any fp32 number t arises, as a
power of two times t over it.  That what is left after the head's factor g lies on
both sides of every border is checked first."""
import numpy as np
import pytest
import torch

from paged import E2M1, E4M3, quantise

F = np.float32


def near(t):
    """t > 0 as a power of two, which bf16 holds, times an fp32 cosine in [1, 2): both exact."""
    x = (np.asarray(t, F).view(np.int32) & 0x7F800000).view(F)
    return x, (t / x).astype(F)


def steps(t, k):
    """The fp32 number k places above t > 0."""
    return (np.asarray(t, F).view(np.int32) + k).view(F)


def ulps(y, border):
    """How many places y is above the border, both positive fp32."""
    return np.asarray(y, F).view(np.int32).astype(np.int64) - np.asarray(border, F).view(np.int32)


def code_rows(g, k):
    """A row for each scale s, d = 64: its blocks of 16 hold 6 s g, the seven borders k places down and
    the seven k places up; elements 32 .. 63 are the same, negated."""
    s = E4M3[1:].astype(F)
    borders = ((E2M1[1:] + E2M1[:-1]) / 2).astype(F)[None] * s[:, None]     # exact
    t = (borders * F(g)).astype(F)
    block = np.concatenate([(6 * s * F(g))[:, None], steps(t, -k), steps(t, k), (s * F(g))[:, None]], 1)
    return near(np.concatenate([block, block], 1))


def scale_rows(g, k):
    """A row for each border between scales: a block with 6 times it k places down, one with k places up."""
    mid = ((E4M3[1:] + E4M3[:-1]) / 2 * 6).astype(F) * F(g)
    half = np.zeros((len(mid), 32), F) + (mid * F(0.25))[:, None]
    half[:, 3], half[:, 20] = steps(mid, -k), steps(mid, k)
    return near(half)


GS = [1.0, 0.7, 3.3e-7, 1536.5]
PLACES = [0, 1, 2, 3]


def rotated(x, c):
    y = (x * c).astype(F)
    return np.concatenate([y, -y], 1)


@pytest.mark.parametrize("g", GS)
def test_the_numbers_lie_on_both_sides(g):
    """Within two places above and below every border of every scale's codes; of the scales (a second
    quotient, by 6, steps up to four places at a time), within four."""
    s = E4M3[1:].astype(F)
    borders = ((E2M1[1:] + E2M1[:-1]) / 2).astype(F)[None] * s[:, None]
    y = np.concatenate([(rotated(*code_rows(g, k))[:, 1:15] / F(g)).reshape(len(s), 2, 7) for k in PLACES], 1)
    off = ulps(y, borders[:, None])
    assert ((off > 0) & (off <= 2)).any(1).all() and ((off < 0) & (off >= -2)).any(1).all()
    mid = ((E4M3[1:] + E4M3[:-1]) / 2).astype(F)
    y = np.stack([(rotated(*scale_rows(g, k))[:, [3, 20]] / F(g)).astype(F) / F(6) for k in PLACES], 1)
    off = ulps(y.reshape(len(mid), -1), mid[:, None])
    assert ((off > 0) & (off <= 4)).any(1).all() and ((off < 0) & (off >= -4)).any(1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("g", GS)
@pytest.mark.parametrize("rows", [code_rows, scale_rows])
def test_codes_and_scales_beside_the_borders(rows, g):
    """Byte for byte those of the definition."""
    from exact_attention_98_gb300 import fa

    d, page = 64, 64
    parts = [rows(g, k) for k in PLACES]
    x, c = (np.concatenate([p[i] for p in parts]) for i in range(2))
    T = len(x)
    k_rows = torch.from_numpy(np.concatenate([x, -x], 1)).to(torch.bfloat16).cuda()[:, None]
    rope = torch.from_numpy(np.concatenate([c, np.zeros_like(c)], 1)).cuda()     # [T, 64]: cosines, sines
    n = -(-T // page)
    pages = fa.paged_pages(n, 1, page, d, "fp4")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    lens, cu = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([T], [0, T]))
    f = torch.tensor([g], dtype=torch.float32, device="cuda")
    fa.paged_append(k_rows, torch.zeros_like(k_rows), pages, table, lens, cu, rope=rope, k_scale=f, v_scale=f)
    assert fa.fa_last_device_status() == fa.FA_OK
    raw = pages[:, 0, 0].cpu().numpy()
    codes, scales = raw[:, : page * 32].reshape(-1, 32)[:T], raw[:, page * 32:].reshape(-1, 4)[:T]
    want, byte = quantise(rotated(x, c), g)
    assert np.array_equal(scales, byte)
    assert np.array_equal(codes, want[:, 0::2] | (want[:, 1::2] << 4))
