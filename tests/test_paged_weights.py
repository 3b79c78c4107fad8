"""4-bit paged attention with weights spread over many powers of two: one
dominating position over a long even tail, as a first token that a model rests
its attention on.

The cache is written by hand, so that every score is exact: Q is 1 in its first
element, K is 0 but for the dominating position, whose score is `bits` ln 2.
Then a tail position weighs 2^-bits of the dominating one, O is
n 2^-bits / (1 + n 2^-bits) where V is 1 in the tail and 0 in the dominating
position, and LSE is bits ln 2 + ln(1 + n 2^-bits).  The sequence is in the batch often
enough for a warp to hold it whole (parts of one that is cut up are joined in fp32).

Tolerances.  Weights are held to 2^-11 of themselves and, below 2^-21 of the
dominating one, to 2^-32 of that one; the score is an fp32 product of about
2^5, off by 2^-17 with the roundings of its factors, which moves the weights by
that share, twice; a lane adds an eighth of a sequence's weights in fp32, to 2^-24 each of
what it has, and so do the products; O is rounded to bf16 (2^-8)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

COPIES = 2000   # of a sequence: more than the warps on the GPU


def tail_cache(fa, d, page, n, at):
    """n tail positions and one dominating position `at`, pages in order, 4 bits."""
    length = n + 1
    pages = -(-length // page)
    raw = torch.zeros(pages, 1, 2, page * (d // 2 + d // 16), dtype=torch.uint8, device="cuda")
    raw[:, :, :, page * d // 2:] = 0x38      # every scale 1
    raw[:, :, 1, : page * d // 2] = 0x22     # V: every code 1
    p, r = at // page, at % page
    raw[p, 0, 0, r * (d // 2)] = 0x07        # K: 6 in the first element
    raw[p, 0, 1, r * (d // 2): (r + 1) * (d // 2)] = 0
    return raw, copies(torch.arange(pages)), copies(torch.tensor(length))


def copies(x):
    return x.to(torch.int32).cuda().expand(COPIES, *x.shape).contiguous()


@pytest.mark.parametrize("n,bits,d,page,group", [
    (40, 3.0, 128, 128, 1), (40, 3.0, 64, 16, 16), (5000, 12.0, 128, 32, 4), (5000, 12.0, 64, 64, 11),
    (131072, 25.0, 128, 128, 1), (131072, 25.0, 64, 64, 16), (40000, 24.5, 64, 16, 3), (40000, 24.5, 128, 32, 12),
    (1 << 20, 23.7, 64, 128, 2), (1 << 20, 25.0, 64, 128, 1), (1 << 20, 29.5, 64, 128, 1)])
def test_tail_under_one_position(n, bits, d, page, group):
    from exact_attention_98_gb300 import fa

    cu = torch.arange(COPIES + 1, dtype=torch.int32, device="cuda")
    q = torch.zeros(COPIES, group, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    tail = n * 2.0 ** -bits
    want, l_want = tail / (1 + tail), bits * math.log(2) + math.log1p(tail)
    for at in (0, n // 3, n):
        raw, table, lens = tail_cache(fa, d, page, n, at)
        o, lse = fa.paged_forward(q, raw, table, lens, cu, scale=bits * math.log(2) / 6)
        assert fa.fa_last_device_status() == fa.FA_OK
        sums = n * 2.0 ** -27
        err = (o.double() - want).abs().max().item()
        assert err <= want * (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -17 + 2 * sums) * 1.01 + n * 2.0 ** -32, (at, err, want)
        l_err = (lse.double() - l_want).abs().max().item()
        assert l_err <= 2.0 ** -19 + 2.0 ** -20 * l_want + sums, (at, l_err)


def test_peaks_after_one_another():
    """Positions that outweigh all before them by less than what makes the reference move, by it, and by
    far more, so that O and LSE come from weights far above the reference: within 64 bits' bounds."""
    from exact_attention_98_gb300 import fa

    d, page = 64, 64
    for step in (0.5, 7.0, 8.0, 14.9, 15.0, 15.1, 30.0):   # log2 units between the peaks
        pages = 8
        raw = torch.zeros(pages, 1, 2, page * (d // 2 + d // 16), dtype=torch.uint8, device="cuda")
        raw[:, :, :, page * d // 2:] = 0x38
        rng = np.random.default_rng(1)
        codes = rng.integers(0, 16, (pages, page, d))
        raw[:, 0, 1, : page * d // 2] = torch.from_numpy(
            (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(pages, -1).astype(np.uint8)).cuda()
        peak = np.zeros(pages * page)
        for i in range(pages):      # one in each page, i + 1 steps high: element i + 1 of K is 1, of Q i + 1
            raw[i, 0, 0, 17 * (d // 2) + (i + 1) // 2] = 0x02 << (4 * ((i + 1) % 2))
            peak[i * page + 17] = i + 1
        q = torch.zeros(COPIES, 1, d, dtype=torch.bfloat16, device="cuda")
        q[:, 0, 1:9] = torch.arange(1, 9)
        cu = torch.arange(COPIES + 1, dtype=torch.int32, device="cuda")
        o, lse = fa.paged_forward(q, raw, copies(torch.arange(pages)), copies(torch.tensor(pages * page)), cu,
                                  scale=step * math.log(2))
        assert fa.fa_last_device_status() == fa.FA_OK
        mag = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
        v = (np.where(codes >= 8, -1.0, 1.0) * mag[codes & 7]).reshape(-1, d)
        s = step * peak
        w = np.exp2(s - s.max())
        total = w.sum()
        ref = w @ v / total
        s_err = 2.0 ** -22 * s.max() + 2.0 ** -20     # the largest score's roundings, in log2 units
        bound = (w @ np.abs(v) / total) * (2.0 ** -11 + 2 * s_err) + np.abs(ref) * 2.0 ** -8 * 1.01 + len(s) * 6 * 2.0 ** -32
        err = np.abs(o[:, 0].double().cpu().numpy() - ref)
        assert (err <= bound).all(), (step, (err / bound).max())
        l_ref = (s.max() + np.log2(total)) * math.log(2)
        assert (lse[:, 0].double() - l_ref).abs().max().item() <= s_err + 2.0 ** -20 * abs(l_ref), step
