"""Tables of the paged cache that cannot be followed: what is skipped, what is
recorded, and what the rows that are left get.  Bounds as in test_paged.py."""
import numpy as np
import pytest
import torch

from paged import Batch

pytestmark = pytest.mark.gpu


def q_of(bt, H, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(bt.T, H, bt.d, generator=g).to(torch.bfloat16)


def on_gpu(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def status(fa):
    code = fa.fa_last_device_status()
    return code, fa.fa_last_device_site() if code != fa.FA_OK else 0


def attend_some(q, rows_k, rows_v, length, window, sinks, scale, gone):
    """64-bit attention of a sequence's last rows q [n, H, d] over its positions but those where `gone`
    holds: O, LSE, and the bounds' sum p |v| and largest sum |q k| (zeros where nothing is left)."""
    n, H, d = q.shape
    Hkv = rows_k.shape[1]
    o, mag = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, dot = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        p = length - n + i
        j = np.arange(max(p + 1, 0))
        keep = ~gone[j]
        if window:
            keep &= (p - j < window) | (j < sinks)
        j = j[keep]
        if len(j) == 0:
            continue
        for h in range(H):
            k, v = rows_k[j, h * Hkv // H], rows_v[j, h * Hkv // H]
            s = scale * (k @ q[i, h])
            w = np.exp(s - s.max())
            lse[i, h] = s.max() + np.log(w.sum())
            w /= w.sum()
            o[i, h], mag[i, h] = w @ v, w @ np.abs(v)
            dot[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return o, lse, mag, dot


def check_some(bt, q, o, lse, window, sinks, gone):
    p_eps = 2.0 ** -8 if bt.fmt == "bf16" else 2.0 ** -11
    o, lse, q64 = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for b, length in enumerate(bt.lens):
        at = slice(bt.cu_list[b], bt.cu_list[b + 1])
        ref, l_ref, mag, dot = attend_some(q64[at], bt.rows[0][b], bt.rows[1][b], length, window, sinks,
                                           bt.fa.default_scale(bt.d), gone[b])
        s_err = 2.0 ** -17 * dot + 2.0 ** -20
        bound = mag * (p_eps + 2 * s_err[..., None]) + 2.0 ** -8 * np.abs(ref) * 1.01 + length * 2.0 ** -32 * 6.0
        assert (np.abs(o[at] - ref) <= bound).all(), (b, np.nanmax(np.abs(o[at] - ref) / bound))
        empty = np.isinf(l_ref)
        assert np.array_equal(np.isneginf(lse[at]), empty), b
        assert (np.abs(lse[at][~empty] - l_ref[~empty]) <= (s_err + 2.0 ** -20 * np.abs(l_ref))[~empty]).all(), b


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("d,page,group,lens,new,window,sinks,bad", [
    # bad: (sequence, page of the sequence)
    (64, 16, 2, [200, 150], [1, 1], 0, 0, [(1, 2), (1, 9)]),
    (128, 16, 12, [333, 50, 90], [2, 1, 1], 0, 0, [(0, 0), (0, 3), (0, 7), (2, 4), (2, 5)]),
    (128, 32, 4, [700, 260], [1, 3], 200, 5, [(0, 0), (0, 20), (1, 3)]),
    (64, 64, 1, [900, 64], [1, 1], 0, 0, [(0, 3), (1, 0)]),                 # nothing left of the second
    (128, 128, 4, [2000, 40], [4, 1], 0, 0, [(0, 0), (0, 15), (1, 0)]),
    (64, 16, 1, [17], [17], 0, 0, [(0, 0)]),                                # the first rows see nothing
])
def test_positions_on_pages_outside_the_cache_are_left_out(fmt, d, page, group, lens, new, window, sinks, bad):
    """They count as masked, in every row of every call, whatever the kernel's memory held before."""
    Hkv = 2
    bt = Batch(fmt, d, page, Hkv, lens, new, seed=sum(lens))
    fa = bt.fa
    q = q_of(bt, Hkv * group)
    other = Batch(fmt, d, page, Hkv, [5000, 300], [1, 1], seed=99)      # leaves rows of its own behind
    q_other = q_of(other, Hkv * group)
    gone = [np.zeros(n, bool) for n in lens]
    for b, i in bad:
        gone[b][i * page: (i + 1) * page] = True
    first = None
    for number in (-1, bt.num_pages, 2 ** 31 - 1, -2 ** 31):
        table = bt.table.copy()
        for b, i in bad:
            table[b, i] = number
        bt.page_table = on_gpu(table)
        other.forward(q_other.cuda())
        assert status(fa) == (fa.FA_OK, 0)
        o, lse = bt.forward(q.cuda(), window=window, sinks=sinks)
        assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x503)
        check_some(bt, q, o, lse, window, sinks, gone)
        first = (o, lse) if first is None else first
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_a_sequence_longer_than_its_pages_is_empty(fmt, window, sinks):
    """Its rows see nothing, as one of a negative length: its pages cannot say where they are.  The others
    are as before.  Append and read go by row: one whose position is past the pages has no place."""
    bt = Batch(fmt, 64, 16, 1, [40, 64, 33], [1, 2, 1], seed=3, max_pages=4)
    fa = bt.fa
    q = q_of(bt, 3)
    want = bt.forward(q.cuda(), window=window, sinks=sinks)
    assert status(fa) == (fa.FA_OK, 0)
    for length in (65, 66, 1000, 2 ** 31 - 1, -1, -2 ** 31):
        bt.seq_lens = on_gpu([40, length, 33])
        o, lse = bt.forward(q.cuda(), window=window, sinks=sinks)
        assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x502)
        assert (o[1:3] == 0).all() and torch.isneginf(lse[1:3]).all(), length
        for i in (0, 3):
            assert torch.equal(o[i], want[0][i]) and torch.equal(lse[i], want[1][i])
    bt.seq_lens = on_gpu([40, 65, 33])       # new rows at 63, which has a place, and 64
    x = torch.randn(4, 1, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    before = bt.pages.clone()
    fa.paged_append(x, x, *bt.tables(), **bt.kw)
    assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x502)
    places = [int(bt.table[0, 2]), int(bt.table[1, 3]), int(bt.table[2, 2])]
    others = [i for i in range(bt.num_pages) if i not in places]
    assert torch.equal(before[others].view(torch.uint8), bt.pages[others].view(torch.uint8))
    k, v = fa.paged_read(*bt.tables(), 4, 64, **bt.kw)
    assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x502)
    assert (k[2] == 0).all() and (v[2] == 0).all()
    bt.seq_lens = on_gpu([40, 64, 33])
    k2, v2 = fa.paged_read(bt.pages, bt.page_table, bt.seq_lens, on_gpu([0, 1, 2, 3]), 3, 64, **bt.kw)
    assert status(fa) == (fa.FA_OK, 0)
    for i, j in ((0, 0), (1, 1), (3, 2)):
        assert torch.equal(k[i], k2[j]) and torch.equal(v[i], v2[j])
    if fmt == "bf16":
        assert torch.equal(k[1], x[1]) and torch.equal(v[1], x[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks,new", [(40, 4, [1, 1]), (40, 0, [1, 1]), (100, 20, [3, 2]), (1, 1, [1, 1]),
                                              (130, 64, [17, 1])])
def test_pages_that_no_row_sees_may_be_freed(fmt, page, window, sinks, new):
    """A server that gives pages back as the window moves on leaves entries that name no page: nothing is
    recorded, and the results keep their bits."""
    lens = [777, 250]
    bt = Batch(fmt, 128, page, 2, lens, new, seed=page + window, max_pages=60)
    fa = bt.fa
    q = q_of(bt, 4)
    want = bt.forward(q.cuda(), window=window, sinks=sinks)
    assert status(fa) == (fa.FA_OK, 0)
    freed = 0
    for number in (-1, bt.num_pages):
        table = bt.table.copy()
        for b, n in enumerate(lens):
            for i in range(bt.max_pages):
                lo, hi = i * page, (i + 1) * page       # positions lo .. hi - 1
                seen = lo < n and (lo < sinks or hi > n - new[b] - window + 1)
                if not seen:
                    freed += lo < n
                    table[b, i] = number
        bt.page_table = on_gpu(table)
        o, lse = bt.forward(q.cuda(), window=window, sinks=sinks)
        assert status(fa) == (fa.FA_OK, 0)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert freed > 0


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_rows_that_do_not_fit_are_recorded_by_append_and_read(fmt):
    """A sequence whose rows reach past the tensors, start before them or run backwards: append and read
    leave it out and say so, as the attention does; what fits keeps its place."""
    bt = Batch(fmt, 64, 16, 1, [40, 50], [1, 1], seed=23, poison=False)
    fa = bt.fa
    x = torch.randn(2, 1, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    before = bt.pages.clone()
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    # offsets, and those of the sequences that are left (none said where a table runs backwards)
    for cu, left in (([0, 1, 3], [0, 1, 1]), ([0, 1, 2 ** 31 - 1], [0, 1, 1]), ([0, 2, 5], [0, 2, 2]),
                     ([0, 0, 3], [0, 0, 0]), ([-3, 1, 2], [1, 1, 2]), ([-1, -1, 2], [0, 0, 0]), ([0, 1, -5], None),
                     ([0, 5, 2], None)):
        c = on_gpu(cu)
        bt.pages.copy_(before)
        fa.paged_append(x, x, bt.pages, bt.page_table, bt.seq_lens, c, q=x, **bt.kw)
        assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x501), cu
        got = bt.pages.clone()
        k, v = fa.paged_read(bt.pages, bt.page_table, bt.seq_lens, c, 2, 64, **bt.kw)
        assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x501), cu
        if left is None:
            continue
        bt.pages.copy_(before)
        fa.paged_append(x, x, bt.pages, bt.page_table, bt.seq_lens, on_gpu(left), **bt.kw)
        want_k, want_v = fa.paged_read(bt.pages, bt.page_table, bt.seq_lens, on_gpu(left), 2, 64, **bt.kw)
        assert status(fa) == (fa.FA_OK, 0)
        assert torch.equal(raw(got), raw(bt.pages)), cu
        for i in range(left[0], left[2]):
            assert torch.equal(k[i], want_k[i]) and torch.equal(v[i], want_v[i]), cu
    # more sequences than a block has threads, the last of which does not fit
    n = 700
    bt = Batch(fmt, 64, 16, 1, [1] * n, [1] * n, seed=1, poison=False)
    x = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    c = bt.cu.clone()
    c[n] += 1
    fa.paged_append(x, x, bt.pages, bt.page_table, bt.seq_lens, c, **bt.kw)
    assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x501)
    fa.paged_read(bt.pages, bt.page_table, bt.seq_lens, c, n, 64, **bt.kw)
    assert status(fa) == (fa.FA_ERR_INVALID_ARG, 0x501)
