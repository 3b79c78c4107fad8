"""The paged cache on the GPU: appending and reading rows, and attention over
the cache, against plain 64-bit implementations.

Tolerances.  A rounding to bf16 is off by 2^-8 of the value at most, to fp16 by
2^-11 (and by 2^-25 below 2^-14).  O: each weight of P rounded (bf16 cache:
2^-8, 4-bit cache: 2^-11) against sum p|v|, then O itself to bf16; scores are
fp32 sums of up to 128 products, off by 2^-17 of their largest sum |q k| (128
roundings of 2^-24), which moves weights by that share, twice (the weight and
the sum of weights).  LSE: the scores' error and a few fp32 roundings."""
import numpy as np
import pytest
import torch

from paged import Batch, attend, quantise, values

pytestmark = pytest.mark.gpu


def rand_q(T, H, d, seed=1, amplitude=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, d, generator=g) * amplitude).to(torch.bfloat16)


def ok(fa):
    assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())


def check_attention(bt, q, o, lse, window, sinks, scale, only=None):
    o, lse, q64 = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    p_eps = 2.0 ** -8 if bt.fmt == "bf16" else 2.0 ** -11
    for b, length in enumerate(bt.lens):
        if only is not None and b not in only:
            continue
        at = slice(bt.cu_list[b], bt.cu_list[b + 1])
        ref, l_ref, mag, dot = attend(q64[at], bt.rows[0][b], bt.rows[1][b], length, window, sinks, scale)
        s_err = 2.0 ** -17 * dot + 2.0 ** -20
        vmax = np.abs(bt.rows[1][b]).max() if length else 0.0
        bound = mag * (p_eps + 2 * s_err[..., None]) + 2.0 ** -8 * np.abs(ref) * 1.01 + length * 2.0 ** -25 * vmax + 1e-30
        err = np.abs(o[at] - ref)
        assert (err <= bound).all(), (b, float((err / bound).max()))
        empty = np.isinf(l_ref)
        assert np.array_equal(np.isneginf(lse[at]), empty)
        l_bound = s_err + 2.0 ** -20 * np.abs(np.where(empty, 0, l_ref))
        assert (np.abs(lse[at][~empty] - l_ref[~empty]) <= l_bound[~empty]).all()


CASES = [
    # fmt, d, page, Hkv, group, lens, new, window, sinks
    ("bf16", 128, 64, 2, 4, [1, 63, 64, 65, 700], [1] * 5, 0, 0),
    ("fp4", 128, 64, 2, 4, [1, 63, 64, 65, 700], [1] * 5, 0, 0),
    ("bf16", 64, 16, 1, 1, [5, 130, 16], [1, 1, 1], 0, 0),
    ("fp4", 64, 16, 1, 1, [5, 130, 16], [1, 1, 1], 0, 0),
    ("bf16", 128, 128, 3, 5, [300, 129, 64], [3, 1, 2], 0, 0),
    ("fp4", 128, 128, 3, 5, [300, 129, 64], [3, 1, 2], 0, 0),
    ("fp4", 64, 128, 2, 8, [513, 127], [4, 5], 0, 0),
    ("bf16", 64, 32, 2, 8, [513, 127], [4, 5], 0, 0),
    # windows and first tokens: window shorter than a tile, sinks across tiles, overlapping the window
    ("bf16", 128, 32, 2, 4, [1000, 40, 257], [1, 1, 1], 100, 4),
    ("fp4", 128, 32, 2, 4, [1000, 40, 257], [1, 1, 1], 100, 4),
    ("fp4", 128, 16, 1, 2, [1000, 333], [5, 3], 1, 0),
    ("bf16", 64, 64, 1, 2, [1000, 333], [5, 3], 1, 70),
    ("fp4", 64, 64, 1, 3, [777, 64], [2, 2], 300, 500),
    ("bf16", 128, 16, 1, 3, [777, 64], [2, 2], 640, 130),
    # sequences without positions, without new rows, with more new rows than positions before
    ("bf16", 128, 64, 1, 4, [0, 90, 0, 33], [1, 0, 0, 33], 0, 0),
    ("fp4", 128, 64, 1, 4, [0, 90, 0, 33], [1, 0, 0, 33], 16, 2),
    # a chunk of new rows longer than the tile
    ("bf16", 128, 64, 1, 2, [260], [200], 50, 3),
    ("fp4", 64, 32, 2, 1, [260], [200], 0, 0),
]


@pytest.mark.parametrize("fmt,d,page,Hkv,group,lens,new,window,sinks", CASES)
def test_attention(fmt, d, page, Hkv, group, lens, new, window, sinks):
    bt = Batch(fmt, d, page, Hkv, lens, new, seed=len(lens) + d)
    q = rand_q(bt.T, Hkv * group, d)
    o, lse = bt.forward(q.cuda(), window=window, sinks=sinks)
    ok(bt.fa)
    check_attention(bt, q, o, lse, window, sinks, bt.fa.default_scale(d))


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_many_sequences_of_all_lengths(fmt):
    """More sequences than a CTA has threads, a few of them long: pieces that hold many segments,
    segments that go through many CTAs."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 397)]
    lens[0], lens[200], lens[396] = 6000, 2500, 3001
    bt = Batch(fmt, 64, 16, 1, lens, [int(n > 0) for n in lens], seed=5)
    q = rand_q(bt.T, 2, 64)
    o, lse = bt.forward(q.cuda(), window=0, sinks=0)
    ok(bt.fa)
    check_attention(bt, q, o, lse, 0, 0, 0.125)


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_one_long_sequence(fmt):
    """One segment per key head, cut through all CTAs; peaked scores (Q of 6 standard deviations)
    move the running maxima."""
    bt = Batch(fmt, 128, 64, 2, [40001], [1], seed=7)
    q = rand_q(1, 6, 128, amplitude=6.0)
    o, lse = bt.forward(q.cuda())
    ok(bt.fa)
    check_attention(bt, q, o, lse, 0, 0, bt.fa.default_scale(128))


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("amplitude", [2.0 ** -60, 2.0 ** 40])
def test_magnitudes_of_q(fmt, amplitude):
    """Q far outside fp16's range, with a scale that brings the scores back."""
    bt = Batch(fmt, 128, 32, 1, [150], [2], seed=9)
    q = rand_q(2, 4, 128, amplitude=amplitude)
    scale = 0.1 / amplitude
    o, lse = bt.forward(q.cuda(), scale=scale)
    ok(bt.fa)
    check_attention(bt, q, o, lse, 0, 0, scale)


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_masked_places_hold_anything(fmt):
    """Cached positions that no row sees are NaN, the ones after the sequence too (see Batch):
    the result is that of a clean cache, bit for bit."""
    lens, new, window, sinks = [500, 131], [2, 1], 70, 5
    outs = []
    for dirty in (False, True):
        bt = Batch(fmt, 128, 32, 1, lens, new, seed=11, poison=dirty)
        if dirty:
            for b, n in enumerate(lens):
                for j in range(sinks, n - new[b] - window + 1):
                    at, off = bt.table[b, j // 32], j % 32
                    if fmt == "bf16":
                        bt.pages[at, :, :, off] = float("nan")
                    else:  # the scales
                        bt.pages[at, :, :, 32 * 64 + off * 8: 32 * 64 + off * 8 + 8] = 0x7F
        q = rand_q(bt.T, 3, 128)
        outs.append(bt.forward(q.cuda(), window=window, sinks=sinks))
        ok(bt.fa)
        check_attention(bt, q, *outs[-1], window, sinks, bt.fa.default_scale(128))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_nan_that_is_seen_is_reported(fmt):
    """A NaN in a visible row reaches O and LSE of the rows that see it, and of no other."""
    bt = Batch(fmt, 64, 16, 1, [80, 80], [1, 1], seed=13)
    at, off = bt.table[1, 2], 3
    if fmt == "bf16":
        bt.pages[at, 0, 0, off, 5] = float("nan")
    else:
        bt.pages[at, 0, 0, 16 * 32 + off * 4] = 0x7F
    q = rand_q(2, 2, 64)
    o, lse = bt.forward(q.cuda())
    ok(bt.fa)
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    check_attention(bt, q, o, lse, 0, 0, 0.125, only=[0])


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_strided_q_and_padding_rows(fmt):
    """Q as a slice of a fused projection, with padding rows behind the last sequence: the results of
    contiguous rows, and the padding of O and LSE as it was."""
    d, Hkv, H = 128, 2, 6
    bt = Batch(fmt, d, 64, Hkv, [130, 77], [2, 1], seed=15)
    q = rand_q(bt.T, H, d)
    want = bt.forward(q.cuda())
    fused = torch.randn(bt.T + 4, H + 2 * Hkv, d, dtype=torch.float32).to(torch.bfloat16).cuda()
    fused[: bt.T, Hkv: Hkv + H] = q.cuda()
    part = fused[:, Hkv: Hkv + H]
    fa = bt.fa
    o = torch.full((bt.T + 4, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bt.T + 4, H), 5.0, device="cuda")
    cache = fa._paged_cache(bt.pages, bt.page_table, bt.seq_lens, d, **bt.kw)
    ws = torch.full((fa.fa_fwd_paged_workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
    fa.fa_fwd_paged(cache, part, part.stride(0), part.stride(1), o, lse, bt.cu, bt.T + 4, 2, H,
                    fa.default_scale(d), 0, 0, ws)
    ok(fa)
    assert torch.equal(o[: bt.T], want[0]) and torch.equal(lse[: bt.T], want[1])
    assert (o[bt.T:] == 3.0).all() and (lse[bt.T:] == 5.0).all()


# --- append and read ---------------------------------------------------------------


def turn(x, pos, table, rot, interleaved):
    """fp32 rotation of rows [T, heads, d] at positions pos, each product and sum rounded."""
    x = x.astype(np.float32).copy()
    half = rot // 2
    a = np.arange(half) * (2 if interleaved else 1)
    b = a + (1 if interleaved else half)
    cos, sin = table[pos][:, None, :half], table[pos][:, None, half:]
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = xa * cos - xb * sin, xb * cos + xa * sin
    return x


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("d,page,rot,interleaved,Hkv,group,lens,new", [
    (128, 64, 128, False, 2, 4, [70, 1, 200], [5, 1, 130]),
    (128, 16, 64, True, 1, 3, [70, 1, 200], [5, 1, 130]),
    (64, 128, 16, False, 3, 1, [300, 128], [299, 1]),
    (64, 32, 64, True, 8, 8, [33, 0, 32, 31], [1, 0, 32, 31]),
    (128, 32, 0, False, 2, 2, [6000], [5500]),  # several tokens to a block of threads
])
def test_append_and_read(fmt, d, page, rot, interleaved, Hkv, group, lens, new):
    """Every byte of the cache after an append: the new rows' as rounded by the definition, all others
    as before; Q rotated; strided inputs with padding rows; and the rows read back."""
    bt = Batch(fmt, d, page, Hkv, lens, new, seed=d + rot)
    fa, H, T = bt.fa, Hkv * group, bt.T
    fused = torch.randn(T + 3, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    if T > 4:
        fused[0] = 0.0                      # blocks of zeros
        fused[1] *= 2.0 ** -40              # scales that round to zero
        fused[2] *= 2.0 ** 30               # scales at their largest
        fused[3, H:, : d // 2: 16] = 24.0   # exact borders: block scale 4
        fused[3, H:, 1: d // 2: 16] = 1.0
        fused[3, H:, 2: d // 2: 16] = 14.0
    q_big = fused.cuda()
    q, k, v = q_big[:, :H], q_big[:, H:H + Hkv], q_big[:, H + Hkv:]
    rope = fa.rope_table(max(lens) + 1, rot) if rot else None
    before = bt.pages.clone()
    q_out = fa.paged_append(k, v, *bt.tables(), q=q, rope=rope, interleaved=interleaved, **bt.kw)
    ok(fa)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]).astype(int)
    seq = np.concatenate([np.full(m, b) for b, m in enumerate(new)]).astype(int)
    host = fused[:T].float().numpy()
    table = None if rope is None else rope.cpu().numpy()
    t = (lambda x: turn(x, pos, table, rot, interleaved)) if rot else (lambda x: x)
    assert torch.equal(q_out[:T].cpu(), bf16(t(host[:, :H])))
    want = before.cpu().clone()
    k_read, v_read = (torch.zeros(T, Hkv, d) for _ in range(2))
    for kv, x, out in ((0, t(host[:, H:H + Hkv]), k_read), (1, host[:, H + Hkv:], v_read)):
        for h in range(Hkv):
            g = 1.0 if bt.k_scale is None else float((bt.k_scale, bt.v_scale)[kv][h])
            if fmt == "fp4":
                code, byte = quantise(x[:, h], g)
                f32 = values(code, byte, 1.0).astype(np.float32) * np.float32(g)
                out[:, h] = torch.from_numpy(f32)
            else:
                out[:, h] = bf16(x[:, h]).float()
            for i in range(T):
                at, off = bt.table[seq[i], pos[i] // page], pos[i] % page
                if fmt == "bf16":
                    want[at, h, kv, off] = bf16(x[i, h])
                else:
                    n = page * d // 2
                    want[at, h, kv, off * (d // 2):(off + 1) * (d // 2)] = torch.from_numpy(code[i, 0::2] | (code[i, 1::2] << 4))
                    want[at, h, kv, n + off * (d // 16): n + (off + 1) * (d // 16)] = torch.from_numpy(byte[i])
    view = lambda x: x.cpu().contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(view(bt.pages), view(want))
    got_k, got_v = fa.paged_read(*bt.tables(), T + 3, d, **bt.kw)
    ok(fa)
    assert torch.equal(got_k[:T].cpu(), k_read.to(torch.bfloat16))
    assert torch.equal(got_v[:T].cpu(), v_read.to(torch.bfloat16))


def test_every_scale():
    """Each e4m3 scale there is, with elements on, just below and just above every border between its
    codes: the codes of the definition, byte for byte."""
    from exact_attention_98_gb300 import fa
    from paged import E2M1, E4M3

    d, T = 64, 0
    rows = []
    for s in E4M3[1:]:
        # largest magnitude 6 s (its sixth is s exactly); the others around the borders
        borders = np.float32((E2M1[1:] + E2M1[:-1]) / 2 * s)
        x = np.concatenate([[6 * s], borders, np.nextafter(borders, np.float32(0))[:4],
                            np.nextafter(borders, np.float32(np.inf))[3:]]).astype(np.float32)
        rows.append(np.concatenate([x, np.zeros(16 - len(x), np.float32)]))
    blocks = np.stack(rows)
    # bf16 holds the borders times a scale (7 bits); what it rounds away from them stays a number to quantise
    k = bf16(np.concatenate([blocks, -blocks, blocks[::-1], blocks], 1)).cuda()[:, None]
    T = k.shape[0]
    pages = fa.paged_pages(8, 1, 16, d, "fp4")
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([T], [0, T]))
    for g in (None, 1.0, 0.7, 3.3e-7):
        f = None if g is None else torch.tensor([g], device="cuda")
        x = k if g is None else (k.float() * g).to(torch.bfloat16)
        fa.paged_append(x, x, pages, table, lens, cu, k_scale=f, v_scale=f)
        ok(fa)
        raw = pages[:, 0, 0].cpu().numpy()
        codes, scales = raw[:, : 16 * 32].reshape(-1, 32)[:T], raw[:, 16 * 32:].reshape(-1, 4)[:T]
        want, byte = quantise(x[:, 0].float().cpu().numpy(), 1.0 if g is None else g)
        assert np.array_equal(scales, byte)
        assert np.array_equal(codes, want[:, 0::2] | (want[:, 1::2] << 4))


def test_append_of_what_is_not_finite():
    """4 bits: a block with an infinity or a NaN reads back as NaN, its neighbours as they are."""
    bt = Batch("fp4", 64, 16, 1, [1], [1], scales=False)
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 3], k[0, 0, 40] = float("inf"), float("nan")
    bt.fa.paged_append(k, k, *bt.tables())
    got, _ = bt.fa.paged_read(*bt.tables(), 1, 64)
    ok(bt.fa)
    nan = torch.isnan(got[0, 0])
    # a block of ones: 1/6 lies between the e4m3 values 5/32 and 11/64, nearer to 11/64 (off by 1/192
    # against 1/96); 1 / (11/64) = 5.8 goes to the code of 6, which stands for 6 * 11/64
    assert nan[:16].all() and nan[32:48].all() and (got[0, 0][~nan] == 6 * 11 / 64).all() and int(nan.sum()) == 32


def test_padding_rows_are_left():
    """q_out's, k's and v's rows behind the last sequence keep their bytes (through the C names)."""
    bt = Batch("bf16", 64, 16, 1, [3], [2])
    fa = bt.fa
    x = torch.randn(5, 1, 64).to(torch.bfloat16).cuda()
    out, k, v = (torch.full((5, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    cache = fa._paged_cache(bt.pages, bt.page_table, bt.seq_lens, 64, None, None)
    fa.fa_paged_append(cache, x, 64, 64, x, 64, 64, bt.cu, 5, x, 64, 64, out, 1, None, 0, 0, False)
    fa.fa_paged_read(cache, bt.cu, 5, k, v)
    ok(fa)
    for got in (out, k, v):
        assert torch.equal(got[:2], x[:2]) and (got[2:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_places_past_32_bits(fmt):
    """Pages whose byte offsets pass 2^32: append, read and attention there."""
    from exact_attention_98_gb300 import fa

    d, page, Hkv = 128, 128, 2
    n = 2 ** 33 // (Hkv * fa.fa_paged_block_bytes(fa.FA_CACHE_FP4 if fmt == "fp4" else 0, page, d)) + 3
    pages = fa.paged_pages(n, Hkv, page, d, fmt)
    table = torch.tensor([[n - 1, 0], [n // 2, n - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([130, 200], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 130, 330], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(330, Hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    fa.paged_append(k, v, pages, table, lens, cu)
    k2, v2 = fa.paged_read(pages, table, lens, cu, 330, d)
    q = torch.randn(2, 4, d, generator=g).to(torch.bfloat16).cuda()
    cu1 = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    o, lse = fa.paged_forward(q, pages, table, lens, cu1)
    ok(fa)
    if fmt == "bf16":
        assert torch.equal(k2, k) and torch.equal(v2, v)
    small = fa.paged_pages(4, Hkv, page, d, fmt)
    table2 = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    fa.paged_append(k, v, small, table2, lens, cu)
    o2, lse2 = fa.paged_forward(q, small, table2, lens, cu1)
    k3, v3 = fa.paged_read(small, table2, lens, cu, 330, d)
    ok(fa)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(k2, k3) and torch.equal(v2, v3)


# --- together, in graphs, on streams -------------------------------------------------


@pytest.mark.parametrize("fmt,window,sinks", [("bf16", 0, 0), ("fp4", 0, 0), ("bf16", 40, 3), ("fp4", 40, 3)])
def test_prompt_then_steps(fmt, window, sinks):
    """A prompt and then tokens one by one, as a model serves them: append (rotating Q and K), attend;
    against 64-bit attention over the rows that the cache then reads back."""
    from exact_attention_98_gb300 import fa

    d, page, Hkv, H, B = 64, 16, 2, 4, 2
    prompt, steps = [37, 5], 12
    rope = fa.rope_table(128, d)
    pages = fa.paged_pages(12, Hkv, page, d, fmt)
    table = torch.arange(12, dtype=torch.int32, device="cuda").flip(0).view(2, 6).contiguous()
    g = torch.Generator().manual_seed(6)
    lens = [0, 0]
    for step in range(steps + 1):
        new = prompt if step == 0 else [1, 1]
        lens = [a + b for a, b in zip(lens, new)]
        T = sum(new)
        fused = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, new[0], T], dtype=torch.int32, device="cuda")
        q = fa.paged_append(fused[:, H:H + Hkv], fused[:, H + Hkv:], pages, table, sl, cu, q=fused[:, :H], rope=rope)
        o, lse = fa.paged_forward(q, pages, table, sl, cu, max_new=max(new), window=window, sinks=sinks)
        ok(fa)
        every = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
        k, v = fa.paged_read(pages, table, sl, every, sum(lens), d)
        ok(fa)

        class Now:
            pass

        bt = Now()
        bt.fmt, bt.lens, bt.cu_list = fmt, lens, [0, new[0], T]
        split = lambda x: [x[: lens[0]].double().cpu().numpy(), x[lens[0]:].double().cpu().numpy()]  # noqa: E731
        bt.rows = [split(k), split(v)]
        check_attention(bt, q, o, lse, window, sinks, fa.default_scale(d))


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_graph_replays_follow_the_lengths(fmt):
    """A step captured once and replayed while the lengths grow gives the eager step's bits; two graphs
    with workspaces of their own on two streams do not disturb each other."""
    from exact_attention_98_gb300 import fa

    d, page, Hkv, H, B = 128, 32, 2, 4, 3
    n_pages = 20
    table = torch.arange(B * n_pages, dtype=torch.int32, device="cuda").view(B, n_pages)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    rope = fa.rope_table(n_pages * page, d)
    graphs = []
    for which in range(2):
        s = torch.cuda.Stream()
        st = dict(s=s, pages=fa.paged_pages(B * n_pages, Hkv, page, d, fmt),
                  lens=torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda"),
                  fused=torch.zeros(B, H + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda"),
                  ws=torch.empty(fa.fa_fwd_paged_workspace_bytes(d), dtype=torch.uint8, device="cuda"))

        def step(st=st):
            f = st["fused"]
            q = fa.paged_append(f[:, H:H + Hkv], f[:, H + Hkv:], st["pages"], table, st["lens"], cu, q=f[:, :H], rope=rope)
            return fa.paged_forward(q, st["pages"], table, st["lens"], cu, workspace=st["ws"])

        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        st["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(st["graph"], stream=s):
            st["out"] = step()
        st["step"] = step
        st["pages"].zero_()
        graphs.append(st)
    eager = fa.paged_pages(B * n_pages, Hkv, page, d, fmt)
    torch.cuda.synchronize()
    for length in (1, 2, 31, 32, 33, 500, 640):
        for which, st in enumerate(graphs):
            st["lens"].copy_(torch.tensor([length, max(1, length // 2), 1], dtype=torch.int32))
            st["fused"].copy_(torch.randn(B, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(length)).to(torch.bfloat16))
        torch.cuda.synchronize()
        for st in graphs:
            with torch.cuda.stream(st["s"]):
                st["graph"].replay()
        torch.cuda.synchronize()
        ok(fa)
        assert torch.equal(graphs[0]["out"][0], graphs[1]["out"][0])
        assert torch.equal(graphs[0]["pages"], graphs[1]["pages"])
        f = graphs[0]["fused"]
        q = fa.paged_append(f[:, H:H + Hkv], f[:, H + Hkv:], eager, table, graphs[0]["lens"], cu, q=f[:, :H], rope=rope)
        o, lse = fa.paged_forward(q, eager, table, graphs[0]["lens"], cu)
        assert torch.equal(o, graphs[0]["out"][0]) and torch.equal(lse, graphs[0]["out"][1])


def test_a_stream_of_its_own():
    """stream=: work goes to that stream, in order with it, and the results' memory belongs to it."""
    bt = Batch("bf16", 128, 64, 2, [3000, 200], [1, 1], seed=21)
    q = rand_q(2, 8, 128).cuda()
    want = bt.forward(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        o, lse = bt.forward(q, stream=s)
        noise = torch.full_like(o, 9.0)  # takes freed memory of the current stream, if any were shared
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        del noise
    ok(bt.fa)


# --- tables that cannot be followed ----------------------------------------------------


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_bad_tables_are_reported(fmt):
    """A page outside the cache, a sequence longer than its pages, rows that do not fit, a position past
    the rotation's table: the status word says so, nothing outside is touched, and the batch's other
    sequence gets its result."""
    d, page, Hkv, H = 64, 16, 1, 2
    bt = Batch(fmt, d, page, Hkv, [40, 50], [1, 1], seed=23, max_pages=4)
    fa = bt.fa
    q = rand_q(2, H, d)
    want = bt.forward(q.cuda())
    k = torch.randn(2, Hkv, d).to(torch.bfloat16).cuda()
    ok(fa)

    def call(site, table=None, lens=None, cu=None, **kw):
        t = bt.page_table if table is None else table
        n = bt.seq_lens if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        c = bt.cu if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        before = bt.pages.clone()
        o, lse = fa.paged_forward(q.cuda(), bt.pages, t, n, c, **bt.kw)
        assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
        assert fa.fa_last_device_site() == site
        assert torch.equal(before.view(torch.uint8), bt.pages.view(torch.uint8))
        return o, lse

    for bad in (-1, bt.num_pages, 2 ** 31 - 1):
        t = bt.page_table.clone()
        t[1, 3] = bad
        o, lse = call(0x503, table=t)
        assert torch.equal(o[0], want[0][0]) and torch.equal(lse[0], want[1][0])
        before = bt.pages.clone()
        fa.paged_append(k, k, bt.pages, t, bt.seq_lens, bt.cu, **bt.kw)
        assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
        at = bt.table[0, 39 // page]
        others = [i for i in range(bt.num_pages) if i != at]
        assert torch.equal(before[others].view(torch.uint8), bt.pages[others].view(torch.uint8))
        bt.pages.copy_(before)
        r, _ = fa.paged_read(bt.pages, t, bt.seq_lens, bt.cu, 2, d, **bt.kw)
        assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
        assert (r[1] == 0).all()
    o, _ = call(0x502, lens=[40, 65])
    assert torch.equal(o[0], want[0][0])
    o, _ = call(0x502, lens=[40, -7])
    assert torch.equal(o[0], want[0][0])
    call(0x501, cu=[0, 1, 3])      # past the rows
    call(0x501, cu=[0, 1, -5])
    call(0x501, cu=[-3, 1, 2])
    call(0x501, cu=[0, 0, 2])      # two rows where max_new is 1
    before = bt.pages.clone()
    fa.paged_append(k, k, *bt.tables(), rope=fa.rope_table(49, d), **bt.kw)  # position 49 has no angles
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_last_device_site() == 0x502
    assert torch.equal(bt.pages[int(bt.table[1, 3])].view(torch.uint8), before[int(bt.table[1, 3])].view(torch.uint8))


def test_launches_are_counted():
    bt = Batch("bf16", 64, 16, 1, [40], [1])
    fa = bt.fa
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    counts = []
    for call in (lambda: fa.paged_append(x, x, *bt.tables()), lambda: fa.paged_read(*bt.tables(), 1, 64),
                 lambda: bt.forward(x)):
        n0 = fa.fa_launch_count()
        call()
        counts.append(fa.fa_launch_count() - n0)
    ok(fa)
    assert counts == [1, 1, 2]


def test_empty_calls():
    """No sequences, no rows, no heads: nothing runs, nothing is wrong."""
    from exact_attention_98_gb300 import fa

    pages = fa.paged_pages(2, 1, 16, 64)
    none = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    n0 = fa.fa_launch_count()
    assert fa.paged_append(none, none, pages, table, lens, cu, q=none).shape == (0, 1, 64)
    o, lse = fa.paged_forward(none, pages, table, lens, cu)
    assert o.shape == (0, 1, 64) and lse.shape == (0, 1)
    k, v = fa.paged_read(pages, table, lens, cu, 0, 64)
    assert k.shape == v.shape == (0, 1, 64)
    o, lse = fa.paged_forward(none, pages, table[:0], lens[:0], cu[:1])
    assert fa.fa_launch_count() == n0
    ok(fa)
