"""Sliding-window attention with first tokens and shared key heads on the GPU,
against a plain 64-bit implementation.

Tolerances, element by element.  A rounding to bf16 is off by 2^-8 of the value
at most.  Scores and dP are fp32 sums of up to 128 products: off by 2^-17 of
their largest sum of magnitudes (128 roundings of 2^-24).  In the backward at
d = 128 the row's LSE and D enter the products as a pair of bf16 numbers,
the second what the first leaves: off by 2^-16 of them.
  O     P rounded: 2^-8 sum p |v|; scores: twice their error (weight and sum of
        weights); O rounded
  LSE   scores, and a few fp32 roundings
  dV    P rounded, and its relative error from scores and LSE: sum (2^-8 + e) p |do|
  dS    rounded: 2^-8 |dS|; P's relative error e; dP's and D's errors times p
  dQ    scale sum |err dS| |k|, dK the same with |q|; all rounded at the end
with fp32 sums over up to 2^15 terms in any order (2^-24 each, far below)."""
import numpy as np
import pytest
import torch

from exact_attention_98_gb300.inputs import attention_inputs

HALF = 2.0 ** -8


def visible(N, window, sinks):
    i, j = np.arange(N)[:, None], np.arange(N)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def plain_forward(q, k, v, scale, window, sinks):
    """One head in 64 bits: O, LSE and the error bounds of both."""
    see = visible(len(q), window, sinks)
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    lse = (m + np.log(w.sum(1, keepdims=True)))[:, 0]
    p = w / w.sum(1, keepdims=True)
    o = p @ v
    s_err = 2.0 ** -17 * (scale * np.where(see, np.abs(q) @ np.abs(k).T, 0)).max(1) + 2.0 ** -20
    o_err = (HALF + 2 * s_err[:, None]) * (p @ np.abs(v)) + HALF * 1.01 * np.abs(o)
    return o, lse, o_err, s_err + 2.0 ** -20 * np.abs(lse)


def plain_backward(q, k, v, o, lse, do, scale, window, sinks):
    """One query head's gradients in 64 bits from the forward's O and LSE, and their error bounds
    (dK's and dV's before the final rounding: they are summed over a group)."""
    see = visible(len(q), window, sinks)
    s = scale * (q @ k.T)
    p = np.where(see, np.exp(np.where(see, s, -np.inf) - lse[:, None]), 0)
    dp = do @ v.T
    D = (do * o).sum(1, keepdims=True)
    ds = p * (dp - D)
    e = 2.0 ** -17 * scale * (np.abs(q) @ np.abs(k).T) + 2.0 ** -16 * np.abs(lse)[:, None] + 2.0 ** -20
    dp_err = 2.0 ** -17 * (np.abs(do) @ np.abs(v).T) + 2.0 ** -16 * (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
    ds_err = (HALF + e) * np.abs(ds) + p * dp_err
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    dq_err = scale * ds_err @ np.abs(k) + HALF * 1.01 * np.abs(dq)
    dk_err = scale * ds_err.T @ np.abs(q)
    dv_err = ((HALF + e) * p).T @ np.abs(do)
    return (dq, dk, dv), (dq_err, dk_err, dv_err)


def inputs(B, H, Hkv, N, d, seed):
    q, _, _, do = attention_inputs(B, H, N, d, seed=seed)
    _, k, v, _ = attention_inputs(B, Hkv, N, d, seed=seed + 1000)
    return q, k, v, do


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, err, what):
    bad = np.abs(got - ref) > err + 1e-30
    assert not bad.any(), (what, float((np.abs(got - ref) / (err + 1e-30)).max()), int(bad.sum()))


def check(B, H, Hkv, N, d, window, sinks, seed=0, scale=None, heads=None, backward=True):
    from exact_attention_98_gb300 import fa

    q, k, v, do = inputs(B, H, Hkv, N, d, seed)
    scale = fa.default_scale(d) if scale is None else scale
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = fa.window_forward(qd, kd, vd, window, sinks, scale=scale)
    assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
    if backward:
        grads = fa.window_backward(qd, kd, vd, o, lse, dod, window, sinks, scale=scale)
        assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
        dq, dk, dv = (f64(t) for t in grads)
    o, lse = f64(o), f64(lse)
    q, k, v, do = (f64(t) for t in (q, k, v, do))
    G = H // Hkv
    for b in range(B):
        for hk in range(Hkv) if heads is None else heads:
            sums = [np.zeros((N, d)) for _ in range(4)]
            for h in range(hk * G, hk * G + G):
                ref, l_ref, o_err, l_err = plain_forward(q[b, h], k[b, hk], v[b, hk], scale, window, sinks)
                within(o[b, h], ref, o_err, ("o", b, h))
                within(lse[b, h], l_ref, l_err, ("lse", b, h))
                if not backward:
                    continue
                g, err = plain_backward(q[b, h], k[b, hk], v[b, hk], o[b, h], lse[b, h], do[b, h], scale, window, sinks)
                within(dq[b, h], g[0], err[0], ("dq", b, h))
                for i, x in enumerate((g[1], g[2], err[1], err[2])):
                    sums[i] += x
            if backward:
                within(dk[b, hk], sums[0], sums[2] + HALF * 1.01 * np.abs(sums[0]), ("dk", b, hk))
                within(dv[b, hk], sums[1], sums[3] + HALF * 1.01 * np.abs(sums[1]), ("dv", b, hk))


CASES = [
    # B, H, Hkv, N, window, sinks
    (1, 1, 1, 1, 1, 0),
    (1, 2, 1, 1, 5, 3),
    (2, 2, 2, 2, 1, 1),
    (1, 4, 2, 127, 30, 0),
    (1, 3, 1, 128, 128, 4),
    (1, 4, 4, 129, 1, 0),        # a window of the row alone
    (1, 4, 4, 129, 1, 128),
    (1, 2, 2, 300, 129, 1),
    (1, 6, 2, 300, 128, 17),     # odd group: two tiles of one head
    (1, 8, 1, 517, 127, 128),    # first tokens over a whole tile
    (2, 4, 2, 640, 256, 16),
    (1, 4, 4, 777, 200, 3),
    (1, 2, 1, 1100, 1000, 4),    # few queries see first tokens from afar
    (1, 2, 2, 1100, 1100, 4),    # window = N: plain causal
    (1, 2, 1, 400, 5000, 128),   # window > N
    (3, 5, 5, 257, 64, 5),
    (1, 12, 4, 1025, 512, 0),
    (1, 1, 1, 2000, 130, 40),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks", CASES)
def test_against_plain(B, H, Hkv, N, window, sinks, d):
    check(B, H, Hkv, N, d, window, sinks, seed=N + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks", [
    (2, 60, 60, 700, 130, 5),    # 720 key tiles: several to a CTA that walks them, few query tiles each
    (1, 150, 50, 500, 40, 0),    # 200, the last of them split
    (1, 160, 160, 100, 7, 2),    # 160 of one query tile
])
def test_more_key_tiles_than_sms(B, H, Hkv, N, window, sinks, d):
    check(B, H, Hkv, N, d, window, sinks, seed=H + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.02, 0.6])
def test_scales(scale, d):
    """Flat and peaked weights."""
    check(1, 4, 2, 700, d, 150, 4, seed=3, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("d,group", [(128, 4), (64, 1), (128, 3)])
def test_longer_sequences(d, group):
    """Several rounds of work items per SM, the last one split; one key head checked in full."""
    check(2, 8 * group, 8, 2900, d, 600, 6, seed=5, heads=[7])


@pytest.mark.gpu
def test_whole_window_is_causal_attention():
    """window >= N with a head per key head computes fa_fwd's causal attention."""
    from exact_attention_98_gb300 import fa

    q, k, v, do = (t.cuda() for t in attention_inputs(1, 3, 900, 128, seed=8))
    o, lse = fa.forward(q, k, v, causal=True)
    o2, lse2 = fa.window_forward(q, k, v, window=900)
    assert (o.float() - o2.float()).abs().max() <= 2 ** -7 and (lse - lse2).abs().max() <= 1e-5
    g = fa.backward(q, k, v, o, lse, do, causal=True)
    g2 = fa.window_backward(q, k, v, o, lse, do, window=10 ** 9)
    for a, b in zip(g, g2):
        assert (a.float() - b.float()).norm() / a.float().norm() <= 0.004  # two results each 2^-9 rms off
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.gpu
def test_shared_heads_sum():
    """dK and dV of a shared key head are the sums over heads with keys of their own."""
    from exact_attention_98_gb300 import fa

    q, k, v, do = (t.cuda() for t in inputs(2, 6, 2, 500, 64, 4))
    o, lse = fa.window_forward(q, k, v, 100, 3)
    dq, dk, dv = fa.window_backward(q, k, v, o, lse, do, 100, 3)
    k6, v6 = (x.repeat_interleave(3, 1).contiguous() for x in (k, v))
    o6, lse6 = fa.window_forward(q, k6, v6, 100, 3)
    dq6, dk6, dv6 = fa.window_backward(q, k6, v6, o, lse, do, 100, 3)
    assert fa.fa_last_device_status() == fa.FA_OK
    assert torch.equal(o, o6) and torch.equal(lse, lse6)
    assert (dq.float() - dq6.float()).norm() / dq.float().norm() <= 1e-3  # the order of fp32 additions
    for a, b in ((dk, dk6), (dv, dv6)):
        s = b.double().view(2, 2, 3, 500, 64)
        # each of the three and the sum rounded once
        assert ((a.double() - s.sum(2)).abs() <= HALF * (s.abs().sum(2) + a.double().abs()) * 1.02 + 1e-6).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [0, 5, 40])
def test_repeats_and_graph(sinks):
    """O, LSE, dK and dV have the same bits from run to run, in a replayed graph too, on another stream,
    and whatever the workspace held."""
    from exact_attention_98_gb300 import fa

    B, H, Hkv, N, d, W = 1, 8, 4, 1500, 128, 300
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hkv, N, d, 9))
    scale = fa.default_scale(d)

    def buffers():
        o, dq = torch.empty_like(q), torch.empty_like(q)
        return o, torch.empty((B, H, N), device="cuda"), dq, torch.empty_like(k), torch.empty_like(v), torch.full(
            (fa.fa_bwd_window_workspace_bytes(B, H, Hkv, N, d, W, sinks),), 0xFF, dtype=torch.uint8, device="cuda")

    def step(b):
        o, lse, dq, dk, dv, ws = b
        fa.fa_fwd_window(q, k, v, o, lse, scale, W, sinks)
        fa.fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, scale, W, sinks, ws)

    first, second = buffers(), buffers()
    step(first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(second)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    third = buffers()
    with torch.cuda.graph(graph, stream=s):
        step(third)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    for other in (second, third):
        for i in (0, 1, 3, 4):
            assert torch.equal(first[i], other[i]), i
        assert (first[2].float() - other[2].float()).norm() / first[2].float().norm() <= 1e-3


@pytest.mark.gpu
def test_streams_keep_their_memory():
    """stream=: outputs and workspace belong to the stream that uses them."""
    from exact_attention_98_gb300 import fa

    q, k, v, do = (t.cuda() for t in inputs(1, 4, 2, 1200, 128, 2))
    o, lse = fa.window_forward(q, k, v, 200, 4)
    want = fa.window_backward(q, k, v, o, lse, do, 200, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(4):
        o2, lse2 = fa.window_forward(q, k, v, 200, 4, stream=s)
        got = fa.window_backward(q, k, v, o2, lse2, do, 200, 4, stream=s)
        noise = [torch.full_like(q, 7.0) for _ in range(3)]
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        del noise
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.gpu
def test_two_backwards_at_once():
    """Persistent CTAs of one call beside another's, on streams of their own: each
    gives what it gives alone, dk and dv bit for bit."""
    from exact_attention_98_gb300 import fa

    calls = []
    for d, Hkv in ((64, 16), (128, 4)):
        q, k, v, do = (t.cuda() for t in inputs(2, 16, Hkv, 1500, d, d))
        o, lse = fa.window_forward(q, k, v, 400, 3)
        calls.append((q, k, v, o, lse, do))
    alone = [fa.window_backward(*c, 400, 3) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        both = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                both.append(fa.window_backward(*c, 400, 3))
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
        for (dq, dk, dv), ref in zip(both, alone):
            assert torch.equal(dk, ref[1]) and torch.equal(dv, ref[2])
            # the order of dq's fp32 additions varies, which can move a rounding to bf16
            assert (dq.float() - ref[0].float()).abs().max() <= 2 * HALF * ref[0].float().abs().max()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last key head's results are those of that head alone."""
    from exact_attention_98_gb300 import fa

    H, Hkv, N, d, W, S = 264, 132, 64000, 128, 128, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda h: torch.randn(1, h, N, d, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = rand(H), rand(Hkv), rand(Hkv), rand(H)
    assert q.numel() > 2 ** 31
    o, lse = fa.window_forward(q, k, v, W, S)
    dq, dk, dv = fa.window_backward(q, k, v, o, lse, do, W, S)
    one = lambda x, n: x[:, -n:].contiguous()  # noqa: E731
    o1, lse1 = fa.window_forward(one(q, 2), one(k, 1), one(v, 1), W, S)
    g1 = fa.window_backward(one(q, 2), one(k, 1), one(v, 1), o1, lse1, one(do, 2), W, S)
    assert fa.fa_last_device_status() == fa.FA_OK
    assert torch.equal(o[:, -2:], o1) and torch.equal(lse[:, -2:], lse1)
    for a, b in zip((dq[:, -2:], dk[:, -1:], dv[:, -1:]), g1):
        assert (a.float() - b.float()).norm() / b.float().norm() <= 2e-3  # parts are cut elsewhere


@pytest.mark.gpu
def test_prompt_both_ways():
    """A prompt through window_forward, and appended to a bf16 cache and attended to there: both within
    their bounds of the 64-bit result."""
    from exact_attention_98_gb300 import fa

    H, Hkv, N, d, W, S = 4, 2, 150, 128, 40, 3
    q, k, v, _ = inputs(1, H, Hkv, N, d, 6)
    o, lse = fa.window_forward(q.cuda(), k.cuda(), v.cuda(), W, S)
    rows = lambda x: x[0].transpose(0, 1).contiguous().cuda()  # noqa: E731
    pages = fa.paged_pages(3, Hkv, 64, d)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([N], [0, N]))
    fa.paged_append(rows(k), rows(v), pages, table, lens, cu)
    o2, lse2 = fa.paged_forward(rows(q), pages, table, lens, cu, max_new=N, window=W, sinks=S)
    assert fa.fa_last_device_status() == fa.FA_OK
    for h in range(H):
        ref, l_ref, o_err, l_err = plain_forward(f64(q)[0, h], f64(k)[0, h // 2], f64(v)[0, h // 2], d ** -0.5, W, S)
        within(f64(o)[0, h], ref, o_err, h)
        within(f64(o2)[:, h], ref, o_err, h)
        within(f64(lse)[0, h], l_ref, l_err, h)
        within(f64(lse2)[:, h], l_ref, l_err, h)


@pytest.mark.gpu
def test_launches_are_counted():
    from exact_attention_98_gb300 import fa

    q, k, v, do = (t.cuda() for t in inputs(1, 2, 1, 200, 64, 1))
    n0 = fa.fa_launch_count()
    o, lse = fa.window_forward(q, k, v, 50)
    assert fa.fa_launch_count() - n0 == 1
    fa.window_backward(q, k, v, o, lse, do, 50)
    assert fa.fa_launch_count() - n0 == 4
    assert fa.fa_last_device_status() == fa.FA_OK


# --- no GPU ---------------------------------------------------------------------------


def test_plain_gradients_by_differences():
    """The tests' own formulas: central differences of sum(O dO), through shared heads."""
    rng = np.random.default_rng(0)
    N, d, G, W, S, scale = 9, 4, 2, 3, 2, 0.5
    q, do = rng.standard_normal((2, G, N, d))
    k, v = rng.standard_normal((2, N, d))

    def loss(q, k, v):
        return sum((plain_forward(q[h], k, v, scale, W, S)[0] * do[h]).sum() for h in range(G))

    grads = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for h in range(G):
        o, lse, _, _ = plain_forward(q[h], k, v, scale, W, S)
        (dq, dk, dv), _ = plain_backward(q[h], k, v, o, lse, do[h], scale, W, S)
        grads[0][h] += dq
        grads[1] += dk
        grads[2] += dv
    step = 1e-5
    for which, (x, g) in enumerate(zip((q, k, v), grads)):
        for at in np.ndindex(x.shape):
            args = [[q, k, v], [q, k, v]]
            for sign, a in ((1, args[0]), (-1, args[1])):
                a[which] = x.copy()
                a[which][at] += sign * step
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * step)
            assert abs(diff - g[at]) <= 1e-7, (which, at)


@pytest.fixture(scope="module")
def fa():
    from exact_attention_98_gb300 import build

    build.build()
    from exact_attention_98_gb300 import fa

    return fa


def fwd(fa, q=0x1000, k=0x1000, v=0x1000, o=0x1000, lse=0x1000, B=1, H=4, Hkv=2, N=300, d=64, scale=0.1, window=9,
        sinks=1):
    return fa.lib.fa_fwd_window(q, k, v, o, lse, B, H, Hkv, N, d, scale, window, sinks, None)


def bwd(fa, q=0x1000, k=0x1000, v=0x1000, o=0x1000, lse=0x1000, B=1, H=4, Hkv=2, N=300, d=64, scale=0.1, window=9,
        sinks=1, dout=0x1000, dq=0x1000, dk=0x1000, dv=0x1000, ws=0x10000, nbytes=1 << 40):
    return fa.lib.fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, N, d, scale, window, sinks, ws, nbytes,
                                None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(fa, call):
    bad, un = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw, want in ((dict(B=-1), bad), (dict(N=-1), bad), (dict(Hkv=-1), bad), (dict(Hkv=0), bad), (dict(Hkv=3), bad),
                     (dict(d=96), un), (dict(scale=0.0), bad), (dict(scale=float("nan")), bad), (dict(window=0), bad),
                     (dict(window=-4), bad), (dict(sinks=-1), bad), (dict(sinks=129), un), (dict(N=2 ** 30 + 1), un),
                     (dict(q=None), bad), (dict(k=None), bad), (dict(v=0x1008), bad), (dict(o=None), bad),
                     (dict(lse=0x1002), bad)):
        assert call(fa, **kw) == want, kw
    for kw in (dict(B=0), dict(N=0), dict(H=0), dict(H=0, Hkv=0)):
        assert call(fa, q=None, k=None, v=None, o=None, lse=None, **kw) == fa.FA_OK, kw


def test_backward_refusals(fa):
    for kw in (dict(dout=None), dict(dq=None), dict(dk=0x1004), dict(dv=None)):
        assert bwd(fa, **kw) == fa.FA_ERR_INVALID_ARG
    need = fa.fa_bwd_window_workspace_bytes(1, 4, 2, 300, 64, 9, 1)
    for kw in (dict(ws=None), dict(nbytes=need - 1), dict(ws=0x10010)):
        assert bwd(fa, **kw) == fa.FA_ERR_WORKSPACE


def test_workspace_bytes(fa):
    n = fa.fa_bwd_window_workspace_bytes
    assert n(1, 4, 2, 0, 64, 9, 1) == 0 and n(1, 4, 3, 300, 64, 9, 1) == 0 and n(1, 4, 2, 300, 64, 9, 129) == 0
    base = fa.fa_bwd_workspace_bytes(1, 4, 300, 64)
    assert n(1, 4, 2, 300, 64, 300, 4) == n(1, 4, 2, 300, 64, 9, 0)  # no query's window leaves a first token
    # 19 parts of 16 rows and the main kernel's, 2 key heads, dK and dV, 16 rows
    assert n(1, 4, 2, 300, 64, 9, 4) - n(1, 4, 2, 300, 64, 9, 0) == 20 * 2 * 2 * 16 * 64 * 4
    assert n(1, 4, 2, 300, 64, 9, 0) >= base


def test_binding_refuses(fa):
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.window_forward(q, q, q, 4)
    with pytest.raises(ValueError, match="expected"):
        fa.window_forward(q[0], q, q, 4)
