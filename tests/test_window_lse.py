"""Window backward with LSE and D far from 0.

Q and K share a large element, which adds the same to every score and so to
LSE; their other elements are multiples of 1/8 up to 1, and so are V and dO.
Products are then multiples of 2^-6 and their sums below 2^14, exact in fp32:
what is off is what the kernels make of LSE and D."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def eighths(rng, *shape):
    return torch.from_numpy(rng.integers(-8, 9, shape) / 8.0)


def inputs(N, d, G, lift, seed):
    rng = np.random.default_rng(seed)
    q, k, v, do = eighths(rng, G, N, d), eighths(rng, 1, N, d), eighths(rng, 1, N, d), eighths(rng, G, N, d)
    q[..., 24:] = 0          # scores of 23 random products: softmax over a few of them
    q[..., 0], k[..., 0] = 64.0, lift / 64.0
    v[..., 0], do[..., 0] = 40.0, 100.0     # D about 4000
    return q, k, v, do


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lift", [512, 8192])
def test_a_row_that_sees_itself_alone(d, lift):
    """Window 1: P = 1, so dV = dO and dS = P (dP - D) = 0 exactly: both sides of exp(S - LSE) and of
    dP - D are the same fp32 number."""
    from exact_attention_98_gb300 import fa

    N = 300
    q, k, v, do = inputs(N, d, 1, lift, d + lift)
    lse = (q * k).sum(-1)
    assert torch.equal(lse, lse.float().double())
    dev = lambda x: x.to(torch.bfloat16)[None].cuda()  # noqa: E731
    dq, dk, dv = fa.window_backward(dev(q), dev(k), dev(v), dev(v), lse.float()[None].cuda(), dev(do), 1, 0, scale=1.0)
    assert fa.fa_last_device_status() == fa.FA_OK
    assert torch.equal(dv.cpu(), do.to(torch.bfloat16)[None])
    assert (dq == 0).all() and (dk == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lift,window,sinks", [(512, 40, 0), (8192, 40, 0), (8192, 130, 5)])
def test_large_lse(d, lift, window, sinks):
    """Element by element: P is off by what the sum S - LSE loses, four alignments of fp32 terms, and by
    its rounding for dV; dP - D by four alignments too."""
    from exact_attention_98_gb300 import fa

    N, G = 400, 2
    q, k, v, do = inputs(N, d, G, lift, 7 + lift)
    i, j = np.arange(N)[:, None], np.arange(N)[None]
    see = (j <= i) & ((i - j < window) | (j < sinks))
    n = lambda x: x.numpy()  # noqa: E731
    K, V = n(k)[0], n(v)[0]
    o, lse = np.zeros((G, N, d)), np.zeros((G, N))
    for h in range(G):
        s = np.where(see, n(q)[h] @ K.T, -np.inf)
        m = s.max(1, keepdims=True)
        w = np.exp(s - m)
        lse[h] = (m + np.log(w.sum(1, keepdims=True)))[:, 0]
        o[h] = (w / w.sum(1, keepdims=True)) @ V
    o = torch.from_numpy(o).to(torch.bfloat16)
    lse = torch.from_numpy(lse).float()
    dev = lambda x: x.to(torch.bfloat16)[None].cuda()  # noqa: E731
    got = fa.window_backward(dev(q), dev(k), dev(v), o[None].cuda(), lse[None].cuda(), dev(do), window, sinks, scale=1.0)
    assert fa.fa_last_device_status() == fa.FA_OK
    dq, dk, dv = (x[0].double().cpu().numpy() for x in got)
    half = 2.0 ** -8
    sums = [np.zeros((N, d)) for _ in range(4)]
    for h in range(G):
        L, O, Q, DO = lse[h].double().numpy(), o[h].double().numpy(), n(q)[h], n(do)[h]
        p = np.where(see, np.exp(np.where(see, Q @ K.T, -np.inf) - L[:, None]), 0)
        dp, D = DO @ V.T, (DO * O).sum(1, keepdims=True)
        ds = p * (dp - D)
        e = 2.0 ** -21 * np.abs(L)[:, None] + 2.0 ** -20
        # D itself: an fp32 sum of up to 128 products, 4000 and small ones
        dp_err = (2.0 ** -21 + 2.0 ** -20) * (np.abs(DO) * np.abs(O)).sum(1, keepdims=True) + 2.0 ** -21 * np.abs(dp)
        ds_err = (half + e) * np.abs(ds) + p * dp_err
        dq_ref = ds @ K
        assert (np.abs(dq[h] - dq_ref) <= ds_err @ np.abs(K) + half * 1.01 * np.abs(dq_ref) + 1e-30).all(), h
        for at, x in enumerate((ds.T @ Q, p.T @ DO, ds_err.T @ np.abs(Q), ((half + e) * p).T @ np.abs(DO))):
            sums[at] += x
    assert (np.abs(dk[0] - sums[0]) <= sums[2] + half * 1.01 * np.abs(sums[0]) + 1e-30).all()
    assert (np.abs(dv[0] - sums[1]) <= sums[3] + half * 1.01 * np.abs(sums[1]) + 1e-30).all()
