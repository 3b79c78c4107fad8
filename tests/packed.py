"""Plain 64-bit attention over packed sequences, with error bounds, for the tests.

Bounds, element by element (e a score's error).  A rounding to bf16 is off by 2^-8
of the value at most.  Scores and dP are fp32 sums of up to 128 products: off by
2^-17 of their largest sum of magnitudes (128 roundings of 2^-24); the row's LSE
and D enter the backward with all their fp32 bits, exponentials and the
accumulators' sums are far below.
  O     P rounded: 2^-8 sum p |v|; scores: twice their error (weight and sum of
        weights); O rounded
  LSE   scores, and a few fp32 roundings
  dV    P rounded, and its relative error e from scores and LSE: sum (2^-8 + e) p |do|
  dS    rounded: 2^-8 |dS|; P's relative error e; dP's and D's errors times p
  dQ    scale sum |err dS| |k|, dK the same with |q|; all rounded at the end"""
import numpy as np
import torch

HALF = 2.0 ** -8


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, err, what):
    bad = ~(np.abs(got - ref) <= err + 1e-30)  # a NaN is bad
    assert not bad.any(), (what, float(np.nanmax(np.abs(got - ref) / (err + 1e-30))), int(bad.sum()))


def visible(n, causal):
    return np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)


def plain_forward(q, k, v, scale, causal):
    """One head of one sequence: O, LSE and the error bounds of both."""
    see = visible(len(q), causal)
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    lse = (m + np.log(w.sum(1, keepdims=True)))[:, 0]
    p = w / w.sum(1, keepdims=True)
    o = p @ v
    s_err = 2.0 ** -17 * (scale * np.where(see, np.abs(q) @ np.abs(k).T, 0)).max(1) + 2.0 ** -20
    o_err = (HALF + 2 * s_err[:, None]) * (p @ np.abs(v)) + HALF * 1.01 * np.abs(o)
    return o, lse, o_err, s_err + 2.0 ** -20 * np.abs(lse)


def plain_backward(q, k, v, o, lse, do, scale, causal):
    """One query head's gradients from the forward's O and LSE, and their error bounds
    (dK's and dV's before the final rounding: they are summed over a group)."""
    see = visible(len(q), causal)
    p = np.where(see, np.exp(np.where(see, scale * (q @ k.T), -np.inf) - lse[:, None]), 0)
    dp = do @ v.T
    ds = p * (dp - (do * o).sum(1, keepdims=True))
    e = 2.0 ** -17 * scale * (np.abs(q) @ np.abs(k).T) + 2.0 ** -20 * (1 + np.abs(lse))[:, None]
    dp_err = 2.0 ** -17 * (np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1, keepdims=True))
    ds_err = (HALF + e) * np.abs(ds) + p * dp_err
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    dq_err = scale * ds_err @ np.abs(k) + HALF * 1.01 * np.abs(dq)
    return (dq, dk, dv), (dq_err, scale * ds_err.T @ np.abs(q), ((HALF + e) * p).T @ np.abs(do))


def batch(lengths, before=0, after=0):
    """cu_seqlens (a list) and the rows of sequences of these lengths with padding rows around them."""
    cu = [before]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu, cu[-1] + after


def rows(n, heads, d, seed, layout="fused"):
    """bf16 rows [n, heads, d] on the GPU: 'fused' (a wider row's part), 'dense', or 'heads' (head by head)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g).to(torch.bfloat16).cuda()
    if layout == "dense":
        return x
    if layout == "heads":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((n, heads + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1: heads + 1] = x
    return wide[:, 1: heads + 1]


def check_forward(o, lse, q, k, v, cu, scale, causal, skip=()):
    """Every sequence's O and LSE against the plain ones."""
    o, lse, q, k, v = (f64(t) for t in (o, lse, q, k, v))
    G = q.shape[1] // k.shape[1]
    for b in range(len(cu) - 1):
        r = slice(cu[b], cu[b + 1])
        if b in skip or cu[b] == cu[b + 1]:
            continue
        for h in range(q.shape[1]):
            ref, l_ref, o_err, l_err = plain_forward(q[r, h], k[r, h // G], v[r, h // G], scale, causal)
            within(o[r, h], ref, o_err, ("o", b, h))
            within(lse[r, h], l_ref, l_err, ("lse", b, h))


def check_backward(grads, q, k, v, o, lse, do, cu, scale, causal, skip=()):
    dq, dk, dv, q, k, v, o, lse, do = (f64(t) for t in (*grads, q, k, v, o, lse, do))
    G = q.shape[1] // k.shape[1]
    for b in range(len(cu) - 1):
        r = slice(cu[b], cu[b + 1])
        if b in skip or cu[b] == cu[b + 1]:
            continue
        for hk in range(k.shape[1]):
            sums = [0, 0, 0, 0]
            for h in range(hk * G, hk * G + G):
                g, err = plain_backward(q[r, h], k[r, hk], v[r, hk], o[r, h], lse[r, h], do[r, h], scale, causal)
                within(dq[r, h], g[0], err[0], ("dq", b, h))
                sums = [a + x for a, x in zip(sums, (g[1], g[2], err[1], err[2]))]
            within(dk[r, hk], sums[0], sums[2] + HALF * 1.01 * np.abs(sums[0]), ("dk", b, hk))
            within(dv[r, hk], sums[1], sums[3] + HALF * 1.01 * np.abs(sums[1]), ("dv", b, hk))
