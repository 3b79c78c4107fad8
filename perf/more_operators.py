"""Cases of the attention over packed sequences and of the rotation of their rows.

Kinds of case:
  packed_fwd   attention within each of several sequences whose rows follow one
               another in one tensor, shared key heads: O and LSE
  packed_bwd   its gradients dQ, dK, dV from the forward's O and LSE
  rotate       Q and K rows rotated by their positions, or (backward) the
               gradients of rotated rows turned back

`run` is the plain form in elementary torch operations, or, with `own`, the
library's calls.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # a few short prompts: latency
        dict(name="packed_fwd_short", kind="packed_fwd", rows=300, seqs=3, first=130, H=16, Hkv=4, d=128, causal=True),
        # the prompts of a serving batch, none padded
        dict(name="packed_fwd_prompts", kind="packed_fwd", rows=24001, seqs=24, first=2000, H=32, Hkv=8, d=128,
             causal=True),
        # one long prompt among short ones
        dict(name="packed_fwd_long", kind="packed_fwd", rows=36001, seqs=9, first=32768, H=16, Hkv=4, d=128,
             causal=True),
        # texts that are encoded in both directions, three query heads per key head
        dict(name="packed_fwd_full_d64", kind="packed_fwd", rows=9999, seqs=17, first=1500, H=12, Hkv=4, d=64,
             causal=False),
        # fine-tuning on a few short odd sequences, a key head for each query head
        dict(name="packed_bwd_small", kind="packed_bwd", rows=777, seqs=3, first=300, H=4, Hkv=4, d=128, causal=True),
        # a training step's layer over packed documents
        dict(name="packed_bwd_train", kind="packed_bwd", rows=16384, seqs=11, first=4096, H=16, Hkv=4, d=128,
             causal=True),
        # the same with d = 64 and a key head for each query head
        dict(name="packed_bwd_d64", kind="packed_bwd", rows=16384, seqs=13, first=3000, H=16, Hkv=16, d=64,
             causal=True),
        # one long document of odd length
        dict(name="packed_bwd_long", kind="packed_bwd", rows=16001, seqs=1, first=16001, H=8, Hkv=2, d=128,
             causal=True),
        # one decode step of a few sequences: latency
        dict(name="rotate_step", kind="rotate", rows=8, H=32, Hkv=8, d=128, rot=128, interleaved=False, backward=False,
             length=5000, packed=False),
        # a training step's layer
        dict(name="rotate_train", kind="rotate", rows=16384, H=32, Hkv=8, d=128, rot=128, interleaved=False,
             backward=False, length=4096, packed=True),
        # its gradients, interleaved pairs over half of the head, d = 64
        dict(name="rotate_grad_d64", kind="rotate", rows=16383, H=16, Hkv=16, d=64, rot=32, interleaved=True,
             backward=True, length=3000, packed=True),
        # prompts at far positions of a long context, half of the head
        dict(name="rotate_far", kind="rotate", rows=4999, H=16, Hkv=4, d=128, rot=64, interleaved=False,
             backward=False, length=131072, packed=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["packed_fwd", "packed_fwd", "packed_bwd", "packed_bwd", "rotate"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 8) if g * Hkv <= 32])
    if kind == "rotate":
        return dict(kind=kind, rows=_spread(rng, 1, 16384), H=H, Hkv=Hkv, d=d, rot=rng.choice([d // 4, d // 2, d]),
                    interleaved=rng.random() < 0.5, backward=rng.random() < 0.5, length=_spread(rng, 16, 131072),
                    packed=rng.random() < 0.5)
    forward = kind == "packed_fwd"
    # a sequence of a single row has a constant softmax, whose gradient is nothing but
    # rounding: the backward's first has some rows
    least = 1 if forward else 64
    most = 32768 if forward else 12000
    first = min(_spread(rng, least, most), most * 8 // H if H > 8 else most)
    seqs = rng.choice([1, _spread(rng, 1, 64)])
    others = (seqs - 1) * _spread(rng, 1, max(2, min(2000, 65536 // (seqs * H) + 2)))
    return dict(kind=kind, rows=first + others, seqs=seqs, first=first, H=H, Hkv=Hkv, d=d, causal=rng.random() < 0.75)


# --- the layout of a case ------------------------------------------------------


def _lengths(case):
    """Rows of each sequence: `first` of the first, the rest spread over the others (some may be empty)."""
    r = random.Random("%(rows)d %(seqs)d %(first)d" % case)
    rest, n = case["rows"] - case["first"], case["seqs"] - 1
    if n == 0:
        return [case["rows"]]
    share = [r.uniform(0.2, 1.0) for _ in range(n)]
    out = [int(rest * s / sum(share)) for s in share]
    out[-1] += rest - sum(out)
    return [case["first"]] + out


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lengths(case))


def work(case):
    c = case
    if c["kind"] == "rotate":
        tables = c["length"] if c["packed"] else c["rows"]  # rows of the table that are read
        return {"bytes": c["rows"] * (c["H"] + c["Hkv"]) * c["d"] * 4 + 4 * c["rows"]
                + min(tables, c["rows"], c["length"]) * c["rot"] * 4,
                "flops": 3 * c["rows"] * (c["H"] + c["Hkv"]) * c["rot"]}
    rows, kv_rows = c["rows"] * c["H"], c["rows"] * c["Hkv"]
    flops = 2.0 * c["d"] * c["H"] * _pairs(c)
    if c["kind"] == "packed_fwd":
        return {"bytes": 2 * c["d"] * (2 * rows + 2 * kv_rows) + 4 * rows, "flops": 2 * flops}
    return {"bytes": 2 * c["d"] * (4 * rows + 4 * kv_rows) + 4 * rows, "flops": 5 * flops}


# --- inputs ----------------------------------------------------------------------


def _table(length, rot):
    """fp32 [length, rot]: cosines, then sines, of each position's angles (taken in 64 bits)."""
    rate = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    angle = torch.arange(length, dtype=torch.float64, device=DEVICE)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device=DEVICE, dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
    T, H, Hkv, d = c["rows"], c["H"], c["Hkv"], c["d"]
    # rows as a fused projection leaves them: [T, (H + 2 Hkv) d]
    fused = randn(T, (H + 2 * Hkv) * d).unflatten(1, (-1, d))
    st = dict(case=c, q=fused[:, :H], k=fused[:, H: H + Hkv])
    if c["kind"] == "rotate":
        if c["packed"]:  # sequences of `length` rows, one after another
            pos = torch.arange(T, device=DEVICE) % c["length"]
        else:
            pos = torch.randint(0, c["length"], (T,), generator=g, device=DEVICE)
        st.update(pos=pos.to(torch.int32), rope=_table(c["length"], c["rot"]))
        return st
    cu = [0]
    for n in _lengths(c):
        cu.append(cu[-1] + n)
    st.update(v=fused[:, H + Hkv:], cu=torch.tensor(cu, dtype=torch.int32, device=DEVICE))
    if own:
        from exact_attention_98_gb300 import fa

        # made once for a batch, used by every layer's forward and backward
        st["plan"] = fa.packed_plan(st["cu"], T, causal=c["causal"])
    if c["kind"] == "packed_bwd":
        o, lse = _packed_forward(st)
        st.update(o=o, lse=lse, dout=randn(T, H, d))
    return st


# --- plain forms -----------------------------------------------------------------


def _sequences(c):
    at = 0
    for n in _lengths(c):
        if n:
            yield at, n
        at += n


def _grouped(x, heads):
    """[n, heads * G, d] -> fp32 [heads, G, n, d]"""
    return x.float().unflatten(1, (heads, -1)).permute(1, 2, 0, 3)


def _scores(c, q, k, i0):
    """Scaled scores of query rows i0.. against a sequence's keys, -inf where a key is not visible."""
    s = (q @ k.mT).div_(math.sqrt(c["d"]))
    if c["causal"]:
        i = i0 + torch.arange(q.shape[2], device=DEVICE)[:, None]
        s.masked_fill_(torch.arange(k.shape[2], device=DEVICE) > i, -math.inf)
    return s


STEP = 2048  # query rows at a time


def _packed_forward(st):
    c = st["case"]
    o = torch.empty(c["rows"], c["H"], c["d"], dtype=torch.bfloat16, device=DEVICE)
    lse = torch.empty(c["rows"], c["H"], dtype=torch.float32, device=DEVICE)
    for at, n in _sequences(c):
        k, v = (_grouped(st[x][at: at + n], c["Hkv"]) for x in "kv")
        for i0 in range(0, n, STEP):
            i1 = min(n, i0 + STEP)
            seen = i1 if c["causal"] else n
            q = _grouped(st["q"][at + i0: at + i1], c["Hkv"])
            s = _scores(c, q, k[:, :, :seen], i0)
            m = s.amax(-1, keepdim=True)
            p = s.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            out = (p @ v[:, :, :seen]) / total
            o[at + i0: at + i1] = out.permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
            lse[at + i0: at + i1] = (m + total.log())[..., 0].permute(2, 0, 1).flatten(1)
    return o, lse


def _packed_backward(st):
    c = st["case"]
    shapes = [st[x].shape for x in ("q", "k", "v")]
    dq, dk, dv = (torch.empty(s, dtype=torch.bfloat16, device=DEVICE) for s in shapes)
    for at, n in _sequences(c):
        k, v = (_grouped(st[x][at: at + n], c["Hkv"]) for x in "kv")
        gk, gv = torch.zeros_like(k[:, 0]), torch.zeros_like(v[:, 0])
        for i0 in range(0, n, STEP):
            i1 = min(n, i0 + STEP)
            seen = i1 if c["causal"] else n
            q, o, do = (_grouped(st[x][at + i0: at + i1], c["Hkv"]) for x in ("q", "o", "dout"))
            lse = st["lse"][at + i0: at + i1].unflatten(1, (c["Hkv"], -1)).permute(1, 2, 0)[..., None]
            p = _scores(c, q, k[:, :, :seen], i0).sub_(lse).exp_()
            ds = (do @ v[:, :, :seen].mT).sub_((do * o).sum(-1, keepdim=True)).mul_(p).div_(math.sqrt(c["d"]))
            dq[at + i0: at + i1] = (ds @ k[:, :, :seen]).permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
            gk[:, :seen] += (ds.mT @ q).sum(1)
            gv[:, :seen] += (p.mT @ do).sum(1)
        dk[at: at + n] = gk.transpose(0, 1).to(torch.bfloat16)
        dv[at: at + n] = gv.transpose(0, 1).to(torch.bfloat16)
    return dq, dk, dv


def _rotate(st, x):
    c = st["case"]
    half = c["rot"] // 2
    row = st["rope"][st["pos"].long()][:, None]
    cos, sin = row[..., :half], row[..., half:]
    if c["backward"]:
        sin = -sin
    x = x.float()
    y, rest = x[..., : c["rot"]], x[..., c["rot"]:]
    a, b = (y[..., 0::2], y[..., 1::2]) if c["interleaved"] else (y[..., :half], y[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1).to(torch.bfloat16)


def run(st):
    c = st["case"]
    if own:
        from exact_attention_98_gb300 import fa

        if c["kind"] == "packed_fwd":
            return fa.packed_forward(st["q"], st["k"], st["v"], st["plan"])
        if c["kind"] == "packed_bwd":
            return fa.packed_backward(st["q"], st["k"], st["v"], st["o"], st["lse"], st["dout"], st["plan"])
        return fa.rotate(st["q"], st["k"], st["pos"], st["rope"], interleaved=c["interleaved"],
                         backward=c["backward"])
    if c["kind"] == "packed_fwd":
        return _packed_forward(st)
    if c["kind"] == "packed_bwd":
        return _packed_backward(st)
    return _rotate(st, st["q"]), _rotate(st, st["k"])


# --- the definition in 64 bits -----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["kind"] == "rotate":
        return tuple(_exact_rotate(st, c, st[x]) for x in "qk")
    if float(_pairs(c)) * c["H"] * c["d"] > 5e11:
        return None
    return _exact_packed(st, c, 1.0 / math.sqrt(c["d"]))


def _exact_rotate(st, c, x):
    rot, sign = c["rot"], -1.0 if c["backward"] else 1.0
    out = x.double().clone()
    table = st["rope"].double()
    pos = st["pos"].long()
    for p in range(rot // 2):
        a, b = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + rot // 2)
        turn = torch.complex(table[pos, p], sign * table[pos, p + rot // 2])[:, None]
        z = torch.complex(x[..., a].double(), x[..., b].double()) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_packed(st, c, scale):
    G, d = c["H"] // c["Hkv"], c["d"]
    f64 = dict(dtype=torch.float64, device=DEVICE)
    o, lse = torch.zeros(c["rows"], c["H"], d, **f64), torch.zeros(c["rows"], c["H"], **f64)
    dq = torch.zeros_like(o)
    dk = torch.zeros(c["rows"], c["Hkv"], d, **f64)
    dv = torch.zeros_like(dk)
    seq = torch.repeat_interleave(torch.arange(len(_lengths(c))), torch.tensor(_lengths(c))).to(DEVICE)
    t = torch.arange(c["rows"], device=DEVICE)
    for i0 in range(0, c["rows"], 1024):
        i = t[i0: i0 + 1024]
        # the keys of all sequences that these rows belong to
        j = t[(seq >= seq[i[0]]) & (seq <= seq[i[-1]])]
        if c["causal"]:
            j = j[j <= i[-1]]
        hidden = seq[i][:, None] != seq[j][None]
        if c["causal"]:
            hidden |= j[None] > i[:, None]
        for h in range(c["H"]):
            k, v = st["k"][j, h // G].double(), st["v"][j, h // G].double()
            q = st["q"][i, h].double()
            s = (scale * (q @ k.T)).masked_fill(hidden, -math.inf)
            if c["kind"] == "packed_fwd":
                lse[i, h] = torch.logsumexp(s, 1)
                o[i, h] = torch.softmax(s, 1) @ v
                continue
            do = st["dout"][i, h].double()
            p = torch.exp(s - st["lse"][i, h].double()[:, None])
            ds = scale * p * (do @ v.T - (do * st["o"][i, h].double()).sum(1, keepdim=True))
            dq[i, h] = ds @ k
            dk[:, h // G].index_add_(0, j, ds.T @ q)
            dv[:, h // G].index_add_(0, j, p.T @ do)
    return (dq, dk, dv) if c["kind"] == "packed_bwd" else (o, lse)
