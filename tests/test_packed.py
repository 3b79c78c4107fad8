"""Attention over packed sequences on the GPU against a plain 64-bit
implementation (tests/packed.py has the bounds), and its plans."""
import pytest
import torch

from packed import batch, check_forward, rows

NAN = float("nan")

CASES = [
    # lengths, H, Hkv, causal
    ([1], 1, 1, True),
    ([1], 2, 1, False),
    ([2, 1, 3], 4, 2, True),
    ([127], 2, 2, True),
    ([128], 2, 1, True),
    ([129], 3, 1, True),          # odd group: two tiles of one head
    ([128, 128, 256], 4, 4, False),
    ([5, 0, 130, 165], 8, 2, True),
    ([5, 0, 130, 165], 8, 2, False),
    ([255, 1, 257], 6, 2, True),
    ([257, 513, 64], 3, 3, False),
    ([0, 0, 300, 0], 2, 1, True),
    ([1] * 70, 2, 2, True),       # more sequences than a warp has lanes
    ([40, 700, 3, 129, 16, 17, 15], 4, 1, True),
    ([1025, 384], 12, 4, True),
    ([640, 127, 640], 5, 5, False),
]


def run(lengths, H, Hkv, d, causal, layout="fused", before=0, after=0, seed=0, scale=None):
    from exact_attention_98_gb300 import fa

    cu, n = batch(lengths, before, after)
    q, k, v = rows(n, H, d, seed, layout), rows(n, Hkv, d, seed + 1, layout), rows(n, Hkv, d, seed + 2, layout)
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    o, lse = fa.packed_forward(q, k, v, plan, scale=scale)
    assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
    check_forward(o, lse, q, k, v, cu, fa.default_scale(d) if scale is None else scale, causal)
    return cu, n, q, k, v, o, lse, plan


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,H,Hkv,causal", CASES)
def test_forward(lengths, H, Hkv, causal, d):
    run(lengths, H, Hkv, d, causal, seed=len(lengths) + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_forward_more_items_than_sms(d):
    # odd group (blocks) and even group (tiles), several rounds of every CTA
    run([300, 520, 77, 1, 900, 256], 48, 16, d, True, seed=1)
    run([300, 520, 77, 1, 900, 256], 48, 24, d, True, seed=2)


# Few items: cut into key ranges and joined.  The bounds hold for that too: a range's LSE, of
# up to 9, is off by its rounding, 2^-21, and weights by exponentials' few ulps, so a
# joined O by less than the 2 * 2^-20 sum p |v| that scores' errors are given.
SPLIT = [
    ([1408], 1, 1, True),
    ([2000], 4, 2, True),             # an even group: one tile of two heads
    ([1537], 3, 1, True),                # an odd one: two tiles of one head, the last without a second
    ([3300, 1, 0, 2400], 2, 2, True),
    ([1281, 1700, 1300], 2, 1, True),
    ([4225], 1, 1, True),
    ([100, 4000], 4, 2, True),
    ([100, 4000], 6, 3, False),    # one item too many
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,H,Hkv,split", SPLIT)
def test_forward_split(lengths, H, Hkv, split, d, causal):
    from exact_attention_98_gb300 import fa

    assert (fa.fa_fwd_packed_workspace_bytes(len(lengths), sum(lengths), H, Hkv, d) > 0) == split
    run(lengths, H, Hkv, d, causal, layout="fused" if H % 2 else "heads", seed=d + H)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths,H,Hkv", [([8200, 8350], 1, 1), ([9000], 2, 1), ([16000, 30], 1, 1), ([1500] * 5, 2, 2)])
def test_forward_split_as_without(lengths, H, Hkv, causal):
    """Longer sequences, with the workspace and without: both round P (2^-8 of sum p v, v > 0, so of O) and O
    once, and nothing else beyond fp32, so they differ by 2 * 2^-8 (1 + 1) |O|, and a little."""
    from ctypes import byref

    from exact_attention_98_gb300 import fa

    cu, n = batch(lengths, 1, 2)
    d = 128
    q, k, v = rows(n, H, d, 1, "dense"), rows(n, Hkv, d, 2, "dense"), rows(n, Hkv, d, 3, "dense")
    v = v.abs() + torch.linspace(0, 1, n, device="cuda").to(torch.bfloat16)[:, None, None]
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    need = fa.fa_fwd_packed_workspace_bytes(len(lengths), n, H, Hkv, d)
    assert need > 0
    got = []
    # (what the workspace holds on entry does not matter)
    for ws in (None, torch.full((need,), 255, dtype=torch.uint8, device="cuda")):
        o = torch.full((n, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, H), 7.0, device="cuda")
        r = [byref(fa.Rows(t.data_ptr(), t.stride(0), t.stride(1))) for t in (q, k, v, o)]
        fa.fa_fwd_packed(plan.plan, len(lengths), n, *r, lse, H, Hkv, d, fa.default_scale(d), ws)
        assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
        got.append((o.double(), lse.double()))
    (o0, l0), (o1, l1) = got
    for t in (o0, l0, o1, l1):
        assert (t[:1] == 7).all() and (t[cu[-1]:] == 7).all()
    r = slice(1, cu[-1])
    assert ((o0 - o1).abs()[r] <= 2.0 ** -8 * 4.1 * o0.abs()[r]).all()
    # scores alike in both; sums and logarithms in fp32
    assert ((l0 - l1).abs()[r] <= 2.0 ** -18 * (1 + l0.abs()[r])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_forward_split_other_rows_do_not_matter(d, causal):
    from exact_attention_98_gb300 import fa

    cu, n = batch([1500, 1300, 1700], 3, 200)
    q, k, v = rows(n, 2, d, 5), rows(n, 2, d, 6), rows(n, 2, d, 7)
    for t, bad in ((q, NAN), (k, float("inf")), (v, NAN)):
        for a, b in ((0, 3), (cu[1], cu[2]), (cu[-1], n)):
            t[a:b] = bad
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    assert fa.fa_fwd_packed_workspace_bytes(3, n, 2, 2, d) > 0
    wide = torch.full((n, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.packed_forward(q, k, v, plan, out=wide[:, 1:3])
    assert fa.fa_last_device_status() == fa.FA_OK
    check_forward(o, lse, q, k, v, cu, fa.default_scale(d), causal, skip=(1,))
    assert (wide[:, 0] == 7).all() and (wide[:, 3] == 7).all()
    assert (wide[:3] == 7).all() and (wide[cu[-1]:] == 7).all()


@pytest.mark.gpu
def test_forward_split_plans():
    """A plan remade in a captured graph, of one sequence, of many and of none; bits do not vary;
    memory that is no plan."""
    from exact_attention_98_gb300 import fa

    n, d = 3000, 128
    cu = torch.tensor([0, 0, n], dtype=torch.int32, device="cuda")
    q, k, v = (rows(n, 2, d, s) for s in range(3))
    plan = fa.packed_plan(cu, n)
    assert fa.fa_fwd_packed_workspace_bytes(2, n, 2, 2, d) > 0
    out = torch.empty(n, 2, d, dtype=torch.bfloat16, device="cuda")
    first = fa.packed_forward(q, k, v, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.packed_plan(cu, n, out=plan)
        _, lse = fa.packed_forward(q, k, v, plan, out=out)
    for offsets in ([0, 0, n], [0, 130, 140], [7, 7, 7], [1, 1500, n - 1]):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK
        check_forward(out, lse, q, k, v, offsets, fa.default_scale(d), True)
        assert (out[: offsets[0]] == 7).all() and (out[offsets[-1]:] == 7).all()
        if offsets == [0, 0, n]:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    out.fill_(7.0)
    fa.packed_forward(q, k, v, fa.PackedPlan(torch.zeros_like(plan.plan), n, 2, True), out=out)
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
    assert (out == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["dense", "heads"])
def test_forward_layouts(layout):
    run([200, 129], 4, 2, 128, True, layout=layout)
    run([200, 129], 3, 3, 64, True, layout=layout)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, 0.002])
def test_forward_scale(scale):
    run([200, 129, 31], 4, 2, 128, True, scale=scale)


def positions(cu, n):
    out = [-1] * n
    for b in range(len(cu) - 1):
        out[cu[b]: cu[b + 1]] = range(cu[b + 1] - cu[b])
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [[7], [0, 5, 0], [128, 1, 300], [3] * 100, [20000, 77, 9000, 8200, 1, 8191, 8193],
                                     [], [1] * 3000])
def test_plan(lengths, causal):
    """Positions, and the lists: every tile once, those that see the most keys first."""
    import struct

    from exact_attention_98_gb300 import fa

    cu, n = batch(lengths, 2, 3)
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    assert fa.fa_last_device_status() == fa.FA_OK
    assert plan.positions.tolist() == positions(cu, n)
    raw = plan.plan.cpu().numpy().tobytes()
    _, r, s, c, n_tiles, n_blocks, begin, end = struct.unpack("8i", raw[:32])
    assert (r, s, c) == (n, len(lengths), int(causal))
    if lengths:
        assert (begin, end) == (cu[0], cu[-1])
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    cap = lambda size: up(16 * (n // size + min(n, len(lengths))))  # noqa: E731
    at = 256 + up(4 * n)
    seqs = [(cu[b], x) for b, x in enumerate(lengths) if x]
    for size, count, by_tile in ((128, n_tiles, causal), (256, n_blocks, causal), (128, n_tiles, False)):
        got = [struct.unpack_from("4i", raw, at + 16 * i) for i in range(count)]
        want = sorted((a, x, t) for a, x in seqs for t in range(-(-x // size)))
        assert sorted(e[:3] for e in got) == want
        cost = [e[2] + 1 if by_tile else -(-e[1] // size) for e in got]
        # costs that share a bucket may come in any order: 1/32 of an octave from 64 on
        bucket = [x if x < 64 else (64 << 5) + ((x.bit_length() - 7) << 5) + ((x >> (x.bit_length() - 6)) & 31)
                  for x in cost]
        assert bucket == sorted(bucket, reverse=True)
        if not by_tile:
                # a sequence's tiles follow one another, from its first on
                assert all(got[i - 1][0] == e[0] and got[i - 1][2] == e[2] - 1 for i, e in enumerate(got) if e[2])
        at += cap(size)


@pytest.mark.gpu
def test_plan_bits_do_not_vary():
    from exact_attention_98_gb300 import fa

    cu, n = batch([300, 5, 5, 700, 129, 129, 0, 64])
    dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    plans = [fa.packed_plan(dev, n) for _ in range(3)]
    # (bytes behind the lists' ends are not written)
    fa.packed_plan(dev, n, out=plans[1])
    for p in plans:
        p.plan.zero_()
        fa.packed_plan(dev, n, out=p)
    assert torch.equal(plans[0].plan, plans[1].plan) and torch.equal(plans[0].plan, plans[2].plan)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 40, 30, 60], [-1, 20, 60], [0, 61], [70, 80], [0, 50, 20]])
def test_bad_offsets(cu):
    """Recorded; the plan is of no sequence, so nothing is written."""
    from exact_attention_98_gb300 import fa

    q = rows(60, 2, 64, 0)
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), 60)
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
    assert plan.positions.tolist() == [-1] * 60
    out = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.packed_forward(q, q, q, plan, out=out)
    assert fa.fa_last_device_status() == fa.FA_OK
    assert (out == 7).all()


@pytest.mark.gpu
def test_not_a_plan():
    """Memory that holds no plan, or one of other rows: recorded, nothing is written."""
    from exact_attention_98_gb300 import fa

    cu, n = batch([30, 30])
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
    other = fa.PackedPlan(torch.zeros_like(plan.plan), n, 2, True)
    q = rows(n, 2, 64, 0)
    out = torch.full((n, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.packed_forward(q, q, q, other, out=out)
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
    fa.packed_forward(q[:59], q[:59], q[:59], fa.PackedPlan(plan.plan, 59, 2, True), out=out[:59])
    assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
    assert (out == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_forward_other_rows_do_not_matter(H, Hkv, d, causal):
    """Infinities and NaN in padding rows and in a sequence between; padding rows of the output keep
    what they held."""
    from exact_attention_98_gb300 import fa

    cu, n = batch([100, 70, 200, 1, 128], 3, 200)
    q, k, v = rows(n, H, d, 5), rows(n, Hkv, d, 6), rows(n, Hkv, d, 7)
    for t, bad in ((q, NAN), (k, float("inf")), (v, NAN)):
        for a, b in ((0, 3), (cu[1], cu[2]), (cu[-1], n)):
            t[a:b] = bad
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    wide = torch.full((n, H + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.packed_forward(q, k, v, plan, out=wide[:, 1: H + 1])
    assert fa.fa_last_device_status() == fa.FA_OK
    check_forward(o, lse, q, k, v, cu, fa.default_scale(d), causal, skip=(1,))
    assert (wide[:, 0] == 7).all() and (wide[:, H + 1] == 7).all()
    assert (wide[:3] == 7).all() and (wide[cu[-1]:] == 7).all()
