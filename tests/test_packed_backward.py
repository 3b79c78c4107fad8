"""Gradients of the attention over packed sequences on the GPU against a plain
64-bit implementation (tests/packed.py has the bounds), and a training
step's and a serving step's calls together."""
import numpy as np
import pytest
import torch

from packed import batch, check_backward, check_forward, f64, plain_backward, plain_forward, rows, within
from test_packed import CASES, run

NAN = float("nan")


def check(lengths, H, Hkv, d, causal, layout="fused", before=0, after=0, seed=0, scale=None):
    from exact_attention_98_gb300 import fa

    cu, n, q, k, v, o, lse, plan = run(lengths, H, Hkv, d, causal, layout, before, after, seed, scale)
    do = rows(n, H, d, seed + 3, layout)
    grads = fa.packed_backward(q, k, v, o, lse, do, plan, scale=scale)
    assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
    check_backward(grads, q, k, v, o, lse, do, cu, fa.default_scale(d) if scale is None else scale, causal)
    return cu, n, q, k, v, o, lse, do, plan, grads


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,H,Hkv,causal", CASES)
def test_backward(lengths, H, Hkv, causal, d):
    check(lengths, H, Hkv, d, causal, seed=len(lengths) + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(48, 16), (48, 24)])
def test_more_items_than_sms(H, Hkv, d):
    check([300, 520, 77, 1, 900, 256], H, Hkv, d, True, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,H,Hkv,causal", [
    ([2000], 1, 1, True),           # parts without a query tile (d = 128)
    ([1030], 3, 1, True),           # parts that begin within a head
    ([1500, 3, 700], 8, 1, True),
    ([700, 1, 640], 16, 2, True),
    ([900], 8, 1, False),
    ([130] * 5, 8, 1, True),
])
def test_split_items(lengths, H, Hkv, causal, d):
    """Few items: each is split, its parts joined afterwards."""
    from exact_attention_98_gb300 import fa

    n = sum(lengths)
    whole = 256 + 2 * ((n * H * 4 + 255) // 256 * 256) + (n * H * d * 4 + 255) // 256 * 256
    parts = (fa.fa_bwd_packed_workspace_bytes(len(lengths), n, H, Hkv, d) - whole) // (2 * Hkv * n * d * 4)
    assert parts > 1 or (d == 64 and H == Hkv)
    check(lengths, H, Hkv, d, causal, seed=n)
    check(lengths, H, Hkv, d, causal, before=70, after=200, seed=n + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(d):
    check([1 + 7 * (i % 5) for i in range(700)], 2, 1, d, True)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_offsets_past_32_bits(d):
    """The sequences are the last rows of tensors of more than 2^31 elements."""
    from exact_attention_98_gb300 import fa

    H, Hkv, lengths = 256, 2, [300, 77]
    n = 2 ** 31 // (H * d) + 1000
    cu, n = batch(lengths, n - sum(lengths), 5)
    end = slice(cu[0], n)
    q, k, v, do = (torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv, H))
    for i, t in enumerate((q, k, v, do)):
        t[end] = rows(n - cu[0], t.shape[1], d, i, "dense")
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
    table = fa.rope_table(300, d)
    turned, _ = fa.rotate(q, None, plan.positions, table)
    want = fa.rotate(q[end].clone(), None, plan.positions[end].clone(), table)[0]
    live = slice(cu[0], cu[-1])
    assert torch.equal(turned[live], want[: cu[-1] - cu[0]])
    del turned, want
    o, lse = fa.packed_forward(q, k, v, plan)
    grads = fa.packed_backward(q, k, v, o, lse, do, plan)
    assert fa.fa_last_device_status() == fa.FA_OK
    cu = [x - cu[0] for x in cu]
    heads = [0, 1, 127, 128, 255]  # (the bounds of every head would take minutes)
    small = [t[end] for t in (q, k, v, o, lse, do, *grads)]
    q, k, v, o, lse, do, dq, dk, dv = small
    for h in heads:
        one = [t[:, h: h + 1] for t in (q, o, do, dq)]
        kv = [t[:, h // 128: h // 128 + 1] for t in (k, v)]
        check_forward(one[1], lse[:, h: h + 1], one[0], *kv, cu, fa.default_scale(d), True)
        for b in range(2):
            s = slice(cu[b], cu[b + 1])
            g, err = plain_backward(f64(one[0][s, 0]), f64(kv[0][s, 0]), f64(kv[1][s, 0]), f64(one[1][s, 0]),
                                    f64(lse[s, h]), f64(one[2][s, 0]), fa.default_scale(d), True)
            within(f64(one[3][s, 0]), g[0], err[0], ("dq", h))
    # dK and dV as those of a batch of the last rows alone (whose items are split otherwise)
    m = cu[-1]
    alone = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), m)
    again = fa.packed_backward(q[:m], k[:m], v[:m], o[:m], lse[:m].contiguous(), do[:m], alone)
    for a, b in zip((dk, dv), again[1:]):
        assert np.abs(f64(a[:m]) - f64(b)).max() <= 2.0 ** -7 * np.abs(f64(b)).max()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["dense", "heads"])
def test_layouts(layout):
    check([200, 129], 4, 2, 128, True, layout=layout)
    check([200, 129], 3, 3, 64, True, layout=layout)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 0.002])
def test_scale(scale, d):
    check([200, 129, 31], 4, 2, d, True, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_other_rows_do_not_matter(H, Hkv, d, causal):
    """Infinities and NaN in padding rows and in a sequence between; the gradients go to parts of a fused
    gradient, whose other parts and padding rows keep what they held."""
    from exact_attention_98_gb300 import fa

    cu, n = batch([100, 70, 200, 1, 128], 3, 200)
    q, k, v, do = rows(n, H, d, 5), rows(n, Hkv, d, 6), rows(n, Hkv, d, 7), rows(n, H, d, 8)
    for t, bad in ((q, NAN), (k, float("inf")), (v, NAN), (do, float("-inf"))):
        for a, b in ((0, 3), (cu[1], cu[2]), (cu[-1], n)):
            t[a:b] = bad
    plan = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, causal)
    o, lse = fa.packed_forward(q, k, v, plan)
    for t in (o, lse):
        t[:3], t[cu[-1]:] = NAN, NAN
    wide = torch.full((n, H + 2 * Hkv + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :H], wide[:, H: H + Hkv], wide[:, H + Hkv: H + 2 * Hkv]
    grads = fa.packed_backward(q, k, v, o, lse, do, plan, out=out)
    assert fa.fa_last_device_status() == fa.FA_OK, hex(fa.fa_last_device_site())
    check_backward(grads, q, k, v, o, lse, do, cu, fa.default_scale(d), causal, skip=(1,))
    assert (wide[:, -1] == 7).all() and (wide[:3] == 7).all() and (wide[cu[-1]:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_bits_and_workspace(d):
    """dK and dV have the same bits from run to run, whatever the workspace holds."""
    from exact_attention_98_gb300 import fa

    cu, n, q, k, v, o, lse, do, plan, first = check([700, 130, 513], 8, 2, d, True)
    nbytes = fa.fa_bwd_packed_workspace_bytes(3, n, 8, 2, d)
    for fill in (0, 255):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")
        again = fa.packed_backward(q, k, v, o, lse, do, plan, workspace=ws)
        assert fa.fa_last_device_status() == fa.FA_OK
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
        check_backward(again, q, k, v, o, lse, do, cu, fa.default_scale(d), True)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_against_differences(d, causal):
    """Single elements of Q, K and V moved in the plain forward: the slope of sum(O dO), within the
    gradients' bounds, those of a D from the rounded O, and the difference's own error."""
    cu, n, q, k, v, o, lse, do, plan, grads = check([37, 140], 2, 1, d, causal, seed=11)
    scale = 1 / np.sqrt(d)
    r = np.random.default_rng(3)
    grads = [f64(g) for g in grads]
    for s in (slice(cu[0], cu[1]), slice(cu[1], cu[2])):
        x = [f64(t)[s] for t in (q, k, v)]
        dof, of, lsef = f64(do)[s], f64(o)[s], f64(lse)[s]
        err = [np.zeros_like(t) for t in x]
        for h in range(2):
            args = x[0][:, h], x[1][:, 0], x[2][:, 0]
            g, e = plain_backward(*args, of[:, h], lsef[:, h], dof[:, h], scale, causal)
            _, l_ref, o_err, _ = plain_forward(*args, scale, causal)
            # D's error is that of O times dO; a row's weights carry it to dQ and dK
            see = np.tril(np.ones((len(l_ref),) * 2, bool)) | (not causal)
            w = np.exp(np.where(see, scale * args[0] @ args[1].T, -np.inf) - l_ref[:, None])
            w *= scale * (np.abs(dof[:, h]) * o_err).sum(1, keepdims=True)
            err[0][:, h] += e[0] + 1.01 * w @ np.abs(args[1])
            err[1][:, 0] += e[1] + 1.01 * w.T @ np.abs(args[0])
            err[2][:, 0] += e[2]
        for i in (1, 2):  # rounded after the sum over the heads
            err[i] += 2.0 ** -8 * 1.02 * np.abs(grads[i][s])

        def loss(which, at, step):
            y = [t.copy() for t in x]
            y[which][at] += step
            return sum((plain_forward(y[0][:, h], y[1][:, 0], y[2][:, 0], scale, causal)[0] * dof[:, h]).sum()
                       for h in range(2))

        for which in range(3):
            for _ in range(12):
                at = tuple(int(r.integers(0, m)) for m in x[which].shape)
                fine, wide = ((loss(which, at, h) - loss(which, at, -h)) / (2 * h) for h in (1e-3, 2e-3))
                got = grads[which][s][at]
                # a central difference's error falls with the square of its step: a third of what doubling adds
                assert abs(got - fine) <= err[which][at] + abs(wide - fine) + 1e-9, (which, at, got, fine)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_training_step(d):
    """Rotation, attention and their gradients in one run on a stream of its own, captured into a graph and replayed
    with other sequences and inputs."""
    from exact_attention_98_gb300 import fa

    H, Hkv, n = 4, 2, 500
    table = fa.rope_table(n, d // 2)
    fused, do = rows(n, H + 2 * Hkv, d, 0, "dense"), rows(n, H, d, 1, "dense")
    cu = torch.tensor([0, 100, 100, 430], dtype=torch.int32, device="cuda")
    grad = torch.zeros_like(fused)
    split = lambda t: (t[:, :H], t[:, H: H + Hkv], t[:, H + Hkv:])  # noqa: E731
    plan = fa.packed_plan(cu, n)

    def step(stream=None):
        fa.packed_plan(cu, n, out=plan, stream=stream)
        q, k, v = split(fused)
        q, k = fa.rotate(q, k, plan.positions, table, stream=stream)
        o, lse = fa.packed_forward(q, k, v, plan, stream=stream)
        dq, dk, dv = fa.packed_backward(q, k, v, o, lse, do, plan, out=split(grad), stream=stream)
        fa.rotate(dq, dk, plan.positions, table, backward=True, out=(dq, dk), stream=stream)
        return q, k, v, o, lse

    def verify(state, lengths):
        q, k, v, o, lse = state
        offsets, _ = batch(lengths)
        check_forward(o, lse, q, k, v, offsets, fa.default_scale(d), True)
        # the rotation undone by the table's own: a rotation's transpose is its inverse
        dq, dk, dv = split(grad)
        dq, dk = fa.rotate(dq, dk, plan.positions, table)
        # (rounded twice more on the way)
        slack = [g.double().cpu().numpy() for g in (dq, dk, dv)]
        exact = fa.packed_backward(q, k, v, o, lse, do, plan)
        check_backward(exact, q, k, v, o, lse, do, offsets, fa.default_scale(d), True)
        end = offsets[-1]
        for a, b in zip(slack, exact):
            b = f64(b)
            pair = np.abs(b).max(-1, keepdims=True)
            assert (np.abs(a - b)[:end] <= 2.0 ** -6 * pair[:end] + 1e-4).all()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = step(side)
    torch.cuda.current_stream().wait_stream(side)
    verify(state, [100, 0, 330])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        state = step()
    for offsets, lengths in (([0, 100, 100, 430], [100, 0, 330]), ([0, 1, 257, 500], [1, 256, 243])):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        fused.copy_(rows(n, H + 2 * Hkv, d, offsets[1], "dense"))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK
        verify(state, lengths)


@pytest.mark.gpu
def test_two_at_once():
    """Backwards on two streams with workspaces of their own; one plan."""
    from exact_attention_98_gb300 import fa

    for d in (64, 128):
        cu, n, q, k, v, o, lse, do, plan, want = check([900, 300, 129], 8, 4, d, True)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = [[fa.packed_backward(q, k, v, o, lse, do, plan, stream=s) for s in streams] for _ in range(3)]
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK
        for pair in got:
            for g in pair:
                assert torch.equal(g[1], want[1]) and torch.equal(g[2], want[2])
                check_backward(g, q, k, v, o, lse, do, cu, fa.default_scale(d), True)


@pytest.mark.gpu
def test_not_a_plan():
    from exact_attention_98_gb300 import fa

    for d in (64, 128):
        n = 60
        plan = fa.PackedPlan(torch.zeros(fa.fa_packed_plan_bytes(2, n), dtype=torch.uint8, device="cuda"), n, 2, True)
        q = rows(n, 2, d, 0)
        lse = torch.zeros(n, 2, device="cuda")
        out = tuple(torch.full((n, 2, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        fa.packed_backward(q, q, q, q, lse, q, plan, out=out)
        assert fa.fa_last_device_status() == fa.FA_ERR_INVALID_ARG
        assert all((t == 7).all() for t in out)


@pytest.mark.gpu
def test_as_plain_attention():
    """One sequence of all rows is the plain causal attention, bit for bit."""
    from exact_attention_98_gb300 import fa

    n, H, d = 1000, 4, 128
    q, k, v, do = (rows(n, H, d, i, "heads") for i in range(4))
    plan = fa.packed_plan(torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    o, lse = fa.packed_forward(q, k, v, plan)
    one = lambda t: t.transpose(0, 1)[None]  # noqa: E731
    o2, lse2 = fa.forward(one(q), one(k), one(v), causal=True)
    assert torch.equal(one(o), o2) and torch.equal(lse.T[None], lse2)
