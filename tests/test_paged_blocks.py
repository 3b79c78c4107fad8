"""Append and read of batches around the sizes where a block takes four tokens
instead of one: the bytes do not depend on it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("more", [-1, 0, 1, 2, 3, 3650])
def test_one_call_as_several(fmt, more):
    from exact_attention_98_gb300 import fa

    T = torch.cuda.get_device_properties(0).multi_processor_count * 8 + more
    d, page, Hkv, H = 64, 32, 2, 4
    n = -(-T // page)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    rope = fa.rope_table(T, d)
    table = torch.randperm(n, generator=g).to(torch.int32).cuda()[None]
    ints = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for size in (T, 500):
        pages = fa.paged_pages(n, Hkv, page, d, fmt)
        q, k, v = [], [], []
        for at in range(0, T, size):
            part = x[at:at + size]
            m = len(part)
            lens, cu = ints(at + m), ints(0, m)
            q.append(fa.paged_append(part[:, H:H + Hkv], part[:, H + Hkv:], pages, table, lens, cu, q=part[:, :H],
                                     rope=rope))
            kv = fa.paged_read(pages, table, lens, cu, m, d)
            k.append(kv[0])
            v.append(kv[1])
        assert fa.fa_last_device_status() == fa.FA_OK
        outs.append([pages.view(torch.uint8)] + [torch.cat(y) for y in (q, k, v)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
