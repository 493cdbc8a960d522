"""Calls that write what the next call of the stream reads, with nothing in between."""
import pytest
import torch

import kv_cache_quantize_b200 as kvq

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("cache", [torch.int8, torch.bfloat16])
def test_attention_sees_what_the_page_calls_before_it_wrote(cache):
    """Rows freed, forked from another parent and attended to, step by step: tables, lengths and pages change under the
    attention's reads.  The same steps with a wait after every call give the same outputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    pages, block, rows, cols = 400, 16, 24, 12
    shape = (pages, block, 2, 128)
    caches = [torch.randint(-128, 128, shape, dtype=torch.int8, generator=g, device="cuda") if cache == torch.int8 else
              torch.randn(shape, generator=g, device="cuda").to(cache) for _ in range(2)]
    scales = [torch.rand((256,), generator=g, device="cuda") / 64 for _ in range(2)] if cache == torch.int8 else []
    q = torch.randn((rows, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    prefix = torch.arange(pages - 4, pages, dtype=I32, device="cuda")
    steps = [[torch.randint(0, 8, (16,), generator=g, device="cuda"), torch.randperm(16, generator=g, device="cuda") + 8]
             for _ in range(40)]

    def run(wait):
        kc, vc = (c.clone() for c in caches)
        table = torch.full((rows, cols), -1, dtype=I32, device="cuda")
        lens = torch.zeros((rows,), dtype=I32, device="cuda")
        refs = torch.zeros((pages,), dtype=I32, device="cuda")
        refs[pages - 4:] = 1
        for i in range(8):                                   # the parents
            table[i, :i + 3] = torch.arange(12 * i, 12 * i + i + 3, dtype=I32, device="cuda")
            refs[12 * i:12 * i + i + 3] = 1
            lens[i] = 16 * (i + 2) + 2 * i + 1
        outs = [torch.empty_like(q) for _ in steps]
        torch.cuda.synchronize()
        done = torch.cuda.synchronize if wait else lambda: None
        for (parents, children), out in zip(steps, outs):
            kvq.free_pages(table, lens, refs, children, block)
            done()
            kvq.fork_pages([kc, vc], table, lens, refs, parents, children, block)
            done()
            kvq.shared_prefix_attention(q, kc, vc, table, lens, prefix, 60, *scales, out=out)
            done()
        assert kvq.get_error() == 0
        return outs, table, lens, refs

    for a, b in zip(run(True), run(False)):
        assert all(torch.equal(x, y) for x, y in zip(a, b)) if isinstance(a, list) else torch.equal(a, b)
