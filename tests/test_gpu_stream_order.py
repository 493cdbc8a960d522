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


def handle(kind, stream):
    return {"object": stream, "handle": stream.cuda_stream, "default handle": 0}[kind]


@pytest.mark.parametrize("kind", ["object", "handle", "default handle"])
def test_streams_given_as_objects_and_handles(kind):
    """Outputs and workspaces that the calls allocate belong to the stream given: memory that the current stream hands
    on at once, and writes, does not meet them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(52)
    side = torch.cuda.Stream()
    q = torch.randn((64, 16, 128), generator=g, device="cuda").to(torch.bfloat16)
    caches = [torch.randn((200, 64, 4, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    table = torch.randint(0, 200, (64, 9), generator=g, device="cuda").to(I32)
    lens = torch.randint(0, 9 * 64, (64,), generator=g, device="cuda").to(I32)
    prefix = torch.arange(60, dtype=I32, device="cuda")
    cu = torch.tensor([0, 20, 64], dtype=I32, device="cuda")
    k = torch.randn((64, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    parents, children = torch.zeros((1,), dtype=I32, device="cuda"), torch.ones((1,), dtype=I32, device="cuda")
    st = handle(kind, side)

    def calls(stream):
        refs, rows, row_lens = torch.zeros((200,), dtype=I32, device="cuda"), table[:2].clone(), torch.zeros((2,), dtype=I32, device="cuda")
        rows[0, :2] = torch.tensor([180, 190], dtype=I32, device="cuda")
        refs[[180, 190]] = 1
        row_lens[0] = 100
        pages = [c.clone() for c in caches]
        torch.cuda.synchronize()
        out = [kvq.shared_prefix_attention(q, *caches, table, lens, prefix, 3800, stream=stream),
               kvq.prompt_attention(q, k, k, cu, stream=stream),
               kvq.fork_pages(pages, rows, row_lens, refs, parents, children, 64, stream=stream)]
        kvq.copy_pages(pages, children, parents, stream=stream)
        kvq.free_pages(rows, row_lens, refs, parents, 64, stream=stream)
        out += kvq.compact_pages(pages, rows, refs, stream=stream)
        for n in (1 << 12, 1 << 16, 1 << 18, 1 << 22, 1 << 24):          # what the allocator may hand on
            torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        return out + pages + [refs, rows, row_lens]

    want = calls(None)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(calls(st), want))
    assert kvq.get_error() == 0 and kvq.get_error(side) == 0


def test_calls_of_several_threads():
    """Each thread on a stream of its own: no state of a call is shared on the host."""
    import threading
    g = torch.Generator(device="cuda")
    g.manual_seed(53)
    caches = [torch.randn((100, 16, 2, 64), generator=g, device="cuda").to(torch.float16) for _ in range(2)]
    table = torch.randint(0, 100, (6, 8), generator=g, device="cuda").to(I32)
    lens = torch.tensor([0, 1, 50, 128, 77, -1], dtype=I32, device="cuda")
    qs = [torch.randn((6, 4, 64), generator=g, device="cuda").to(torch.float16) for _ in range(4)]
    cu = torch.tensor([0, 2, 6], dtype=I32, device="cuda")

    def once(q, stream=None):
        return (kvq.shared_prefix_attention(q, *caches, table, lens, stream=stream)[:5],
                kvq.prompt_attention(q, q[:, :2].contiguous(), q[:, 2:].contiguous(), cu, stream=stream))

    want = [once(q) for q in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                if not all(torch.equal(a, b) for a, b in zip(once(qs[i]), want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and kvq.get_error() == 0
