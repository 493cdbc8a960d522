"""The cache epilogue, the attention and the page operations together, as a serving loop runs them."""
import pytest
import torch

import kv_cache_quantize_b200 as kvq
from _attention import check_rows, prompt64, shared64

pytestmark = pytest.mark.gpu
NQ, NKV, D, BLOCK, PAGES = 8, 2, 128, 16, 96
H = (NQ + 2 * NKV) * D


class Server:
    """int8 caches, a block table and one layer's projections of random tokens."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        c = lambda: torch.zeros((PAGES, BLOCK, NKV, D), dtype=torch.int8, device="cuda")  # noqa: E731
        self.k, self.v = c(), c()
        self.scale_k = 0.02 + 0.02 * torch.rand(NKV * D, generator=self.g, device="cuda")
        self.scale_v = 0.02 + 0.02 * torch.rand(NKV * D, generator=self.g, device="cuda")
        self.offset_k = torch.randn(NKV * D, generator=self.g, device="cuda").round()
        self.offset_v = torch.randn(NKV * D, generator=self.g, device="cuda").round()
        self.table = torch.full((6, 24), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(6, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(PAGES, dtype=torch.int32, device="cuda")

    def tokens(self, n):
        x = torch.randn((n, H), generator=self.g, device="cuda").to(torch.bfloat16)
        angle = 6.28 * torch.rand((n, 1, D // 2), generator=self.g, device="cuda")
        angle = torch.cat([angle, angle], -1)
        return x, angle.cos().to(torch.bfloat16), angle.sin().to(torch.bfloat16)

    def write(self, x, cos, sin, slots):
        return kvq.dequant_rope_quant_kvcache(x, cos, sin, self.k, self.v, slots, self.scale_k, self.scale_v, self.offset_k,
                                              self.offset_v, size_splits=(NQ * D, NKV * D, NKV * D), kv_output=True,
                                              cache_mode="page")

    def decode(self, q, rows, shared):
        """Attention of one token of each row; the first `shared` pages are common to all."""
        return kvq.shared_prefix_attention(q, self.k, self.v, self.table[rows, shared:], self.lens[rows] - shared * BLOCK,
                                           self.table[rows[0], :shared].contiguous(), shared * BLOCK, scale_k=self.scale_k,
                                           scale_v=self.scale_v, offset_k=self.offset_k, offset_v=self.offset_v)

    def want(self, q, rows, shared):
        return shared64(q, self.k, self.v, self.table[rows, shared:], self.lens[rows] - shared * BLOCK,
                        self.table[rows[0], :shared], shared * BLOCK, self.scale_k, self.scale_v, self.offset_k,
                        self.offset_v)


def prefilled(seed, n):
    """A server whose row 0 holds a prompt of n tokens, after checking the prompt's attention."""
    s = Server(seed)
    held = -(-n // BLOCK)
    pages = torch.randperm(PAGES, generator=s.g, device="cuda")[:held].to(torch.int32)
    s.table[0, :held] = pages
    s.lens[0] = n
    s.ref[pages.long()] = 1
    t = torch.arange(n, device="cuda")
    q, k, v = s.write(*s.tokens(n), (pages[t // BLOCK] * BLOCK + t % BLOCK).to(torch.int32))
    out = kvq.prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), check=True)
    want, _, bound, _ = prompt64(q, k, v, [(0, n, 0, n)])
    check_rows(out, want, bound, "prompt")
    return s


def slots_of(s, rows):
    """The place of each row's next token."""
    n = s.lens[rows].long()
    return s.table[rows, n // BLOCK] * BLOCK + (n % BLOCK).to(torch.int32)


def test_prompt_fork_decode_free_compact():
    s = prefilled(1, 300)                                     # 18 full pages, 12 tokens in the last one
    rows = torch.tensor([0, 2, 3, 5], device="cuda")
    fresh = kvq.fork_pages([s.k, s.v], s.table, s.lens, s.ref, torch.zeros(3, dtype=torch.int32, device="cuda"),
                           rows[1:], BLOCK, check=True)
    assert bool((fresh >= 0).all()) and len(set(fresh.tolist())) == 3 and s.ref[s.table[0, :18].long()].tolist() == [4] * 18
    for _ in range(3):
        q, _, _ = s.write(*s.tokens(4), slots_of(s, rows))
        s.lens[rows] += 1
        out = s.decode(q, rows, 18)
        want, _, bound, _ = s.want(q, rows, 18)
        check_rows(out, want, bound, "decode")
    # without sharing: every request over its own row
    alone = kvq.shared_prefix_attention(q, s.k, s.v, s.table[rows], s.lens[rows], scale_k=s.scale_k, scale_v=s.scale_v,
                                        offset_k=s.offset_k, offset_v=s.offset_v, check=True)
    check_rows(alone, want, bound, "unshared")
    # one row ends; the pool closes its holes; the others' tokens are where their table says
    kvq.free_pages(s.table, s.lens, s.ref, rows[2:3], BLOCK, check=True)
    kvq.compact_pages([s.k, s.v], s.table, s.ref, new_table=s.table, new_ref_count=s.ref, check=True)
    used = int((s.ref > 0).sum())
    assert used == 18 + 3 and bool((s.ref[:used] > 0).all()) and int(s.table.max()) == used - 1
    keep = torch.tensor([0, 1, 3], device="cuda")
    again = s.decode(q[keep], rows[keep], 18)
    check_rows(again, want[keep], bound[keep], "after compaction")
    assert kvq.get_error() == 0


def test_a_step_captured_and_replayed():
    """The epilogue and the attention in one graph, replayed as the rows grow, against eager calls; two graphs of the
    same calls replayed one after the other have workspaces of their own."""
    s = prefilled(2, 130)
    rows = torch.tensor([0, 1, 4], device="cuda")
    kvq.fork_pages([s.k, s.v], s.table, s.lens, s.ref, torch.zeros(2, dtype=torch.int32, device="cuda"), rows[1:], BLOCK)
    x, cos, sin = s.tokens(3)
    slots = slots_of(s, rows)
    own_table = s.table[rows, 8:].contiguous()
    own_lens = (s.lens[rows] + 1 - 128).contiguous()
    prefix = s.table[0, :8].contiguous()

    def step():
        q, _, _ = s.write(x, cos, sin, slots)
        return kvq.shared_prefix_attention(q, s.k, s.v, own_table, own_lens, prefix, 128, scale_k=s.scale_k,
                                           scale_v=s.scale_v, offset_k=s.offset_k, offset_v=s.offset_v)

    def prompt():
        q, k, v = s.write(*big, torch.full((200,), -1, dtype=torch.int32, device="cuda"))
        return kvq.prompt_attention(q[None], k[None], v[None])

    big = s.tokens(200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(), prompt()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (step, step, prompt):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for _ in range(3):
        for y, src in zip((x, cos, sin), s.tokens(3)):
            y.copy_(src)
        slots.copy_(slots_of(s, rows))
        for g, out in graphs:
            out.zero_()
            g.replay()
        s.lens[rows] += 1
        eager, eager_prompt = step(), prompt()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], eager) and torch.equal(graphs[1][1], eager)
        assert torch.equal(graphs[2][1], eager_prompt)
        own_lens += 1
    assert kvq.get_error() == 0
    del graphs


def test_two_streams_at_once():
    """Calls that run side by side on two streams give what they give alone."""
    s = prefilled(3, 200)
    n = torch.tensor([0, 1500, 1501, 2600], dtype=torch.int32, device="cuda")
    g = s.g
    q, k, v = (torch.randn((2600, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (NQ, NKV, NKV))
    dq = torch.randn((64, NQ, D), generator=g, device="cuda").to(torch.bfloat16)
    table, prefix = s.table[:1, 4:].expand(64, -1), s.table[0, :4].contiguous()
    lens = (torch.arange(64, device="cuda") % 130).to(torch.int32)

    def prompt(stream=None):
        return kvq.prompt_attention(q, k, v, n, stream=stream)

    def decode(stream=None):
        return kvq.shared_prefix_attention(dq, s.k, s.v, table, lens, prefix, 64, scale_k=s.scale_k, scale_v=s.scale_v,
                                           stream=stream)

    a, b = prompt(), decode()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (one, two):
        st.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(10):
        outs.append((prompt(one), decode(two), decode(one), prompt(two)))
    torch.cuda.synchronize()
    for p1, d1, d2, p2 in outs:
        assert torch.equal(p1, a) and torch.equal(p2, a) and torch.equal(d1, b) and torch.equal(d2, b)
    assert kvq.get_error() == 0
