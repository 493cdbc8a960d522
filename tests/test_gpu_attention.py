"""prompt_attention and shared_prefix_attention on the GPU against the definition in 64 bits."""
import math

import pytest
import torch

import kv_cache_quantize_b200 as kvq
from _attention import check_rows, prompt64, shared64

pytestmark = pytest.mark.gpu
BF, F16, I8 = torch.bfloat16, torch.float16, torch.int8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(shape, dtype, g, mul=1.0):
    return (mul * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def spans(lq, lk):
    a, b = cu(lq), cu(lk)
    return [(a[i], lq[i], b[i], lk[i]) for i in range(len(lq))]


def run_prompt(q, k, v, lq, lk, causal=True, scale=None, what="", **kw):
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    out = torch.full_like(q, 3.0)
    kvq.get_error()
    kvq.prompt_attention(q, k, v, i32(cu(lq)), i32(cu(lk)), out=out, lse=lse, causal=causal, softmax_scale=scale,
                         check=True, **kw)
    want, wl, bound, lb = prompt64(q, k, v, spans(lq, lk), causal, scale)
    check_rows(out, want, bound, what + " out")
    check_rows(lse, wl, lb, what + " lse")
    untouched = torch.isnan(want)
    assert bool((out[untouched] == 3.0).all()) and bool((lse[torch.isnan(wl)] == 7.0).all())
    return out, lse


LENGTHS = [[1], [45], [128], [127, 129, 1, 64], [0, 5, 0, 300, 1, 0], [32, 33, 31, 95, 96, 97], [511, 640]]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [(4, 1), (14, 7), (3, 3), (6, 2)])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_prompt_lengths(dtype, dim, heads, lens):
    g = gen(1)
    nq, nkv = heads
    t = sum(lens)
    q, k, v = rnd((t, nq, dim), dtype, g, 2.0), rnd((t, nkv, dim), dtype, g), rnd((t, nkv, dim), dtype, g)
    run_prompt(q, k, v, lens, lens)


@pytest.mark.parametrize("heads", [(1, 1), (5, 1), (7, 1), (48, 2), (128, 1), (65, 1), (16, 4)])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_head_groups(heads, dim):
    g = gen(2)
    nq, nkv = heads
    lens = [70, 3, 200]
    t = sum(lens)
    q, k, v = rnd((t, nq, dim), BF, g, 2.0), rnd((t, nkv, dim), BF, g), rnd((t, nkv, dim), BF, g)
    run_prompt(q, k, v, lens, lens)


@pytest.mark.parametrize("lq,lk", [([1, 1, 1], [1, 300, 128]), ([5, 40], [700, 41]), ([50, 200, 3], [20, 200, 0]),
                                   ([130, 64], [1000, 129])], ids=str)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_prompt_other_keys_than_queries(lq, lk, causal, dtype):
    """A cached context in front of the queries; fewer keys than queries leave rows that see nothing: 0 and -inf."""
    g = gen(3)
    q, k, v = rnd((sum(lq), 8, 128), dtype, g, 2.0), rnd((sum(lk), 2, 128), dtype, g), rnd((sum(lk), 2, 128), dtype, g)
    out, lse = run_prompt(q, k, v, lq, lk, causal)
    for q0, n, _, m in spans(lq, lk):
        blind = max(0, n - m) if causal else (n if m == 0 else 0)
        assert bool((out[q0:q0 + blind] == 0).all()) and bool((lse[q0:q0 + blind] == -math.inf).all())


@pytest.mark.parametrize("s,sk", [(1, 1), (77, 77), (128, 128), (300, 333)])
def test_prompt_equal_lengths(s, sk):
    """The 4-D form is the packed one."""
    g = gen(4)
    q, k, v = rnd((3, s, 8, 64), F16, g), rnd((3, sk, 4, 64), F16, g), rnd((3, sk, 4, 64), F16, g)
    got = kvq.prompt_attention(q, k, v, check=True)
    packed = kvq.prompt_attention(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), i32(cu([s] * 3)), i32(cu([sk] * 3)))
    assert torch.equal(got.flatten(0, 1), packed)
    want, _, bound, _ = prompt64(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), spans([s] * 3, [sk] * 3))
    check_rows(packed, want, bound)


def test_prompt_strides_and_unused_rows():
    """q, k and v as slices of one projection, an output with other strides, rows behind the last sequence."""
    g = gen(5)
    lens = [130, 7, 64]
    t = sum(lens) + 37
    qkv = rnd((t, (8 + 2 + 2) * 128), BF, g, 1.5)
    q = qkv[:, :1024].view(t, 8, 128)
    k = qkv[:, 1024:1280].view(t, 2, 128)
    v = qkv[:, 1280:].view(t, 2, 128)
    want, _, bound, _ = prompt64(q, k, v, spans(lens, lens))
    store = torch.full((t, 8, 136), 3.0, dtype=BF, device="cuda")
    kvq.prompt_attention(q, k, v, i32(cu(lens)), out=store[..., :128], check=True)
    check_rows(store[..., :128], want, bound)
    assert bool((store[sum(lens):] == 3.0).all()) and bool((store[..., 128:] == 3.0).all())
    # heads outermost
    kt, vt = k.transpose(0, 1).contiguous().transpose(0, 1), v.transpose(0, 1).contiguous().transpose(0, 1)
    ot = torch.full((8, t, 128), 3.0, dtype=BF, device="cuda").transpose(0, 1)
    kvq.prompt_attention(q, kt, vt, i32(cu(lens)), out=ot, check=True)
    assert torch.equal(ot[:sum(lens)], store[:sum(lens), :, :128]) and bool((ot[sum(lens):] == 3.0).all())
    # one token's keys for all (stride 0) are refused
    with pytest.raises(kvq.KvqError):
        kvq.prompt_attention(q, k[:1].expand(t, 2, 128), v, i32(cu(lens)))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_values_in_places_nobody_sees(bad, dim):
    """NaN and infinities in another sequence, behind the last one and at later tokens stay there."""
    g = gen(6)
    lens = [50, 200, 9, 130]
    t = sum(lens) + 30
    q, k, v = rnd((t, 8, dim), BF, g), rnd((t, 2, dim), BF, g), rnd((t, 2, dim), BF, g)
    want, _, bound, _ = prompt64(q, k, v, spans(lens, lens))
    for x in (k, v):
        x[50:250] = bad                       # the whole second sequence
        x[sum(lens):] = bad                   # behind the last one
        x[259 + 100:, 1] = bad                # the fourth one's last tokens, one head
    q[50:250] = bad
    out = kvq.prompt_attention(q, k, v, i32(cu(lens)), check=True)
    live = torch.ones_like(want, dtype=torch.bool)
    live[50:250] = False
    live[259 + 100:, 4:] = False
    check_rows(out, torch.where(live, want, torch.full_like(want, math.nan)), bound)
    if math.isnan(bad):
        assert bool(torch.isnan(out[259 + 100:sum(lens), 4:].float()).all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_prompt_infinite_values_that_are_seen(bad):
    """An infinite value at a later token of the tile reaches exactly the rows that see it."""
    g = gen(7)
    n = 90
    q, k, v = rnd((n, 4, 128), BF, g), rnd((n, 1, 128), BF, g), rnd((n, 1, 128), BF, g)
    v[40, 0, 5] = bad
    out = kvq.prompt_attention(q, k, v, i32([0, n]), check=True)
    assert bool((out[40:, :, 5] == bad).all()) and bool(torch.isfinite(out[:40].float()).all())
    keep = [c for c in range(128) if c != 5]
    assert bool(torch.isfinite(out[:, :, keep].float()).all())


def test_prompt_offsets_beyond_32_bits():
    """Token rows a megabyte apart: q, k, v and out in one buffer of more than 2^32 elements."""
    t, step = 4500, 1 << 20
    big = torch.empty((t * step,), dtype=BF, device="cuda")
    at = [big[1024 * i:].as_strided((t, h, 64), (step, 64, 1)) for i, h in enumerate((4, 2, 2, 4))]
    g = gen(14)
    for x in at[:3]:
        x.copy_(rnd(x.shape, BF, g))
    q, k, v, out = at
    kvq.prompt_attention(q, k, v, i32([0, 4200, t]), out=out, check=True)
    want, _, bound, _ = prompt64(q[4200:], k[4200:], v[4200:], [(0, 300, 0, 300)])
    check_rows(out[4200:], want, bound)


def test_prompt_large_scores_and_scale():
    g = gen(8)
    q, k, v = rnd((200, 4, 64), BF, g, 30.0), rnd((200, 4, 64), BF, g, 30.0), rnd((200, 4, 64), BF, g)
    run_prompt(q, k, v, [200], [200], scale=1.0)
    run_prompt(q, k, v, [200], [200], scale=-0.01)
    run_prompt(q, k, v, [200], [200], scale=0.0)


def test_prompt_nan_scores_reach_their_row_alone():
    """A NaN query, and a NaN key for the rows that see it."""
    g = gen(13)
    for dtype in (BF, F16):
        q, k, v = rnd((300, 4, 128), dtype, g), rnd((300, 2, 128), dtype, g), rnd((300, 2, 128), dtype, g)
        want, _, bound, _ = prompt64(q, k, v, [(0, 300, 0, 300)])
        q[70, 1, 3] = math.nan
        k[200, 1, 7] = math.nan
        out = kvq.prompt_attention(q, k, v, i32([0, 300]), check=True)
        assert bool(torch.isnan(out[70, 1].float()).all()) and bool(torch.isnan(out[200:, 2:].float()).all())
        want[70, 1] = math.nan
        want[200:, 2:] = math.nan
        check_rows(out, want, bound)


def test_prompt_bad_spans_are_reported_and_left_out():
    g = gen(9)
    q, k, v = rnd((100, 4, 64), BF, g), rnd((100, 4, 64), BF, g), rnd((100, 4, 64), BF, g)
    for offsets in ([0, 40, 101], [-5, 40, 100], [50, 40, 100]):
        out = torch.full_like(q, 3.0)
        kvq.get_error()
        kvq.prompt_attention(q, k, v, i32(offsets), out=out)
        assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
        for b in range(2):
            lo, hi = offsets[b], offsets[b + 1]
            if 0 <= lo <= hi <= 100:
                want, _, bound, _ = prompt64(q, k, v, [(lo, hi - lo, lo, hi - lo)])
                check_rows(out, want, bound)
        if offsets[0] == 0:
            assert bool((out[40:] == 3.0).all())


@pytest.mark.parametrize("n", [4096])
def test_prompt_long(n):
    g = gen(10)
    q, k, v = rnd((n, 4, 128), BF, g, 2.0), rnd((n, 2, 128), BF, g), rnd((n, 2, 128), BF, g)
    run_prompt(q, k, v, [n], [n])


def test_prompt_many_sequences():
    g = gen(11)
    lens = [(7 * i * i + 3) % 61 for i in range(700)]
    t = sum(lens)
    q, k, v = rnd((t, 4, 64), F16, g), rnd((t, 2, 64), F16, g), rnd((t, 2, 64), F16, g)
    run_prompt(q, k, v, lens, lens)


def test_prompt_is_the_same_each_time_and_on_another_stream():
    g = gen(12)
    lens = [300, 1, 77, 1000]
    t = sum(lens)
    q, k, v = rnd((t, 8, 128), BF, g), rnd((t, 2, 128), BF, g), rnd((t, 2, 128), BF, g)
    c = i32(cu(lens))
    a = kvq.prompt_attention(q, k, v, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = [kvq.prompt_attention(q, k, v, c, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, x) for x in b)


# ---------------------------------------------------------------------------
# the paged form
# ---------------------------------------------------------------------------
def paged(seed, lens, prefix, nq, nkv, dim, block, dtype, cache, pad_pages=3, offsets=True):
    g = gen(seed)
    held = [-(-max(n, 0) // block) for n in lens]
    npre = -(-prefix // block)
    total = npre + sum(held) + pad_pages
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(held + [1]) + 1), -1, dtype=torch.int32, device="cuda")
    at = npre
    for b, m in enumerate(held):
        table[b, :m] = order[at:at + m]
        at += m
    d = dict(q=rnd((len(lens), nq, dim), dtype, g, 2.0), table=table, lens=i32(lens), prefix_table=order[:npre].clone(),
             prefix_len=prefix)
    shape = (total, block, nkv, dim)
    if cache == I8:
        d["kc"] = torch.randint(-128, 128, shape, dtype=I8, generator=g, device="cuda")
        d["vc"] = torch.randint(-128, 128, shape, dtype=I8, generator=g, device="cuda")
        d["scale_k"] = (0.5 + torch.rand(nkv * dim, generator=g, device="cuda")) / 60
        d["scale_v"] = (0.5 + torch.rand(nkv, dim, generator=g, device="cuda")) / 60
        if offsets:
            d["offset_k"] = torch.randn(nkv * dim, generator=g, device="cuda") * 5
            d["offset_v"] = torch.randn(nkv, dim, generator=g, device="cuda") * 5
    else:
        d["kc"], d["vc"] = rnd(shape, cache, g), rnd(shape, cache, g)
    return d


def call_shared(d, **kw):
    par = {n: d[n] for n in ("scale_k", "scale_v", "offset_k", "offset_v") if n in d}
    return kvq.shared_prefix_attention(d["q"], d["kc"], d["vc"], d["table"], d["lens"], d["prefix_table"],
                                       d["prefix_len"], **par, **kw)


def want_shared(d, scale=None):
    par = {n: d.get(n) for n in ("scale_k", "scale_v", "offset_k", "offset_v")}
    return shared64(d["q"], d["kc"], d["vc"], d["table"], d["lens"], d["prefix_table"], d["prefix_len"], **par,
                    scale=scale)


def run_shared(d, scale=None):
    out = torch.full_like(d["q"], 3.0)
    lse = torch.full(d["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    kvq.get_error()
    call_shared(d, out=out, lse=lse, softmax_scale=scale, check=True)
    want, wl, bound, lb = want_shared(d, scale)
    check_rows(out, want, bound, "out")
    check_rows(lse, wl, lb, "lse")
    assert bool((out[torch.isnan(want)] == 3.0).all()) and bool((lse[torch.isnan(wl)] == 7.0).all())
    return out


KINDS = [(BF, I8), (F16, I8), (BF, BF), (F16, F16)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [(4, 1), (14, 7), (6, 2), (3, 3), (16, 1)])
@pytest.mark.parametrize("lens,prefix", [([1], 0), ([0, 17, -1, 64], 0), ([0, 0], 1), ([5, -1, 130], 100),
                                         ([33, 1], 333), ([0, 700, 31], 1024)], ids=str)
def test_shared_lengths(dtype, cache, dim, heads, lens, prefix):
    run_shared(paged(21, lens, prefix, *heads, dim, 16, dtype, cache))


@pytest.mark.parametrize("block", [1, 3, 16, 48, 64, 100, 256])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_page_sizes(block, dtype, cache):
    run_shared(paged(22, [block, 2 * block + 1, 5, 301], 2 * block + block // 2 + 150, 8, 2, 128, block, dtype, cache))


@pytest.mark.parametrize("heads", [(1, 1), (5, 1), (40, 2), (128, 1), (17, 1), (33, 1), (65, 1)])
@pytest.mark.parametrize("dtype,cache", [(BF, I8), (F16, F16)])
def test_shared_head_groups(heads, dtype, cache):
    run_shared(paged(23, [3, 70, 0, 129], 200, *heads, 64, 32, dtype, cache))


@pytest.mark.parametrize("batch", [1, 2, 7, 31, 64, 65, 130])
@pytest.mark.parametrize("dtype,cache", [(BF, I8), (BF, BF)])
def test_shared_batches(batch, dtype, cache):
    lens = [(i * 37) % 90 for i in range(batch)]
    run_shared(paged(24, lens, 1000, 8, 2, 128, 32, dtype, cache))


@pytest.mark.parametrize("heads", [(4, 1), (40, 1), (6, 1)])
@pytest.mark.parametrize("batch", [3, 5, 33, 43, 67])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_groups_of_few_rows(heads, batch, dtype, cache):
    """Batches of up to 32 rows, and batches whose last group of requests has so few."""
    lens = [(i * 53) % 300 - 1 for i in range(batch)]
    run_shared(paged(35, lens, 900, *heads, 64, 16, dtype, cache))


def test_shared_nan_reaches_its_request_alone():
    for dtype, cache in KINDS:
        d = paged(36, [100, 40, 300, 7], 300, 8, 2, 128, 16, dtype, cache)
        want, _, bound, _ = want_shared(d)
        d["q"][1, 3, 5] = math.nan
        out = call_shared(d, check=True)
        assert bool(torch.isnan(out[1, 3].float()).all())
        want[1, 3] = math.nan                              # not compared
        check_rows(out, want, bound)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_many_requests(dtype, cache):
    """More pieces of work than multiprocessors: every one of them takes several, of all kinds."""
    run_shared(paged(34, [(i * 53) % 400 for i in range(150)], 700, 8, 4, 64, 16, dtype, cache))


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_long(dtype, cache):
    run_shared(paged(25, [3000, 20, 1500], 5000, 16, 4, 128, 64, dtype, cache))
    run_shared(paged(26, [9000], 0, 4, 1, 128, 64, dtype, cache))


def test_shared_without_offsets_and_other_scales():
    d = paged(27, [10, 200], 300, 8, 2, 128, 32, BF, I8, offsets=False)
    run_shared(d)
    run_shared(d, scale=0.0)
    run_shared(d, scale=-0.3)
    d["scale_k"] = d["scale_k"] * 2.0 ** -40           # keys far below and above the range of f16
    d["q"] = d["q"] * 2.0 ** 40
    run_shared(d)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_values_in_places_nobody_sees(bad, dim):
    """Tokens of a page behind a request's last one, and pages of nobody."""
    d = paged(28, [3, 17, 100], 37, 8, 2, dim, 16, BF, BF)
    want, _, bound, _ = want_shared(d)
    seen = torch.zeros(d["kc"].shape[:2], dtype=torch.bool, device="cuda")
    t = torch.arange(16, device="cuda")
    for row, n in [(d["prefix_table"], 37)] + [(d["table"][b], int(d["lens"][b])) for b in range(3)]:
        for e in range(-(-n // 16)):
            seen[int(row[e])] |= t < n - 16 * e
    d["kc"][~seen] = bad
    d["vc"][~seen] = bad
    check_rows(call_shared(d, check=True), want, bound)


def test_shared_strides_and_views():
    """Table rows that are views, caches with padding between pages, strided queries and outputs, any table row twice."""
    d = paged(29, [40, 40, 100, 7], 64, 8, 2, 128, 16, BF, I8)
    plain = call_shared(d, check=True)
    wide = torch.full((4, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + d["table"].shape[1]] = d["table"]
    d["table"] = wide[:, 5:5 + d["table"].shape[1]]
    for n in ("kc", "vc"):
        c = d[n]
        padded = torch.zeros((c.shape[0], c[0].numel() + 64), dtype=I8, device="cuda")
        padded[:, :c[0].numel()] = c.flatten(1)
        d[n] = padded[:, :c[0].numel()].view(c.shape)
    q = torch.zeros((4, 24, 128), dtype=BF, device="cuda")
    q[:, 8:16] = d["q"]
    d["q"] = q[:, 8:16]
    out = torch.zeros((4, 8, 160), dtype=BF, device="cuda")[..., :128]
    call_shared(d, out=out, check=True)
    assert torch.equal(out, plain)
    d["table"] = d["table"][:1].expand(4, -1)              # all requests on one row, stride 0
    d["lens"] = i32([40, 12, 33, 0])
    run_shared(d)


@pytest.mark.parametrize("block", [64, 24])
def test_shared_offsets_beyond_32_bits(block):
    """Pages at the end of a cache of more than 4 GB."""
    d = paged(37, [300, 10], 200, 8, 4, 128, block, BF, I8)
    few = d["kc"].shape[0]
    pages = (9 << 29) // (block * 4 * 128)                       # 4.5 GB
    far = torch.zeros((pages, block, 4, 128), dtype=I8, device="cuda")
    far[pages - few:] = d["kc"]
    want, wl, bound, lb = want_shared({**d, "vc": d["kc"]})
    d["table"] = torch.where(d["table"] >= 0, d["table"] + pages - few, -1).to(torch.int32)
    d["prefix_table"] = d["prefix_table"] + pages - few
    check_rows(call_shared({**d, "kc": far, "vc": far}, check=True), want, bound)


def test_shared_without_pages_or_requests():
    for dtype, cache in KINDS:
        d = paged(38, [0, -1, 0], 0, 8, 2, 64, 16, dtype, cache)
        out = run_shared(d)
        assert bool((out[[0, 2]] == 0).all())
        empty = {**d, "kc": d["kc"][:0], "vc": d["vc"][:0]}
        assert bool((call_shared(empty, check=True)[[0, 2]] == 0).all())
        none = {**d, "q": d["q"][:0], "table": d["table"][:0], "lens": d["lens"][:0]}
        assert call_shared(none, check=True).shape == (0, 8, 64)


def test_shared_bad_pages_and_lengths_are_reported_and_left_out():
    d = paged(30, [40, 40, 40, 20], 32, 8, 2, 64, 16, BF, I8)
    full, _, bound, _ = want_shared(d)
    d["table"][1, 2] = d["kc"].shape[0]                    # the third page of request 1: its 8 tokens are left out
    d["lens"] = i32([40, 40, 40000, 20])
    out = torch.full_like(d["q"], 3.0)
    kvq.get_error()
    call_shared(d, out=out)
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    check_rows(out[[0, 3]], full[[0, 3]], bound[[0, 3]])
    assert bool((out[2] == 3.0).all())
    d["lens"] = i32([40, 32, -7, 20])
    want, _, bound, _ = want_shared({**d, "lens": i32([40, 32, -1, 20])})
    check_rows(out[1], want[1], bound[1])
    out.fill_(3.0)
    call_shared(d, out=out)
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    check_rows(out, want, bound)
    # a page of the prefix that is not there: its tokens are left out for everybody
    d["lens"] = i32([40, 32, 40, 20])
    d["prefix_table"][1] = -1
    want, _, bound, _ = want_shared({**d, "prefix_len": 16})
    out = call_shared(d)
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    check_rows(out, want, bound)


def test_shared_equals_every_request_on_its_own():
    """The prefix shared, and the same tokens listed in each request's own row."""
    d = paged(31, [40, 7, 0, 90], 64, 8, 2, 128, 16, BF, BF)
    own = torch.cat([d["prefix_table"][None].expand(4, -1), d["table"]], 1)
    alone = {**d, "table": own, "lens": d["lens"] + 64, "prefix_len": 0}
    want, _, bound, _ = want_shared(d)
    check_rows(call_shared(alone, check=True), want, bound)
    check_rows(call_shared(d, check=True), want, bound)


def test_shared_is_the_same_each_time_and_on_another_stream():
    d = paged(32, [i * 11 % 200 for i in range(40)], 1500, 16, 4, 128, 64, BF, I8)
    a = call_shared(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = [call_shared(d, stream=side) for _ in range(3)]
    c = call_shared(d)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, x) for x in (*b, c))


def test_shared_with_a_workspace_of_the_caller():
    d = paged(33, [100, 300], 2000, 8, 2, 128, 64, F16, I8)
    need = kvq.shared_prefix_attention_workspace(2, 8, 2, 128, 2000, d["table"].shape[1] * 64)
    a = call_shared(d)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    b = call_shared(d, workspace=ws[:need])
    assert torch.equal(a, b) and bool((ws[need:] == 0xFF).all())
    if need:
        with pytest.raises(kvq.KvqError):
            call_shared(d, workspace=ws[:need - 1])
