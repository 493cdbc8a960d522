"""Measured cases of the operators that read and manage the paged cache.

Three families, as a serving loop uses them next to the cache epilogue:
  prompt   attention over whole prompts: causal, grouped heads, packed sequences of different lengths;
  shared   attention of one new token per request over a paged cache whose long prefix all requests share;
  copy, fork, compact   the pages of a cache: copying them, freeing rows and forking others from them
           (shared full pages, a copy of the last, partly filled one), and closing the holes of a pool.

A case is a dict of plain values; prepare() makes its inputs from a seed, run() makes one pass, in plain torch or
(with `own` true) through the framework's calls, and exact() gives the definition's values in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short question: the call's latency counts
        dict(name="prompt_short", op="prompt", batch=1, longest=45, context=0, nq=14, nkv=7, dim=64, dtype="f16"),
        # a batch of prompts of very different lengths, packed without padding
        dict(name="prompt_packed", op="prompt", batch=24, longest=2048, context=0, nq=16, nkv=4, dim=128, dtype="bf16"),
        # one long document
        dict(name="prompt_long", op="prompt", batch=1, longest=16384, context=0, nq=16, nkv=4, dim=128, dtype="bf16"),
        # a handful of requests behind a short system prompt: latency again
        dict(name="shared_small", op="shared", batch=3, prefix=500, longest=40, nq=12, nkv=3, dim=128, page=16,
             dtype="bf16", cache="i8"),
        # a chat server's step with 16-bit pages
        dict(name="shared_chat", op="shared", batch=40, prefix=2000, longest=1500, nq=16, nkv=4, dim=128, page=64,
             dtype="bf16", cache="bf16"),
        # many requests over one long document in int8 pages
        dict(name="shared_large", op="shared", batch=256, prefix=32768, longest=1024, nq=16, nkv=4, dim=128, page=64,
             dtype="bf16", cache="i8"),
        # a few pages of one request
        dict(name="copy_few", op="copy", pairs=7, pages=512, page=64, nkv=4, dim=128, caches=2),
        # the whole working set of a server, moved to other pages
        dict(name="copy_many", op="copy", pairs=4001, pages=8192, page=64, nkv=4, dim=128, caches=2),
        # beam search: every beam's row freed and forked again in each step
        dict(name="fork_beams", op="fork", parents=4, children=12, longest=900, pages=512, page=16, nkv=3, dim=128,
             caches=2),
        # one document's row forked for many samples, over the caches of several layers
        dict(name="fork_samples", op="fork", parents=16, children=480, longest=6000, pages=4096, page=64, nkv=4,
             dim=128, caches=8),
        # a pool with few holes
        dict(name="compact_small", op="compact", pages=300, used=170, moves=40, rows=20, page=16, nkv=7, dim=128,
             caches=2),
        # a long-running pool, a third of it free
        dict(name="compact_large", op="compact", pages=8192, used=5400, moves=1800, rows=128, page=64, nkv=4,
             dim=128, caches=2),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(("prompt", "shared", "copy", "fork", "compact"))
    nq, nkv = rng.choice(((16, 4), (12, 3), (14, 7), (8, 8), (8, 1)))
    dim = rng.choice((64, 128, 128))
    page = rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("bf16", "f16"))
    if op == "prompt":
        longest = _spread(rng, 1, 6000)
        batch = min(_spread(rng, 1, 48), max(1, 100_000_000 // longest ** 2))
        context = rng.choice((0, 0, _spread(rng, 1, 2000)))
        return dict(op=op, batch=batch, longest=longest, context=context, nq=nq, nkv=nkv, dim=dim, dtype=dtype)
    if op == "shared":
        return dict(op=op, batch=_spread(rng, 1, 200), prefix=_spread(rng, 16, 24000), longest=_spread(rng, 1, 1000),
                    nq=nq, nkv=nkv, dim=dim, page=page, dtype=dtype, cache=rng.choice(("i8", "i8", dtype)))
    if op == "copy":
        pairs = _spread(rng, 1, 1500)
        return dict(op=op, pairs=pairs, pages=2 * pairs + rng.randint(0, 500), page=page, nkv=nkv, dim=dim,
                    caches=rng.randint(1, 4))
    if op == "fork":
        parents, children, longest = _spread(rng, 1, 12), _spread(rng, 1, 200), _spread(rng, 1, 3000)
        return dict(op=op, parents=parents, children=children, longest=longest,
                    pages=parents * -(-longest // page) + children + rng.randint(0, 300), page=page, nkv=nkv, dim=dim,
                    caches=rng.randint(1, 4))
    used = _spread(rng, 8, 2500)
    moves = rng.randint(0, used // 3)
    return dict(op=op, pages=used + moves + rng.randint(0, used), used=used, moves=moves,
                rows=min(used, _spread(rng, 1, 100)), page=page, nkv=nkv, dim=dim, caches=rng.randint(1, 4))


def _lengths(case):
    """The sequences' lengths, from the case alone: the longest, then others between 1 and it."""
    r = random.Random("%d %d" % (case["batch"], case["longest"]))
    return [case["longest"]] + [r.randint(1, case["longest"]) for _ in range(case["batch"] - 1)]


def _parent_lengths(case):
    r = random.Random("%d %d" % (case["parents"], case["longest"]))
    return [case["longest"]] + [r.randint(1, case["longest"]) for _ in range(case["parents"] - 1)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _prepare_prompt(case, g):
    lens = _lengths(case)
    ctx = case["context"]
    dt = DTYPES[case["dtype"]]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    cuk = [c + ctx * i for i, c in enumerate(cu)]
    # queries scaled so that scores spread over a few units, as trained heads' scores do
    q = (2.0 * torch.randn(cu[-1], case["nq"], case["dim"], generator=g, device=DEVICE)).to(dt)
    k = torch.randn(cuk[-1], case["nkv"], case["dim"], generator=g, device=DEVICE).to(dt)
    v = torch.randn(cuk[-1], case["nkv"], case["dim"], generator=g, device=DEVICE).to(dt)
    return dict(q=q, k=k, v=v, cu_q=_ints(cu), cu_k=_ints(cuk))


def _codes(shape, g):
    return torch.randn(shape, generator=g, device=DEVICE).mul_(36.0).round_().clamp_(-128, 127).to(torch.int8)


def _prepare_shared(case, g):
    lens = _lengths(case)
    page, nkv, dim = case["page"], case["nkv"], case["dim"]
    own_pages = [-(-n // page) for n in lens]
    width = max(own_pages)
    npre = -(-case["prefix"] // page)
    total = npre + sum(own_pages) + 5
    order = torch.randperm(total, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    at = npre
    for b, n in enumerate(own_pages):
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(table=table, lens=_ints(lens), prefix_table=order[:npre].clone())
    shape = (total, page, nkv, dim)
    if case["cache"] == "i8":
        # the static int8 form that the cache epilogue writes: a scale and an offset for each head and channel
        s["k"], s["v"] = _codes(shape, g), _codes(shape, g)
        for n in ("scale_k", "scale_v"):
            s[n] = (0.5 + torch.rand(nkv, dim, generator=g, device=DEVICE)) / 36.0
        for n in ("offset_k", "offset_v"):
            s[n] = torch.randn(nkv, dim, generator=g, device=DEVICE).mul_(3.0).round_()
    else:
        s["k"] = torch.randn(shape, generator=g, device=DEVICE).to(DTYPES[case["cache"]])
        s["v"] = torch.randn(shape, generator=g, device=DEVICE).to(DTYPES[case["cache"]])
    s["q"] = (2.0 * torch.randn(len(lens), case["nq"], dim, generator=g, device=DEVICE)).to(DTYPES[case["dtype"]])
    return s


def _caches(case, g):
    shape = (case["pages"], case["page"], case["nkv"], case["dim"])
    return [torch.randint(-128, 128, shape, dtype=torch.int8, generator=g, device=DEVICE)
            for _ in range(case["caches"])]


def _prepare_copy(case, g):
    order = torch.randperm(case["pages"], generator=g, device=DEVICE).to(torch.int32)
    n = case["pairs"]
    return dict(caches=_caches(case, g), src=order[:n].clone(), dst=order[n:2 * n].clone())


def _prepare_fork(case, g):
    page, lens = case["page"], _parent_lengths(case)
    n = [-(-x // page) for x in lens]
    rows = case["parents"] + case["children"]
    order = torch.randperm(case["pages"], generator=g, device=DEVICE).to(torch.int32)
    names = torch.randperm(rows, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((rows, max(n)), -1, dtype=torch.int32, device=DEVICE)
    seq_lens = torch.zeros(rows, dtype=torch.int32, device=DEVICE)
    ref = torch.zeros(case["pages"], dtype=torch.int32, device=DEVICE)
    at = 0
    for i, (x, m) in enumerate(zip(lens, n)):
        row = int(names[i])
        table[row, :m] = order[at:at + m]
        seq_lens[row] = x
        at += m
    ref[order[:at].long()] = 1
    pick = torch.randint(0, case["parents"], (case["children"],), generator=g, device=DEVICE)
    return dict(caches=_caches(case, g), table=table, lens=seq_lens, ref=ref, parents=names[pick].clone(),
                children=names[case["parents"]:].clone())


def _prepare_compact(case, g):
    pages, used, moves, rows = case["pages"], case["used"], case["moves"], case["rows"]
    low = torch.randperm(used, generator=g, device=DEVICE)[moves:]                          # kept below the border
    high = used + torch.randperm(pages - used, generator=g, device=DEVICE)[:moves]          # to be moved down
    live = torch.cat([low, high])[torch.randperm(used, generator=g, device=DEVICE)]
    width = -(-used // rows) + 3
    flat = torch.full((rows, width), -1, dtype=torch.int32, device=DEVICE)
    at = torch.arange(used, device=DEVICE)
    flat[at % rows, at // rows] = live.to(torch.int32)
    ref = torch.zeros(pages, dtype=torch.int32, device=DEVICE)
    ref[live] = 1
    return dict(caches=_caches(case, g), table=flat, ref=ref)


def prepare(case, seed):
    g = _generator(seed)
    make = dict(prompt=_prepare_prompt, shared=_prepare_shared, copy=_prepare_copy, fork=_prepare_fork,
                compact=_prepare_compact)[case["op"]]
    state = make(case, g)
    state["case"] = dict(case)
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _softmax_rows(scores):
    """exp(s - max) and its sum along the last dimension; rows of -inf alone give zeros."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    return p, p.sum(-1, keepdim=True)


def _plain_prompt(s):
    q, k, v, case = s["q"], s["k"], s["v"], s["case"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    batch, nq, nkv, dim = case["batch"], case["nq"], case["nkv"], case["dim"]
    iq = torch.arange(case["longest"], device=q.device)
    ik = torch.arange(case["longest"] + case["context"], device=q.device)
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    qp = q[(cu_q[:-1, None] + iq).clamp_(max=q.shape[0] - 1)].float()
    kp = k[(cu_k[:-1, None] + ik).clamp_(max=k.shape[0] - 1)].float()
    vp = v[(cu_k[:-1, None] + ik).clamp_(max=k.shape[0] - 1)].float()
    qp = qp.view(batch, -1, nkv, nq // nkv, dim).permute(0, 2, 3, 1, 4).reshape(batch, nkv, -1, dim)
    scores = qp @ (kp.permute(0, 2, 3, 1) * dim ** -0.5)
    scores = scores.view(batch, nkv, nq // nkv, iq.numel(), ik.numel())
    hidden = ik > (iq[:, None] + (lk - lq)[:, None, None])
    hidden |= (ik >= lk[:, None])[:, None, :]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    p, total = _softmax_rows(scores)
    o = p.view(batch, nkv, -1, ik.numel()) @ vp.permute(0, 2, 1, 3)
    o = o.view(batch, nkv, nq // nkv, -1, dim) / total
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu_q[1:].contiguous(), t, right=True)
    o = o.permute(0, 3, 1, 2, 4)[b, t - cu_q[b]]
    return o.reshape(q.shape).to(q.dtype)


def _values(cache, pages, scale, offset):
    """The stored values of these pages, tokens in order."""
    x = cache[pages.long()].float()
    if scale is not None:
        x = (x - offset) * scale
    return x.flatten(-4, -3)


def _plain_shared(s):
    q, case = s["q"], s["case"]
    batch, nkv, dim = case["batch"], case["nkv"], case["dim"]
    sk, sv, ok, ov = (s.get(n) for n in ("scale_k", "scale_v", "offset_k", "offset_v"))
    qf = q.float().view(batch, nkv, -1, dim) * dim ** -0.5
    kp = _values(s["k"], s["prefix_table"], sk, ok)[: case["prefix"]]
    vp = _values(s["v"], s["prefix_table"], sv, ov)[: case["prefix"]]
    table = s["table"].clamp(min=0)
    ko, vo = _values(s["k"], table, sk, ok), _values(s["v"], table, sv, ov)
    shared = (qf.transpose(0, 1).reshape(nkv, -1, dim) @ kp.permute(1, 2, 0)).view(nkv, batch, -1, kp.shape[0])
    alone = qf @ ko.permute(0, 2, 3, 1)
    hidden = torch.arange(ko.shape[1], device=q.device) >= s["lens"][:, None]
    alone.masked_fill_(hidden[:, None, None], -math.inf)
    p, total = _softmax_rows(torch.cat([shared.transpose(0, 1), alone], -1))
    ps, pa = p[..., : kp.shape[0]], p[..., kp.shape[0]:]
    o = (ps.transpose(0, 1).reshape(nkv, -1, kp.shape[0]) @ vp.transpose(0, 1)).view(nkv, batch, -1, dim)
    o = (o.transpose(0, 1) + pa @ vo.transpose(1, 2)) / total
    return o.reshape(q.shape).to(q.dtype)


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for c in s["caches"]:
        c[dst] = c[src]
    return s["caches"]


def _plain_fork(s):
    table, lens, ref, page = s["table"], s["lens"], s["ref"], s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    pos = torch.arange(table.shape[1], device=table.device)
    # free the children's rows
    held = pos < ((lens[children] + page - 1) // page)[:, None]
    ref.index_add_(0, table[children].clamp(min=0).flatten().long(), -held.flatten().to(torch.int32))
    table[children] = -1
    lens[children] = 0
    # fork: share the full pages, copy the last one where it is partly filled
    n = lens[parents]
    full, part = (n // page).long(), n % page > 0
    vacant = torch.sort((ref > 0).to(torch.int32), stable=True)[1]
    nth = part.cumsum(0) - 1
    fresh = torch.where(part, vacant[nth.clamp(min=0)], -1)
    row = table[parents]
    last = row.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    src = torch.where(part, last, row[:, 0].long())
    dst = torch.where(part, fresh, row[:, 0].long())
    shared = pos < full[:, None]
    ref.index_add_(0, row.clamp(min=0).flatten().long(), shared.flatten().to(torch.int32))
    ref.index_add_(0, fresh.clamp(min=0), part.to(torch.int32))
    row = torch.where(shared, row, -1)
    row = torch.where((pos == full[:, None]) & part[:, None], fresh[:, None].to(torch.int32), row)
    table[children] = row
    lens[children] = n
    for c in s["caches"]:
        c[dst] = c[src]
    return s["caches"], table, lens, ref, fresh.to(torch.int32)


def _plain_compact(s):
    table, ref = s["table"], s["ref"]
    pages = ref.numel()
    p = torch.arange(pages, device=ref.device)
    used = ref > 0
    count = used.sum()
    hole = ~used & (p < count)
    moved = used & (p >= count)
    holes = torch.sort((~hole).to(torch.int32), stable=True)[1]
    target = torch.where(moved, holes[(moved.cumsum(0) - 1).clamp(min=0)], p)
    page_map = torch.where(used, target, -1)
    new_ref = torch.zeros(pages + 1, dtype=ref.dtype, device=ref.device)
    new_ref[torch.where(used, target, pages)] = ref
    new_table = torch.where(table >= 0, page_map[table.clamp(min=0).long()], -1).to(torch.int32)
    src = moved.nonzero()[:, 0]
    dst = target[src]
    for c in s["caches"]:
        c[dst] = c[src]
    return s["caches"], new_table, new_ref[:pages], page_map.to(torch.int32)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_run(s):
    import kv_cache_quantize_b200 as kvq

    op = s["case"]["op"]
    if op == "prompt":
        return kvq.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    if op == "shared":
        return kvq.shared_prefix_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix_table"],
                                           s["case"]["prefix"], scale_k=s.get("scale_k"), scale_v=s.get("scale_v"),
                                           offset_k=s.get("offset_k"), offset_v=s.get("offset_v"))
    if op == "copy":
        kvq.copy_pages(s["caches"], s["src"], s["dst"])
        return s["caches"]
    if op == "fork":
        page = s["case"]["page"]
        kvq.free_pages(s["table"], s["lens"], s["ref"], s["children"], page)
        fresh = kvq.fork_pages(s["caches"], s["table"], s["lens"], s["ref"], s["parents"], s["children"], page)
        return s["caches"], s["table"], s["lens"], s["ref"], fresh
    new_table, new_ref, page_map = kvq.compact_pages(s["caches"], s["table"], s["ref"])
    return s["caches"], new_table, new_ref, page_map


def run(state):
    if own:
        return _own_run(state)
    plain = dict(prompt=_plain_prompt, shared=_plain_shared, copy=_plain_copy, fork=_plain_fork,
                 compact=_plain_compact)
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("prompt", "shared"):
        nq, nkv, dim, lens = case["nq"], case["nkv"], case["dim"], _lengths(case)
    if op == "prompt":
        ctx = case["context"]
        seen = sum(n * ctx + n * (n + 1) // 2 for n in lens)
        tokens = sum(lens)
        return dict(bytes=2 * dim * (2 * nq * tokens + 2 * nkv * (tokens + ctx * len(lens))) + 8 * (len(lens) + 1),
                    flops=4 * nq * dim * seen)
    if op == "shared":
        width = 1 if case["cache"] == "i8" else 2
        keys = case["prefix"] + sum(lens)
        entries = -(-case["prefix"] // case["page"]) + sum(-(-n // case["page"]) for n in lens)
        scales = 16 * nkv * dim if case["cache"] == "i8" else 0
        return dict(bytes=2 * nkv * dim * width * keys + 4 * nq * dim * len(lens) + 4 * (entries + len(lens)) + scales,
                    flops=4 * nq * dim * (len(lens) * case["prefix"] + sum(lens)))
    page_bytes = case["page"] * case["nkv"] * case["dim"] * case["caches"]
    if op == "copy":
        return dict(bytes=2 * page_bytes * case["pairs"] + 8 * case["pairs"], flops=0)
    if op == "fork":
        lens = _parent_lengths(case)
        partial = sum(n % case["page"] > 0 for n in lens) / len(lens) * case["children"]
        entries = sum(-(-n // case["page"]) for n in lens) / len(lens) * case["children"]
        # the freed rows' and the parents' entries read, the children's written, the counts of the pages read
        return dict(bytes=2 * page_bytes * partial + 4 * (4 * entries + 5 * case["children"] + case["pages"]), flops=0)
    return dict(bytes=2 * page_bytes * case["moves"] + 4 * (2 * case["used"] + 3 * case["pages"]), flops=0)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _attend(q, k, v, visible):
    """Rows of q over the keys that visible (a truth value for each row and key) shows them."""
    w = torch.einsum("id,jd->ij", q, k) / math.sqrt(q.shape[1])
    w = torch.where(visible, w, torch.full_like(w, -math.inf))
    w = torch.exp(w - w.max(dim=1, keepdim=True).values)
    return torch.einsum("ij,jd->id", w, v) / w.sum(dim=1, keepdim=True)


def exact(case, seed):
    if case["op"] not in ("prompt", "shared"):
        return None                     # bytes and page numbers are copied, not computed
    s = prepare(case, seed)
    group = case["nq"] // case["nkv"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    if case["op"] == "prompt":
        starts_q, starts_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["batch"]):
            a, e, ka, ke = starts_q[b], starts_q[b + 1], starts_k[b], starts_k[b + 1]
            i = torch.arange(e - a, device=q.device)[:, None] + (ke - ka) - (e - a)
            visible = torch.arange(ke - ka, device=q.device)[None] <= i
            for h in range(case["nq"]):
                out[a:e, h] = _attend(q[a:e, h], s["k"][ka:ke, h // group].double(),
                                      s["v"][ka:ke, h // group].double(), visible)
        return out
    n_pre = case["prefix"]
    for b in range(case["batch"]):
        n = int(s["lens"][b])
        for h in range(case["nkv"]):
            parts = []
            for c, sc, of in (("k", "scale_k", "offset_k"), ("v", "scale_v", "offset_v")):
                first = s[c][s["prefix_table"].long(), :, h].reshape(-1, case["dim"])[:n_pre]
                rest = s[c][s["table"][b].clamp(min=0).long(), :, h].reshape(-1, case["dim"])[:n]
                x = torch.cat([first, rest]).double()
                if sc in s:
                    x = (x - s[of][h].double()) * s[sc][h].double()
                parts.append(x)
            rows = slice(h * group, (h + 1) * group)
            everything = torch.ones((group, n_pre + n), dtype=torch.bool, device=q.device)
            out[b, rows] = _attend(q[b, rows], parts[0], parts[1], everything)
    return out
