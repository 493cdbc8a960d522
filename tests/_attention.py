"""Plain 64-bit attention and page bookkeeping for the tests, and how far an fp32-accumulating kernel may be from it."""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}       # half a rounding step, relative


def attend64(q, k, v, see, scale, u_out, u_p, kmag=None, vmag=None, u_q=0.0):
    """One head: rows q [n, D] over keys k [m, D], v [m, D] (float64); row i sees the keys that see[i] marks.
    Returns (out, lse, the bound of |out|'s error, the bound of lse's error).

    The bounds count, for a kernel with exact products and fp32 sums:
      ds    the scores: D + 8 roundings (2^-23 each, of the running sum) of sum |q| |k|, and of the score itself
            when it is scaled, shifted by the maximum and exponentiated (2^-22 each of its magnitude); over int8
            codes also u_q of sum |q| |k|, the rounding of q times the key scale (plus, for each channel, half a
            subnormal f16 step, 2^-25 of the row's largest, which D of them bring to less than 2^-17 of it);
      sums  each of the m terms of the weights' sum and of the product with v: 2^-23 of the sum of magnitudes;
      u_p   the weights' rounding for the product with v (and, where they are f16, 2^-33 of the largest |v| for each
            key: half a subnormal step of weights that the kernels scale up by 2^8);
      u_out the output's rounding.
    kmag, vmag: magnitudes of the terms that k and v are sums of (|code| + |offset|, scaled), where they are."""
    kmag = k.abs() if kmag is None else kmag
    vmag = v.abs() if vmag is None else vmag
    n, m = q.shape[0], k.shape[0]
    s = (q @ k.T) * scale
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    top = s.max(1, keepdim=True).values if m else s.new_full((n, 1), -math.inf)
    some = top > -math.inf
    p = torch.where(some, torch.exp(s - torch.where(some, top, torch.zeros_like(top))), torch.zeros_like(s))
    l = p.sum(1, keepdim=True)
    w = torch.where(some, p / l.clamp(min=1e-300), torch.zeros_like(p))
    vz = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))          # rows nobody sees may hold anything
    vm = torch.where(see.any(0)[:, None], vmag, torch.zeros_like(vmag))
    out = w @ vz
    lse = torch.where(some[:, 0], top[:, 0] + torch.log(l[:, 0].clamp(min=1e-300)), top[:, 0])
    mag = torch.where(see, (q.abs() @ kmag.T) * abs(scale), torch.zeros_like(s))
    smax = torch.where(see, s.abs(), torch.zeros_like(s))
    zero = s.new_zeros(n)
    ds = (q.shape[1] + 8) * 2.0 ** -23 * (mag.max(1).values if m else zero) + \
        2.0 ** -21 * (1 + (smax.max(1).values if m else zero))
    if u_q:
        big = (q.abs().max(1).values if n else zero) * (kmag.max() if m else 0.0) * abs(scale)
        ds = ds + u_q * (mag.max(1).values if m else zero) + 2.0 ** -25 * q.shape[1] * big
    sums = (m + 64) * 2.0 ** -23
    a = w @ vm
    sub = m * 2.0 ** -33 * (vm.max() if m else 0.0) if u_p < 2.0 ** -9 else 0.0
    bound = u_out * out.abs() + a * (u_p * (1 + u_out) + 2 * ds[:, None] + sums) + sub
    if u_out < 2.0 ** -9:
        bound = bound + 2.0 ** -25                             # an f16 output below its normal range
    return out, lse, bound, ds + sums + 2.0 ** -22 * torch.where(some[:, 0], lse.abs(), zero)


def prompt64(q, k, v, spans, causal=True, scale=None):
    """q [T, Nq, D], k, v [Tk, Nkv, D]; spans: (q0, lq, k0, lk) of each sequence.  Returns out, lse and their bounds
    in float64; rows of no sequence are NaN (not written)."""
    T, Nq, D = q.shape
    G = Nq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    u = U[q.dtype]
    out = torch.full((T, Nq, D), math.nan, dtype=torch.float64, device=q.device)
    bound, lse, lb = out.clone(), out[..., 0].clone(), out[..., 0].clone()
    for q0, lq, k0, lk in spans:
        i = torch.arange(lq, device=q.device)[:, None]
        j = torch.arange(lk, device=q.device)[None]
        see = (j <= i + lk - lq) if causal else torch.ones((lq, lk), dtype=torch.bool, device=q.device)
        for h in range(Nq):
            r = attend64(q[q0:q0 + lq, h].double(), k[k0:k0 + lk, h // G].double(), v[k0:k0 + lk, h // G].double(),
                         see, scale, u, u)
            out[q0:q0 + lq, h], lse[q0:q0 + lq, h], bound[q0:q0 + lq, h], lb[q0:q0 + lq, h] = r
    return out, lse, bound, lb


def check_rows(got, want, bound, what=""):
    """got (any type) within bound of want where want is a number; rows that want leaves out are not looked at."""
    live = ~torch.isnan(want)
    d = (got.double() - want).abs()
    d = torch.where(torch.isinf(want) & (got.double() == want), torch.zeros_like(d), d)
    bad = live & ~(d <= bound)
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(live.sum())} values off, first at {at}: got "
                             f"{float(got[at])}, want {float(want[at])}, bound {float(bound[at]):.3g}")


def page_values(cache, pages, n, h, scale=None, offset=None):
    """The first n tokens' values of head h in these pages, and the magnitudes of what they are computed from."""
    if n == 0:
        z = torch.zeros((0, cache.shape[3]), dtype=torch.float64, device=cache.device)
        return z, z
    x = cache[pages.long().clamp(min=0), :, h].reshape(-1, cache.shape[3])[:n].double()
    if scale is None:
        return x, x.abs()
    sc = scale.view(cache.shape[2], cache.shape[3])[h].double()
    of = torch.zeros_like(sc) if offset is None else offset.view(cache.shape[2], cache.shape[3])[h].double()
    return (x - of) * sc, (x.abs() + of.abs()) * sc.abs()


def shared64(q, kc, vc, table, lens, prefix_table, prefix_len, scale_k=None, scale_v=None, offset_k=None,
             offset_v=None, scale=None):
    B, Nq, D = q.shape
    Nkv = kc.shape[2]
    G = Nq // Nkv
    scale = D ** -0.5 if scale is None else scale
    u_out = U[q.dtype]
    u_p = U[torch.float16] if kc.dtype == torch.int8 else U[kc.dtype]
    u_q = 0.0 if kc.dtype != torch.int8 else 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22
    out = torch.full((B, Nq, D), math.nan, dtype=torch.float64, device=q.device)
    bound, lse, lb = out.clone(), out[..., 0].clone(), out[..., 0].clone()
    block = kc.shape[1]
    for h in range(Nkv):
        pre = [page_values(c, prefix_table[: -(-prefix_len // block)], prefix_len, h, s, o) if prefix_len else
               page_values(c, None, 0, h) for c, s, o in ((kc, scale_k, offset_k), (vc, scale_v, offset_v))]
        for b in range(B):
            n = int(lens[b])
            if n < 0:
                continue
            own = [page_values(c, table[b, : -(-n // block)], n, h, s, o)
                   for c, s, o in ((kc, scale_k, offset_k), (vc, scale_v, offset_v))]
            k, km, v, vm = (torch.cat([pre[i][j], own[i][j]]) for i in (0, 1) for j in (0, 1))
            rows = slice(h * G, (h + 1) * G)
            see = torch.ones((G, k.shape[0]), dtype=torch.bool, device=q.device)
            out[b, rows], lse[b, rows], bound[b, rows], lb[b, rows] = attend64(q[b, rows].double(), k, v, see, scale, u_out,
                                                                              u_p, km, vm, u_q)
    return out, lse, bound, lb


# ---------------------------------------------------------------------------
# page bookkeeping, one step at a time
# ---------------------------------------------------------------------------
def free_plain(table, lens, ref, rows, block):
    """On lists of numpy arrays, in place; returns whether anything was out of range."""
    fault = False
    for r in rows:
        if r == -1:
            continue
        if not 0 <= r < len(lens):
            fault = True
            continue
        n, lens[r] = int(lens[r]), 0
        if n == 0:
            continue
        held = -(-n // block)
        if n < 0 or held > table.shape[1]:
            fault, held = True, 0 if n < 0 else table.shape[1]
        for e in range(held):
            p = table[r, e]
            if not 0 <= p < len(ref) or ref[p] <= 0:
                fault = True
            else:
                ref[p] -= 1
        table[r] = -1
    return fault


def fork_plain(caches, table, lens, ref, parents, children, block):
    """Returns (fresh, fault bits)."""
    fresh, bits = [], 0
    lens0, taken = lens.copy(), {}
    ok = []
    for i, (p, c) in enumerate(zip(parents, children)):
        good = 0 <= p < len(lens) and 0 <= c < len(lens) and p != c and \
            0 <= lens0[p] <= table.shape[1] * block and lens0[c] == 0
        ok.append(good)
        if not good and not (p == -1 and c == -1):
            bits |= 1
        if good:
            taken.setdefault(c, i)
    vacant = iter([p for p in range(len(ref)) if ref[p] <= 0])
    for i, (p, c) in enumerate(zip(parents, children)):
        if not ok[i]:
            fresh.append(-2)
            continue
        if taken[c] != i or p in taken:
            bits |= 1
            fresh.append(-2)
            continue
        n = int(lens0[p])
        full, page = n // block, -1
        if n % block:
            page = next(vacant, None)
            if page is None:
                bits |= 4
                fresh.append(-2)
                continue
        row = [-1] * table.shape[1]
        for e in range(full):
            row[e] = table[p, e]
            ref[table[p, e]] += 1
        if page >= 0:
            row[full] = page
            ref[page] = 1
            for ca in caches:
                ca[page] = ca[table[p, full]]
        table[c] = row
        lens[c] = n
        fresh.append(page)
    return fresh, bits


def compact_plain(caches, table, ref):
    used = [p for p in range(len(ref)) if ref[p] > 0]
    u = len(used)
    holes = [p for p in range(u) if ref[p] <= 0]
    page_map = [-1] * len(ref)
    new_ref = ref * 0
    for p in used:
        to = p if p < u else holes.pop(0)
        page_map[p] = to
        new_ref[to] = ref[p]
        if to != p:
            for c in caches:
                c[to] = c[p]
    new_table = table.copy()
    for r in range(table.shape[0]):
        for e in range(table.shape[1]):
            if table[r, e] >= 0:
                new_table[r, e] = page_map[table[r, e]]
    return new_table, new_ref, page_map
