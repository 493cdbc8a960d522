"""shared_prefix_attention over 16-bit pages with values that are not finite, on the GPU against the definition in 64 bits."""
import math

import pytest
import torch

import kv_cache_quantize_b200 as kvq
from _attention import check_rows, shared64
from test_gpu_attention import call_shared, paged, want_shared

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def place(d, b, key):
    """Where key `key` of request b (of the prefix: b None) lies: page and token."""
    block = d["kc"].shape[1]
    row = d["prefix_table"] if b is None else d["table"][b]
    return int(row[key // block]), key % block


def check(d, odd, **kw):
    """odd: (request or None, key, head, channel, value) of the values put in.  Channels they reach are the definition's
    infinities and NaNs; the others are within the bound of the same call without them."""
    want, wl, bound, lb = want_shared(d)
    for b, key, head, channel, value in odd:
        page, token = place(d, b, key)
        d["vc"][page, token, head, channel] = value
    full = want_shared(d)[0]
    out = torch.full_like(d["q"], 3.0)
    lse = torch.full(d["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    call_shared(d, out=out, lse=lse, check=True, **kw)
    reached = ~torch.isfinite(full)
    assert bool(reached.any()) and not bool(reached.all())
    got = out.double()[reached]
    assert torch.equal(torch.isnan(got), torch.isnan(full[reached]))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(full[reached], nan=0.0))
    check_rows(out, torch.where(reached, math.nan, want), bound, "out")
    check_rows(lse, wl, lb, "lse")


INF = math.inf


@pytest.mark.parametrize("value", [INF, -INF, math.nan])
@pytest.mark.parametrize("own", [20, 100, 300])
@pytest.mark.parametrize("block", [16, 64, 24])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_own_value_that_is_not_finite(dtype, block, own, value):
    for dim, heads in ((128, (8, 2)), (64, (3, 3))):
        for key in (0, own - 1, own // 2):
            d = paged(41, [own, 5, own], 0, *heads, dim, block, dtype, dtype)
            check(d, [(0, key, 1, dim // 2 + 3, value)])


@pytest.mark.parametrize("batch", [1, 3, 40])
@pytest.mark.parametrize("prefix", [20, 100, 300])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_prefix_value_that_is_not_finite(dtype, prefix, batch):
    """Groups of few rows (four times in a tile) and of many."""
    for value in (INF, -INF, math.nan):
        for key in (0, prefix - 1, prefix // 3):
            d = paged(42, [3 + i % 150 for i in range(batch)], prefix, 8, 2, 128, 16, dtype, dtype)
            check(d, [(None, key, 0, 77, value)])


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("block", [32, 12])
def test_several_values_that_are_not_finite(dtype, block):
    """Infinities of both signs that meet in a channel, in one quarter of a step, in two, in two steps, in prefix and own."""
    for pairs in ([(0, 3, INF), (0, 20, -INF)], [(0, 3, INF), (0, 50, -INF)], [(0, 3, INF), (0, 200, -INF)],
                  [(None, 7, INF), (0, 9, -INF)], [(0, 3, INF), (0, 120, INF)], [(0, 10, -INF), (0, 290, -INF)]):
        d = paged(43, [300, 40], 64, 8, 2, 64, block, dtype, dtype)
        check(d, [(b, key, 1, 9, value) for b, key, value in pairs] + [(0, 130, 1, 33, INF), (1, 39, 0, 0, -INF)])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_values_that_are_not_finite_over_many_steps(dtype):
    """Pieces of several steps for each tile, cut over many CTAs, the maxima moving as they go."""
    d = paged(44, [5000, 10], 4000, 8, 2, 128, 64, dtype, dtype)
    d["q"] = d["q"] * 0.5
    check(d, [(0, 4999, 0, 1, INF), (0, 31, 0, 2, -INF), (None, 1000, 1, 127, INF), (0, 700, 1, 127, -INF), (None, 0, 0, 5, math.nan)])


def test_values_that_are_not_finite_beside_pages_that_are_not_there():
    """A missing page's keys are no one's; a seen infinity beside them stays one."""
    d = paged(45, [100, 60], 0, 8, 2, 128, 16, BF, BF)
    d["table"][0, 2] = -1
    keep = torch.tensor([k for k in range(100) if not 32 <= k < 48], device="cuda")
    d["vc"][int(d["table"][0, 4]), 3, 1, 9] = INF
    out = torch.full_like(d["q"], 3.0)
    kvq.get_error()
    call_shared(d, out=out)
    assert kvq.get_error() == kvq.FAULT_SLOT_RANGE
    # the same keys in pages of their own
    k, v = (d[n][d["table"][0, :7].long().clamp(min=0)].reshape(-1, 2, 128)[keep] for n in ("kc", "vc"))
    pages = [torch.zeros((6, 16, 2, 128), dtype=BF, device="cuda") for _ in range(2)]
    for p, x in zip(pages, (k, v)):
        p.view(-1, 2, 128)[:84] = x
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([84], dtype=torch.int32, device="cuda")
    full = shared64(d["q"][:1], *pages, table, lens, None, 0)[0]
    reached = ~torch.isfinite(full)
    assert int(reached.sum()) == 4 and torch.equal(out[:1].double()[reached], full[reached])
    pages[1] = torch.where(torch.isfinite(pages[1].float()), pages[1], 0)
    want, _, bound, _ = shared64(d["q"][:1], *pages, table, lens, None, 0)
    check_rows(out[:1], torch.where(reached, math.nan, want), bound)


def test_calls_answer_with_their_device():
    d = paged(46, [5], 0, 8, 2, 64, 16, BF, BF)
    page = torch.zeros((1,), dtype=torch.int32, device="cuda")
    answer = kvq._calls().copy_pages([d["kc"]], page, page, None)
    assert answer[0] == 0 and answer[2] == d["kc"].get_device()


@pytest.mark.parametrize("heads", [(8, 2), (40, 1)])
@pytest.mark.parametrize("dtype,cache", [(BF, torch.int8), (F16, torch.int8), (F16, F16)])
@pytest.mark.parametrize("cols", [0, 1, 8, 9, 20])
def test_workspace_of_just_the_size_that_is_asked_for(cols, dtype, cache, heads):
    """Tables without columns, of one step of 128 keys and of more; the bytes behind the workspace stay as they are,
    and what stood in it (NaN) does not matter."""
    for batch, prefix in ((5, 300), (150, 1000), (3, 0)):
        lens = [min(cols * 16, i * 29 % (cols * 16 + 1) + (i % 3 == 0) * 40) for i in range(batch)]
        d = paged(47, lens, prefix, *heads, 64, 16, dtype, cache)
        d["table"] = d["table"][:, :cols] if cols <= d["table"].shape[1] else torch.nn.functional.pad(
            d["table"], (0, cols - d["table"].shape[1]), value=-1)
        assert d["table"].shape == (batch, cols)
        want, wl, bound, lb = want_shared(d)
        need = kvq.shared_prefix_attention_workspace(batch, *heads, 64, prefix, cols * 16)
        ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        lse = torch.zeros((batch, heads[0]), dtype=torch.float32, device="cuda")
        out = call_shared(d, workspace=ws[:need], lse=lse, check=True)
        check_rows(out, want, bound, "out")
        check_rows(lse, wl, lb, "lse")
        assert bool((ws[need:] == 0xFF).all())
        with pytest.raises(kvq.KvqError):
            call_shared(d, workspace=ws[:need - 1])
