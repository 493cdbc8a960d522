"""The attention calls with the queries' own memory as output."""
import pytest
import torch

import kv_cache_quantize_b200 as kvq
from _attention import check_rows, prompt64
from test_gpu_attention import call_shared, gen, i32, paged, rnd, want_shared

pytestmark = pytest.mark.gpu
BF, F16, I8 = torch.bfloat16, torch.float16, torch.int8


@pytest.mark.parametrize("dtype,cache", [(BF, I8), (F16, I8), (BF, BF), (F16, F16)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch", [3, 70])
def test_shared_into_its_queries(batch, dim, dtype, cache):
    """lse too, whose share of the key offsets comes from the queries."""
    d = paged(61, [i * 31 % 200 for i in range(batch)], 150, 8, 2, dim, 16, dtype, cache)
    want, wl, bound, lb = want_shared(d)
    lse = torch.zeros((batch, 8), dtype=torch.float32, device="cuda")
    out = call_shared(d, out=d["q"], lse=lse, check=True)
    assert out.data_ptr() == d["q"].data_ptr()
    check_rows(out, want, bound, "out")
    check_rows(lse, wl, lb, "lse")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_into_its_queries(dim, dtype):
    g = gen(62)
    lens = [1, 300, 77, 0, 640, 33]
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    q, k, v = (rnd((at[-1], heads, dim), dtype, g) for heads in (6, 2, 2))
    want, wl, bound, lb = prompt64(q, k, v, [(at[i], n, at[i], n) for i, n in enumerate(lens)])
    lse = torch.zeros((at[-1], 6), dtype=torch.float32, device="cuda")
    kvq.prompt_attention(q, k, v, i32(at), out=q, lse=lse, check=True)
    check_rows(q, want, bound, "out")
    check_rows(lse, wl, lb, "lse")
