"""The attention and page calls without a GPU: what they refuse, and with which status.

Descriptors carry NULL data: every refusal comes before the pointers are looked at, and a valid set stops at
KVQ_ERR_NULL, so no call here can reach a launch.
"""
import ctypes

import pytest
import torch

import kv_cache_quantize_b200 as kvq

OK, ENULL, ENDIM, ESHAPE, EDTYPE, EATTR, ELAYOUT, ECAP, ECUDA, EUNSUP = range(10)
BF, F16, F32, I8, I32, I64, U8 = (torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.int32, torch.int64,
                                  torch.uint8)


@pytest.fixture(scope="module")
def L():
    from kv_cache_quantize_b200 import build
    build.build()
    return kvq.lib()


def t(shape, dtype, stride=None):
    x = torch.empty_strided(shape, stride, dtype=dtype, device="meta") if stride else \
        torch.empty(shape, dtype=dtype, device="meta")
    d = kvq.KvqTensor()
    d.data, d.dtype, d.ndim = 0, kvq._DTYPES[dtype], x.dim()
    for i, (s, st) in enumerate(zip(x.shape, x.stride())):
        d.shape[i], d.stride[i] = s, st
    return d


def ref(x):
    return None if x is None else ctypes.addressof(x)


def array(items):
    return (kvq.KvqTensor * max(1, len(items)))(*items)


# ---------------------------------------------------------------------------
PROMPT = dict(q=t((50, 8, 128), BF), k=t((60, 2, 128), BF), v=t((60, 2, 128), BF), cu_q=t((4,), I32), cu_k=t((4,), I32),
              out=t((50, 8, 128), BF), lse=t((50, 8), F32), scale=0.1)
EQUAL = dict(q=t((2, 50, 8, 64), F16), k=t((2, 60, 2, 64), F16), v=t((2, 60, 2, 64), F16), cu_q=None, cu_k=None,
             out=t((2, 50, 8, 64), F16), lse=t((2, 50, 8), F32), scale=0.1)


def prompt(L, base=PROMPT, **kw):
    a = {**base, **kw}
    return L.kvq_prompt_attention(*(ref(a[n]) for n in ("q", "k", "v", "cu_q", "cu_k", "out", "lse")), 1, a["scale"], None)


@pytest.mark.parametrize("kw,status", [
    ({}, ENULL), ({"lse": None}, ENULL), ({"cu_k": None, "k": t((50, 2, 128), BF), "v": t((50, 2, 128), BF)}, ENULL),
    ({"q": None}, ENULL), ({"k": None}, ENULL), ({"v": None}, ENULL), ({"out": None}, ENULL),
    ({"cu_q": None}, ENDIM), ({"q": t((50, 1024), BF)}, ENDIM), ({"k": t((1, 60, 2, 128), BF)}, ENDIM),
    ({"q": t((50, 8, 128), F32)}, EDTYPE), ({"k": t((60, 2, 128), F16)}, EDTYPE), ({"v": t((60, 2, 128), I8)}, EDTYPE),
    ({"out": t((50, 8, 128), F32)}, EDTYPE),
    ({"q": t((50, 8, 96), BF), "k": t((60, 2, 96), BF), "v": t((60, 2, 96), BF), "out": t((50, 8, 96), BF)}, EUNSUP),
    ({"k": t((60, 2, 64), BF)}, ESHAPE), ({"v": t((61, 2, 128), BF)}, ESHAPE), ({"v": t((60, 1, 128), BF)}, ESHAPE),
    ({"k": t((60, 3, 128), BF), "v": t((60, 3, 128), BF)}, ESHAPE), ({"out": t((49, 8, 128), BF)}, ESHAPE),
    ({"out": t((50, 4, 128), BF)}, ESHAPE),
    ({"q": t((50, 129, 128), BF), "out": t((50, 129, 128), BF), "k": t((60, 1, 128), BF), "v": t((60, 1, 128), BF)}, EUNSUP),
    ({"q": t((50, 8, 128), BF, (2048, 256, 2))}, ELAYOUT), ({"q": t((50, 8, 128), BF, (1028, 128, 1))}, ELAYOUT),
    ({"k": t((60, 2, 128), BF, (300, 132, 1))}, ELAYOUT), ({"k": t((60, 2, 128), BF, (0, 128, 1))}, ELAYOUT),
    ({"v": t((60, 2, 128), BF, (256, 0, 1))}, ELAYOUT), ({"q": t((50, 8, 128), BF, (1024, 120, 1))}, ELAYOUT), ({"out": t((50, 8, 128), BF, (0, 128, 1))}, ELAYOUT),
    ({"out": t((50, 8, 128), BF, (1024, 64, 1))}, ELAYOUT),
    ({"cu_q": t((4,), I64)}, EDTYPE), ({"cu_k": t((5,), I32)}, ESHAPE), ({"cu_q": t((1, 4), I32)}, ENDIM),
    ({"cu_q": t((0,), I32), "cu_k": t((0,), I32)}, ESHAPE), ({"cu_q": t((4,), I32, (2,))}, ELAYOUT),
    ({"lse": t((50, 8), BF)}, EDTYPE), ({"lse": t((50, 7), F32)}, ESHAPE), ({"lse": t((50, 8), F32, (1, 50))}, ELAYOUT),
    ({"lse": t((400,), F32)}, ENDIM), ({"scale": float("nan")}, EATTR), ({"scale": float("inf")}, EATTR),
    ({"q": t((0, 8, 128), BF), "out": t((0, 8, 128), BF), "lse": None}, OK), ({"cu_q": t((1,), I32), "cu_k": t((1,), I32)}, OK),
])
def test_prompt_refusals(L, kw, status):
    assert prompt(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({}, ENULL), ({"cu_k": t((3,), I32)}, ENULL), ({"k": t((1, 60, 2, 64), F16), "v": t((1, 60, 2, 64), F16)}, ESHAPE),
    ({"k": t((3, 40, 2, 64), F16), "v": t((3, 40, 2, 64), F16)}, ESHAPE), ({"v": t((2, 59, 2, 64), F16)}, ESHAPE),
    ({"q": t((2, 50, 8, 64), F16, (26000, 512, 64, 1))}, ELAYOUT), ({"lse": t((2, 8, 50), F32)}, ESHAPE),
    ({"q": t((2, 0, 8, 64), F16), "out": t((2, 0, 8, 64), F16), "lse": None}, OK),
])
def test_prompt_refusals_of_the_equal_length_form(L, kw, status):
    assert prompt(L, EQUAL, **kw) == status


SHARED = dict(q=t((5, 8, 128), BF), k=t((40, 16, 2, 128), I8), v=t((40, 16, 2, 128), I8), table=t((5, 6), I32),
              lens=t((5,), I32), pt=t((4,), I32), prefix=60, sk=t((2, 128), F32), sv=t((256,), F32), ok=None, ov=None,
              out=t((5, 8, 128), BF), lse=None, scale=0.1, ws=t((1 << 24,), U8))


def shared(L, **kw):
    a = {**SHARED, **kw}
    return L.kvq_shared_prefix_attention(*(ref(a[n]) for n in ("q", "k", "v", "table", "lens", "pt")), a["prefix"],
                                         *(ref(a[n]) for n in ("sk", "sv", "ok", "ov", "out", "lse")), a["scale"],
                                         ref(a["ws"]), None)


@pytest.mark.parametrize("kw,status", [
    ({}, ENULL), ({"ok": t((256,), F32), "ov": t((2, 128), F32)}, ENULL), ({"pt": None, "prefix": 0}, ENULL),
    ({"k": t((40, 16, 2, 128), BF), "v": t((40, 16, 2, 128), BF), "sk": None, "sv": None}, ENULL),
    ({"table": t((5, 6), I32, (0, 1))}, ENULL), ({"table": t((5, 0), I32)}, ENULL),
    ({"q": None}, ENULL), ({"k": None}, ENULL), ({"table": None}, ENULL), ({"lens": None}, ENULL), ({"out": None}, ENULL),
    ({"sk": None}, ENULL), ({"sv": None}, ENULL), ({"pt": None}, ENULL),
    ({"q": t((5, 1, 8, 128), BF)}, ENDIM), ({"k": t((40, 16, 256), I8)}, ENDIM), ({"table": t((30,), I32)}, ENDIM),
    ({"pt": t((1, 4), I32)}, ENDIM), ({"lse": t((40,), F32)}, ENDIM),
    ({"q": t((5, 8, 128), F32)}, EDTYPE), ({"k": t((40, 16, 2, 128), U8)}, EDTYPE), ({"v": t((40, 16, 2, 128), BF)}, EDTYPE),
    ({"k": t((40, 16, 2, 128), F16), "v": t((40, 16, 2, 128), F16)}, EDTYPE), ({"out": t((5, 8, 128), F16)}, EDTYPE),
    ({"table": t((5, 6), I64)}, EDTYPE), ({"lens": t((5,), I64)}, EDTYPE), ({"pt": t((4,), I64)}, EDTYPE),
    ({"sk": t((256,), F16)}, EDTYPE), ({"lse": t((5, 8), BF)}, EDTYPE), ({"ws": t((1 << 22,), F32)}, EDTYPE),
    ({"k": t((40, 16, 2, 128), BF), "v": t((40, 16, 2, 128), BF)}, EATTR), ({"prefix": -1}, EATTR),
    ({"scale": float("inf")}, EATTR), ({"prefix": 65}, ESHAPE), ({"k": t((40, 16, 3, 128), I8)}, ESHAPE),
    ({"k": t((40, 16, 2, 64), I8)}, ESHAPE), ({"v": t((41, 16, 2, 128), I8)}, ESHAPE), ({"table": t((6, 6), I32)}, ESHAPE),
    ({"lens": t((4,), I32)}, ESHAPE), ({"sk": t((128,), F32)}, ESHAPE), ({"out": t((5, 4, 128), BF)}, ESHAPE),
    ({"lse": t((8, 5), F32)}, ESHAPE),
    ({"q": t((5, 8, 32), BF), "out": t((5, 8, 32), BF)}, EUNSUP),
    ({"k": t((40, 16, 2, 128), I8, (4096, 256, 129, 1))}, ELAYOUT), ({"k": t((40, 16, 2, 128), I8, (4100, 256, 128, 1))}, ELAYOUT),
    ({"v": t((40, 16, 2, 128), I8, (4095, 256, 128, 1))}, ELAYOUT),
    ({"v": t((40, 16, 2, 128), I8, (4160, 256, 128, 1))}, ELAYOUT),
    ({"k": t((40, 16, 2, 128), I8, (4112, 256, 128, 1)), "v": t((40, 16, 2, 128), I8, (4112, 256, 128, 1))}, ELAYOUT),
    ({"k": t((1 << 27, 16, 2, 128), I8), "v": t((1 << 27, 16, 2, 128), I8)}, ESHAPE), ({"table": t((5, 6), I32, (12, 2))}, ELAYOUT),
    ({"lens": t((5,), I32, (2,))}, ELAYOUT), ({"out": t((5, 8, 128), BF, (0, 128, 1))}, ELAYOUT),
    ({"sk": t((2, 128), F32, (1, 2))}, ELAYOUT),
])
def test_shared_refusals(L, kw, status):
    assert shared(L, **kw) == status


def test_shared_workspace_sizes(L):
    f = kvq.shared_prefix_attention_workspace
    for bad in ((-1, 8, 2, 128, 0, 0), (1, 8, 3, 128, 0, 0), (1, 8, 0, 128, 0, 0), (1, 8, 2, 96, 0, 0), (1, 8, 2, 128, -1, 0),
                (1, 8, 2, 128, 0, -1)):
        assert f(*bad) == -1
    assert f(0, 8, 2, 128, 0, 0) >= 0
    if f(256, 16, 4, 128, 32768, 1024) > 0:
        assert shared(L, q=t((256, 16, 128), BF), out=t((256, 16, 128), BF), k=t((4000, 64, 4, 128), I8), v=t((4000, 64, 4, 128), I8),
                      table=t((256, 16), I32), lens=t((256,), I32), pt=t((512,), I32), prefix=32768, sk=t((512,), F32),
                      sv=t((512,), F32), ws=t((f(256, 16, 4, 128, 32768, 1024) - 1,), U8)) == ECAP


# ---------------------------------------------------------------------------
CACHES = [t((40, 16, 2, 128), I8), t((40, 16, 2, 128), BF), t((40, 3), F32, (5, 1))]


@pytest.mark.parametrize("caches,src,dst,status", [
    (CACHES, t((4,), I32), t((4,), I64), ENULL), (CACHES, t((0,), I32), t((0,), I32), OK), ([], t((4,), I32), t((4,), I32), EATTR),
    (CACHES * 22, t((4,), I32), t((4,), I32), EATTR), (CACHES + [t((41, 16), I8)], t((4,), I32), t((4,), I32), ESHAPE),
    ([t((40,), I8)], t((4,), I32), t((4,), I32), ENDIM), (CACHES, t((4,), I32), t((5,), I32), ESHAPE),
    (CACHES, t((4,), F32), t((4,), I32), EDTYPE), (CACHES, t((4,), I32), t((4, 1), I32), ENDIM),
    (CACHES, t((4,), I32, (2,)), t((4,), I32), ELAYOUT), ([t((40, 16, 2, 128), I8, (4096, 256, 1, 2))], t((4,), I32), t((4,), I32), ELAYOUT),
    ([t((40, 16), I8, (15, 1))], t((4,), I32), t((4,), I32), ELAYOUT), ([t((40, 0, 16), I8)], t((4,), I32), t((4,), I32), OK),
    ([t((2, 1 << 29), F32)], t((4,), I32), t((4,), I32), ESHAPE), ([t((2, 1 << 32), I8)], t((4,), I32), t((4,), I32), ESHAPE),
])
def test_copy_refusals(L, caches, src, dst, status):
    assert L.kvq_copy_pages(array(caches), len(caches), ref(src), ref(dst), None) == status


def test_copy_null(L):
    i = t((4,), I32)
    assert L.kvq_copy_pages(None, 2, ref(i), ref(i), None) == ENULL
    assert L.kvq_copy_pages(array(CACHES), 3, None, ref(i), None) == ENULL


FREE = dict(table=t((9, 5), I32), lens=t((9,), I32), refs=t((40,), I32), rows=t((3,), I64), block=16)


@pytest.mark.parametrize("kw,status", [
    ({}, ENULL), ({"table": None}, ENULL), ({"lens": None}, ENULL), ({"refs": None}, ENULL), ({"rows": None}, ENULL),
    ({"table": t((9, 5), I64)}, EDTYPE), ({"lens": t((9,), I64)}, EDTYPE), ({"refs": t((40,), F32)}, EDTYPE),
    ({"rows": t((3,), F32)}, EDTYPE), ({"table": t((45,), I32)}, ENDIM), ({"lens": t((9, 1), I32)}, ENDIM),
    ({"lens": t((8,), I32)}, ESHAPE), ({"block": 0}, EATTR), ({"block": -3}, EATTR), ({"table": t((9, 5), I32, (10, 2))}, ELAYOUT),
    ({"table": t((9, 5), I32, (0, 1))}, ELAYOUT), ({"refs": t((40,), I32, (2,))}, ELAYOUT), ({"rows": t((0,), I32)}, OK),
    ({"table": t((0, 5), I32), "lens": t((0,), I32)}, OK), ({"table": t((9, 0), I32)}, OK),
])
def test_free_refusals(L, kw, status):
    a = {**FREE, **kw}
    assert L.kvq_free_pages(ref(a["table"]), ref(a["lens"]), ref(a["refs"]), ref(a["rows"]), a["block"], None) == status


FORK = dict(caches=CACHES, table=t((9, 5), I32), lens=t((9,), I32), refs=t((40,), I32), parents=t((3,), I64),
            children=t((3,), I32), block=16, fresh=t((3,), I32))


@pytest.mark.parametrize("kw,status", [
    ({}, ENULL), ({"caches": []}, ENULL), ({"table": None}, ENULL), ({"fresh": None}, ENULL), ({"children": None}, ENULL),
    ({"refs": t((41,), I32)}, ESHAPE), ({"children": t((4,), I32)}, ESHAPE), ({"fresh": t((4,), I32)}, ESHAPE),
    ({"lens": t((10,), I32)}, ESHAPE), ({"fresh": t((3,), I64)}, EDTYPE), ({"parents": t((3,), F32)}, EDTYPE),
    ({"table": t((9, 5), I64)}, EDTYPE), ({"block": 0}, EATTR), ({"caches": CACHES * 22}, EATTR), ({"table": t((9,), I32)}, ENDIM),
    ({"parents": t((0,), I32), "children": t((0,), I32), "fresh": t((0,), I32)}, OK), ({"table": t((9, 0), I32)}, ESHAPE),
])
def test_fork_refusals(L, kw, status):
    a = {**FORK, **kw}
    assert L.kvq_fork_pages(array(a["caches"]), len(a["caches"]), ref(a["table"]), ref(a["lens"]), ref(a["refs"]),
                            ref(a["parents"]), ref(a["children"]), a["block"], ref(a["fresh"]), None) == status


COMPACT = dict(caches=CACHES, table=t((9, 5), I32), refs=t((40,), I32), nt=t((9, 5), I32), nr=t((40,), I32), pm=t((40,), I32))


@pytest.mark.parametrize("kw,status", [
    ({}, ENULL), ({"caches": []}, ENULL), ({"nt": None}, ENULL), ({"nr": None}, ENULL), ({"pm": None}, ENULL), ({"refs": None}, ENULL),
    ({"nt": t((9, 6), I32)}, ESHAPE), ({"nr": t((41,), I32)}, ESHAPE), ({"pm": t((39,), I32)}, ESHAPE), ({"refs": t((39,), I32)}, ESHAPE),
    ({"caches": [t((41, 4), I8)]}, ESHAPE), ({"pm": t((40,), I64)}, EDTYPE), ({"nt": t((9, 5), I64)}, EDTYPE),
    ({"nr": t((40,), I32, (2,))}, ELAYOUT), ({"table": t((9, 5), I32, (0, 1))}, ELAYOUT),
    ({"caches": [], "table": t((0, 5), I32), "nt": t((0, 5), I32), "refs": t((0,), I32), "nr": t((0,), I32), "pm": t((0,), I32)}, OK),
])
def test_compact_refusals(L, kw, status):
    a = {**COMPACT, **kw}
    assert L.kvq_compact_pages(array(a["caches"]), len(a["caches"]), ref(a["table"]), ref(a["refs"]), ref(a["nt"]), ref(a["nr"]),
                               ref(a["pm"]), None) == status


# ---------------------------------------------------------------------------
def test_binding_refuses_host_tensors_and_other_types(L):
    q = torch.zeros((4, 2, 64), dtype=BF)
    cu = torch.tensor([0, 4], dtype=I32)
    with pytest.raises(ValueError, match="CUDA device"):
        kvq.prompt_attention(q, q, q, cu)
    with pytest.raises(ValueError, match="CUDA device"):
        kvq.copy_pages([torch.zeros((4, 4))], cu, cu)
    with pytest.raises(ValueError, match="CUDA device"):
        kvq.shared_prefix_attention(q, q[None], q[None], cu[None], cu, scale_k=None)
    with pytest.raises(TypeError):
        kvq.prompt_attention(q.double(), q, q, cu)
    with pytest.raises(TypeError):
        kvq.free_pages([[1, 2]], cu, cu, cu, 16)


def test_descriptors_of_the_extension_are_those_of_desc():
    """Field for field the ones of the ctypes binding."""
    for x in (torch.zeros((3, 0), dtype=I8), torch.empty((0,) * 8, dtype=I64), torch.empty((0, 2), dtype=torch.float8_e8m0fnu)):
        assert kvq._calls().descriptor(x) == bytes(kvq.desc(x))
    for dt in kvq._DTYPES:
        assert kvq._calls().descriptor(torch.empty((0,), dtype=dt)) == bytes(kvq.desc(torch.empty((0,), dtype=dt)))
    with pytest.raises(ValueError):
        kvq._calls().descriptor(torch.empty((0,) * 9))


def test_extension_refuses_wrong_arguments():
    c = kvq._calls()
    e = torch.empty((0, 2, 64), dtype=BF)
    with pytest.raises(TypeError):
        c.prompt_attention(e, e)
    with pytest.raises(TypeError):
        kvq.prompt_attention(e, e, e, softmax_scale="x")
    with pytest.raises(TypeError):
        kvq.copy_pages([None], e, e)
    with pytest.raises(TypeError):
        kvq.copy_pages(3, e, e)
    with pytest.raises(TypeError):
        kvq.free_pages(e, e, e, e, "sixteen")
    with pytest.raises(kvq.KvqError):
        kvq.prompt_attention(e, e, e)
