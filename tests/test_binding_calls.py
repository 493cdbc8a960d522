"""The binding of the attention and page calls without a GPU: what it does around the library's calls."""
import contextlib
import ctypes

import pytest
import torch

import kv_cache_quantize_b200 as kvq


class Extension:
    """Stands in for the extension module: every call ran on device 1, its default stream."""

    def __getattr__(self, name):
        return lambda *args: (0, 0, 1, name)


class Library:
    """Stands in for the library: get_error answers from the fault word of the device that is current."""

    def __init__(self):
        self.current, self.words = 0, {0: kvq.FAULT_TIMEOUT, 1: kvq.FAULT_NO_PAGE}

    def kvq_get_error(self, stream, bits):
        ctypes.cast(bits, ctypes.POINTER(ctypes.c_uint32))[0] = self.words[self.current]
        self.words[self.current] = 0
        return 0


E = torch.empty((0,), dtype=torch.int32)
CALLS = {"prompt_attention": (E, E, E), "shared_prefix_attention": (E, E, E, E, E), "copy_pages": ([E], E, E),
         "free_pages": (E, E, E, E, 16), "fork_pages": ([E], E, E, E, E, E, 16), "compact_pages": ([E], E, E)}


@pytest.mark.parametrize("name", CALLS)
def test_check_reads_the_fault_word_of_the_calls_device(name, monkeypatch):
    """Tensors on device 1 while device 0 is current: the fault of device 1 is raised, that of device 0 stays."""
    library = Library()

    @contextlib.contextmanager
    def on(dev):
        before, library.current = library.current, library.current if dev is None else dev.index
        yield
        library.current = before

    monkeypatch.setattr(kvq, "_calls", Extension)
    monkeypatch.setattr(kvq, "lib", lambda: library)
    monkeypatch.setattr(kvq, "_on", on)
    call = getattr(kvq, name)
    assert call(*CALLS[name]) in (name, None)
    with pytest.raises(kvq.KvqFault) as e:
        call(*CALLS[name], check=True)
    assert e.value.args and "FAULT_NO_PAGE" in str(e.value)
    assert library.words == {0: kvq.FAULT_TIMEOUT, 1: 0}
    assert call(*CALLS[name], check=True) in (name, None)


def test_calls_answer_with_their_device():
    """Where every tensor is empty there is none."""
    c = torch.empty((0, 4), dtype=torch.int8)
    status, stream, device, result = kvq._calls().copy_pages([c], E, E, None)
    assert (status, stream, device, result) == (0, 0, -1, None)


def test_workspace_follows_the_own_keys_a_call_can_have():
    """No own keys: no room for them.  One step of 128 keys: one tile's rows.  More: two tiles'."""
    f = kvq.shared_prefix_attention_workspace
    for args in ((2048, 64, 8, 128), (3, 12, 3, 64), (64, 128, 1, 128), (1, 40, 1, 64)):
        none, one, full, more = (f(*args, 4096, own) for own in (0, 128, 129, 1 << 20))
        assert 0 < none < one < full == more and f(*args, 4096, 1) == one
        b, nq, nkv, d = args
        rows = 4 * nq // nkv if nq // nkv <= 32 else nq // nkv
        assert one - none == full - one == (b * nkv + 148) * rows * (d + 2) * 4
        assert f(*args, 0, 0) == 4 * (b + 1) + f(0, *args[1:], 0, 0) - 4
    assert f(256, 16, 4, 128, 32768, 1024) > 0


def descriptor(shape, dtype):
    """With NULL data: a set that is accepted stops there (status 1) and reaches no launch."""
    d = kvq.KvqTensor()
    d.data, d.dtype, d.ndim = 0, kvq._DTYPES[dtype], len(shape)
    stride = 1
    for i in reversed(range(len(shape))):
        d.shape[i], d.stride[i] = shape[i], stride
        stride *= shape[i]
    return d


SHAPE, LAYOUT, NULL = 3, 6, 1


@pytest.mark.parametrize("sequences,heads,status", [
    ((1 << 29) + 7, 8, SHAPE),               # 2^32 + 56 work items, 56 in 32 bits
    (1 << 29, 8, SHAPE), (1 << 28, 8, SHAPE), ((1 << 28) - 1, 8, NULL), (1 << 30, 1, NULL), ((1 << 30) - 1, 2, NULL), (4, 8, NULL)])
def test_prompt_refuses_more_work_than_a_grid_holds(sequences, heads, status):
    q = descriptor((50, heads, 64), torch.bfloat16)
    cu = descriptor((sequences + 1 if sequences < 1 << 30 else 1 << 30,), torch.int32)
    ref = lambda x: ctypes.addressof(x)  # noqa: E731
    assert kvq.lib().kvq_prompt_attention(ref(q), ref(q), ref(q), ref(cu), None, ref(q), None, 1, 0.1, None) == status


@pytest.mark.parametrize("heads,status", [((1 << 32) + 8, LAYOUT), ((1 << 31) + 8, SHAPE), ((1 << 30) + 8, SHAPE)])
def test_prompt_refuses_more_heads_than_32_bits_hold(heads, status):
    """The largest by its stride, 2^38 elements and more."""
    q = descriptor((1, heads, 64), torch.bfloat16)
    cu = descriptor((2,), torch.int32)
    ref = lambda x: ctypes.addressof(x)  # noqa: E731
    assert kvq.lib().kvq_prompt_attention(ref(q), ref(q), ref(q), ref(cu), None, ref(q), None, 1, 0.1, None) == status


@pytest.mark.parametrize("batch,cols,status", [
    (300, 1 << 19, SHAPE),                   # 300 x 2^23 steps of 128 keys, more than 2^31
    (256, 1 << 19, SHAPE), (255, 1 << 19, NULL), (300, 1 << 12, NULL)])
def test_shared_refuses_more_own_steps_than_32_bits_count(batch, cols, status):
    """One table row for all requests (stride 0), pages of 2048 tokens."""
    q, caches = descriptor((batch, 4, 64), torch.bfloat16), descriptor((8, 2048, 1, 64), torch.bfloat16)
    table, lens, ws = descriptor((batch, cols), torch.int32), descriptor((batch,), torch.int32), descriptor((1 << 33,), torch.uint8)
    table.stride[0] = 0
    ref = lambda x: None if x is None else ctypes.addressof(x)  # noqa: E731
    got = kvq.lib().kvq_shared_prefix_attention(*(ref(x) for x in (q, caches, caches, table, lens)), None, 0, None, None, None,
                                                None, ref(q), None, 0.1, ref(ws), None)
    assert got == status
    assert (kvq.shared_prefix_attention_workspace(batch, 4, 1, 64, 0, cols * 2048) == -1) == (status == SHAPE)


@pytest.mark.parametrize("prefix,status", [
    ((1 << 63) - 1, SHAPE), ((1 << 63) - 1 - 0x7FFFFF00, SHAPE), ((1 << 32) + 5, SHAPE), ((1 << 30) + 1, SHAPE), (8 * 2048, NULL)])
def test_shared_refuses_prefixes_whose_length_leaves_its_type(prefix, status):
    """Lengths near 2^63 wrapped to small and negative ones, those above 2^31 lost their upper bits."""
    q, caches = descriptor((2, 4, 64), torch.bfloat16), descriptor((8, 2048, 1, 64), torch.bfloat16)
    table, lens, ws = descriptor((2, 3), torch.int32), descriptor((2,), torch.int32), descriptor((1 << 33,), torch.uint8)
    pages = descriptor((8,), torch.int32)
    ref = lambda x: None if x is None else ctypes.addressof(x)  # noqa: E731
    got = kvq.lib().kvq_shared_prefix_attention(*(ref(x) for x in (q, caches, caches, table, lens, pages)), prefix, None, None,
                                                None, None, ref(q), None, 0.1, ref(ws), None)
    assert got == status
    assert (kvq.shared_prefix_attention_workspace(2, 4, 1, 64, prefix, 3 * 2048) == -1) == (status == SHAPE)
