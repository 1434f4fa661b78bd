"""What the binding of the paged calls checks, with tensors that only claim to lie on a device and a
library that only notes its calls."""
import types

import pytest
import torch

import fourier_basis_attention_b200 as fa

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32
B, HQ, HKV, PAGE, TOTAL, KEEP = 2, 8, 2, 16, 5, 20


class Claimed(torch.Tensor):
    """A host tensor that says it lies on CUDA device `index`."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def on(index, *shape, dtype=BF):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(Claimed)
    t.index = index
    return t


@pytest.fixture
def gpus(monkeypatch):
    """.current: the current device; .calls: (name, arguments) of the library calls made."""
    state = types.SimpleNamespace(current=0, calls=[])
    fa._import_torch()
    note = lambda name: lambda *a: state.calls.append((name, a)) or 0  # noqa: E731
    monkeypatch.setattr(fa, "_device", lambda: state.current)
    monkeypatch.setattr(fa, "_raw_stream", lambda stream, device: None)
    monkeypatch.setattr(fa, "LIB", types.SimpleNamespace(**{n: note(n) for n in fa.EXPORTED}))
    return state


def cache_on(index, page=PAGE, pages=8, max_pages=4):
    return fa.PagedCache(on(index, pages, HKV, page, 128), on(index, pages, HKV, page, 128),
                         on(index, B, max_pages, dtype=I32))


def batch_on(index, cache=None, **kw):
    kw = dict(dict(total_q=TOTAL, max_q=4), **kw)
    return fa.PagedBatch(cache or cache_on(index), HQ, on(index, B + 1, dtype=I32), on(index, B, dtype=I32), **kw)


def append(index, batch, **kw):
    fa.fa_paged_append(batch, on(index, TOTAL, HKV, 128), on(index, TOTAL, HKV, 128), **kw)


def attend(index, batch, **kw):
    fa.fa_paged_attend(batch, on(index, TOTAL, HQ, 128), on(index, TOTAL, HQ, 128), **kw)


def weights(index, batch, **kw):
    fa.fa_paged_weights(batch, on(index, TOTAL, HQ, 128), on(index, TOTAL, HQ, dtype=F32),
                        on(index, B, HKV, 64, dtype=F32), **kw)


def evict(index, batch, dst=None, **kw):
    fa.fa_evict(batch, on(index, B, HKV, 64, dtype=F32), KEEP, dst or cache_on(index),
                on(index, B, HKV, KEEP, dtype=I32), on(index, B, dtype=I32), **kw)


CALLS = {"fa_paged_append": append, "fa_paged_attend": attend, "fa_paged_weights": weights, "fa_evict": evict}


def refused(call, *args, **kw):
    with pytest.raises(fa.FaError) as e:
        call(*args, **kw)
    assert e.value.code == fa.FA_ERR_INVALID
    return str(e.value)


@pytest.mark.parametrize("name", CALLS)
def test_a_batch_of_another_device_is_refused(gpus, name):
    """A batch holds pointers: with another device current, tensors of that device would go with
    pages of the first."""
    batch = batch_on(0)
    CALLS[name](0, batch)
    assert [n for n, _ in gpus.calls] == [name]
    gpus.current = 1
    assert "the batch is on cuda:0" in refused(CALLS[name], 1, batch)
    CALLS[name](1, batch_on(1))
    assert len(gpus.calls) == 2


def test_a_cache_of_another_device_is_refused(gpus):
    cache = cache_on(0)
    gpus.current = 1
    assert "the cache is on cuda:0" in refused(batch_on, 1, cache)
    assert "dst is on cuda:0" in refused(evict, 1, batch_on(1), cache)
    assert not gpus.calls


@pytest.mark.parametrize("call", [attend, weights])
@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32 + 5])
def test_windows_past_32_bits_are_refused(gpus, call, window):
    """Cut to 32 bits, 2^32 + 5 would be a window of 5 keys."""
    assert "does not fit 32 bits" in refused(call, 0, batch_on(0), window=window)
    assert "does not fit 32 bits" in refused(fa.fa_paged_attend_workspace_size, batch_on(0), window=window)
    assert not gpus.calls
    call(0, batch_on(0), window=2 ** 31 - 1)
    assert len(gpus.calls) == 1


@pytest.mark.parametrize("call", [attend, weights])
@pytest.mark.parametrize("scale", [1e-46, 1e-300, -1e-300])
def test_scales_that_vanish_in_fp32_are_refused(gpus, call, scale):
    """0 would pick the default scale."""
    with pytest.raises(fa.FaError) as e:
        call(0, batch_on(0), scale=scale)
    assert e.value.code == fa.FA_ERR_UNSUPPORTED and not gpus.calls


@pytest.mark.parametrize("kw", [dict(max_kv=2 ** 32 + 64), dict(max_kv=2 ** 31), dict(max_kv=None)], ids=str)
def test_bounds_past_32_bits_are_refused(gpus, kw):
    """A table of 2^17 entries over pages of 2^15 tokens has room for 2^32."""
    table = on(0, B, 2 ** 17, dtype=I32) if kw["max_kv"] is None else None
    cache = cache_on(0)
    if table is not None:
        cache.page_table, cache.max_pages, cache.page_size = table, 2 ** 17, 2 ** 15
    assert "max_kv" in refused(batch_on, 0, cache, **kw)


def test_eviction_into_a_table_with_room_for_more_than_32_bits(gpus):
    """What counts is the room for `keep` tokens; 2^17 pages of 2^15 tokens would be cut to none."""
    dst = cache_on(0)
    dst.max_pages, dst.page_size = 2 ** 17, 2 ** 15
    evict(0, batch_on(0), dst)
    shape = gpus.calls[0][1][7]._obj
    assert (shape.max_pages, shape.page_size, shape.max_kv) == (2 ** 17, 2 ** 15, KEEP)
    for kw in (dict(sink=2 ** 32), dict(recent=2 ** 32 + 1)):
        assert "does not fit 32 bits" in refused(evict, 0, batch_on(0), **kw)
    small = cache_on(0, page=4, max_pages=2)  # room for 8 tokens: the library refuses it
    evict(0, batch_on(0), small)
    assert gpus.calls[1][1][7]._obj.max_kv == 8


@pytest.mark.parametrize("kw", [dict(rot_dim=2 ** 32 + 64), dict(original_len=2 ** 32 + 1)], ids=str)
def test_rope_sizes_past_32_bits_are_refused(kw):
    assert "does not fit 32 bits" in refused(fa.fa_rope_init, scaling="bands", factor=2.0, **kw)
