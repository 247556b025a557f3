"""A KVCache's C handle names the arrays that the cache holds now (host)."""
import copy
import dataclasses
import pickle

import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep

ARRAYS = ("k", "v", "k_scale", "v_scale", "page_table")


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    """Addresses of host tensors stand for device ones: no call reads them here."""
    def address(t, what, dtype, shape=None):
        assert t.dtype is dtype and (shape is None or t.shape == shape) and t.is_contiguous(), what
        return t.data_ptr()
    monkeypatch.setattr(ep, "_address", address)


def new_cache(seqs=3, most=4, pages=5, heads=2, size=16, dim=64):
    return ep.new_kv_cache(pages, heads, size, dim, torch.zeros((seqs, most), dtype=torch.int32))


def handle_is_of(cache):
    c = cache.c_struct()
    return all(getattr(c, n) == getattr(cache, n).data_ptr() for n in ARRAYS) and (
        c.num_pages, c.num_heads, c.page_size, c.head_dim) == tuple(cache.k.shape) and (
        c.num_seqs, c.max_pages) == tuple(cache.page_table.shape) and cache.c_ref._obj is c


def test_the_handle_is_built_once():
    cache = new_cache()
    assert handle_is_of(cache) and cache.c_struct() is cache.c_struct()
    assert (cache.heads, cache.dim, cache.seqs, cache.cu_shape) == (2, 64, (3,), (4,))


@pytest.mark.parametrize("name", ARRAYS)
def test_a_replaced_array_reaches_the_next_call(name):
    cache = new_cache()
    assert handle_is_of(cache)
    setattr(cache, name, getattr(cache, name).clone())
    assert handle_is_of(cache)


def test_a_grown_batch_and_pool():
    cache = new_cache()
    assert handle_is_of(cache)
    cache.page_table = torch.zeros((7, 9), dtype=torch.int32)
    assert handle_is_of(cache) and cache.seqs == (7,) and cache.cu_shape == (8,)
    for name in ("k", "v"):
        setattr(cache, name, torch.zeros((11, 2, 16, 64), dtype=torch.uint8))
        setattr(cache, name + "_scale", torch.zeros((11, 2)))
    assert handle_is_of(cache) and cache.c_struct().num_pages == 11


def test_arrays_that_do_not_fit_are_refused_at_the_next_call():
    cache = new_cache()
    cache.c_struct()
    cache.page_table = torch.zeros(7, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.c_struct()


@pytest.mark.parametrize("copied", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c)),
                                    lambda c: dataclasses.replace(c)])
@pytest.mark.parametrize("used", [False, True])
def test_a_copy_has_a_handle_of_its_own(copied, used):
    cache = new_cache()
    if used:
        cache.c_struct()
    other = copied(cache)
    assert handle_is_of(other) and handle_is_of(cache) and other.c_struct() is not cache.c_struct()
    other.page_table = torch.zeros((1, 2), dtype=torch.int32)
    assert handle_is_of(other) and handle_is_of(cache)


def test_the_handle_is_seen_only_once_it_is_whole(monkeypatch):
    """What a call reads beside the handle is there whenever the handle is."""
    cache = new_cache()
    seen = []
    plain = ep.KVCache.__setattr__

    def watch(self, name, value):
        plain(self, name, value)
        if self._c is not None:
            seen.append(all(hasattr(self, n) for n in ("c_ref", "heads", "dim", "seqs", "cu_shape")))
    monkeypatch.setattr(ep.KVCache, "__setattr__", watch)
    cache.c_struct()
    assert seen and all(seen)


@pytest.mark.parametrize("table", [torch.zeros((3, 4), dtype=torch.int64), torch.zeros((4, 3), dtype=torch.int32).t(),
                                   torch.zeros(4, dtype=torch.int32), torch.zeros((3, 8), dtype=torch.int32)[:, ::2]])
def test_new_kv_cache_refuses_a_table_that_it_would_have_to_copy(table):
    with pytest.raises(ValueError):
        ep.new_kv_cache(2, 2, 16, 64, table)


def test_new_kv_cache_holds_the_callers_table():
    table = torch.zeros((3, 4), dtype=torch.int32)
    assert ep.new_kv_cache(2, 2, 16, 64, table).page_table is table
