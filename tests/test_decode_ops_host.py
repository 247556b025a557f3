"""Refusals of the decode step's operators, on the host before any CUDA call."""
import ctypes

import pytest

import combine_ep_get_dispatch_gb300 as ep

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from combine_ep_get_dispatch_gb300 import build
    build.build()
    return ep.lib()


def cache(**kw):
    f = dict(k=256, v=256, k_scale=256, v_scale=256, page_table=256, num_pages=10, num_heads=4, page_size=64,
             head_dim=128, num_seqs=3, max_pages=5)
    f.update(kw)
    return ctypes.byref(ep.ep_kv_cache_t(*f.values()))


BAD_CACHES = [dict(page_size=48), dict(page_size=0), dict(head_dim=96), dict(head_dim=256), dict(num_heads=0),
              dict(num_pages=-1), dict(num_seqs=2), dict(max_pages=-1), dict(max_pages=1 << 26), dict(k=None),
              dict(v_scale=None), dict(page_table=None)]


def append(L, c, n=3, lens=256, cu=None, k=256, ks=512, v=256, vs=512, q=256, qs=1024, qo=256, qos=1024, qh=8, rope=256,
           rows=100, dim=128):
    return L.ep_kv_append(c, P(lens), P(cu), n, P(k), ks, P(v), vs, P(q), qs, P(qo), qos, qh, P(rope), rows, dim, 0,
                          None, None)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_append_refuses_caches(L, bad):
    assert append(L, cache(**bad)) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=2), dict(lens=None), dict(k=None), dict(v=None), dict(ks=511), dict(ks=516), dict(vs=504),
    dict(q=None), dict(qo=None), dict(qs=1016), dict(qos=1020), dict(qh=0), dict(rope=None), dict(dim=8), dict(dim=144),
    dict(dim=0), dict(dim=-16), dict(rows=-1)])
def test_append_refuses_arguments(L, bad):
    assert append(L, cache(), **bad) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(k=264), dict(v=258), dict(q=264), dict(qo=264), dict(rope=260)])
def test_append_refuses_alignment(L, bad):
    assert append(L, cache(), **bad) == ep.EP_ERR_ALIGNMENT


def test_append_refuses_a_misaligned_cache_and_accepts_nothing(L):
    assert append(L, cache(k=264)) == ep.EP_ERR_ALIGNMENT
    assert append(L, None) == ep.EP_ERR_INVALID_ARG
    assert append(L, cache(num_seqs=0), n=0) == ep.EP_OK


def attend(L, c, n=3, lens=256, q=256, qs=1024, qh=8, scale=0.1, window=0, out=256, ws=256, size=1 << 30):
    return L.ep_kv_attention(c, P(lens), None, n, P(q), qs, qh, scale, window, P(out), None, P(ws), size, None, None)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_attention_refuses_caches(L, bad):
    assert attend(L, cache(**bad)) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=4), dict(lens=None), dict(q=None), dict(out=None), dict(qs=1000), dict(qs=1028), dict(qh=6),
    dict(qh=0), dict(qh=8192), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_attention_refuses_arguments(L, bad):
    assert attend(L, cache(), **bad) == ep.EP_ERR_INVALID_ARG


def test_attention_refuses_alignment_and_workspaces(L):
    need = ep.ep_kv_attention_workspace_bytes(3, 8, 4, 128)
    assert need > 0
    assert attend(L, cache(), size=need - 1) == ep.EP_ERR_WORKSPACE
    assert attend(L, cache(), ws=None) == ep.EP_ERR_WORKSPACE
    assert attend(L, cache(), ws=264) == ep.EP_ERR_ALIGNMENT
    assert attend(L, cache(), q=264) == ep.EP_ERR_ALIGNMENT
    assert attend(L, cache(), out=264) == ep.EP_ERR_ALIGNMENT
    assert attend(L, cache(num_seqs=0), n=0) == ep.EP_OK
    for bad in ((-1, 8, 4, 128), (3, 6, 4, 128), (3, 8, 0, 128), (3, 8, 4, 80)):
        assert ep.ep_kv_attention_workspace_bytes(*bad) == 0


def linear(L, x=256, xs=None, rows=10, K=256, count=256, off=256, region=0, E=4, most=10, w=256, ws=256, M=64, flags=0,
           y=256, work=256, size=1 << 40):
    return L.ep_expert_linear(P(x), P(xs), rows, K, P(count), P(off), region, E, most, P(w), P(ws), M, flags, P(y),
                              P(work), size, None, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(K=0), dict(K=192), dict(K=16512), dict(E=0), dict(E=1025), dict(most=-1), dict(M=0), dict(M=12),
    dict(M=8, flags=1), dict(M=(1 << 20) + 8), dict(flags=2), dict(count=None), dict(w=None), dict(ws=None),
    dict(x=None), dict(y=None), dict(off=None, region=-1), dict(off=None, region=1 << 31)])
def test_expert_linear_refuses_arguments(L, bad):
    assert linear(L, **bad) == ep.EP_ERR_INVALID_ARG


def test_expert_linear_refuses_alignment_and_workspaces(L):
    for bad in (dict(x=264), dict(y=264), dict(w=272), dict(ws=264), dict(work=384)):
        assert linear(L, **bad) == ep.EP_ERR_ALIGNMENT
    need = ep.ep_expert_linear_workspace_bytes(4, 10, 256, False)
    assert need > 0 and linear(L, size=need - 1) == ep.EP_ERR_WORKSPACE
    assert linear(L, work=None) == ep.EP_ERR_WORKSPACE
    assert linear(L, most=0) == ep.EP_OK and linear(L, rows=0, x=None, y=None) == ep.EP_OK
    for bad in ((0, 10, 256, False), (4, -1, 256, False), (4, 10, 100, False)):
        assert ep.ep_expert_linear_workspace_bytes(*bad) == 0
