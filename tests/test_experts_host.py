"""Refusals of the router and the 8-bit experts, on the host before any CUDA call; and their stream argument."""
import ctypes
import inspect

import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from combine_ep_get_dispatch_gb300 import build
    build.build()
    return ep.lib()


def route(L, z=256, stride=64, N=3, E=64, K=8, bias=256, G=8, kept=4, best=2, flags=0, scale=1.0, idx=256, w=256, s=None):
    return L.ep_route(P(z), stride, N, E, K, P(bias), G, kept, best, flags, scale, P(idx), P(w), P(s), None)


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(E=0), dict(E=1032), dict(E=60), dict(K=0), dict(K=33), dict(E=8, K=9, G=1, kept=1), dict(G=0),
    dict(G=64, kept=4), dict(kept=0), dict(kept=9), dict(best=0), dict(best=3), dict(flags=8), dict(stride=63),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(z=None), dict(idx=None), dict(w=None)])
def test_route_refuses_arguments(L, bad):
    assert route(L, **bad) == ep.EP_ERR_INVALID_ARG


def test_route_refuses_alignment_and_accepts_nothing(L):
    for bad in (dict(z=258), dict(z=257, flags=ep.EP_ROUTE_BF16), dict(bias=258), dict(idx=257), dict(w=258), dict(s=258)):
        assert route(L, **bad) == ep.EP_ERR_ALIGNMENT
    assert route(L, N=0, z=None, idx=None, w=None, bias=None) == ep.EP_OK


def route_backward(L, dw=256, ds=None, z=256, stride=64, idx=256, N=3, E=64, K=8, flags=0, scale=1.0, dz=256):
    return L.ep_route_backward(P(dw), P(ds), P(z), stride, P(idx), N, E, K, flags, scale, P(dz), None, None)


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=33), dict(E=8, K=9), dict(flags=8), dict(stride=63),
    dict(scale=float("nan")), dict(z=None), dict(idx=None), dict(dw=None), dict(dz=None)])
def test_route_backward_refuses_arguments(L, bad):
    assert route_backward(L, **bad) == ep.EP_ERR_INVALID_ARG


def test_route_backward_refuses_alignment_and_accepts_nothing(L):
    for bad in (dict(z=258), dict(dw=258), dict(ds=257), dict(idx=258), dict(dz=258),
                dict(dz=257, flags=ep.EP_ROUTE_BF16)):
        assert route_backward(L, **bad) == ep.EP_ERR_ALIGNMENT
    assert route_backward(L, N=0, z=None, idx=None, dw=None, dz=None) == ep.EP_OK


def linear(L, x=256, xs=256, rows=10, K=256, count=256, off=256, region=0, E=4, most=10, w=256, ws=256, M=256, flags=0,
           y=256, ys=None, work=256, size=1 << 40):
    return L.ep_expert_linear_fp8(P(x), P(xs), rows, K, P(count), P(off), region, E, most, P(w), P(ws), M, flags, P(y),
                                  P(ys), P(work), size, None, None)


GLU, T, FP8, ROUND, UE8M0 = (ep.EP_LINEAR_GLU, ep.EP_LINEAR_TRANSPOSED, ep.EP_LINEAR_OUT_FP8,
                             ep.EP_LINEAR_OUT_ROUND_SCALE, ep.EP_LINEAR_OUT_UE8M0)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=1 << 31), dict(K=0), dict(K=192), dict(K=16512), dict(E=0), dict(E=1025), dict(most=-1),
    dict(M=0), dict(M=12), dict(M=8, flags=GLU), dict(M=(1 << 20) + 8), dict(flags=64), dict(flags=GLU | T),
    dict(flags=ROUND), dict(flags=UE8M0), dict(M=136, flags=T), dict(M=136, flags=FP8, ys=256),
    dict(M=128, flags=GLU | FP8, ys=256), dict(flags=FP8), dict(count=None), dict(w=None), dict(ws=None), dict(x=None),
    dict(xs=None), dict(y=None), dict(off=None, region=-1), dict(off=None, region=1 << 31),
    dict(most=(1 << 27) - 1, M=1 << 20)])
def test_expert_linear_fp8_refuses_arguments(L, bad):
    assert linear(L, **bad) == ep.EP_ERR_INVALID_ARG


def test_expert_linear_fp8_refuses_alignment_and_workspaces(L):
    for bad in (dict(x=264), dict(y=264), dict(w=264), dict(ws=258), dict(xs=258), dict(work=384),
                dict(flags=FP8, ys=258)):
        assert linear(L, **bad) == ep.EP_ERR_ALIGNMENT
    need = ep.ep_expert_linear_fp8_workspace_bytes(4, 10)
    assert need > 0 and linear(L, size=need - 1) == ep.EP_ERR_WORKSPACE
    assert linear(L, work=None) == ep.EP_ERR_WORKSPACE
    assert linear(L, most=0) == ep.EP_OK and linear(L, rows=0, x=None, xs=None, y=None) == ep.EP_OK
    for bad in ((0, 10), (4, -1), (1025, 10)):
        assert ep.ep_expert_linear_fp8_workspace_bytes(*bad) == 0


CALLS = [ep.route, ep.route_backward, ep.expert_linear_fp8, ep.expert_linear_fp8_backward]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_the_whole_call_goes_to_its_stream(call, monkeypatch):
    seen = []
    monkeypatch.setattr(ep, "_on_stream", lambda stream, f, *args: seen.append((stream, f, args)))
    sig = inspect.signature(call)
    given = {name: object() for name in sig.parameters}
    call(**given)
    (stream, f, args), = seen
    assert stream is given.pop("stream") and f is call
    bound = sig.bind(*args).arguments
    assert bound.pop("stream", None) is None
    assert bound == given


def test_shapes_and_types_are_checked():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="score"):
        ep.route(z, 2, score="tanh")
    with pytest.raises(ValueError, match="logits"):
        ep.route(z, 2)  # not on a GPU
    with pytest.raises(ValueError, match="score"):
        ep.route_backward(z, z, z, score="tanh")
    x, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    w, ws = torch.zeros(3, 384, 256, dtype=torch.uint8), torch.zeros(3, 3, 2)
    n, off = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    good = dict(x=x, x_scale=s, weight=w, weight_scale=ws, row_count=n, row_offset=off)
    for bad, what in ((dict(weight=w[0]), "weight"), (dict(x=x[:, :128]), "x, x_scale"), (dict(x_scale=s[:, :1]), "x_scale"),
                      (dict(row_count=n[:2]), "row_count"), (dict(weight_scale=ws[:, :2]), "weight_scale"),
                      (dict(row_offset=None), "without row_offset"), (dict(row_offset=off[:2]), "row_offset"),
                      (dict(glu=True), "weight_scale"), (dict(out=torch.zeros(4, 256)), "out"),
                      (dict(round_scale=True), "use_fp8"), (dict(use_ue8m0=True), "use_fp8"), (dict(out_scale=s), "use_fp8"),
                      (dict(use_fp8=True, out_scale=s), "out_scale")):
        with pytest.raises(ValueError, match=what):
            ep.expert_linear_fp8(**(good | bad))
    with pytest.raises(ValueError, match="x, x_scale"):  # the gradient's rows have the outputs' channels
        ep.expert_linear_fp8_backward(x, s, w, ws, n, off)


def test_no_channels_are_refused():
    u8 = dict(dtype=torch.uint8)
    n, off = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for call in (ep.expert_linear_fp8, ep.expert_linear_fp8_backward):
        w = torch.zeros(3, 0, 0, **u8)
        with pytest.raises((ValueError, ep.EPError)):
            call(torch.zeros(4, 0, **u8), torch.zeros(4, 0), w, torch.zeros(3, 0, 0), n, off)
