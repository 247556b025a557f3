"""The page-level calls on a stream of their own, beside a caller's stream with half a second of work ahead."""
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep

pytestmark = pytest.mark.gpu
N, K, H, E, R = 300, 4, 512, 16, 4
T = -(-N // R)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(scope="module")
def batch():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(N, 2 * H, generator=g, device="cuda").to(torch.bfloat16)[:, ::2]  # copied within the calls
    idx = torch.rand(N, E, generator=g, device="cuda").topk(K).indices               # int64: converted within the calls
    ones = torch.ones(E, R * T, H, dtype=torch.bfloat16, device="cuda")
    return x, idx, torch.rand(N, K, generator=g, device="cuda"), ones


def normal(batch, stream=None):
    x, idx, w, _ = batch
    lay = ep.get_dispatch_layout(idx, E, R, stream=stream)
    res = ep.dispatch(x, lay, w, stream=stream)
    y = res.expert_x  # worst case and exact: a token's K slots
    out = ep.combine(y, lay, w, stream=stream)
    lay2, res2 = ep.get_layout_and_dispatch(x, idx, E, R, w, use_fp8=True, stream=stream)
    two, rows = ep.combine_two_level(y, lay, w, stream=stream)
    gy, gw = ep.combine_backward(x, lay, y, w, stream=stream)
    gx = ep.dispatch_backward(y, lay, stream=stream)
    return [lay.expert_slot, lay.rank_slot, res.expert_x, res.expert_src, out, lay2.expert_slot, res2.expert_x,
            res2.expert_scales, two, rows, gy, gw, gx]


def low_latency(batch, stream=None):
    x, idx, w, y = batch
    (rx, rs), count, handle, hook = ep.low_latency_dispatch(x, idx, T, E, R, stream=stream)
    hook()
    out = ep.low_latency_combine(y, w, handle, stream=stream)
    late, hook2 = ep.low_latency_combine(y, w, handle, return_recv_hook=True, stream=stream)
    hook2()
    mask = ep.low_latency_query_mask_buffer(handle, stream=stream)
    return [count, handle.recv_src, out, late, mask, rx, rs]


@pytest.mark.parametrize("calls", [normal, low_latency])
def test_beside_a_busy_caller(batch, calls):
    want = calls(batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    if calls is normal:
        calls(batch, side)  # (its sizes are asked for on the host; code and memory are there from now on)
        side.synchronize()
    dirty = [torch.full((t.numel() * t.element_size(),), 0xFF, dtype=torch.uint8, device="cuda") for t in want] + \
        [torch.full((1 << 16,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    del dirty
    torch.cuda.synchronize()
    torch.cuda._sleep(int(1e9))
    got = calls(batch, side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the caller's work is still ahead
    torch.cuda.synchronize()
    if calls is low_latency:  # rows that nobody received are anything
        live = torch.arange(R * T, device="cuda")[None] < want[0][:, None]
        for i in (1, 5, 6):
            want[i], got[i] = want[i][live], got[i][live]
    else:
        n = N * K
        for i in (2, 3, 6, 7):
            want[i], got[i] = want[i][:n], got[i][:n]
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(a.view(torch.uint8) if a.dtype is torch.bfloat16 else a,
                           b.view(torch.uint8) if b.dtype is torch.bfloat16 else b), i
