"""The decode step's operators as a serving loop calls them: arrays replaced between calls, other streams, padding."""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_a_replaced_page_table_and_pool_reach_the_next_call():
    """A cache whose table and pool grow between calls gives the bits of one made with the final ones."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kv = torch.randn(40, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    k, v = kv[:, :2], kv[:, 2:]
    q = torch.randn(1, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    small, large = ints(3).view(1, 1), ints(3, 0, 6).view(1, 3)
    cache, whole = ep.new_kv_cache(4, 2, 16, 64, small), ep.new_kv_cache(8, 2, 16, 64, large)
    ep.kv_append(k[:16], v[:16], cache, ints(16), cu_tokens=ints(0, 16))
    ep.kv_append(k[:16], v[:16], whole, ints(16), cu_tokens=ints(0, 16))
    assert torch.equal(ep.kv_attention(q, cache, ints(16)), ep.kv_attention(q, whole, ints(16)))
    cache.page_table = large
    for name in ("k", "v", "k_scale", "v_scale"):
        old = getattr(cache, name)
        setattr(cache, name, torch.cat([old, torch.zeros_like(old)]))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.kv_append(k[16:], v[16:], cache, ints(40), cu_tokens=ints(0, 24), status=st)
    ep.kv_append(k[16:], v[16:], whole, ints(40), cu_tokens=ints(0, 24))
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(cache, name), getattr(whole, name)), name
    assert torch.equal(ep.kv_attention(q, cache, ints(40), status=st), ep.kv_attention(q, whole, ints(40)))
    assert int(st.item()) == 0


def busy_caller(need):
    """The caller's stream has half a second of work ahead, and memory that it let go holds ones everywhere."""
    torch.cuda.synchronize()
    for size in {512, *need}:
        dirty = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del dirty
    torch.cuda.synchronize()
    torch.cuda._sleep(int(1e9))


def test_attention_on_a_stream_of_its_own_beside_a_busy_one():
    """What a call makes for its stream waits for nothing on the caller's, and is not given out while it is in use."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    P, pages, KH, D = 64, 300, 2, 128
    cache = ep.new_kv_cache(pages, KH, P, D, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages))
    n = pages * P - 5  # long enough to be shared by many blocks, whose counters lie in the workspace
    kv = torch.randn(n, 2 * KH, D, generator=g, device="cuda").to(torch.bfloat16)
    ep.kv_append(kv[:, :KH], kv[:, KH:], cache, ints(n), cu_tokens=ints(0, n))
    q = torch.randn(1, 16, D, generator=g, device="cuda").to(torch.bfloat16)
    lens = ints(n)
    want, want_lse = ep.kv_attention(q, cache, lens, return_lse=True)
    need = ep.ep_kv_attention_workspace_bytes(1, 16, KH, D)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        busy_caller((need, want.numel() * 2, want_lse.numel() * 4))
        got, lse = ep.kv_attention(q, cache, lens, return_lse=True, stream=stream)
        with torch.cuda.stream(side):  # the next ones to ask for memory there
            after = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
        side.synchronize()
        assert not torch.cuda.current_stream().query()  # the caller's work is still ahead
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(lse, want_lse) and all((t == 0xFF).all() for t in after)


def test_append_and_experts_on_a_stream_of_their_own_beside_a_busy_one():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k = torch.randn(30, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    table = ints(0, 1).view(1, 2)
    rope = torch.randn(30, 64, generator=g, device="cuda")
    lens, cu = ints(30), ints(0, 30)
    want = ep.kv_append(k, k, ep.new_kv_cache(2, 2, 16, 64, table), lens, cu_tokens=cu, rope=rope, q=k)
    cache = ep.new_kv_cache(2, 2, 16, 64, table)
    w = torch.randint(0, 256, (3, 64, 512), generator=g, dtype=torch.uint8, device="cuda")
    s = torch.full((3, 64, 32), 120, dtype=torch.uint8, device="cuda")
    x = torch.randn(3, 7, 1024, generator=g, device="cuda").to(torch.bfloat16)
    count = ints(7, 7, 7)
    want_y = ep.expert_linear(x, w, s, count)
    side = torch.cuda.Stream()
    busy_caller((want.numel() * 2, want_y.numel() * 2, ep.ep_expert_linear_workspace_bytes(3, 21, 1024, False)))
    q = ep.kv_append(k, k, cache, lens, cu_tokens=cu, rope=rope, q=k, stream=side)
    y = ep.expert_linear(x, w, s, count, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(y, want_y)


@pytest.mark.parametrize("D,P,QH,rot,cu", [(64, 16, 3, 64, (0, 4, 4, 9)), (128, 64, 8, 0, (0, 1, 2, 3)),
                                           (64, 32, 5, 32, (3, 4, 6, 9)), (128, 16, 2, 128, (13, 13, 13, 13)),
                                           (64, 16, 4, 16, (0, 0, 0, 0))])
def test_tokens_that_no_sequence_covers_are_padding(D, P, QH, rot, cu):
    """They append nothing, their queries are zeros and their attention rows are empty; the others are as without them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    n, lo, hi = 13, cu[0], cu[-1]
    lens = ints(*(20 + b - a for a, b in zip(cu, cu[1:])))
    qkv = torch.randn(n, QH + 2, D, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([QH, 1, 1], 1)
    rope = torch.randn(40, rot, generator=g, device="cuda") if rot else None
    table = torch.arange(3 * 4, dtype=torch.int32, device="cuda").view(3, 4)
    caches = []
    for _ in range(2):
        c = ep.new_kv_cache(12, 1, P, D, table)
        c.k.fill_(0x38), c.v.fill_(0x30), c.k_scale.fill_(0.125), c.v_scale.fill_(0.125)
        caches.append(c)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    G = QH + QH % 2  # (in place: a strided slice whose other heads stay)
    out = torch.full((n, G, D), 9.0, dtype=torch.bfloat16, device="cuda")
    ep.kv_append(k, v, caches[0], lens, cu_tokens=ints(*cu), rope=rope, q=q, q_out=out[:, :QH], status=st)
    assert not out[:lo, :QH].any() and not out[hi:, :QH].any() and (out[:, QH:] == 9.0).all()
    if hi > lo:
        want = ep.kv_append(k[lo:hi], v[lo:hi], caches[1], lens, cu_tokens=ints(*(x - lo for x in cu)), rope=rope,
                            q=q[lo:hi])
        assert torch.equal(out[lo:hi, :QH], want)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    o, lse = ep.kv_attention(out[:, :QH], caches[0], lens, cu_tokens=ints(*cu), return_lse=True, status=st)
    inside = np.zeros(n, bool)
    inside[lo:hi] = True
    inside = torch.from_numpy(inside).cuda()
    assert not o[~inside].any() and torch.isneginf(lse[~inside]).all() and torch.isfinite(lse[inside]).all()
    assert int(st.item()) == 0
