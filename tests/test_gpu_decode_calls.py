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
