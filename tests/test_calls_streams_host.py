"""Every page-level call hands its whole self over to the stream that it is given (host)."""
import inspect

import pytest

import combine_ep_get_dispatch_gb300 as ep

CALLS = [ep.get_dispatch_layout, ep.dispatch, ep.get_layout_and_dispatch, ep.combine, ep.dispatch_backward,
         ep.combine_backward, ep.combine_two_level, ep.low_latency_dispatch, ep.low_latency_combine,
         ep.low_latency_query_mask_buffer, ep.kv_append, ep.kv_attention, ep.expert_linear]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_the_whole_call_goes_to_its_stream(call, monkeypatch):
    seen = []

    def on_stream(stream, f, *args):
        seen.append((stream, f, args))
        return ("first", "second")
    monkeypatch.setattr(ep, "_on_stream", on_stream)
    sig = inspect.signature(call)
    given = {name: object() for name in sig.parameters}
    result = call(**given)
    (stream, f, args), = seen
    assert stream is given.pop("stream") and f is call
    bound = sig.bind(*args).arguments
    assert bound.pop("stream", None) is None
    assert bound == given
    # a phase that is launched later goes there as well
    if call in (ep.low_latency_dispatch, ep.low_latency_combine):
        assert result[0] == "first"
        result[1]()
        assert seen[1] == (stream, "second", ())


def test_parts_of_a_result_are_found(monkeypatch):
    class T:
        def __init__(self):
            self.on = []

        def record_stream(self, s):
            self.on.append(s)
    t = [T() for _ in range(6)]
    ep._record(((t[0], t[1]), None, ep.DispatchResult(rank_x=t[2], expert_src=t[3]),
                ep.LLHandle(t[4], 1, 2, 3, 4, 5, 6, t[5], None), lambda: None), "stream")
    assert all(x.on == ["stream"] for x in t)
