"""Tensors that a call on a named stream takes: the stream's work may read them
after their last reference is gone, so their memory stays theirs until then."""
import contextlib
import types

import pytest
import torch

import bit_level_weight_gb300 as cas


class Recorded(torch.Tensor):
    """A CPU tensor that says it is a device tensor and notes the streams that it is told of."""
    is_cuda = True

    def record_stream(self, stream):
        self.streams = getattr(self, "streams", []) + [stream]


def test_arguments_are_recorded_on_the_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    a, b, c = (torch.zeros(3).as_subclass(Recorded) for _ in range(3))
    st = types.SimpleNamespace(device=a.device)
    seen = []
    cas._with_stream(st, a, lambda *args: seen.append(args), a, None, 3, b, 1.5)
    assert seen == [(a, None, 3, b, 1.5)]
    assert a.streams == [st] and b.streams == [st] and not hasattr(c, "streams")


def test_arguments_of_a_refused_stream_are_left_alone():
    a = torch.zeros(3).as_subclass(Recorded)
    with pytest.raises(ValueError, match="device"):
        cas._with_stream(types.SimpleNamespace(device=torch.device("meta")), a, None, a)
    assert not hasattr(a, "streams")


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["rules", "append", "plan"])
def test_memory_of_dropped_arguments_is_not_reused_under_a_call(which):
    """A call waits behind other work of its stream while its arguments are
    dropped: new tensors of their size lie elsewhere until it is through."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_level_weight_gb300 import build
    build.build()
    dev, n = "cuda", 3 << 20  # sizes of blocks that hold nothing else
    make = {"rules": lambda: torch.zeros(1, 1, n, device=dev), "append": lambda: torch.zeros(n // 512, 512, device=dev),
            "plan": lambda: torch.zeros(n, dtype=torch.int32, device=dev)}[which]
    cache = cas.paged4_cache(3, 16, 1)
    few = [torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev),
           torch.zeros(1, 3, dtype=torch.int32, device=dev)]
    more = [torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(2)]
    call = {"rules": lambda t, st: cas.adjust_logits(t, stream=st),
            "append": lambda t, st: cas.paged4_append(t, 2, cache, *few, stream=st),
            "plan": lambda t, st: cas.paged_plan(few[2], few[1], t, more[0], 16, more[1], 4, stream=st)}[which]
    call(make(), torch.cuda.current_stream())  # (the library is loaded, memory is there)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    t = make()
    at = t.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(400_000_000)  # a fifth of a second
    out = call(t, st)
    del t
    assert not st.query()  # (the call has not begun)
    assert make().data_ptr() != at
    st.synchronize()
    del out
    again = [make() for _ in range(4)]  # behind the call the memory is free again
    assert at in [x.data_ptr() for x in again]


@pytest.mark.gpu
def test_a_call_on_a_named_stream_is_captured():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_level_weight_gb300 import build
    build.build()
    x = torch.randn(3, 1, 5000, device="cuda")
    bias = (torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda"), torch.tensor([7, 4000], dtype=torch.int32, device="cuda"),
            torch.tensor([2.0, float("-inf")], device="cuda"))
    want = cas.adjust_logits(x, bias_start=bias[0], bias_token=bias[1], bias_value=bias[2])
    out, st, graph = torch.zeros_like(x), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        cas.adjust_logits(x, bias_start=bias[0], bias_token=bias[1], bias_value=bias[2], out=out, stream=st)
    assert not out.any()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.isneginf(out[2, 0, 4000]) and out[0, 0, 7] == x[0, 0, 7] + 2
