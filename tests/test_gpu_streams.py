"""What a call allocates itself comes from the pool of the stream that it runs on.

The allocator hands a freed block on in the order of the stream it belongs to.  A call on another stream that
took its output or its workspace from the current stream's pool could write a block on which the current
stream's work is still queued.  No race is provoked here: the tests read which stream's pool a block is from."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


def pool_of(t):
    """The stream whose pool holds t's memory."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.fixture
def allocations(pkv, monkeypatch):
    """The streams that were current when the binding allocated something."""
    seen = []

    def spy(make):
        def made(*args, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return make(*args, **kw)
        return made

    class Torch:
        """torch, with the functions the binding allocates with recorded."""
        empty, empty_like = staticmethod(spy(torch.empty)), staticmethod(spy(torch.empty_like))

        def __getattr__(self, name):
            return getattr(torch, name)

    monkeypatch.setattr(pkv, "torch", Torch())
    return seen


def inputs():
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    b = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    codes = lambda: torch.zeros(3, 256, 8, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    scales = lambda: torch.full((3, 8, 256), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)  # noqa: E731
    return dict(q=b(2, 16, D), k=b(2, 8, D), v=b(2, 8, D), k16=b(3, 256, 8, D), v16=b(3, 256, 8, D), k8=codes(), v8=codes(),
                ks=scales(), vs=scales(), pos=i(4, 9), slots=i(4, 300), tables=i(0, 1).view(2, 1), lens=i(5, 45), cu_q=i(0, 1, 2),
                cu_k=i(0, 5, 50), x=torch.randn(2, 1000, device="cuda"), T=torch.ones(2, device="cuda"),
                so=torch.tensor([1, 2], device="cuda"))


CALLS_8_BIT = {
    "rope_store_fp8": lambda p, a, s: p.pkv_rope_store_kvcache_fp8(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["k8"], a["v8"], a["ks"],
                                                                   a["vs"], 1e4, stream=s),
    "decode_fp8": lambda p, a, s: p.pkv_decode_fp8(a["q"], a["k8"], a["v8"], a["ks"], a["vs"], a["tables"], a["lens"], 45, 0.1, stream=s),
    "prefill_fp8": lambda p, a, s: p.pkv_prefill_varlen_fp8(a["q"], a["k8"], a["v8"], a["ks"], a["vs"], a["cu_q"], a["cu_k"], a["tables"],
                                                            1, 45, 50, 0.1, stream=s),
    "sample_filtered": lambda p, a, s: p.pkv_sample_filtered(a["x"], a["T"], None, None, None, 1, stream=s),
    "sample_filtered_dev": lambda p, a, s: p.pkv_sample_filtered_dev(a["x"], a["T"], None, None, None, a["so"], stream=s),
}


def check_call(pkv, call, allocations, monkeypatch):
    a = inputs()
    ref = call(pkv, a, None)
    torch.cuda.synchronize()                              # the inputs are ready on any stream
    side = torch.cuda.Stream()
    held = []
    record = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: (held.append((t.data_ptr(), s.cuda_stream)), record(t, s))[1])
    allocations.clear()
    out = call(pkv, a, side)
    monkeypatch.undo()
    assert allocations and set(allocations) == {side.cuda_stream}
    assert pool_of(out) == side.cuda_stream
    # and the caller's stream, on which the result will be read, holds it after the caller lets go of it
    assert (out.data_ptr(), torch.cuda.current_stream().cuda_stream) in held
    side.synchronize()
    assert torch.equal(out, ref)
    same = call(pkv, a, torch.cuda.current_stream())      # the current stream, named
    assert pool_of(same) == torch.cuda.current_stream().cuda_stream and torch.equal(same, ref)


@pytest.mark.parametrize("name", CALLS_8_BIT)
def test_8_bit_and_filtered_calls_allocate_on_their_stream(pkv, name, allocations, monkeypatch):
    check_call(pkv, CALLS_8_BIT[name], allocations, monkeypatch)


CALLS = {
    "rope_store": lambda p, a, s: p.pkv_rope_store_kvcache(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["k16"], a["v16"], 1e4, stream=s),
    "decode": lambda p, a, s: p.pkv_decode(a["q"], a["k16"], a["v16"], a["tables"], a["lens"], 45, 0.1, stream=s),
    "decode_append": lambda p, a, s: p.pkv_decode_append(a["q"], a["k"], a["v"], a["k16"], a["v16"], a["tables"], a["lens"], 45, 0.1, stream=s),
    "prefill": lambda p, a, s: p.pkv_prefill_varlen(a["q"], a["k16"], a["v16"], a["cu_q"], a["cu_k"], a["tables"], 1, 45, 0.1, stream=s),
    "sample": lambda p, a, s: p.pkv_sample(a["x"], a["T"], 1, stream=s),
    "sample_dev": lambda p, a, s: p.pkv_sample_dev(a["x"], a["T"], a["so"], stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_bf16_cache_calls_allocate_on_their_stream(pkv, name, allocations, monkeypatch):
    check_call(pkv, CALLS[name], allocations, monkeypatch)


def test_plans_and_call_objects_allocate_on_their_stream(pkv, allocations):
    a = inputs()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = pkv.pkv_prefill_plan(a["cu_q"], a["cu_k"], 2, 1, 45, 16, 8, D, 256, 1, stream=side)
    assert pool_of(ws) == side.cuda_stream
    out = torch.empty_like(a["q"])
    torch.cuda.synchronize()
    allocations.clear()
    call = pkv.DecodeAppendCall(a["q"], a["k"], a["v"], a["k16"], a["v16"], a["tables"], a["lens"], 45, 0.1, out, stream=side)
    call()
    assert allocations and set(allocations) == {side.cuda_stream}
    side.synchronize()
    assert torch.equal(out, pkv.pkv_decode(a["q"], a["k16"], a["v16"], a["tables"], a["lens"], 45, 0.1))


def test_calls_on_a_forked_stream_are_captured(pkv):
    """A call on a stream that a capture has forked to, with everything it allocates."""
    a = inputs()
    for name, call in {**CALLS_8_BIT, **CALLS}.items():
        ref = call(pkv, a, None)
        torch.cuda.synchronize()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            out = call(pkv, a, side)
            torch.cuda.current_stream().wait_stream(side)
        out.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), name
        del graph
