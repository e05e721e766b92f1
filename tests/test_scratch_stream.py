"""A workspace that a call makes for itself comes from the memory of the stream
that the call runs on.  From the current stream's it would be handed out again,
and written, while the kernels on the other stream still read it (CPU)."""
import contextlib

import pytest
import torch

import paged_kv_cache_69_gb300 as pa

from test_binding_host import _decode_inputs, _pool, rec  # noqa: F401  (the recording stand-in)


class _Stream:
    cuda_stream = 77


def _calls():
    k, v = _pool()
    q, out, bt, sl = _decode_inputs()
    w = torch.zeros(10, 2, 16)
    return {
        "decode": lambda **kw: pa.pa_decode(out, q, k, v, bt, sl, 0.1, **kw),
        "attention": lambda **kw: pa.pa_attention(out, q, k, v, bt, sl, torch.arange(4, dtype=torch.int32), 0.1, 1, **kw),
        "weights": lambda **kw: pa.pa_decode_weights(out, w, q, k, v, bt, sl, 0.1, **kw),
        "evict": lambda **kw: pa.pa_evict(k, v, w, bt, sl, sl, 32, **kw),
    }


@pytest.mark.parametrize("name", ["decode", "attention", "weights", "evict"])
@pytest.mark.parametrize("given", ["none", "stream", "handle", "default"])
def test_scratch_is_allocated_on_the_calls_stream(rec, monkeypatch, name, given):  # noqa: F811
    current, seen = [None], []

    @contextlib.contextmanager
    def on(stream):
        current[0] = stream
        yield
        current[0] = None

    empty = torch.empty

    def watched(*a, **kw):
        seen.append(current[0])
        return empty(*a, **kw)

    external, default, stream = object(), object(), _Stream()
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: external if h == 55 else None)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: default)
    call = _calls()[name]
    monkeypatch.setattr(torch, "empty", watched)
    arg = {"none": None, "stream": stream, "handle": 55, "default": 0}[given]
    call(stream=arg)
    assert seen == [{"none": None, "stream": stream, "handle": external, "default": default}[given]]
    call(stream=arg, workspace=torch.zeros(4096, dtype=torch.uint8))
    assert len(seen) == 1


@pytest.mark.parametrize("name", ["decode", "attention", "weights", "evict"])
def test_bounds_that_give_no_workspace_are_refused(rec, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(type(rec), "__getattr__", lambda self, n: lambda *a: b"" if "string" in n else 0)
    with pytest.raises(pa.PaError):
        _calls()[name]()


@pytest.mark.gpu
def test_memory_of_a_busy_stream_is_not_handed_out():
    """Tensors made on the current stream while the call waits on another one."""
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(300, 16, 2, 128, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(3, 8, 128, generator=g).half().cuda()
    bt = torch.arange(300, dtype=torch.int32, device="cuda").view(3, 100)
    sl = torch.tensor([1600, 900, 1500], dtype=torch.int32, device="cuda")
    n = pa.pa_decode_workspace_size(3, 8, 1600, 128)
    ref, out = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode(ref, q, k, v, bt, sl, 0.09)
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        busy = s if isinstance(s, torch.cuda.Stream) else torch.cuda.ExternalStream(s)
        torch.cuda.synchronize()
        for _ in range(20):
            with torch.cuda.stream(busy):
                torch.cuda._sleep(200000)
            pa.pa_decode(out, q, k, v, bt, sl, 0.09, stream=s)
            [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
