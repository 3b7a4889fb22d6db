"""Life of the scratch buffers that the binding keeps per stream (no GPU: the
stream calls are stood in for)."""
import contextlib
import gc
import types
import weakref

import pytest
import torch


@pytest.fixture
def bs(monkeypatch):
    import fp8_quantized_gemm_q4_gb300 as bs
    state = types.SimpleNamespace(capturing=False)
    monkeypatch.setattr(bs, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    return types.SimpleNamespace(state=state, get=lambda n: bs._workspace_of(torch.device("cpu"), 7, n))


def test_kept_and_shared(bs):
    a = bs.get(1000)
    assert a.numel() >= 1000 and not a.any()
    assert bs.get(500) is a and bs.get(1000) is a


def test_an_outgrown_buffer_stays(bs):
    """A graph captured with it may still be replayed."""
    held = weakref.ref(bs.get(1000))
    assert bs.get(3000).numel() >= 3000
    gc.collect()
    assert held() is not None


def test_growth_is_bounded(bs):
    """Ever larger calls, each a little above the last, take at most twice the largest in all."""
    seen = []
    for n in range(1000, 60000, 100):
        ws = bs.get(n)
        if not any(ws is x for x in seen):
            seen.append(ws)
    assert sum(x.numel() for x in seen) <= 2 * seen[-1].numel() <= 4 * 60000


def test_made_in_a_capture(bs):
    """Zeroed only when the graph runs: nothing that another call may rely on."""
    bs.state.capturing = True
    a = bs.get(1000)
    bs.state.capturing = False
    b = bs.get(1000)
    assert b is not a
    bs.state.capturing = True
    assert bs.get(800) is b      # there before the capture, and zero
    c = bs.get(5000)
    bs.state.capturing = False
    assert c.numel() >= 5000 and bs.get(1000) is b


def test_stream_handle_without_the_raw_one(monkeypatch):
    """A torch without the function that gives the bare handle."""
    import fp8_quantized_gemm_q4_gb300 as bs
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(bs, "_raw_stream", None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=11))
    assert bs._stream() == 11
    assert bs._stream(types.SimpleNamespace(cuda_stream=5)) == 5
