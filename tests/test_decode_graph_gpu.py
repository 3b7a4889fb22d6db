"""A captured step of DecodeAttention among other steps."""
import pytest
import torch

from tests.test_decode_step_gpu import layer, tokens, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_captured_step_between_prompts(cuda_lib):
    """A one-token step captured on a stream that has run nothing, replayed after
    prompts on that stream and with junk in memory allocated since, against
    the same steps without a graph."""
    bs = cuda_lib
    (a, gen), (b, _) = layer(bs, pages=18), layer(bs, pages=18)
    x, one = tokens(3, gen), i32([1, 1, 1])
    side = torch.cuda.Stream()
    prompts = [(tokens(45, gen), [20, 5, 20]), (tokens(40, gen), [1, 38, 1])]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        out = b.step(x, one, 1)
    keep = []
    for p, new in prompts:
        want = a.step(p, i32(new), max(new))
        with torch.cuda.stream(side):
            got = b.step(p, i32(new), max(new))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        keep.append(torch.full((32 << 20,), 0x5a, dtype=torch.uint8, device=DEV))
        for _ in range(2):
            g.replay()
            want = a.step(x, one, 1)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(a.lens, b.lens)
            assert all(torch.equal(s, t) for s, t in zip(a.cache, b.cache))
    assert all(bool((k == 0x5a).all()) for k in keep)


def test_the_layer_owns_its_scratch(cuda_lib, monkeypatch):
    """Attention of a step does not touch the stream's buffer; a workspace given by hand must hold what is needed."""
    bs = cuda_lib
    monkeypatch.setattr(bs, "_workspaces", {})
    a, gen = layer(bs)
    a.step(tokens(12, gen), i32([5, 4, 3]), 5)
    assert not bs._workspaces
    q = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device=DEV)
    cu, kv = i32([0, 1]), i32([2])
    with pytest.raises(bs.BSError):
        bs.kv_attention(q, a.cache, a.table[:1], cu, kv, 1, workspace=a.workspace[:4096])
    with pytest.raises(TypeError):
        bs.kv_attention(q, a.cache, a.table[:1], cu, kv, 1, workspace=a.workspace.view(torch.int32))
    with pytest.raises(ValueError):
        bs.kv_attention_workspace(96)
