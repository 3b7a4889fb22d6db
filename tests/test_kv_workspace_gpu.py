"""The scratch of kv_attention as the binding keeps it: its size, its life, and
calls captured in CUDA graphs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def case(bs, kv_lens, q_lens, Hq=16, Hkv=4, D=128, page=64, seed=0):
    """Arguments of kv_attention for requests with these lengths, each with pages of its own."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pages = [-(-m // page) for m in kv_lens]
    cache = bs.KVCache.empty(sum(pages), Hkv, page, D)
    for codes in (cache.k, cache.v):
        codes.copy_(torch.randn(codes.shape, device=DEV, generator=gen).to(torch.float8_e4m3fn).view(torch.uint8))
    table, at = [], 0
    for n in pages:
        table.append(list(range(at, at + n)) + [-1] * (max(pages) - n))
        at += n
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], Hq, D), device=DEV, generator=gen).to(torch.bfloat16)
    return q, cache, i32(table), i32(cu), i32(kv_lens), max(q_lens)


def test_a_refused_call_leaves_later_ones_alone(cuda_lib, monkeypatch):
    """A call without heads is turned away; the next valid one, of the same head size, is served."""
    bs = cuda_lib
    for name in ("_kv_workspace_bytes", "_kv_workspace_sizes"):   # as in a new process
        if isinstance(getattr(bs, name, None), dict):
            monkeypatch.setattr(bs, name, {})
    q, cache, table, cu, kv, most = case(bs, [300, 70], [1, 1])
    with pytest.raises(bs.BSError):
        bs.kv_attention(q[:, :0], cache, table, cu, kv, most)
    out = bs.kv_attention(q, cache, table, cu, kv, most)
    assert bool((out != 0).any())


@pytest.mark.parametrize("D", [64, 128])
def test_one_size_serves_every_call(cuda_lib, D):
    """What the binding keeps is at least what the library asks for, for few and many rows, short and long calls."""
    bs = cuda_lib
    lib = bs.load()
    q, cache, table, cu, kv, most = case(bs, [300, 70], [1, 1], D=D)
    bs.kv_attention(q, cache, table, cu, kv, most)
    kept = bs._kv_workspace_sizes[(q.get_device(), D)]
    for T, Hq, Hkv, most in ((1, 8, 8, 1), (64, 32, 8, 1), (4096, 32, 8, 4096), (5000, 64, 1, 3), (300, 8, 1, 300)):
        a = bs._KV_ATTENTION_ARGS.pack(*(0,) * 19, T, Hq, Hkv, D, most, *(0,) * 4)
        assert 0 < int(lib.bs_kv_attention_workspace_bytes(a)) <= kept


def graph_of(call, stream):
    g = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=stream):
        out = call()
    return g, out


def test_replay_after_the_buffer_grew(cuda_lib, monkeypatch):
    """Captured with the stream's buffer, which a later call then replaces by a
    larger one; memory allocated since is filled with junk before the replays."""
    bs = cuda_lib
    monkeypatch.setattr(bs, "_workspaces", {})
    side = torch.cuda.Stream()
    small, large = case(bs, [5000, 900], [1, 1], D=64), case(bs, [3000, 700], [150, 90])
    want = bs.kv_attention(*small).clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        bs.kv_attention(*small)
    g, out = graph_of(lambda: bs.kv_attention(*small), side)
    before = bs._workspaces[(out.get_device(), side.cuda_stream)]
    with torch.cuda.stream(side):
        wide = bs.kv_attention(*large)
    torch.cuda.synchronize()
    assert bs._workspaces[(out.get_device(), side.cuda_stream)] is not before
    del before
    junk = [torch.full((1 << 20,), 0x5a, dtype=torch.uint8, device=DEV) for _ in range(64)]
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((x == 0x5a).all()) for x in junk)
    assert torch.equal(wide, bs.kv_attention(*large))


def test_capture_without_a_first_call(cuda_lib, monkeypatch):
    """Two graphs captured on a stream that has no buffer yet, the second replayed
    first, with calls on the stream between them."""
    bs = cuda_lib
    monkeypatch.setattr(bs, "_workspaces", {})
    side = torch.cuda.Stream()
    few, many = case(bs, [5000, 900], [1, 1]), case(bs, [3000, 700], [150, 90])
    want = [bs.kv_attention(*few).clone(), bs.kv_attention(*many).clone()]
    torch.cuda.synchronize()
    g0, out0 = graph_of(lambda: [bs.kv_attention(*few), bs.kv_attention(*few)], side)
    g1, out1 = graph_of(lambda: bs.kv_attention(*many), side)
    with torch.cuda.stream(side):
        eager = bs.kv_attention(*few)
    torch.cuda.synchronize()
    assert torch.equal(eager, want[0])
    for g in (g1, g0, g0, g1, g0):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[0]) for o in out0) or g is g1
        assert torch.equal(out1, want[1])
