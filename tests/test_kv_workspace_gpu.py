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
