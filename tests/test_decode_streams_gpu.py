"""Outputs that a serving call makes itself are of the stream that it is given: memory of the
current stream's may still be written to by what was started there before."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def calls(bs):
    """(call with a stream, an output's shape and type); outputs too large for memory that others share."""
    bf = torch.bfloat16
    T, D = 4096, 128
    q = torch.randn((T, 4, D), device=DEV).to(bf)
    k = torch.randn((T, 2, D), device=DEV).to(bf)
    lens, table = (i32([T]), i32([0]), i32([0, T])), torch.arange(T // 64, device=DEV, dtype=torch.int32)[None]
    for kind in (bs.KVCache, bs.KVCacheFP4):
        c = kind.empty(T // 64, 2, 64, D)
        bs.kv_append(k, k, torch.arange(T, device=DEV, dtype=torch.int32), c)
        yield lambda s, c=c: bs.kv_attention(q, c, table, lens[2], lens[0], T, stream=s), q.shape, bf
        angles = bs.rotary_angles(T, D)
        at = torch.arange(T, device=DEV, dtype=torch.int32)
        yield lambda s, c=c, a=angles, at=at: bs.kv_append_rotary(q, k, k, at, at, a, c, stream=s), q.shape, bf
        yield lambda s, c=c, at=at: bs.kv_gather(c, at, stream=s)[0], k.shape, bf
    n = 1 << 20
    yield lambda s: bs.kv_plan(lens[1], i32([0]), table.clone(), table[0].clone(), i32([64]), 64, n, stream=s)[2], (n,), torch.int32
    yield lambda s: bs.kv_positions(lens[1], i32([0, n]), n, stream=s), (n,), torch.int32
    x = torch.randn((16, 128), device=DEV).to(bf)
    codes, sf = torch.zeros((1 << 17, 64), device=DEV, dtype=torch.uint8), torch.zeros(1 << 20, device=DEV, dtype=torch.uint8)
    yield lambda s: bs.matvec_fp4(x, codes, sf, stream=s), (16, 1 << 17), bf
    y, a, b = (torch.randn(s, device=DEV).to(bf) for s in ((T, 512), (1, 8, 512), (1, 512, 8)))
    yield lambda s: bs.lora_add(y, y, a, b, i32([0, T]), i32([0]), stream=s), y.shape, bf


def test_outputs_are_of_the_stream_of_the_call(cuda_lib):
    """What the current stream has given back, and may still be at work on, is not taken for another stream's output."""
    bs = cuda_lib
    side = torch.cuda.Stream()
    for i, (call, shape, dt) in enumerate(calls(bs)):
        torch.cuda.synchronize()
        want = call(None)
        side.wait_stream(torch.cuda.current_stream())
        held = [torch.empty(shape, dtype=dt, device=DEV) for _ in range(4)]
        mine = {t.data_ptr() for t in held}
        del held
        got = call(side)
        assert got.data_ptr() not in mine, i
        side.synchronize()
        assert got.shape == tuple(shape) and torch.equal(got, want), i
    assert bs.device_status()[0] == bs.BS_OK
