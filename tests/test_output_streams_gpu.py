"""Outputs and scratch that the quantizers', products' and MoE calls make themselves are of the
stream that the call is given (as test_decode_streams_gpu has it for the serving calls)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
M, N, K = 2048, 1024, 2048


def calls(bs):
    """(call with a stream, whose outputs are a tuple; the inputs that they are made from live on)."""
    x, w = torch.randn((M, K), device=DEV).bfloat16(), torch.randn((N, K), device=DEV).bfloat16()
    gather = torch.arange(M, device=DEV, dtype=torch.int32)
    (xc, xs, _), (wc, ws, _) = bs.q4_quantize(x), bs.q4_quantize(w)
    xs16 = bs.q4_quantize(x[:16])[1]
    (x8, s8), (w8, b8) = bs.q8_quantize(x), bs.q8_quantize(w, bs.Q8_BLOCK)
    logits = torch.randn((M, 64), device=DEV)
    ids, tw = bs.moe_router_topk(logits, 8)
    d = bs.moe_dispatch(ids, tw, 64)
    rows = torch.randn((bs.moe_rows_bound(M, 8, 64), 256), device=DEV)
    return [lambda s: bs.q4_quantize(x, stream=s)[:2], lambda s: bs.q4_quantize_two_level(x, stream=s),
            lambda s: (bs.tensor_amax(x, stream=s),), lambda s: bs.fp4_gather_rows(xc, xs, K, gather, stream=s),
            lambda s: bs.fp8_gather_rows(x8, s8, gather, stream=s), lambda s: bs.q8_quantize(x, stream=s),
            lambda s: (bs.gemm_fp4(xc, xs, wc, ws, K, stream=s),), lambda s: (bs.gemm_fp8(x8, s8, w8, b8, stream=s),),
            lambda s: tuple(bs.gemm_fp4_multi(xc[:16], xs16, [(wc, ws)] * 2, K, stream=s)),
            lambda s: bs.moe_router_topk(logits, 8, stream=s), lambda s: (bs.moe_dispatch(ids, tw, 64, stream=s)["counts"],),
            lambda s: (bs.moe_combine(rows, d["pair_of_row"], M, 8, stream=s),)]


def test_outputs_are_of_the_stream_of_the_call(cuda_lib):
    bs = cuda_lib
    side = torch.cuda.Stream()
    for i, call in enumerate(calls(bs)):
        want = call(None)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        held = [torch.empty_like(t) for t in want for _ in range(4)] + [torch.empty(1 << 20, device=DEV, dtype=torch.uint8)]
        mine = {t.data_ptr() for t in held}
        del held
        got = call(side)
        assert not mine & {t.data_ptr() for t in got}, i
        side.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, want)), i
    assert bs.device_status()[0] == bs.BS_OK
