"""Tensors that are not on the GPU are refused by the binding of the decode-step
calls, before anything asks for a stream (no GPU needed: the stream is stood in
for, and a call that went on would reach the stand-in)."""
import pytest
import torch


@pytest.fixture
def bs(monkeypatch):
    import fp8_quantized_gemm_q4_gb300 as bs

    def reached(stream=None):
        raise AssertionError("the call went on to the library")

    monkeypatch.setattr(bs, "_stream", reached)
    monkeypatch.setattr(bs, "_lib", object())
    return bs


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_host_tensors(bs):
    c = bs.KVCache.empty(4, 2, 16, 64, device="cpu")
    x, q = torch.zeros(3, 2, 64), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    w, sf, xb = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.zeros(2, 64).bfloat16()
    for call in (lambda: bs.kv_plan(i32(2), i32(2), i32(2, 3), i32(9), i32(1), 16, 4),
                 lambda: bs.kv_release(i32(2), i32(2), i32(2, 3), i32(9), i32(1), 16),
                 lambda: bs.kv_append(x, x, i32(3), c),
                 lambda: bs.kv_attention(q, c, i32(1, 4), i32(2), i32(1), 3),
                 lambda: bs.matvec_fp4(xb, w, sf),
                 lambda: bs.matvec_fp4(xb, w, sf, out_dtype=torch.float32, bias=torch.zeros(8).bfloat16())):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_one_host_tensor_among_others(cuda_lib, bs):
    """Each argument in turn left on the host."""
    dev = "cuda"
    c = bs.KVCache.empty(4, 2, 16, 64)
    k = torch.zeros(3, 2, 64, device=dev)
    q, lse = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=dev), torch.zeros(3, 4, device=dev)
    w, sf = torch.zeros(8, 32, dtype=torch.uint8, device=dev), torch.zeros(512, dtype=torch.uint8, device=dev)
    xb, b, ts = torch.zeros(2, 64, device=dev).bfloat16(), torch.zeros(8, device=dev).bfloat16(), torch.ones(1, device=dev)
    n = lambda *shape: i32(*shape).to(dev)
    plan_out = (n(3), n(2), n(4), n(1))
    calls = [(lambda *a: bs.kv_plan(*a[:5], 16, 4, out=a[5:]), [n(2), n(2), n(2, 3), n(9), n(1), *plan_out]),
             (lambda *a: bs.kv_release(*a, 16), [n(2), n(2), n(2, 3), n(9), n(1)]),
             (lambda k, v, s, *c: bs.kv_append(k, v, s, c), [k, k.clone(), n(3), *c]),
             (lambda q, t, cu, kv, out, lse, ws, *c: bs.kv_attention(q, c, t, cu, kv, 3, out=out, lse=lse, workspace=ws),
              [q, n(1, 4), n(2), n(1), q.clone(), lse, w.new_zeros(64), *c]),
             (lambda x, w, s, b, ts, out: bs.matvec_fp4(x, w, s, bias=b, tensor_scale=ts, out=out),
              [xb, w, sf, b, ts, torch.zeros(2, 8, device=dev)])]
    for f, args in calls:
        for i in range(len(args)):
            a = list(args)
            a[i] = a[i].cpu()
            with pytest.raises(ValueError, match="GPU"):
                f(*a)
