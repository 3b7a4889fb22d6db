"""The decode step (plan, projections, append, attention) as a user runs it.

Attention over the step's own cache has the bound of its kernel (weights rounded
to fp16, output to bf16); the output projection multiplies that error by
|W_out| and adds its own fp32 accumulation and bf16 rounding:
    |y - ref| <= |W| (2^-8 |o| + (2^-11 + 2 e) A + m 2^-25 vmax)
                 + (K + 8) 2^-24 |W| |o| + 2^-8 |y|."""
import pytest
import torch

from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
HID, HQ, HKV, D, PAGE = 256, 8, 2, 64, 16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def weights(bs, rows, cols, gen):
    codes, sf, _ = bs.q4_quantize((torch.randn(rows, cols, device=DEV, generator=gen) * 0.05).to(torch.bfloat16))
    return codes, sf


def layer(bs, requests=3, pages=12):
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    gen = torch.Generator(device=DEV).manual_seed(5)
    w_qkv = weights(bs, (HQ + 2 * HKV) * D, HID, gen)
    w_out = weights(bs, HID, HQ * D, gen)
    return DecodeAttention(w_qkv, w_out, HQ, HKV, D, requests, pages, PAGE, 6), gen


def tokens(n, gen):
    return torch.randn(n, HID, device=DEV, generator=gen).to(torch.bfloat16)


def reference(bs, a, x, new):
    """The step in 64 bits from the cache that it left, and its bound."""
    T = x.shape[0]
    from fp8_quantized_gemm_q4_gb300.decode import fp4_linear
    q = fp4_linear(x, *a.w_qkv)[:, :HQ * D].reshape(T, HQ, D).double()
    table = ref.e4m3_table().to(DEV)
    k = table[a.cache.k.long()] * a.cache.k_scale.double()[..., None, None]
    v = table[a.cache.v.long()] * a.cache.v_scale.double()[..., None, None]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    lens = [m if n else 0 for m, n in zip(a.lens.tolist(), new)]
    o, _, A, S = ref.attention(q, k, v, a.table.tolist(), cu, lens, PAGE, D ** -0.5)
    e = (D + 16) * 2.0 ** -24 * S[..., None]
    do = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * e) * A + max(lens) * 2.0 ** -25 * 448 * float(a.cache.v_scale.max())
    W = ref.fp4_weights(*a.w_out, HID, HQ * D).to(DEV)
    o, do = o.reshape(T, -1), do.reshape(T, -1)
    y = o @ W.T
    bound = (do + (HQ * D + 8) * 2.0 ** -24 * (o.abs() + do)) @ W.abs().T
    return y, bound * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs() + 1e-30


def check(bs, a, x, new, got):
    want, bound = reference(bs, a, x, new)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def test_requests_come_and_go(cuda_lib):
    """Prompts of different lengths, single tokens, a request that ends and one
    that takes its place."""
    bs = cuda_lib
    bs.clear_device_status()
    a, gen = layer(bs)
    for new in ([1, 16 - 2, 1], [1, 1, 1], [0, 3, 1]):   # at most 16 tokens: activations in bf16 all the way
        x = tokens(sum(new), gen)
        check(bs, a, x, new, a.step(x, i32(new), max(new)))
    assert a.lens.tolist() == [2, 18, 3] and int(a.n_free) == 12 - 4
    a.release(i32([0, 1, 0]))
    assert a.lens.tolist() == [2, 0, 3] and int(a.n_free) == 12 - 2
    for new in ([1, 5, 1], [1, 1, 1]):
        x = tokens(sum(new), gen)
        check(bs, a, x, new, a.step(x, i32(new), max(new)))
    assert bs.device_status()[0] == bs.BS_OK


def test_same_as_the_calls_and_as_its_graph(cuda_lib):
    bs = cuda_lib
    a, gen = layer(bs)
    b, _ = layer(bs)
    x0, x1, new = tokens(45, gen), tokens(3, gen), i32([1, 1, 1])
    y0 = a.step(x0, i32([20, 5, 20]), 20)
    assert torch.equal(b.step(x0, i32([20, 5, 20]), 20), y0)
    # one call after the other
    y1 = a.step(x1, new, 1)
    cu, kv, slots, left = bs.kv_plan(b.lens, new, b.table, b.free, b.n_free, PAGE, 3)
    qkv = bs.matvec_fp4(x1, *b.w_qkv)
    q, k, v = (t.contiguous() for t in qkv.view(3, HQ + 2 * HKV, D).split([HQ, HKV, HKV], 1))
    bs.kv_append(k, v, slots, b.cache)
    y = bs.matvec_fp4(bs.kv_attention(q, b.cache, b.table, cu, kv, 1).view(3, -1), *b.w_out)
    assert torch.equal(y, y1) and torch.equal(kv, a.lens)
    assert all(torch.equal(s, t) for s, t in zip(a.cache, b.cache))
    # the same step captured and replayed: lengths go on by one a replay
    b.n_free.copy_(left)
    b.lens.copy_(kv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, _ = layer(bs)
    with torch.cuda.stream(side):
        c.step(x1, new, 1)   # the stream's workspace, before the capture
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = b.step(x1, new, 1)
    for _ in range(4):
        g.replay()
        want = a.step(x1, new, 1)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(a.lens, b.lens)


def test_pages_run_out(cuda_lib):
    bs = cuda_lib
    a, gen = layer(bs, pages=2)
    x = tokens(12, gen)
    bs.clear_device_status()
    y = a.step(x, i32([5, 4, 3]), 5)
    assert bs.device_status()[0] == bs.BS_ERR_PAGES
    bs.clear_device_status()
    assert a.lens.tolist() == [5, 4, 0] and int(a.n_free) == 0
    assert bool((y[9:] == 0).all()) and bool((y[:9] != 0).any(1).all())


def test_refusals(cuda_lib):
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    a, gen = layer(bs)
    with pytest.raises(ValueError):
        DecodeAttention(a.w_qkv, a.w_out, HQ, HKV, 128, 3, 12, PAGE, 6)
    with pytest.raises(ValueError):
        a.step(tokens(2, gen), i32([1, 1]), 1)   # two lengths for three requests
