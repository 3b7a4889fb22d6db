"""The products around the attention of DecodeAttention."""
import pytest
import torch

from tests import decode_reference as ref
from tests.test_decode_step_gpu import i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weights(bs, N, K, gen):
    codes, sf, _ = bs.q4_quantize((torch.randn(N, K, device=DEV, generator=gen) * 0.05).to(torch.bfloat16))
    return codes, sf


def off(y, x, w, scale=1.0):
    """Largest |y - x W^T| over its bound: fp32 sums over K, terms of x below 2^-29 of the row's largest, bf16 output."""
    N, K = w[0].shape[0], w[0].shape[1] * 2
    W = ref.fp4_weights(*w[:2], N, K).to(DEV) * scale
    want, S = x.double() @ W.T, x.double().abs() @ W.abs().T
    low = 2.0 ** -39 * K * x.double().abs().amax(1, keepdim=True) * W.abs().amax(1)[None]
    bound = (K + 8) * 2.0 ** -24 * S + low + 2.0 ** -8 * want.abs()
    return float(((y.double() - want).abs() / bound).max())


@pytest.mark.parametrize("T", [1, 16, 17, 45])
@pytest.mark.parametrize("N,K", [(320, 192), (129, 256)])
def test_any_number_of_columns(cuda_lib, T, N, K):
    """Weights whose rows are no multiple of 128, for any number of tokens."""
    from fp8_quantized_gemm_q4_gb300.decode import fp4_linear
    gen = torch.Generator(device=DEV).manual_seed(T + N)
    w = weights(cuda_lib, N, K, gen)
    x = torch.randn(T, K, device=DEV, generator=gen).to(torch.bfloat16)
    assert off(fp4_linear(x, *w), x, w) <= 1
    out = torch.full((T, N), 9.0, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(fp4_linear(x, *w, out=out), fp4_linear(x, *w)) and bool((out != 9.0).any())


def test_layer_of_odd_width(cuda_lib):
    """An odd number of heads of 64 and a hidden size of 192: prompts and single tokens."""
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    gen = torch.Generator(device=DEV).manual_seed(1)
    Hq, Hkv, D, hidden = 3, 1, 64, 192
    a = DecodeAttention(weights(bs, (Hq + 2 * Hkv) * D, hidden, gen), weights(bs, hidden, Hq * D, gen), Hq, Hkv, D, 2, 8,
                        16, 4)
    bs.clear_device_status()
    prompt = torch.randn(50, hidden, device=DEV, generator=gen).to(torch.bfloat16)
    y = a.step(prompt, i32([30, 20]), 30)
    assert y.shape == (50, hidden) and bool(y.isfinite().all()) and a.lens.tolist() == [30, 20]
    y = a.step(prompt[:2], i32([1, 1]), 1)
    assert bool(y.isfinite().all()) and a.lens.tolist() == [31, 21] and bs.device_status()[0] == bs.BS_OK


def test_two_level_weights(cuda_lib):
    """Weights of q4_quantize_two_level, as it returns them, for few and many tokens and in a layer."""
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention, fp4_linear
    gen = torch.Generator(device=DEV).manual_seed(2)
    Hq, Hkv, D, hidden = 4, 2, 64, 256
    raw = [(torch.randn(n, k, device=DEV, generator=gen) * 2.0 ** -9).to(torch.bfloat16)
           for n, k in (((Hq + 2 * Hkv) * D, hidden), (hidden, Hq * D))]
    two = [bs.q4_quantize_two_level(w) for w in raw]
    x = torch.randn(40, hidden, device=DEV, generator=gen).to(torch.bfloat16)
    codes, sf, ts = two[0]
    assert float(ts) != 1.0
    assert off(fp4_linear(x[:9], codes, sf, tensor_scale=ts), x[:9], two[0], float(ts)) <= 1
    # a power of two on the product is exact: few tokens and many against the same without it
    for n in (9, 40):
        plain = fp4_linear(x[:n], codes, sf)
        assert torch.equal(fp4_linear(x[:n], codes, sf, tensor_scale=ts), plain * ts.to(torch.bfloat16))
    a = DecodeAttention(*two, Hq, Hkv, D, 2, 12, 16, 6)
    bs.clear_device_status()
    y = a.step(x[:13], i32([9, 4]), 9)
    q, k, v = fp4_linear(x[:13], codes, sf, tensor_scale=ts).split([Hq * D, Hkv * D, Hkv * D], 1)
    table = ref.e4m3_table().to(DEV)
    kk, vv = (table[c.long()] * s.double()[..., None, None] for c, s in ((a.cache.k, a.cache.k_scale), (a.cache.v, a.cache.v_scale)))
    o, _, A, S = ref.attention(q.reshape(13, Hq, D).double(), kk, vv, a.table.tolist(), [0, 9, 13], [9, 4], 16, D ** -0.5)
    do = 2.0 ** -8 * o.abs() + (2.0 ** -11 + (D + 16) * 2.0 ** -23 * S[..., None]) * A + 9 * 2.0 ** -25 * 448 * float(a.cache.v_scale.max())
    W = ref.fp4_weights(*two[1][:2], hidden, Hq * D).to(DEV) * float(two[1][2])
    o, do = o.reshape(13, -1), do.reshape(13, -1)
    bound = (do + (Hq * D + 8) * 2.0 ** -24 * (o.abs() + do)) @ W.abs().T * (1 + 2.0 ** -8) + 2.0 ** -8 * (o @ W.T).abs() + 1e-30
    assert bool(((y.double() - o @ W.T).abs() <= bound).all())
    y = a.step(x, i32([20, 20]), 20)     # more than 16 tokens
    assert bool(y.isfinite().all()) and a.lens.tolist() == [29, 24] and bs.device_status()[0] == bs.BS_OK


@pytest.mark.parametrize("N,K", [(512, 256), (1024, 4160)])
def test_activations(cuda_lib, N, K):
    """Which rows of x are quantized is the caller's choice: "bf16" and "fp4" give a
    row the same result among few rows and many, "auto" is the one up to 16 rows and the
    other from 17 on, and those differ by far more than either's own error."""
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import fp4_linear
    gen = torch.Generator(device=DEV).manual_seed(N)
    w = weights(bs, N, K, gen)
    x = torch.randn(40, K, device=DEV, generator=gen).to(torch.bfloat16)
    xc, xsf, _ = bs.q4_quantize(x)
    rounded = ref.fp4_weights(xc, xsf, 40, K).to(DEV)
    full = {mode: fp4_linear(x, *w, activations=mode) for mode in ("bf16", "fp4", "auto")}
    assert off(full["bf16"], x, w) <= 1 and off(full["fp4"], rounded, w) <= 1
    assert off(full["fp4"], x, w) > 10 and torch.equal(full["auto"], full["fp4"])
    for n in (1, 3, 8, 16, 17, 33):
        assert torch.equal(fp4_linear(x[:n], *w, activations="bf16"), full["bf16"][:n])
        assert off(fp4_linear(x[:n], *w, activations="fp4"), rounded[:n], w) <= 1
        assert torch.equal(fp4_linear(x[:n], *w), fp4_linear(x[:n], *w, activations="bf16" if n <= 16 else "fp4"))


def test_a_token_alone_and_in_a_batch(cuda_lib):
    """With bf16 activations, the step of request 0 is the same whether two requests run or 20."""
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    gen = torch.Generator(device=DEV).manual_seed(4)
    Hq, Hkv, D, hidden = 8, 2, 64, 256
    w = weights(bs, (Hq + 2 * Hkv) * D, hidden, gen), weights(bs, hidden, Hq * D, gen)
    prompt = torch.randn(20, 5, hidden, device=DEV, generator=gen).to(torch.bfloat16)
    caches = []
    for B in (2, 20):
        a = DecodeAttention(*w, Hq, Hkv, D, B, 64, 16, 3, activations="bf16")
        a.step(prompt[:B].reshape(-1, hidden), i32([5] * B), 5)
        a.step(prompt[:B, 0], i32([1] * B), 1)
        caches.append([(c[int(a.table[0, 0])], s[int(a.table[0, 0])]) for c, s in ((a.cache.k, a.cache.k_scale), (a.cache.v, a.cache.v_scale))])
    for (c0, s0), (c1, s1) in zip(*caches):
        assert torch.equal(c0, c1) and torch.equal(s0, s1)


def test_refusals(cuda_lib):
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention, fp4_linear
    gen = torch.Generator(device=DEV).manual_seed(5)
    w = weights(bs, 320, 192, gen)
    x = torch.zeros(3, 192, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        fp4_linear(x, *w, activations="fp4")
    with pytest.raises(ValueError):
        fp4_linear(x, *w, activations="fp8")
    for mode in ("fp4", "bf8"):
        with pytest.raises(ValueError):
            DecodeAttention(w, weights(bs, 192, 192, gen), 3, 1, 64, 2, 8, 16, 4, activations=mode)
