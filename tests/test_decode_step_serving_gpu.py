"""The decode step with a rotation, a 4-bit cache and adapters, as a user runs it.

Attention over the step's own cache has the bound of its kernel; the output projection
multiplies that error by |W_out|, and its adapter's by |A| |B| (as in
test_decode_step_gpu, with the adapter's matrix beside the weight):
    |y - ref| <= (|W| + s |B| |A|) (2^-8 |o| + (2^-11 + 2 e) A + m 2^-25 vmax)
                 + (2^-16 + (K + 8) 2^-23) (|W| + s |B| |A|) |o| + 2^-7 |y|
(two roundings of y: the product's and the adapter's, the first on a part of it that may
be larger than the sum: 2^-8 of it is in the bound as well)."""
import pytest
import torch

from tests import decode_reference as ref
from tests import serving_reference as sref
from tests.test_decode_step_gpu import D, HID, HKV, HQ, PAGE, i32, tokens, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def adapters(gen, n, r, K, N):
    return ((torch.randn(n, r, K, device=DEV, generator=gen) * 0.05).to(torch.bfloat16),
            (torch.randn(n, N, r, device=DEV, generator=gen) * 0.05).to(torch.bfloat16),
            torch.rand(n, device=DEV, generator=gen) + 0.5)


def layer(bs, bits=4, rot=True, lora=True, mixed=False, requests=3, pages=12):
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    gen = torch.Generator(device=DEV).manual_seed(5)
    w_qkv = weights(bs, (HQ + 2 * HKV) * D, HID, gen)
    w_out = weights(bs, HID, HQ * D, gen)
    kw = dict(lora_qkv=adapters(gen, 2, 16, HID, (HQ + 2 * HKV) * D), lora_out=adapters(gen, 2, 8, HQ * D, HID)) if lora else {}
    a = DecodeAttention(w_qkv, w_out, HQ, HKV, D, requests, pages, PAGE, 6, cache_bits=bits, interleaved=mixed,
                        angles=bs.rotary_angles(6 * PAGE, 32) if rot else None, **kw)
    a.which.copy_(i32([1, -1, 0][:requests]))
    return a, gen


def reference(bs, a, x, new, before):
    """The step in 64 bits from the cache that it left (whose new rows are checked apart), and its bound."""
    from fp8_quantized_gemm_q4_gb300.decode import fp4_linear
    T = x.shape[0]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    which = a.which.tolist()
    qkv = fp4_linear(x, *a.w_qkv)
    if a.lora_qkv:      # the kernel's own, which test_lora_gpu holds to its bound: what follows depends on its rounding
        la, lb, ls = a.lora_qkv
        want, size = sref.lora(x, qkv, la, lb, cu, which, ls)
        got = bs.lora_add(x, qkv, la, lb, i32(cu), a.which, scales=ls)
        assert bool(((got.double() - want).abs() <= 2.0 ** -15 * size + 2.0 ** -8 * want.abs()).all())
        qkv = got
    q, k, v = (t.reshape(T, -1, D) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    pos = torch.cat([torch.arange(m, m + n, device=DEV) for m, n in zip(before, new)])
    if a.angles is not None:
        q = sref.rotate(q, pos, a.angles, a.interleaved).float().to(torch.bfloat16)
        k = sref.rotate(k, pos, a.angles, a.interleaved)
    four = type(a.cache) is bs.KVCacheFP4
    table = a.table.tolist()
    if four:
        kv = [sref.values4(c, s) for c, s in ((a.cache.k, a.cache.k_scale), (a.cache.v, a.cache.v_scale))]
        req = [b for b, n in enumerate(new) for _ in range(n)]
        page = torch.tensor([table[b][p // PAGE] for b, p in zip(req, pos.tolist())], device=DEV)
        for x_new, codes, scale in ((k.double(), a.cache.k, a.cache.k_scale), (v.double(), a.cache.v, a.cache.v_scale)):
            wc, ws = sref.quantize4(x_new)
            assert torch.equal(codes[page, :, pos % PAGE], wc) and torch.equal(scale[page, :, pos % PAGE], ws)
    else:
        t = ref.e4m3_table().to(DEV)
        kv = [t[c.long()] * s.double()[..., None, None] for c, s in ((a.cache.k, a.cache.k_scale), (a.cache.v, a.cache.v_scale))]
    lens = [m if n else 0 for m, n in zip(a.lens.tolist(), new)]
    o, _, A, S = ref.attention(q.double(), *kv, table, cu, lens, PAGE, D ** -0.5)
    e = (D + 16) * 2.0 ** -24 * S[..., None]
    do = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * e) * A + max(lens) * 2.0 ** -25 * float(kv[1].abs().max())
    W = ref.fp4_weights(*a.w_out, HID, HQ * D).to(DEV)
    o, do = o.reshape(T, -1), do.reshape(T, -1)
    y = o @ W.T
    part, mag, dm = y.abs(), o.abs() @ W.abs().T, do @ W.abs().T
    if a.lora_out:
        la, lb, ls = a.lora_out
        y, size = sref.lora(o, y, la, lb, cu, which, ls)
        mag = mag + size
        dm = dm + sref.lora(do, torch.zeros_like(y), la, lb, cu, which, ls)[1]
    bound = dm + (2.0 ** -16 + (HQ * D + 8) * 2.0 ** -23) * (mag + dm) + 2.0 ** -8 * (part + dm) + 2.0 ** -8 * (y.abs() + dm)
    return y, bound + 1e-30


def check(bs, a, x, new, max_new):
    before = a.lens.tolist()
    got = a.step(x, i32(new), max_new)
    want, bound = reference(bs, a, x, new, before)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("bits,rot,lora,mixed", [(4, True, True, False), (4, False, False, False), (8, True, False, True),
                                                 (8, False, True, False), (4, True, False, True)])
def test_requests_come_and_go(cuda_lib, bits, rot, lora, mixed):
    bs = cuda_lib
    bs.clear_device_status()
    a, gen = layer(bs, bits, rot, lora, mixed)
    for new in ([1, 16 - 2, 1], [1, 1, 1], [0, 3, 1]):   # at most 16 tokens: activations in bf16 all the way
        check(bs, a, tokens(sum(new), gen), new, max(new))
    assert a.lens.tolist() == [2, 18, 3] and int(a.n_free) == 12 - 4
    a.release(i32([0, 1, 0]))
    a.which.copy_(i32([1, 1, -1]))
    for new in ([1, 5, 1], [1, 1, 1]):
        check(bs, a, tokens(sum(new), gen), new, max(new))
    assert bs.device_status()[0] == bs.BS_OK


@pytest.mark.parametrize("bits", [4, 8])
def test_same_as_its_graph(cuda_lib, bits):
    """A step captured, replayed between prompts of other shapes, against the same steps without a graph."""
    bs = cuda_lib
    (a, gen), (b, _) = layer(bs, bits, pages=18), layer(bs, bits, pages=18)
    x, one = tokens(3, gen), i32([1, 1, 1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = b.step(x, one, 1)
    for p, new in ((tokens(45, gen), [20, 5, 20]), (tokens(40, gen), [1, 38, 1])):
        want = a.step(p, i32(new), max(new))
        with torch.cuda.stream(side):
            got = b.step(p, i32(new), max(new))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for _ in range(2):
            g.replay()
            want = a.step(x, one, 1)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(a.lens, b.lens)
            assert all(torch.equal(s, t) for s, t in zip(a.cache, b.cache))
    assert bs.device_status()[0] == bs.BS_OK


def test_pages_run_out(cuda_lib):
    """A request for which the pages do not suffice gets zeros and its adapter's nothing; the others are served."""
    bs = cuda_lib
    a, gen = layer(bs, pages=2)
    bs.clear_device_status()
    y = a.step(tokens(12, gen), i32([5, 4, 3]), 5)
    assert bs.device_status()[0] == bs.BS_ERR_PAGES
    bs.clear_device_status()
    assert a.lens.tolist() == [5, 4, 0]
    assert bool((y[9:] == 0).all()) and bool((y[:9] != 0).any(1).all())


def test_rows_behind_the_last_request(cuda_lib):
    """A padded batch: rows past the sum of the lengths change nothing for the others."""
    bs = cuda_lib
    (a, gen), (b, _) = layer(bs), layer(bs)
    x = tokens(16, gen)
    x[7:] = float("nan")
    want = a.step(x[:7], i32([3, 0, 4]), 4)
    got = b.step(x, i32([3, 0, 4]), 4)
    assert torch.equal(got[:7], want) and all(torch.equal(s, t) for s, t in zip(a.cache, b.cache))


def test_positions(cuda_lib):
    bs = cuda_lib
    for seq, new in (([5], [3]), ([0, 7, 100, 3], [2, 0, 5, 1]), (list(range(3000)), [i % 3 for i in range(3000)])):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        want = [s + i for s, n in zip(seq, new) for i in range(n)]
        out = bs.kv_positions(i32(seq), i32(cu), cu[-1] + 4)
        assert out.tolist() == want + [0] * 4
    assert bs.kv_positions(i32([]), i32([0]), 2).tolist() == [0, 0]


def test_refusals(cuda_lib):
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    a, gen = layer(bs)
    for kw in (dict(cache_bits=5), dict(lora_qkv=a.lora_out), dict(lora_out=a.lora_qkv), dict(lora_out=a.lora_out[:2])):
        with pytest.raises(ValueError):
            DecodeAttention(a.w_qkv, a.w_out, HQ, HKV, D, 3, 12, PAGE, 6, **kw)
