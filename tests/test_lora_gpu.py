"""Adapters of many requests against a 64-bit reference.

Bound: with t = x A^T and S = scale |x| |A|^T |B|^T, fp32 sums of exact products over K
(any order: relative K 2^-24 of the sum of magnitudes, at most) and over r, and t as a
pair of bf16 (2^-8 of 2^-9: 2^-16 at most; for fp32 outputs three: 2^-24):
    |out - ref| <= (term + (K + 3 r + 8) 2^-24) S + round |ref|
with term and round 2^-16 and 2^-8 for bf16 outputs, 2^-24 and 2^-23 for fp32."""
import random

import pytest
import torch

from tests import serving_reference as sref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def build(seed, T, K, N, r, n, dt):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, K), device=DEV, generator=gen).to(torch.bfloat16)
    y = torch.randn((T, N), device=DEV, generator=gen).to(dt)
    a = (torch.randn((n, r, K), device=DEV, generator=gen) * 0.05).to(torch.bfloat16)
    b = (torch.randn((n, N, r), device=DEV, generator=gen) * 0.3).to(torch.bfloat16)
    return x, y, a, b, torch.rand(n, device=DEV, generator=gen) + 0.5


def check(bs, x, y, a, b, cu, which, scales, **kw):
    want, size = sref.lora(x, y, a, b, cu, which, scales)
    bs.clear_device_status()
    got = bs.lora_add(x, y, a, b, i32(cu), i32(which), scales=scales, **kw)
    assert bs.device_status()[0] == bs.BS_OK
    n, K, r = cu[-1], x.shape[1], a.shape[1]
    term, step = (2.0 ** -16, 2.0 ** -8) if y.dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -23)
    bound = (term + (K + 3 * r + 8) * 2.0 ** -24) * size[:n] + step * want[:n].abs()
    err = (got[:n].double() - want[:n]).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())
    return got


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


SIZES = [(64, 8, 8), (128, 136, 16), (520, 264, 24), (4096, 1000, 64), (1032, 1536, 128), (8, 72, 40), (192, 4096, 32)]


@pytest.mark.parametrize("K,N,r", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_single_tokens(cuda_lib, K, N, r, dt):
    """One row a request, adapters shared, alone, or none."""
    rng = random.Random(K)
    B, n = 37, 9
    which = [rng.randint(-2, n - 1) for _ in range(B)]
    x, y, a, b, s = build(K + r, B + 2, K, N, r, n, dt)
    out = torch.full_like(y, 9.0)
    check(cuda_lib, x, y, a, b, list(range(B + 1)), which, s, out=out)
    assert bool((out[B:] == 9.0).all())                   # rows past the last request
    bare = [i for i, w in enumerate(which) if w < 0]
    assert torch.equal(out[bare], y[bare])
    check(cuda_lib, x, y, a, b, list(range(B + 1)), which, None)


@pytest.mark.parametrize("K,N,r", SIZES)
@pytest.mark.parametrize("lens", [[1, 0, 5, 17, 64, 2], [300, 3, 130, 1], [16, 16, 16], [1], [129], [65, 63]])
def test_ragged(cuda_lib, K, N, r, lens):
    """Prompts, drafts and single tokens in one call, in place."""
    rng = random.Random(sum(lens))
    which = [rng.randint(0, 2) for _ in lens]
    if len(which) > 2:
        which[2] = -1
    for dt in (torch.bfloat16, torch.float32):
        x, y, a, b, s = build(N, sum(lens), K, N, r, 3, dt)
        got = check(cuda_lib, x, y, a, b, offsets(lens), which, s)
        again = y.clone()
        assert cuda_lib.lora_add(x, again, a, b, i32(offsets(lens)), i32(which), scales=s, out=again) is again
        assert torch.equal(got, again)


def test_many_rows_and_requests(cuda_lib):
    rng = random.Random(3)
    for lens in ([rng.randint(0, 3) for _ in range(1500)], [2000, 1, 900]):
        x, y, a, b, s = build(1, sum(lens), 256, 520, 16, 70, torch.bfloat16)
        check(cuda_lib, x, y, a, b, offsets(lens), [rng.randint(-1, 69) for _ in lens], s)


@pytest.mark.parametrize("lens,r,dt", [([3500, 31], 16, torch.bfloat16), ([2800, 0, 3200], 32, torch.bfloat16),
                                       ([8200], 64, torch.bfloat16), ([11900, 100], 8, torch.bfloat16),
                                       ([1190], 128, torch.bfloat16), ([1000, 3090], 128, torch.float32),
                                       ([4000, 100], 24, torch.float32), ([9000], 40, torch.float32)])
def test_rounds(cuda_lib, lens, r, dt):
    """Rows enough for more than one round of tiles on the GPU: clusters of eight down to two CTAs."""
    x, y, a, b, s = build(r, sum(lens), 328, 264, r, 3, dt)
    check(cuda_lib, x, y, a, b, offsets(lens), [2, 0, 1][:len(lens)], s)


def test_strides(cuda_lib):
    """Rows of x, y and out as slices of wider matrices, what is beside them untouched; another stream."""
    lens, which = [3, 40, 1], [1, 0, 1]
    x, y, a, b, s = build(2, 44, 512, 264, 16, 2, torch.bfloat16)
    want = check(cuda_lib, x, y, a, b, offsets(lens), which, s)
    wx, wy, wo = (torch.full((44, w), 5.0, device=DEV, dtype=torch.bfloat16) for w in (1024, 528, 600))
    wx[:, 256:768], wy[:, 8:272] = x, y
    side = torch.cuda.Stream()
    cu, w = i32(offsets(lens)), i32(which)
    side.wait_stream(torch.cuda.current_stream())
    cuda_lib.lora_add(wx[:, 256:768], wy[:, 8:272], a, b, cu, w, scales=s, out=wo[:, 16:280], stream=side)
    side.synchronize()
    assert torch.equal(wo[:, 16:280], want)
    assert bool((wo[:, :16] == 5).all()) and bool((wo[:, 280:] == 5).all())


def test_repeatable_and_captured(cuda_lib):
    """The same bits again, alone, in a graph, and beside another graph that runs at the same time."""
    bs = cuda_lib
    sets = []
    for seed, lens in ((1, [1] * 40), (2, [300, 70])):
        x, y, a, b, s = build(seed, sum(lens), 2048, 1032, 32, 5, torch.bfloat16)
        args = (x, y, a, b, i32(offsets(lens)), i32([i % 5 for i in range(len(lens))]), s)
        want = bs.lora_add(*args)
        for _ in range(3):
            assert torch.equal(bs.lora_add(*args), want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = bs.lora_add(*args)
        sets.append((g, out, want, torch.cuda.Stream(), args))   # what the graph reads stays alive
    torch.cuda.synchronize()
    for _ in range(5):
        for g, out, _, side, _ in sets:
            with torch.cuda.stream(side):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _ in sets:
            assert torch.equal(out, want)
            out.zero_()
        torch.cuda.synchronize()


def test_contract_breaks(cuda_lib):
    """Offsets and adapters that do not exist set the status and touch nothing outside the call."""
    bs = cuda_lib
    x, y, a, b, s = build(4, 90, 256, 264, 16, 3, torch.bfloat16)
    x3, o3 = torch.zeros((270, 256), device=DEV, dtype=torch.bfloat16), torch.full((270, 264), 9.0, device=DEV, dtype=torch.bfloat16)
    x3[90:180] = x
    bs.clear_device_status()
    for cu, which in (([0, 30, -7, 90], [0, 1, 2]), ([0, 30, 20, 90], [0, 1, 2]), ([0, 30, 60, 95], [0, 1, 2]),
                      ([0, 30, 60, (1 << 31) - 1], [0, 1, 2]), ([-5, 30, 60, 90], [0, 1, 2]), ([0, 30, 60, 90], [0, 3, 2]),
                      ([0, 30, 60, 90], [0, (1 << 31) - 1, 2]), ([0, 95, 200, 300], [0, 1, 2])):
        bs.lora_add(x3[90:180], y, a, b, i32(cu), i32(which), scales=s, out=o3[90:180])
        assert bs.device_status()[0] == bs.BS_ERR_OFFSETS, (cu, which)
        bs.clear_device_status()
        assert bool((o3[:90] == 9).all()) and bool((o3[180:] == 9).all())
    out = bs.lora_add(x, y, a, b, i32([0, 30, 60, 90]), i32([0, 3, 2]), scales=s)
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()
    assert torch.equal(out[30:60], y[30:60])      # an adapter that there is not adds nothing
    want, size = sref.lora(x, y, a, b, [0, 30, 60, 90], [0, -1, 2], s)
    assert bool(((out.double() - want).abs() <= 2.0 ** -12 * size + 2.0 ** -8 * want.abs()).all())


def test_nan_and_infinity(cuda_lib):
    """A NaN or infinite row of x, and adapters that hold one, reach the rows that use them and no other."""
    bs = cuda_lib
    lens, which = [1, 1, 20, 1, 70], [0, 1, 2, -1, 1]
    x, y, a, b, s = build(5, sum(lens), 256, 264, 16, 3, torch.bfloat16)
    want = bs.lora_add(x, y, a, b, i32(offsets(lens)), i32(which), scales=s)
    for value in (float("nan"), float("inf")):
        bad = x.clone()
        bad[[0, 7, 40], 13] = value
        got = bs.lora_add(bad, y, a, b, i32(offsets(lens)), i32(which), scales=s)
        fine = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
        fine[[0, 7, 40]] = False
        assert torch.equal(got[fine], want[fine]) and not bool(got[~fine].isfinite().any())
    a2 = a.clone()
    a2[1, 3, 200] = float("nan")
    got = bs.lora_add(x, y, a2, b, i32(offsets(lens)), i32(which), scales=s)
    uses = torch.zeros(sum(lens), dtype=torch.bool, device=DEV)
    uses[1:2] = uses[23:] = True
    assert bool(got[uses].isnan().all()) and torch.equal(got[~uses], want[~uses])


def test_empty(cuda_lib):
    bs = cuda_lib
    x, y, a, b, s = build(6, 4, 64, 64, 8, 2, torch.bfloat16)
    out = torch.full_like(y, 3.0)
    bs.lora_add(x, y, a, b, i32([0]), i32([]), out=out)
    bs.lora_add(x, y, a, b, i32([0, 0]), i32([1]), out=out)
    assert bool((out == 3).all())
    assert bs.lora_add(x[:0], y[:0], a, b, i32([0, 0]), i32([0])).shape == (0, 64)
    assert torch.equal(bs.lora_add(x, y, a[:0], b[:0], i32([0, 4]), i32([-1])), y)


@pytest.mark.parametrize("lens", [[1, 1, 1], [40, 60, 90]])
def test_rows_past_32_bits(cuda_lib, lens):
    """Rows of x, y and out, and adapters, whose offsets pass 2^32 bytes."""
    bs = cuda_lib
    T, K, N, r = sum(lens), 64, 72, 8
    x, y, a, b, s = build(9, T, K, N, r, 3, torch.bfloat16)
    want = bs.lora_add(x, y, a, b, i32(offsets(lens)), i32([0, 2, 1]), scales=s)
    step = ((1 << 31) // (T - 1) + 64) // 8 * 8
    room = torch.zeros((T * step,), device=DEV, dtype=torch.bfloat16)
    wx, wy, wo = (torch.as_strided(room, (T, n), (step, 1), at) for n, at in ((K, 0), (N, 64), (N, 136)))
    wx.copy_(x), wy.copy_(y)
    bs.lora_add(wx, wy, a, b, i32(offsets(lens)), i32([0, 2, 1]), scales=s, out=wo)
    assert torch.equal(wo, want) and torch.equal(wx, x) and torch.equal(wy, y)
    # an adapter behind 2^32 bytes of others
    n = (1 << 31) // (r * K) + 2
    big = torch.zeros((n, r, K), device=DEV, dtype=torch.bfloat16)
    big[-1] = a[0]
    small_b = torch.zeros((n, N, r), device=DEV, dtype=torch.bfloat16)
    small_b[-1] = b[0]
    got = bs.lora_add(x, y, big, small_b, i32([0, T]), i32([n - 1]))
    assert torch.equal(got, bs.lora_add(x, y, a, b, i32([0, T]), i32([0])))
