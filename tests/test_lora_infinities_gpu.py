"""Adapters with infinities: what the formula gives in 64 bits, the sign of each infinity,
NaN where it says so, and the other rows and columns as if there were none.

Values are chosen so that no fp32 sum meets an infinity that the formula does not have:
A is positive, B small.  Bound of the finite ones as in test_lora_gpu."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = math.inf
TYPES = [torch.bfloat16, torch.float32]
LENS = [[1, 1, 1, 1, 1], [3, 40, 20, 70, 7]]    # tiles of 8 rows, and of 64


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def build(seed, T, K, N, r, n, dt):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16)
    y = torch.randn((T, N), generator=g).to(dt)
    a = (torch.rand((n, r, K), generator=g) * 0.2 + 0.05).to(torch.bfloat16)
    b = (torch.randn((n, N, r), generator=g) * 0.3).to(torch.bfloat16)
    return x, y, a, b, torch.rand(n, generator=g) + 0.5


def check(bs, x, y, a, b, scales, lens, which):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    want, size = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    for i, w in enumerate(which):
        if w < 0:
            continue
        lo, hi = cu[i], cu[i + 1]
        xd, ad, bd, s = x[lo:hi].double(), a[w].double(), b[w].double(), scales[w].double()
        t = (xd[:, None] * ad).sum(-1) * s            # element by element: nothing but the formula's products
        want[lo:hi] += (t[:, None] * bd).sum(-1)
        size[lo:hi] = ((xd[:, None] * ad).abs().sum(-1)[:, None] * bd.abs()).sum(-1) * s
    args = [v.to(DEV) for v in (x, y, a, b)]
    bs.clear_device_status()
    got = bs.lora_add(*args, i32(cu), i32(which), scales=scales.to(DEV)).cpu().double()
    assert bs.device_status()[0] == bs.BS_OK
    assert torch.equal(got.isnan(), want.isnan())
    far = want.isinf()
    assert torch.equal(got.isinf(), far) and torch.equal(got[far], want[far])
    ok = want.isfinite()
    K, r = x.shape[1], a.shape[1]
    term, step = (2.0 ** -16, 2.0 ** -8) if y.dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -23)
    bound = (term + (K + 3 * r + 8) * 2.0 ** -24) * size + step * want.abs()
    assert bool(((got - want).abs()[ok] <= bound[ok]).all())
    return want


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("r", [8, 32, 40, 64, 96, 128])
def test_infinite_products(cuda_lib, lens, r, dt):
    """Rows of x with an infinity (t infinite in all ranks), or in K's tail; B of one sign a column, or of both (NaN)."""
    T, K, N = sum(lens), 104, 72
    x, y, a, b, s = build(r, T, K, N, r, 3, dt)
    b[:, :40] = b[:, :40].abs() * torch.where(torch.arange(40) % 2 == 0, 1.0, -1.0)[:, None].bfloat16()
    b[:, 40:, 0], b[:, 40:, 1] = 0.25, -0.5
    x[0, 5], x[T - 1, K - 1], x[T // 2, 64] = INF, -INF, INF
    want = check(cuda_lib, x, y, a, b, s, lens, [0, 1, 2, 1, 0])
    assert int(want.isinf().sum()) >= 3 * 40 and bool(want[0, 40:].isnan().all())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("r", [8, 24, 64, 128])
def test_infinite_weights(cuda_lib, lens, r, dt):
    """Infinities in B against products of any sign, some exactly a bf16 number, some 0 (NaN); in y; an infinite scale of A."""
    T, K, N = sum(lens), 64, 72
    x, y, a, b, s = build(r + 1, T, K, N, r, 3, dt)
    s[:] = 1.0
    rng = random.Random(r)
    a[0, 3], a[1, r - 1] = 0.0, 0.0
    a[0, 3, :2], a[1, r - 1, 7] = 1.0, 0.5            # ranks whose t is x0 + x1, or x7 / 2
    x[:, 1] = -x[:, 0] * (torch.arange(T) % 2).bfloat16()   # t 0 in every second row, else x0
    for w, k in ((0, 3), (1, r - 1), (2, 2)):
        for n in (0, 7, 33, 64, 71):
            b[w, n, k] = rng.choice([INF, -INF])
    y[T - 1, 5], y[0, 6] = -INF, math.nan
    a[2, 5, 11] = INF
    want = check(cuda_lib, x, y, a, b, s, lens, [0, 1, 2, 0, 1])
    assert bool(want.isinf().any()) and bool(want.isnan().any()) and bool(want.isfinite().any())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", LENS)
def test_products_past_bf16(cuda_lib, lens, dt):
    """t between bf16's largest number and fp32's: 2^128 - 2^118, exact in any order of its sum."""
    T, K, N, r = sum(lens), 64, 40, 16
    x, y, a, b, s = build(9, T, K, N, r, 3, dt)
    s[:] = 1.0
    x[:], a[:] = 0.0, 1.0
    x[:, 3:13] = 2.0 ** torch.arange(118, 128).float()
    x[::2] *= -1
    b[:] = (b.float() * 2.0 ** -120).bfloat16()
    want = check(cuda_lib, x, y, a, b, s, lens, [0, 1, 2, 1, 0])
    assert bool(want.isfinite().all()) and float((want - y.double()).abs().max()) > 1
