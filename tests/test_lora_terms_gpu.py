"""The terms that x A^T enters the second product in, apart from every other rounding.

x = (2^16, 2^8, 1) in three places and A of whole numbers below 2^8 make t = x A^T any whole number
of up to 24 bits, exact in fp32 in every order; a column of B has one power of two, so that out - y
is one t times it.  Then
  fp32  the terms are within 2^-28 of t, and their three products are added in two fp32 sums, each
        off by a step at most (2^-23): |out - t b| <= 2^-21 |t b|, with y = 0
  bf16  the terms are within 2^-16 of t; y = -b t cut to bf16's 8 bits leaves what only the second
        term holds, below 2^-7 |t b|, rounded to bf16 once: |out - ref| <= (2^-16 + 2^-21) |t b| + 2^-8 |ref|
Without its last term a result is off by up to 2^-16 (fp32) and 2^-7 (bf16) of t b."""
import pytest
import torch

from tests.test_lora_gpu import i32, offsets

DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16]


def cut(t):
    """The first 8 significant bits."""
    return (t.float().view(torch.int32) & -65536).view(torch.float32).double()


def inputs(seed, T, K, N, r, dt):
    """x, y, A [1, r, K], B [1, N, r] and, in 64 bits, the products that are added to y and |t b|."""
    g = torch.Generator().manual_seed(seed)
    x, a, b = torch.zeros(T, K), torch.zeros(r, K), torch.zeros(N, r)
    at = torch.randperm(K, generator=g)[:3]
    x[:, at] = torch.tensor([2.0 ** 16, 2.0 ** 8, 1.0]) * torch.exp2(torch.randint(-6, 7, (T, 1), generator=g).float())
    x[::3] *= -1
    a[:, at] = torch.randint(0, 256, (r, 3), generator=g).float()
    a[:, at[0]] += (a[:, at[0]] == 0).float()
    a[0, at], a[1, at] = torch.tensor([255.0, 255, 255]), torch.tensor([128.0, 0, 1])
    which = torch.randint(0, r, (N,), generator=g)
    b[torch.arange(N), which] = torch.exp2(torch.randint(-5, 6, (N,), generator=g).float()) * (1 - 2.0 * (torch.arange(N) % 2))
    t = x.double() @ a.double().T
    assert bool((t == t.float().double()).all())
    tb = t[:, which] * b[torch.arange(N), which].double()
    y = torch.zeros(T, N) if dt == torch.float32 else -cut(tb)
    return x.bfloat16(), y.to(dt), a.bfloat16()[None], b.bfloat16()[None], tb


def close(got, y, tb):
    want = y.double() + tb
    if y.dtype == torch.float32:
        return (got.double() - want).abs() <= 2.0 ** -21 * tb.abs()
    return (got.double() - want).abs() <= (2.0 ** -16 + 2.0 ** -21) * tb.abs() + 2.0 ** -8 * want.abs()


@pytest.mark.parametrize("dt", TYPES)
def test_the_bound_sees_a_missing_term(dt):
    """On the CPU: all terms pass, one less does not, nor do the last two exchanged for twice the first's place."""
    x, y, a, b, tb = inputs(1, 60, 64, 72, 16, dt)
    first = cut(tb)
    second = cut(tb - first) if dt == torch.float32 else (tb - first).bfloat16().double()
    third = (tb - first - second).bfloat16().double()
    terms = [first, second, third] if dt == torch.float32 else [first, second]
    add = lambda parts: (y.double() + sum(parts)).to(dt)
    assert bool(close(add(terms), y, tb).all())
    assert not bool(close(add(terms[:-1]), y, tb).all())
    assert not bool(close(add(terms[:-1] + [terms[-2]]), y, tb).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", [[1] * 30, [200, 150], [2500] + [1] * 90], ids=["few", "many", "both"])
@pytest.mark.parametrize("r", [8, 32, 40, 64, 72, 128])
def test_terms(cuda_lib, r, lens, dt):
    K, N = 200, 136
    x, y, a, b, tb = (v.to(DEV) for v in inputs(r, sum(lens), K, N, r, dt))
    got = cuda_lib.lora_add(x, y, a, b, i32(offsets(lens)), i32([0] * len(lens)))
    ok = close(got, y, tb)
    assert bool(ok.all()), int((~ok).sum())
    assert cuda_lib.device_status()[0] == cuda_lib.BS_OK
