"""FP4 weights times a few bf16 rows against a 64-bit product of the decoded
weights.  Bound: fp32 accumulation over K, |err| <= K 2^-24 sum |x w| (plus
the terms of x below 2^-29 of the row's largest), bf16 outputs 2^-8 |y|."""
import pytest
import torch

from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(bs, M, N, K, out_dtype=torch.float32, bias=False, two_level=False, alpha=1.0, seed=0, ldx=0, ldo=0, xs=None):
    gen = torch.Generator(device=DEV).manual_seed(seed + M * 7 + N + K)
    rows = max(N, 1)
    w = (torch.randn((rows, K), device=DEV, generator=gen) * 0.02).to(torch.bfloat16)
    ts = None
    if two_level:
        codes, sf, ts = bs.q4_quantize_two_level(w)
    else:
        codes, sf, _ = bs.q4_quantize(w)
    codes = codes[:N]
    x = torch.randn((M, K + ldx), device=DEV, generator=gen)
    if xs is not None:
        x = xs(x)
    x = x.to(torch.bfloat16)[:, :K]
    b = torch.randn(N, device=DEV, generator=gen).to(torch.bfloat16) if bias else None
    buf = torch.full((M, N + ldo), 9.0, dtype=out_dtype, device=DEV)
    y = bs.matvec_fp4(x, codes, sf, alpha=alpha, bias=b, tensor_scale=ts, out=buf[:, :N])
    assert bool((buf[:, N:] == 9.0).all())
    W = ref.fp4_weights(codes, sf, N, K).to(DEV)
    a = alpha * (float(ts) if two_level else 1.0)
    X = x.double()
    want = a * (X @ W.T)
    S = abs(a) * (X.abs() @ W.abs().T)
    low = abs(a) * 2.0 ** -40 * K * X.abs().amax(1, keepdim=True) * W.abs().amax(1)[None]
    if bias:
        want = want + b.double()
    bound = (K + 8) * 2.0 ** -24 * S + low + 2.0 ** -23 * want.abs()
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    err = (y.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())
    return y


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 15, 16])
@pytest.mark.parametrize("N,K", [(1, 64), (129, 64), (1000, 192), (77, 1536), (256, 4160), (4096, 1024)])
def test_shapes(cuda_lib, M, N, K):
    run(cuda_lib, M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 7168, 4096), (16, 7168, 4096), (5, 33, 7168), (1, 40000, 256), (16, 20001, 128),
                                   (8, 300, 14336)])
def test_sizes(cuda_lib, M, N, K):
    run(cuda_lib, M, N, K, out_dtype=torch.bfloat16, bias=True, two_level=True)


@pytest.mark.parametrize("M,N,K", [(1, 19457, 64), (8, 24323, 192), (9, 25000, 576), (16, 29185, 640), (2, 50001, 64),
                                   (16, 49153, 192), (13, 130, 4160), (3, 1, 4224), (16, 2049, 8256)])
def test_many_tiles_or_long_rows(cuda_lib, M, N, K):
    """One to five tiles a warp, several blocks of tiles, K that ends inside a
    chunk or before some warps' first chunk."""
    run(cuda_lib, M, N, K, ldx=8, ldo=1)


@pytest.mark.parametrize("M", [1, 4, 16])
def test_epilogue_and_strides(cuda_lib, M):
    for dt in (torch.float32, torch.bfloat16):
        for bias in (False, True):
            run(cuda_lib, M, 130, 320, out_dtype=dt, bias=bias, two_level=bias, alpha=-0.37, ldx=24, ldo=3)


@pytest.mark.parametrize("M", [1, 3, 16])
def test_ranges_of_x(cuda_lib, M):
    """Rows far apart in size, outliers, zero rows, values at the ends of bf16."""
    def outliers(x):
        x[:, ::97] *= 1e4
        return x

    def rows(x):
        return x * torch.logspace(-30, 30, x.shape[0], device=DEV)[:, None]

    def wide(x):
        return x * torch.exp2(torch.randint(-35, 5, x.shape, device=DEV).float())

    def tiny(x):
        return x * 1e-38

    def huge(x):
        return x.clamp(-3, 3) * 1e34

    def zero(x):
        x[0] = 0
        return x

    for f in (outliers, rows, wide, tiny, huge, zero):
        run(cuda_lib, M, 200, 640, xs=f)


def test_repeats_and_streams(cuda_lib):
    bs = cuda_lib
    a = run(bs, 3, 5000, 2048, seed=4)
    assert torch.equal(a, run(bs, 3, 5000, 2048, seed=4))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert torch.equal(a, run(bs, 3, 5000, 2048, seed=4))


def test_row_does_not_depend_on_the_others(cuda_lib):
    """A row's result is the same whichever rows are beside it in its tile of 8."""
    bs = cuda_lib
    w = (torch.randn((500, 1024), device=DEV) * 0.02).to(torch.bfloat16)
    codes, sf, _ = bs.q4_quantize(w)
    x = torch.randn((16, 1024), device=DEV).to(torch.bfloat16)
    y = bs.matvec_fp4(x, codes, sf, out_dtype=torch.float32)
    z = bs.matvec_fp4(x.flip(0).contiguous(), codes, sf, out_dtype=torch.float32)
    assert torch.equal(y, z.flip(0))


def test_weights_past_32_bits(cuda_lib):
    """Codes past byte 2^32: the last rows against the same rows on their own."""
    bs = cuda_lib
    K = 16384
    N = (1 << 32) // (K // 2) + 200
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    rows = (N + 127) // 128 * 128
    sf = torch.randint(0x30, 0x40, (rows * (K // 16),), dtype=torch.uint8, device=DEV)
    x = torch.randn((1, K), device=DEV).to(torch.bfloat16)
    y = bs.matvec_fp4(x, codes, sf, out_dtype=torch.float32)
    lo = (N - 200) // 128 * 128
    z = bs.matvec_fp4(x, codes[lo:], sf[lo * (K // 16):], out_dtype=torch.float32)
    assert torch.equal(y[:, lo:], z)
