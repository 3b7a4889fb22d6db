"""NaN and infinite elements of x in the FP4 matrix-vector product."""
import math

import pytest
import torch

from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,N,K", [(3, 200, 320), (16, 130, 1024), (9, 300, 4160), (2, 19457, 64)])
def test_nonfinite_rows(cuda_lib, M, N, K):
    """A row with a NaN is NaN; one with infinities is what the sum of its infinite
    terms is (NaN where one meets a weight of 0 or they differ in sign); the other rows
    are the same bit for bit."""
    bs = cuda_lib
    gen = torch.Generator(device=DEV).manual_seed(M + K)
    codes, sf, _ = bs.q4_quantize((torch.randn((N, K), device=DEV, generator=gen) * 0.02).to(torch.bfloat16))
    W = ref.fp4_weights(codes, sf, N, K).to(DEV)
    x = torch.randn((M, K), device=DEV, generator=gen).to(torch.bfloat16)
    y = bs.matvec_fp4(x, codes, sf, out_dtype=torch.float32)
    for row, places in ((M - 1, {K - 3: math.nan}), (0, {1: math.inf}), (M // 2, {0: -math.inf, K - 1: math.inf})):
        z, want = x.clone(), y.clone()
        terms = torch.zeros(N, dtype=torch.float64, device=DEV)
        for k, v in places.items():
            z[row, k] = v
            terms += v * W[:, k]
        want[row] = terms.float()
        got = bs.matvec_fp4(z, codes, sf, out_dtype=torch.float32)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(0.25, math.inf, -math.inf), want.nan_to_num(0.25, math.inf, -math.inf))
