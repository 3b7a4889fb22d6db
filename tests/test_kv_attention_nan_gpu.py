"""NaN inputs and codes of kv_attention: they reach what the formula says and nothing else."""
import math

import pytest
import torch

from tests.test_kv_attention_gpu import build, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"

# few rows per KV head; many; many of a unit that is cut between CTAs; both kernels in one call
CALLS = [([3, 5], [70, 300]), ([150, 90], [200, 1300]), ([40], [6000]), ([200, 2, 130], [150, 70, 900])]


def run(bs, q, cache, table, cu, kv):
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    bs.clear_device_status()
    out = bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv), 0, lse=lse)
    assert bs.device_status()[0] == bs.BS_OK
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("q_lens,kv_lens", CALLS)
def test_nan_query(cuda_lib, Hq, Hkv, D, q_lens, kv_lens):
    """A query row with a NaN: its output and its lse are NaN (not the -infinity of a row that sees nothing), the others as without it."""
    q, cache, table, cu = build(cuda_lib, 3, kv_lens, q_lens, Hq, Hkv, D, 64)
    out, lse = run(cuda_lib, q, cache, table, cu, kv_lens)
    at = [(cu[1] - 1, 1), (cu[-1] - 1, Hq - 1)]
    bad = q.clone()
    for t, h in at:
        bad[t, h, 5] = math.nan
        out[t, h], lse[t, h] = math.nan, math.nan
    got, got_lse = run(cuda_lib, bad, cache, table, cu, kv_lens)
    assert torch.equal(got.nan_to_num(77.0), out.nan_to_num(77.0))
    assert torch.equal(got_lse.nan_to_num(77.0), lse.nan_to_num(77.0))
