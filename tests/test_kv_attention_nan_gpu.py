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


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (16, 2, 64, 16), (24, 8, 128, 32), (4, 4, 64, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", CALLS + [([60, 300], [20, 40])])
def test_nan_codes(cuda_lib, Hq, Hkv, D, page, q_lens, kv_lens):
    """NaN codes of new and of old tokens.  Against the same cache with 0 in their
    place: of V, the rows that see the token have NaN in its column and are the same
    bit for bit elsewhere, lse included; the rows before it are untouched, those that
    see nothing 0.  Of K, the rows that see the token are NaN, the others untouched."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 5, kv_lens, q_lens, Hq, Hkv, D, page)
    G = Hq // Hkv
    for which in ("v", "k"):
        codes = getattr(cache, which)
        kept = codes.clone()
        places = []       # request, token, KV head, column
        for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
            for i, t in enumerate(sorted({m - 1, max(0, m - n // 2), max(0, m - n + 1), max(0, m - n), m // 3})):
                places.append((b, t, (i + b) % Hkv, (0, D - 1, 37, 17, 40)[i]))
        for b, t, h, d in places:
            codes[table[b][t // page], h, t % page, d] = 0
        want, want_lse = run(bs, q, cache, table, cu, kv_lens)
        for i, (b, t, h, d) in enumerate(places):
            codes[table[b][t // page], h, t % page, d] = 0xff if i % 2 else 0x7f
            n, m = q_lens[b], kv_lens[b]
            first = max(0, t - (m - n))          # the first new token that sees t
            rows = slice(cu[b] + first, cu[b] + n)
            if which == "v":
                want[rows, h * G:(h + 1) * G, d] = math.nan
            else:
                want[rows, h * G:(h + 1) * G] = math.nan
                want_lse[rows, h * G:(h + 1) * G] = math.nan
        got, got_lse = run(bs, q, cache, table, cu, kv_lens)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got_lse.isnan(), want_lse.isnan())
        assert torch.equal(got.nan_to_num(77.0), want.nan_to_num(77.0))
        assert torch.equal(got_lse.nan_to_num(77.0), want_lse.nan_to_num(77.0))
        codes.copy_(kept)


def test_nan_query_and_nothing_seen(cuda_lib):
    """A row that sees no token gets 0 and -infinity whatever its query holds."""
    q, cache, table, cu = build(cuda_lib, 7, [0, 3], [4, 6], 8, 2, 64, 16)
    q[:] = math.nan
    out, lse = run(cuda_lib, q, cache, table, cu, [0, 3])
    assert bool((out[:7] == 0).all()) and bool((lse[:7] == -math.inf).all())
    assert bool(out[7:].isnan().all()) and bool(lse[7:].isnan().all())
