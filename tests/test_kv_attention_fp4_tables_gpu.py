"""Attention over the 4-bit cache: which kernel takes a request follows from the rows and
tokens of the call, not from the room in its table nor from rows behind the last request, so
neither changes a bit; and calls that are shared out among both kernels whatever their
lengths, for the kernel of many rows.  Bounds of test_kv_attention_fp4_gpu."""
import math

import pytest
import torch

from tests import test_kv_attention_fp4_gpu as base
from tests.test_kv_attention_fp4_gpu import build, check, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(bs, q, cache, table, cu, kv, max_q):
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 7.0, device=DEV)
    bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv), max_q, out=out, lse=lse)
    return out, lse


CALLS = [([104, 104], [4756, 4756], 4, 4, 64), ([75, 75, 75], [2700, 2750, 2600], 3, 1, 128), ([512], [512], 8, 2, 128),
         ([40], [6000], 8, 2, 64), ([130, 2, 1], [2000, 900, 3000], 12, 4, 128), ([200], [100], 16, 2, 64),
         # just below and above the sums that decide, 2^23 over two KV heads and 15 2^18 over more
         ([64, 64], [8192, 8192], 8, 2, 64), ([64, 64, 1], [8192, 8192, 1], 8, 2, 64),
         ([60, 60], [2048, 2048], 16, 4, 64), ([60, 60, 1], [2048, 2048, 5], 16, 4, 64), ([1900, 3], [700, 2000], 4, 1, 64)]


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D", CALLS)
def test_room_changes_nothing(cuda_lib, q_lens, kv_lens, Hq, Hkv, D):
    """Tables from just wide enough to a quarter of a million tokens, a known bound of the rows or none."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, sum(q_lens), kv_lens, q_lens, Hq, Hkv, D, 32)
    want, lse = check(bs, q, cache, table, cu, kv_lens, 32)
    width = max(len(r) for r in table)
    for more in (0, 40, 1000, 8000):
        wide = [r + [-1] * (width + more - len(r)) for r in table]
        for max_q in (max(q_lens), 0):
            out, l = run(bs, q, cache, wide, cu, kv_lens, max_q)
            assert torch.equal(out, want) and torch.equal(l, lse), (more, max_q)
    assert bs.device_status()[0] == bs.BS_OK


def test_room_changes_nothing_in_a_step(cuda_lib):
    """DecodeAttention with tables of other widths: the same outputs."""
    bs = cuda_lib
    from fp8_quantized_gemm_q4_gb300.decode import DecodeAttention
    from tests.test_decode_step_serving_gpu import layer
    from tests.test_decode_step_gpu import D, HKV, HQ, PAGE, tokens
    a, gen = layer(bs, pages=30, lora=False, rot=False)
    b = DecodeAttention(a.w_qkv, a.w_out, HQ, HKV, D, 3, 30, PAGE, 9000, cache_bits=4)
    for new in ([90, 20, 60], [1, 60, 1], [3, 0, 2]):
        x = tokens(sum(new), gen)
        assert torch.equal(a.step(x, i32(new), max(new)), b.step(x, i32(new), max(new)))
    assert bs.device_status()[0] == bs.BS_OK


PAD = {1: 65537, 3: 21846, 4: 16385, 8: 8193, 16: 4097, 32: 2049}   # rows from which a call is too large to be one kernel's whole


@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 64), (8, 8, 64, 16), (16, 2, 64, 128), (3, 1, 128, 32)])
@pytest.mark.parametrize("q_lens,kv_lens", base.RAGGED)
def test_ragged_among_both(cuda_lib, Hq, Hkv, D, page, q_lens, kv_lens):
    bs = cuda_lib
    pad = PAD[Hq] - sum(q_lens) + 2
    q, cache, table, cu = build(bs, sum(q_lens), kv_lens, q_lens, Hq, Hkv, D, page, extra_T=pad)
    out, lse = check(bs, q, cache, table, cu, kv_lens, page, out=torch.full_like(q, 3.0))
    assert bool((out[cu[-1]:] == 3.0).all()) and bool((lse[cu[-1]:] == 7.0).all())


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (16, 2, 64, 16)])
@pytest.mark.parametrize("q_lens,kv_lens", [([150, 90], [200, 1300]), ([200, 2, 130], [150, 70, 900]), ([60, 300], [20, 40])])
def test_nan_scales_among_both(cuda_lib, Hq, Hkv, D, page, q_lens, kv_lens):
    """A NaN scale of V in its 16 columns of the rows that see its token, of K in those rows; sharp scores; a NaN query."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 5, kv_lens, q_lens, Hq, Hkv, D, page, extra_T=PAD[Hq] - sum(q_lens) + 2)
    check(bs, q, cache, table, cu, kv_lens, page, scale=4.0)
    G = Hq // Hkv
    for scales in (cache.v_scale, cache.k_scale):
        kept = scales.clone()
        b = len(q_lens) - 1
        n, m = q_lens[b], kv_lens[b]
        t, h, d = max(0, m - n // 2), Hkv - 1, 1
        scales[table[b][t // page], h, t % page, d] = 0
        want, want_lse = run(bs, q, cache, table, cu, kv_lens, 0)
        scales[table[b][t // page], h, t % page, d] = 0x7f
        rows = slice(cu[b] + max(0, t - (m - n)), cu[b + 1])
        cols = slice(16 * d, 16 * d + 16) if scales is cache.v_scale else slice(0, D)
        want[rows, h * G:(h + 1) * G, cols] = math.nan
        if scales is cache.k_scale:
            want_lse[rows, h * G:(h + 1) * G] = math.nan
        got, got_lse = run(bs, q, cache, table, cu, kv_lens, 0)
        for x, y in ((got, want), (got_lse, want_lse)):
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(77.0), y.nan_to_num(77.0))
        scales.copy_(kept)
    q[cu[0]] = math.nan
    got, got_lse = run(bs, q, cache, table, cu, kv_lens, 0)
    unseen = kv_lens[0] < q_lens[0]
    assert bool((got[cu[0]] == 0).all() if unseen else got[cu[0]].isnan().all()) and not bool(got[cu[0] + 1:].isnan().any())


def test_requests_that_claim_more_than_the_call(cuda_lib):
    """Offsets that break the contract, in calls that one kernel would take whole and in others: the status, no row outside."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 9, [3000, 40], [120, 30], 8, 2, 64, 16)
    T = q.shape[0]
    room, lse = torch.full((3 * T, 8, 64), 3.0, device=DEV, dtype=torch.bfloat16), torch.full((3 * T, 8), 7.0, device=DEV)
    for more in (0, 20000):
        wide = i32([r + [-1] * more for r in table])
        for off in ([0, 1, -7], [0, T, 0], [0, (1 << 31) - 1, T], [-(1 << 31), T, T], [0, T + 1, 2 * T]):
            bs.clear_device_status()
            bs.kv_attention(q, cache, wide, i32(off), i32([3000, 40]), 0, out=room[T:2 * T], lse=lse[T:2 * T])
            assert bs.device_status()[0] == bs.BS_ERR_OFFSETS, (more, off)
            assert bool((room[:T] == 3).all()) and bool((room[2 * T:] == 3).all())
            assert bool((lse[:T] == 7).all()) and bool((lse[2 * T:] == 7).all())
    bs.clear_device_status()
    check(bs, q, cache, table, cu, [3000, 40], 16)
