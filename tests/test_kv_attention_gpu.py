"""Attention over the 8-bit paged cache against a 64-bit reference.

Bound: the weights are rounded to fp16 (relative 2^-11, or 2^-25 absolute
below fp16's normal range), scores carry an fp32 sum over D, the output is
rounded to bf16 (2^-8):
    |out - ref| <= (2^-11 + 2 e) A + m 2^-25 max|v| + 2^-8 |ref|,
    e = (D + 16) 2^-24 S,  |lse - ref| <= e + 2^-20 (1 + |ref|)
with A = sum p |v| / sum p, S = max_t sum_d |q k| * scale, m tokens seen."""
import math
import random

import pytest
import torch

from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def build(bs, seed, kv_lens, q_lens, Hq, Hkv, D, page, spread=1.0, extra_T=0):
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pages = [-(-m // page) for m in kv_lens]
    ids = list(range(sum(pages) + 2))
    rng.shuffle(ids)
    width = max(pages + [1]) + 1
    table, at = [], 0
    for n in pages:
        table.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    cache = bs.KVCache.empty(len(ids), Hkv, page, D)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        s = torch.exp2(torch.randint(-9, -5, scale.shape, device=DEV, generator=gen).float())
        x = torch.randn(codes.shape, device=DEV, generator=gen) / s[..., None, None]
        codes.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scale.copy_(s)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1] + extra_T, Hq, D), device=DEV, generator=gen) * spread
    return q.to(torch.bfloat16), cache, table, cu


def values(codes, scale):
    return ref.e4m3_table().to(DEV)[codes.long()] * scale.double()[..., None, None]


def check(bs, q, cache, table, cu, kv_lens, page, scale=None, **kw):
    T, Hq, D = q.shape
    q_lens = [b - a for a, b in zip(cu, cu[1:])]
    sc = D ** -0.5 if scale is None else scale
    lse = torch.full((T, Hq), 7.0, device=DEV)
    bs.clear_device_status()
    out = bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), kw.pop("max_q", max(q_lens + [0])),
                          softmax_scale=scale, lse=lse, **kw)
    assert bs.device_status()[0] == bs.BS_OK
    n = cu[-1]
    want, wlse, A, S = ref.attention(q[:n].double(), values(cache.k, cache.k_scale), values(cache.v, cache.v_scale),
                                     table, cu, kv_lens, page, sc)
    got = out[:n].double()
    assert not got.isnan().any()
    e = (D + 16) * 2.0 ** -24 * S[..., None]
    vmax = 448 * float(cache.v_scale.max())
    bound = (2.0 ** -11 + 2 * e) * A + max(kv_lens + [0]) * 2.0 ** -25 * vmax + 2.0 ** -8 * want.abs() + 1e-30
    err = (got - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    empty = wlse == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty)
    assert bool((got[empty] == 0).all())
    le = (lse[:n].double() - wlse).abs()[~empty]
    lb = (e[..., 0] + 2.0 ** -20 * (1 + wlse.abs()))[~empty]
    assert bool((le <= lb).all()), float((le / lb).max())
    return out, lse


HEADS = [(1, 1, 64), (4, 1, 128), (8, 2, 64), (32, 8, 128), (6, 2, 128), (16, 16, 64), (32, 2, 128), (40, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode(cuda_lib, Hq, Hkv, D, page):
    """One token a request, caches from empty to long, ends inside pages and tiles."""
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 0, 1000, 2049]
    q, cache, table, cu = build(cuda_lib, Hq + page, kv, [1] * len(kv), Hq, Hkv, D, page)
    check(cuda_lib, q, cache, table, cu, kv, page)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 64), (8, 8, 64, 16), (12, 4, 128, 16), (16, 2, 64, 128),
                                           (16, 1, 128, 32)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([3, 0, 5, 1], [3, 70, 700, 0]), ([1, 17, 2, 64], [500, 17, 1, 64]), ([129, 1, 300], [129, 4000, 900]),
    ([200], [100]), ([9, 9], [4, 5]), ([130, 65, 33, 1, 4], [2000, 66, 1000, 90, 3000])])
def test_ragged(cuda_lib, Hq, Hkv, D, page, q_lens, kv_lens):
    """Drafts, prompts and chunks over a prefix mixed with single tokens; more rows than tokens (rows that see nothing)."""
    q, cache, table, cu = build(cuda_lib, sum(q_lens), kv_lens, q_lens, Hq, Hkv, D, page, extra_T=3)
    out, lse = check(cuda_lib, q, cache, table, cu, kv_lens, page, out=torch.full_like(q, 3.0))
    assert bool((out[-3:] == 3.0).all()) and bool((lse[-3:] == 7.0).all())   # rows past the last request
    # the same rows when no bound on the rows of a request is known
    out2, lse2 = check(cuda_lib, q, cache, table, cu, kv_lens, page, max_q=0)
    n = cu[-1]
    assert torch.equal(out[:n], out2[:n]) and torch.equal(lse[:n], lse2[:n])


def test_long_cache_one_request(cuda_lib):
    """A single request over a long cache is split over the GPU; repeated calls agree bit for bit."""
    kv = [60001]
    q, cache, table, cu = build(cuda_lib, 3, kv, [1], 8, 1, 128, 64, spread=2.0)
    a, la = check(cuda_lib, q, cache, table, cu, kv, 64)
    for _ in range(3):
        b, lb = check(cuda_lib, q, cache, table, cu, kv, 64)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_many_requests(cuda_lib):
    rng = random.Random(5)
    kv = [rng.randint(0, 90) for _ in range(1500)]
    q, cache, table, cu = build(cuda_lib, 5, kv, [1] * 1500, 8, 2, 64, 16)
    check(cuda_lib, q, cache, table, cu, kv, 16)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 70]), ([100, 2], [300, 70])])
def test_sharp_and_flat_scores(cuda_lib, q_lens, kv_lens):
    for spread, scale in ((30.0, 0.5), (1e-3, 1e-3), (1.0, 4.0)):
        q, cache, table, cu = build(cuda_lib, 11, kv_lens, q_lens, 8, 2, 128, 16, spread=spread)
        check(cuda_lib, q, cache, table, cu, kv_lens, 16, scale=scale)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [301, 77]), ([90, 3], [301, 77])])
def test_page_scales_far_apart(cuda_lib, q_lens, kv_lens):
    """Pages of one request with value scales from 2^-30 to 2^20: small pages still weigh in the softmax sum."""
    q, cache, table, cu = build(cuda_lib, 13, kv_lens, q_lens, 4, 2, 64, 16)
    cache.v_scale.copy_(torch.exp2(torch.randint(-30, 21, cache.v_scale.shape, device=DEV).float()))
    check(cuda_lib, q, cache, table, cu, kv_lens, 16)
    cache.k_scale.copy_(torch.exp2(torch.randint(-30, -5, cache.k_scale.shape, device=DEV).float()))
    cache.v_scale.mul_(1.37)       # any positive scale
    check(cuda_lib, q, cache, table, cu, kv_lens, 16)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [300, 70, 1]), ([100, 2, 1], [300, 70, 1])])
def test_nan_where_masked(cuda_lib, q_lens, kv_lens):
    """NaN codes behind a request's last token and in pages that nobody owns, NaN scales of those pages, change nothing."""
    page = 64
    q, cache, table, cu = build(cuda_lib, 17, kv_lens, q_lens, 8, 2, 128, page)
    a, la = check(cuda_lib, q, cache, table, cu, kv_lens, page)
    owned = {i for r in table for i in r if i >= 0}
    for codes in (cache.k, cache.v):
        for r, m in zip(table, kv_lens):
            if m % page:
                codes[r[m // page], :, m % page:] = 0x7f
    ghosts = [i for i in range(cache.k.shape[0]) if i not in owned]
    assert ghosts
    cache.k[ghosts] = 0xff
    cache.v[ghosts] = 0x7f
    cache.k_scale[ghosts] = math.nan
    cache.v_scale[ghosts] = math.inf
    lse = torch.empty_like(la)
    b = cuda_lib.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), max(q_lens), lse=lse)
    assert torch.equal(a, b) and torch.equal(la, lse)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(16, 2, 128, 64), (24, 8, 64, 16)])
def test_edges_in_a_large_call(cuda_lib, Hq, Hkv, D, page):
    """Sharp, flat and far apart scores, NaN where nobody looks, ids outside the pool,
    rows that see nothing, in a call of thousands of rows."""
    bs = cuda_lib
    q_lens, kv_lens = [200, 2, 1, 40, 90], [700, 70, 1, 17, 0]
    for spread, scale in ((30.0, 0.5), (1e-3, 1e-3), (1.0, None)):
        q, cache, table, cu = build(bs, 41, kv_lens, q_lens, Hq, Hkv, D, page, spread=spread)
        check(bs, q, cache, table, cu, kv_lens, page, scale=scale)
    cache.v_scale.copy_(torch.exp2(torch.randint(-30, 21, cache.v_scale.shape, device=DEV).float()))
    a, la = check(bs, q, cache, table, cu, kv_lens, page)
    owned = {i for r in table for i in r if i >= 0}
    for codes in (cache.k, cache.v):
        for r, m in zip(table, kv_lens):
            if m % page:
                codes[r[m // page], :, m % page:] = 0x7f
    ghosts = [i for i in range(cache.k.shape[0]) if i not in owned]
    cache.k[ghosts] = 0xff
    cache.v[ghosts] = 0x7f
    cache.k_scale[ghosts] = math.nan
    cache.v_scale[ghosts] = math.inf
    lse = torch.empty_like(la)
    b = bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), max(q_lens), lse=lse)
    assert torch.equal(a, b) and torch.equal(la, lse)
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1):
        t = [list(r) for r in table]
        t[0][1] = bad
        bs.clear_device_status()
        bs.kv_attention(q, cache, i32(t), i32(cu), i32(kv_lens), max(q_lens))
        assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()


def test_strides_and_streams(cuda_lib):
    """q and out as slices, [H, T, D] in memory, on a stream of their own."""
    kv, ql = [400, 33, 64], [1, 5, 1]
    q, cache, table, cu = build(cuda_lib, 19, kv, ql, 8, 4, 128, 32)
    a, la = check(cuda_lib, q, cache, table, cu, kv, 32)
    s = torch.cuda.Stream()
    wide = torch.empty((q.shape[0], 24, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:16] = q
    o = torch.empty((8, q.shape[0], 128), dtype=torch.bfloat16, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    b = cuda_lib.kv_attention(wide[:, 8:16], cache, i32(table), i32(cu), i32(kv), 5, out=o.transpose(0, 1), stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_bad_page_ids(cuda_lib):
    """Ids outside the pool set the status and leave their page out."""
    bs = cuda_lib
    for ql in ([1], [40]):
        kv = [100]
        q, cache, table, cu = build(bs, 23, kv, ql, 4, 2, 64, 16)
        keep = [i for i in range(7) if i != 2]
        for bad in (-1, cache.k.shape[0], 2 ** 31 - 1):
            t = [list(table[0])]
            t[0][2] = bad
            bs.clear_device_status()
            lse = torch.empty((q.shape[0], 4), device=DEV)
            out = bs.kv_attention(q, cache, i32(t), i32(cu), i32(kv), ql[0], lse=lse)
            assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
            if ql == [1]:
                shorter = [[table[0][i] for i in keep]]
                l2 = torch.empty_like(lse)
                o2 = bs.kv_attention(q, cache, i32(shorter), i32(cu), i32([84]), 1, lse=l2)
                assert (out.float() - o2.float()).abs().max() <= 2.0 ** -6
                assert (lse - l2).abs().max() <= 1e-4
    bs.clear_device_status()


def test_lengths_past_the_table(cuda_lib):
    """A length that the table's width cannot hold is cut to it; rows past T are not touched."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 29, [64], [1], 4, 2, 64, 16)
    t = i32([table[0][:4]])
    a = bs.kv_attention(q, cache, t, i32(cu), i32([64]), 1)
    b = bs.kv_attention(q, cache, t, i32(cu), i32([6400]), 1)
    assert torch.equal(a, b)


def test_cache_past_32_bits(cuda_lib):
    """Pages whose byte offset passes 2^32."""
    bs = cuda_lib
    page, H, D = 128, 8, 128
    pages = (1 << 32) // (page * H * D) + 40
    k = torch.zeros((pages, H, page, D), dtype=torch.uint8, device=DEV)
    cache = bs.KVCache(k, torch.zeros_like(k), torch.ones((pages, H), device=DEV), torch.ones((pages, H), device=DEV))
    ids = list(range(pages - 40, pages, 3))
    kv = [len(ids) * page - 9]
    small = bs.KVCache.empty(len(ids), H, page, D)
    gen = torch.Generator(device=DEV).manual_seed(31)
    for big, sm in ((cache.k, small.k), (cache.v, small.v)):
        x = (torch.randn(sm.shape, device=DEV, generator=gen) * 2).to(torch.float8_e4m3fn).view(torch.uint8)
        sm.copy_(x)
        big[ids] = x
    for n in (1, 40):
        q = torch.randn((n, 16, D), device=DEV, generator=gen).to(torch.bfloat16)
        a = bs.kv_attention(q, cache, i32([ids]), i32([0, n]), i32(kv), n)
        b = bs.kv_attention(q, small, i32([list(range(len(ids)))]), i32([0, n]), i32(kv), n)
        assert torch.equal(a, b)


@pytest.mark.parametrize("q_lens,sites", [([1, 2, 1], {51, 52}), ([140, 90, 33], set(range(60, 77)))], ids=["few", "many"])
def test_waits_that_run_out(cuda_lib, q_lens, sites):
    """With a wait limit of 1 us the kernels end by themselves, either with a right
    result or with the status that says otherwise, and leave the workspace as the
    next call needs it.  The first scores of many rows take longer than that; the
    copies that few rows wait for may not."""
    bs = cuda_lib
    kv = [3000, 700, 2100]
    q, cache, table, cu = build(bs, 23, kv, q_lens, 16, 4, 128, 64)
    args = (q, cache, i32(table), i32(cu), i32(kv), max(q_lens))
    bs.clear_device_status()
    want = bs.kv_attention(*args)
    torch.cuda.synchronize()
    for _ in range(3):
        with bs.kernel_options(wait_timeout_us=1):
            got = bs.kv_attention(*args)
        torch.cuda.synchronize()
        st, detail = bs.device_status()
        if st == bs.BS_OK and max(q_lens) < 10:
            assert torch.equal(got, want)
        else:
            assert st == bs.BS_ERR_TIMEOUT and (detail >> 8) in sites, (st, hex(detail))
        bs.clear_device_status()
        assert torch.equal(bs.kv_attention(*args), want)
        assert bs.device_status()[0] == bs.BS_OK


def test_workspace_shared_with_a_gemm(cuda_lib):
    """A decode GEMM (stream-K) and attention of either kind in turn on one stream."""
    bs = cuda_lib
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, w = (torch.randn(n, 2048, device=DEV, generator=gen).to(torch.bfloat16) for n in (16, 640))
    (xc, xs, _), (wc, ws, _) = bs.q4_quantize(x), bs.q4_quantize(w)
    calls = [lambda: bs.gemm_fp4(xc, xs, wc, ws, 2048)]
    for q_lens in ([1, 1], [77, 40]):
        q, cache, table, cu = build(bs, 31, [2500, 900], q_lens, 16, 4, 128, 64)
        calls.append(lambda a=(q, cache, i32(table), i32(cu), i32([2500, 900]), max(q_lens)): bs.kv_attention(*a))
    want = [f() for f in calls]
    for order in ([0, 1, 2], [2, 0, 1], [1, 1, 0], [2, 2, 0]):
        for i in order:
            assert torch.equal(calls[i](), want[i])


def test_empty_calls(cuda_lib):
    bs = cuda_lib
    q, cache, table, cu = build(bs, 37, [50], [2], 4, 2, 64, 16)
    out = torch.full_like(q, 5.0)
    bs.kv_attention(q, cache, i32(table), i32([0, 0]), i32([50]), 1, out=out)
    assert bool((out == 5.0).all())
    bs.kv_attention(q[:0], cache, i32(table), i32([0, 0]), i32([50]), 1, out=out[:0])
    lse = torch.zeros((2, 4), device=DEV)
    bs.kv_attention(q, cache, i32(table), i32(cu), i32([0]), 2, out=out, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
