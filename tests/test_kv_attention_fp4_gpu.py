"""Attention over the 4-bit paged cache against a 64-bit reference.

Bound: as over the 8-bit cache.  A code times its scale is exact in fp16; the weights are
rounded to fp16 (relative 2^-11, or 2^-25 absolute below fp16's normal range), scores
carry an fp32 sum over D, the output is rounded to bf16 (2^-8):
    |out - ref| <= (2^-11 + 2 e) A + m 2^-25 max|v| + 2^-8 |ref|,
    e = (D + 16) 2^-24 S,  |lse - ref| <= e + 2^-20 (1 + |ref|)
with A = sum p |v| / sum p, S = max_t sum_d |q k| * scale, m tokens seen."""
import math
import random
import sys

import pytest
import torch

from tests import decode_reference as ref
from tests import serving_reference as sref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


ROOM = 0   # tokens that a block table has room for beyond those that are cached


@pytest.fixture(params=[0, 1 << 18], ids=["", "roomy"])
def room(request, monkeypatch):
    """Small calls whose tables leave room for long requests are shared out among both kernels, others are one's."""
    monkeypatch.setattr(sys.modules[__name__], "ROOM", request.param)


def build(bs, seed, kv_lens, q_lens, Hq, Hkv, D, page, spread=1.0, extra_T=0, low=0x20, high=0x30):
    """Random codes; scale codes low .. high - 1 (by default 2^-3 .. 1)."""
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pages = [-(-m // page) for m in kv_lens]
    ids = list(range(sum(pages) + 2))
    rng.shuffle(ids)
    width = max(pages + [1]) + 1 + ROOM // page
    table, at = [], 0
    for n in pages:
        table.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    cache = bs.KVCacheFP4.empty(len(ids), Hkv, page, D)
    for t, lo, hi in ((cache.k, 0, 256), (cache.v, 0, 256), (cache.k_scale, low, high), (cache.v_scale, low, high)):
        t.copy_(torch.randint(lo, hi, t.shape, device=DEV, generator=gen, dtype=torch.uint8))
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1] + extra_T, Hq, D), device=DEV, generator=gen) * spread
    return q.to(torch.bfloat16), cache, table, cu


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
    k, v = sref.values4(cache.k, cache.k_scale), sref.values4(cache.v, cache.v_scale)
    want, wlse, A, S = ref.attention(q[:n].double(), k, v, table, cu, kv_lens, page, sc)
    got = out[:n].double()
    assert not got.isnan().any()
    e = (D + 16) * 2.0 ** -24 * S[..., None]
    bound = (2.0 ** -11 + 2 * e) * A + max(kv_lens + [0]) * 2.0 ** -25 * float(v.abs().max()) + 2.0 ** -8 * want.abs() + 1e-30
    err = (got - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    empty = wlse == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty)
    assert bool((got[empty] == 0).all())
    le = (lse[:n].double() - wlse).abs()[~empty]
    lb = (e[..., 0] + 2.0 ** -20 * (1 + wlse.abs()))[~empty]
    assert bool((le <= lb).all()), float((le / lb).max())
    return out, lse


HEADS = [(1, 1, 64), (4, 1, 128), (32, 8, 128), (6, 2, 128), (16, 16, 64), (32, 2, 128), (40, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode(cuda_lib, Hq, Hkv, D, page):
    """One token a request, caches from empty to long, ends inside pages and tiles."""
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 0, 1000, 2049]
    q, cache, table, cu = build(cuda_lib, Hq + page, kv, [1] * len(kv), Hq, Hkv, D, page)
    check(cuda_lib, q, cache, table, cu, kv, page)


RAGGED = [([3, 0, 5, 1], [3, 70, 700, 0]), ([1, 17, 2, 64], [500, 17, 1, 64]), ([129, 1, 300], [129, 4000, 900]),
          ([200], [100]), ([9, 9], [4, 5]), ([130, 65, 33, 1, 4], [2000, 66, 1000, 90, 3000])]


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 64), (8, 8, 64, 16), (12, 4, 128, 16), (16, 2, 64, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", RAGGED)
def test_ragged(cuda_lib, Hq, Hkv, D, page, q_lens, kv_lens):
    """Drafts, prompts and chunks over a prefix mixed with single tokens; more rows than tokens (rows that see nothing)."""
    q, cache, table, cu = build(cuda_lib, sum(q_lens), kv_lens, q_lens, Hq, Hkv, D, page, extra_T=3)
    out, lse = check(cuda_lib, q, cache, table, cu, kv_lens, page, out=torch.full_like(q, 3.0))
    assert bool((out[-3:] == 3.0).all()) and bool((lse[-3:] == 7.0).all())   # rows past the last request
    # the same rows when no bound on the rows of a request is known
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    cuda_lib.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), 0, out=out2, lse=lse2)
    n = cu[-1]
    assert torch.equal(out[:n], out2[:n]) and torch.equal(lse[:n], lse2[:n])


def test_long_cache_one_request(cuda_lib):
    """A single request over a long cache is split over the GPU; repeated calls agree bit for bit."""
    kv = [60001]
    q, cache, table, cu = build(cuda_lib, 3, kv, [1], 8, 1, 128, 64, spread=2.0)
    a, la = check(cuda_lib, q, cache, table, cu, kv, 64)
    for _ in range(3):
        lse = torch.empty_like(la)
        assert torch.equal(a, cuda_lib.kv_attention(q, cache, i32(table), i32(cu), i32(kv), 1, lse=lse))
        assert torch.equal(la, lse)


def test_many_requests(cuda_lib):
    rng = random.Random(5)
    kv = [rng.randint(0, 90) for _ in range(1500)]
    q, cache, table, cu = build(cuda_lib, 5, kv, [1] * 1500, 8, 2, 64, 16)
    check(cuda_lib, q, cache, table, cu, kv, 16)


def test_many_requests_of_both_kinds(cuda_lib, monkeypatch):
    """More requests than a CTA has threads, single tokens and prompts among one another, some without rows or tokens."""
    monkeypatch.setattr(sys.modules[__name__], "ROOM", 2048)
    rng = random.Random(6)
    q_lens = [rng.choice([1, 1, 1, 1, 1, 1, 0, 5, 33, 70]) for _ in range(1700)]
    kv = [max(0, n + rng.choice([0, 3, 90, -4])) for n in q_lens]
    q, cache, table, cu = build(cuda_lib, 6, kv, q_lens, 8, 2, 64, 16)
    check(cuda_lib, q, cache, table, cu, kv, 16)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 70]), ([100, 2], [300, 70])])
def test_sharp_and_flat_scores(cuda_lib, q_lens, kv_lens):
    for spread, scale in ((30.0, 0.5), (1e-3, 1e-3), (1.0, 4.0)):
        q, cache, table, cu = build(cuda_lib, 11, kv_lens, q_lens, 8, 2, 128, 16, spread=spread)
        check(cuda_lib, q, cache, table, cu, kv_lens, 16, scale=scale)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [301, 77]), ([90, 3], [301, 77])])
def test_every_scale(cuda_lib, q_lens, kv_lens):
    """Scales from 0 and the smallest (2^-9) to 448 beside each other."""
    q, cache, table, cu = build(cuda_lib, 13, kv_lens, q_lens, 4, 2, 64, 16, low=0, high=0x7f, spread=0.05)
    check(cuda_lib, q, cache, table, cu, kv_lens, 16)
    cache.v_scale.clamp_(max=7)       # subnormal ones alone
    check(cuda_lib, q, cache, table, cu, kv_lens, 16)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (16, 2, 64, 16), (24, 8, 128, 32), (4, 4, 64, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", [([3, 5], [70, 300]), ([150, 90], [200, 1300]), ([40], [6000]),
                                            ([200, 2, 130], [150, 70, 900]), ([60, 300], [20, 40])])
def test_nan_scales(cuda_lib, Hq, Hkv, D, page, q_lens, kv_lens):
    """NaN scales of new and of old tokens.  Against the same cache with 0 in their
    place: of V, the rows that see the token have NaN in its 16 columns and are the same
    bit for bit elsewhere, lse included; the rows before it are untouched, those that
    see nothing 0.  Of K, the rows that see the token are NaN, the others untouched.
    Behind the last tokens and in pages that nobody owns, nothing changes."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 5, kv_lens, q_lens, Hq, Hkv, D, page)
    G = Hq // Hkv
    owned = {i for r in table for i in r if i >= 0}
    ghosts = [i for i in range(cache.k.shape[0]) if i not in owned]

    def run():
        lse = torch.full(q.shape[:2], 7.0, device=DEV)
        bs.clear_device_status()
        out = bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), 0, lse=lse)
        assert bs.device_status()[0] == bs.BS_OK
        return out, lse

    a, la = run()
    for s in (cache.k_scale, cache.v_scale):
        s[ghosts] = 0x7f
        for r, m in zip(table, kv_lens):
            if m % page:
                s[r[m // page], :, m % page:] = 0xff
    b, lb = run()
    assert torch.equal(a, b) and torch.equal(la, lb)
    for which in ("v_scale", "k_scale"):
        scales = getattr(cache, which)
        kept = scales.clone()
        places = []       # request, token, KV head, group
        for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
            for i, t in enumerate(sorted({m - 1, max(0, m - n // 2), max(0, m - n + 1), max(0, m - n), m // 3})):
                places.append((b, t, (i + b) % Hkv, (0, D // 16 - 1, 2, 1, 3)[i]))
        for b, t, h, d in places:
            scales[table[b][t // page], h, t % page, d] = 0
        want, want_lse = run()
        for i, (b, t, h, d) in enumerate(places):
            scales[table[b][t // page], h, t % page, d] = 0xff if i % 2 else 0x7f
            n, m = q_lens[b], kv_lens[b]
            first = max(0, t - (m - n))          # the first new token that sees t
            rows = slice(cu[b] + first, cu[b] + n)
            if which == "v_scale":
                want[rows, h * G:(h + 1) * G, 16 * d:16 * d + 16] = math.nan
            else:
                want[rows, h * G:(h + 1) * G] = math.nan
                want_lse[rows, h * G:(h + 1) * G] = math.nan
        got, got_lse = run()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got_lse.isnan(), want_lse.isnan())
        assert torch.equal(got.nan_to_num(77.0), want.nan_to_num(77.0))
        assert torch.equal(got_lse.nan_to_num(77.0), want_lse.nan_to_num(77.0))
        scales.copy_(kept)


@pytest.mark.usefixtures("room")
def test_nan_query(cuda_lib):
    """A row that sees no token gets 0 and -infinity whatever its query holds; NaN rows stay among themselves."""
    for q_lens, kv_lens in (([4, 6], [0, 3]), ([100, 60], [0, 30])):
        q, cache, table, cu = build(cuda_lib, 7, kv_lens, q_lens, 8, 2, 64, 16)
        q[:] = math.nan
        lse = torch.empty(q.shape[:2], device=DEV)
        out = cuda_lib.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), 0, lse=lse)
        none = sum(q_lens) - kv_lens[1]
        assert bool((out[:none] == 0).all()) and bool((lse[:none] == -math.inf).all())
        assert bool(out[none:].isnan().all()) and bool(lse[none:].isnan().all())


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("Hq,Hkv,D,page", [(16, 2, 128, 64), (24, 8, 64, 16)])
def test_contract_breaks(cuda_lib, Hq, Hkv, D, page):
    """Bad page ids, lengths and offsets set the status; rows outside the call are not touched; the next call is served."""
    bs = cuda_lib
    for q_lens, kv_lens in (([1, 2], [320, 100]), ([150, 40], [320, 100])):
        q, cache, table, cu = build(bs, 9, kv_lens, q_lens, Hq, Hkv, D, page)
        T = q.shape[0]
        bs.clear_device_status()
        want = bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), 0)
        assert bs.device_status()[0] == bs.BS_OK
        for bad in (-1, cache.k.shape[0], 2 ** 31 - 1):
            t = [list(r) for r in table]
            t[0][1] = bad
            bs.kv_attention(q, cache, i32(t), i32(cu), i32(kv_lens), max(q_lens))
            assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
            bs.clear_device_status()
        room = torch.zeros((3 * T, Hq, D), dtype=torch.bfloat16, device=DEV)
        room[T:2 * T] = q
        for off in ([0, 1, -7], [0, 2, 1], [0, 1, T + 5], [0, 1, (1 << 31) - 1], [-3, 1, T], [0, T + 100, T + 5000]):
            out, lse = torch.full_like(room, 3.0), torch.full((3 * T, Hq), 7.0, device=DEV)
            bs.kv_attention(room[T:2 * T], cache, i32(table), i32(off), i32(kv_lens), 0, out=out[T:2 * T], lse=lse[T:2 * T])
            assert bs.device_status()[0] == bs.BS_ERR_OFFSETS, off
            bs.clear_device_status()
            for x, v in ((out, 3.0), (lse, 7.0)):
                assert bool((x[:T] == v).all()) and bool((x[2 * T:] == v).all())
        t = i32([r[:-(-320 // page)] for r in table])
        for kv, same in (([320 + page, 100], [320, 100]), ([(1 << 31) - 1, 100], [320, 100]), ([320, -1], [320, 0])):
            same = [-(-320 // page) * page, same[1]]
            kv[0] = same[0] if kv[0] == 320 else kv[0] + page
            if kv[0] > (1 << 31) - 1:
                kv[0] = (1 << 31) - 1
            got = bs.kv_attention(q, cache, t, i32(cu), i32(kv), 0)
            assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
            bs.clear_device_status()
            assert torch.equal(got, bs.kv_attention(q, cache, t, i32(cu), i32(same), 0))
        assert torch.equal(bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv_lens), 0), want)
        assert bs.device_status()[0] == bs.BS_OK


def test_many_requests_claim_the_same_rows(cuda_lib):
    """Offsets that rise and fall, each pair of them the whole call: the status, and no row outside it."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 41, [40], [30], 8, 2, 64, 16)
    T, n = 30, 4000
    room, lse = torch.full((3 * T, 8, 64), 3.0, device=DEV, dtype=torch.bfloat16), torch.full((3 * T, 8), 7.0, device=DEV)
    for B in (n, 5000):     # the few-rows kernel's whole, and shared out
        bs.clear_device_status()
        bs.kv_attention(q, cache, i32(table * B), i32([0, T] * (B // 2) + [0]), i32([40] * B), 0, out=room[T:2 * T], lse=lse[T:2 * T])
        assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
        assert bool((room[:T] == 3).all()) and bool((room[2 * T:] == 3).all())
        assert bool((lse[:T] == 7).all()) and bool((lse[2 * T:] == 7).all())
    bs.clear_device_status()
    check(bs, q, cache, table, cu, [40], 16)


@pytest.mark.usefixtures("room")
def test_strides_streams_and_workspaces(cuda_lib):
    """q and out as slices, [H, T, D] in memory, on a stream of their own, with a workspace of their own; both
    caches and both kernels in turn on one workspace."""
    bs = cuda_lib
    kv, ql = [400, 33, 64], [1, 5, 1]
    q, cache, table, cu = build(bs, 19, kv, ql, 8, 4, 128, 32)
    a, la = check(bs, q, cache, table, cu, kv, 32)
    s = torch.cuda.Stream()
    wide = torch.empty((q.shape[0], 24, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:16] = q
    o = torch.empty((8, q.shape[0], 128), dtype=torch.bfloat16, device=DEV)
    ws = bs.kv_attention_workspace(128)
    s.wait_stream(torch.cuda.current_stream())
    bs.kv_attention(wide[:, 8:16], cache, i32(table), i32(cu), i32(kv), 5, out=o.transpose(0, 1), stream=s, workspace=ws)
    s.synchronize()
    assert torch.equal(a, o.transpose(0, 1))
    calls = []
    for n in ([1, 1], [77, 40]):
        args = build(bs, 31, [2500, 900], n, 16, 4, 128, 64)
        eight = bs.KVCache.empty(args[1].k.shape[0], 4, 64, 128)
        eight.k.copy_(torch.randint(0, 0x60, eight.k.shape, device=DEV, dtype=torch.uint8))
        eight.v.copy_(eight.k)
        for c in (args[1], eight):
            calls.append((args[0], c, i32(args[2]), i32(args[3]), i32([2500, 900]), max(n)))
    want = [bs.kv_attention(*c) for c in calls]
    for order in ([0, 1, 2, 3], [3, 2, 1, 0], [0, 2, 1, 3], [1, 1, 2, 2]):
        for i in order:
            assert torch.equal(bs.kv_attention(*calls[i], workspace=ws), want[i])


def test_cache_past_32_bits(cuda_lib):
    """Pages whose byte offset passes 2^32."""
    bs = cuda_lib
    page, H, D = 128, 8, 128
    pages = (1 << 32) // (page * H * D // 2) + 40
    cache = bs.KVCacheFP4.empty(pages, H, page, D)
    ids = list(range(pages - 40, pages, 3))
    kv = [len(ids) * page - 9]
    small = bs.KVCacheFP4.empty(len(ids), H, page, D)
    gen = torch.Generator(device=DEV).manual_seed(31)
    for big, sm in zip(cache, small):
        sm.copy_(torch.randint(0x20, 0x40, sm.shape, device=DEV, generator=gen, dtype=torch.uint8))
        big[ids] = sm
    for n in (1, 40):
        q = torch.randn((n, 16, D), device=DEV, generator=gen).to(torch.bfloat16)
        a = bs.kv_attention(q, cache, i32([ids]), i32([0, n]), i32(kv), n)
        b = bs.kv_attention(q, small, i32([list(range(len(ids)))]), i32([0, n]), i32(kv), n)
        assert torch.equal(a, b)


@pytest.mark.parametrize("q_lens,sites", [([1, 2, 1], {51, 52}), ([140, 90, 33], set(range(60, 77)))], ids=["few", "many"])
def test_waits_that_run_out(cuda_lib, q_lens, sites):
    """With a wait limit of 1 us the kernels end by themselves, with a right result or with the status that says
    otherwise, and leave the workspace as the next call needs it."""
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
        if st == bs.BS_OK:
            assert torch.equal(got, want)
        else:
            assert st == bs.BS_ERR_TIMEOUT and (detail >> 8) in sites, (st, hex(detail))
        bs.clear_device_status()
        assert torch.equal(bs.kv_attention(*args), want)
        assert bs.device_status()[0] == bs.BS_OK


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
