"""Rotary appends into both caches and rows read back, against 64-bit references.
Codes, scales and rotated queries are exact: the definition rounds every step."""
import random

import pytest
import torch

from tests import decode_reference as ref
from tests import serving_reference as sref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def filled(bs, fp4, pages, Hkv, page, D, gen):
    """A cache that holds something everywhere."""
    cache = (bs.KVCacheFP4 if fp4 else bs.KVCache).empty(pages, Hkv, page, D)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if fp4:
            codes.copy_(torch.randint(0, 256, codes.shape, device=DEV, generator=gen, dtype=torch.uint8))
            scale.copy_(torch.randint(0x20, 0x50, scale.shape, device=DEV, generator=gen, dtype=torch.uint8))
        else:
            x = torch.randn(codes.shape, device=DEV, generator=gen) * 60
            codes.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            scale.copy_(torch.exp2(torch.randint(-9, -5, scale.shape, device=DEV, generator=gen).float()))
    return cache


def layout(seed, olds, news, page):
    """Slots and positions of the new tokens of requests in pages of their own, and the number of pages."""
    rng = random.Random(seed)
    need = [-(-(a + b) // page) for a, b in zip(olds, news)]
    ids = list(range(sum(need) + 3))
    rng.shuffle(ids)
    slots, pos, at = [], [], 0
    for a, b, n in zip(olds, news, need):
        mine = ids[at:at + n]
        at += n
        for i in range(a, a + b):
            slots.append(mine[i // page] * page + i % page)
            pos.append(i)
    return slots, pos, len(ids)


def check(bs, fp4, slots, pos, pages, Hq, Hkv, D, page, R, mixed, dt, seed=0, edit=None, in_place=False):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    T = len(slots)
    cache = filled(bs, fp4, pages, Hkv, page, D, gen)
    before = [t.clone() for t in cache]
    qkv = (torch.randn((T, Hq + 2 * Hkv, D + 8), device=DEV, generator=gen)).to(dt)[..., :D]
    qkv[:, :, ::29] *= 5
    if edit:
        edit(qkv)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    angles = bs.rotary_angles(max(pos) + 1, R) if R else None
    want_q = sref.rotate(q, i32(pos), angles, mixed) if R else q.double()
    want_k = sref.rotate(k, i32(pos), angles, mixed) if R else k.double()
    live = torch.tensor([0 <= s < pages * page for s in slots], device=DEV)
    q_out = q if in_place else torch.full((T, Hq, D), 9.0, device=DEV, dtype=torch.bfloat16)
    old_q = q_out.clone()
    bs.clear_device_status()
    got = bs.kv_append_rotary(q if Hq else None, k, v, i32(slots), i32(pos) if R else None, angles, cache,
                              q_out=q_out if Hq else None, interleaved=mixed)
    if Hq:
        want = torch.where(live[:, None, None], want_q.float().to(torch.bfloat16), old_q)
        assert got is q_out and torch.equal(got.view(torch.int16), want.view(torch.int16))
    for x, codes, scale, c0, s0 in ((want_k, cache.k, cache.k_scale, before[0], before[2]),
                                    (v.double(), cache.v, cache.v_scale, before[1], before[3])):
        if fp4:
            at = torch.tensor([s for s in slots if 0 <= s < pages * page], dtype=torch.long, device=DEV)
            wc, ws = sref.quantize4(x[live])
            for t, w in ((c0, wc), (s0, ws)):
                t[at // page, :, at % page] = w
            assert torch.equal(codes, c0) and torch.equal(scale, s0)
        else:
            val, sc = ref.e4m3_table().to(DEV)[c0.long()].cpu(), s0.double().cpu()
            ref.kv_append(x.cpu(), slots, val, sc, page)
            # a page that a call names twice apart gets either part's scale (the header says so)
            runs = [s // page for i, s in enumerate(slots)
                    if s >= 0 and (s % page == 0 or i == 0 or slots[i - 1] != s - 1)]
            once = [i for i in range(pages) if runs.count(i) < 2]
            assert torch.equal(ref.e4m3_table()[codes.cpu().long()][once], val[once])
            assert torch.equal(scale.double().cpu()[once], sc[once])
    return cache, got


ROT = [(128, 128, False), (128, 128, True), (128, 64, False), (128, 48, False), (128, 16, True), (64, 64, False),
       (64, 48, True), (64, 16, False), (64, 0, False)]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("D,R,mixed", ROT)
@pytest.mark.parametrize("page,dt", [(16, torch.bfloat16), (64, torch.float32), (128, torch.bfloat16)])
def test_ragged(cuda_lib, fp4, D, R, mixed, page, dt):
    """Single tokens, drafts and prompts, begun and carried on inside pages; odd numbers of heads."""
    olds = [0, 5, 15, 16, 63, 100, 0, 127, 40]
    news = [1, 1, 2, 17, 1, 130, 33, 1, 0]
    slots, pos, pages = layout(D + R + page, olds, news, page)
    check(cuda_lib, fp4, slots, pos, pages, 5, 3, D, page, R, mixed, dt, seed=R)
    assert cuda_lib.device_status()[0] == cuda_lib.BS_OK


@pytest.mark.parametrize("page,D,dt", [(16, 128, torch.bfloat16), (64, 64, torch.float32), (128, 128, torch.bfloat16),
                                       (128, 64, torch.bfloat16)])
def test_long_calls(cuda_lib, page, D, dt):
    """More than 2048 rows: the 8-bit form that shares a page's rows among warps; prompts beside single tokens."""
    rng = random.Random(page)
    olds = [rng.randint(0, 300) for _ in range(120)]
    news = [1] * 100 + [rng.randint(1, 12) for _ in range(17)] + [900, 700, 555]
    slots, pos, pages = layout(page, olds, news, page)
    for fp4 in (False, True):
        check(cuda_lib, fp4, slots, pos, pages, 3, 2, D, page, D, False, dt, seed=3)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("B", [1, 5])
def test_one_token(cuda_lib, fp4, B):
    slots, pos, pages = layout(1, [70] * B, [1] * B, 64)
    check(cuda_lib, fp4, slots, pos, pages, 32, 8, 128, 64, 128, False, torch.bfloat16, in_place=True)
    check(cuda_lib, fp4, slots, pos, pages, 0, 1, 64, 64, 64, True, torch.bfloat16)      # no queries
    check(cuda_lib, fp4, slots, pos, pages, 40, 1, 64, 64, 32, True, torch.float32)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T", [40, 2100])
def test_skipped_rows(cuda_lib, fp4, T):
    """Rows with negative slots and slots past the cache are left out with their queries, wherever they stand."""
    bs = cuda_lib
    slots, pos, pages = layout(2, [3, 0], [T // 2, T - T // 2], 16)
    for i in (0, 7, 8, T // 2, T - 1):
        slots[i] = -1 - i
    check(bs, fp4, slots, pos, pages, 2, 2, 64, 16, 64, False, torch.bfloat16)
    assert bs.device_status()[0] == bs.BS_OK
    slots[20] = pages * 16
    check(bs, fp4, slots, pos, pages, 2, 2, 64, 16, 64, False, torch.bfloat16)
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()


def test_positions_outside_the_table(cuda_lib):
    bs = cuda_lib
    k = torch.randn((3, 1, 64), device=DEV)
    angles = bs.rotary_angles(10, 64)
    for fp4 in (False, True):
        cache = (bs.KVCacheFP4 if fp4 else bs.KVCache).empty(2, 1, 16, 64)
        want = (bs.KVCacheFP4 if fp4 else bs.KVCache).empty(2, 1, 16, 64)
        bs.kv_append_rotary(k, k, k, i32([3, 4, 5]), i32([-5, 10, 1 << 30]), angles, cache)
        assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
        bs.clear_device_status()
        bs.kv_append_rotary(k, k, k, i32([3, 4, 5]), i32([0, 9, 9]), angles, want)
        assert all(torch.equal(a, b) for a, b in zip(cache, want))
        assert bs.device_status()[0] == bs.BS_OK


def test_values_beyond_the_format(cuda_lib):
    """4 bits: zero groups, tiny and huge ones, infinities and NaN; each group of 16 is for itself."""
    def edit(x):
        x[0, :, :16] = 0.0
        x[1, :, :16] = 1e-30
        x[2, :, :16] = 3e4
        x[3, :, 5] = float("inf")
        x[4, :, 5] = -float("inf")
        x[4, :, 20] = float("nan")
        x[5, :, 16:32] = 6 * 2.0 ** -10 * 1.0001   # the smallest scale
        x[6, :, 16:32] = 6 * 2.0 ** -10            # half of it: to the even one, 0
        x[7, :, 0:16] = -0.0
    slots, pos, pages = layout(4, [0], [9], 16)
    check(cuda_lib, True, slots, pos, pages, 0, 2, 64, 16, 0, False, torch.float32, edit=edit)
    check(cuda_lib, True, slots, pos, pages, 0, 2, 64, 16, 0, False, torch.bfloat16, edit=edit)


def test_every_bf16_value(cuda_lib):
    """All finite bf16 values beside an element that sets the group's scale, and as the element that sets it."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = bits[bits.isfinite()]
    v = torch.cat([v, v.new_zeros(-len(v) % 32)]).view(-1, 1, 4, 8)
    T = len(v)
    for top in (0.0, 0.01, 1.0, 100.0, 2600.0):
        def edit(x):
            x[:, 1:] = torch.cat([v, torch.full_like(v, top)], -1).view(T, 1, 64).to(DEV)
        check(cuda_lib, True, list(range(T)), [0] * T, -(-T // 16), 1, 1, 64, 16, 0, False, torch.bfloat16, edit=edit)


def test_plain_append_takes_both_caches(cuda_lib):
    bs = cuda_lib
    slots, pos, pages = layout(5, [0, 9], [20, 3], 16)
    x = torch.randn((23, 2, 64), device=DEV, dtype=torch.bfloat16)
    cache = bs.KVCacheFP4.empty(pages, 2, 16, 64)
    bs.kv_append(x, -x, i32(slots), cache)
    wc, ws = sref.quantize4(x.double())
    at = torch.tensor(slots, device=DEV)
    assert torch.equal(cache.k[at // 16, :, at % 16], wc) and torch.equal(cache.k_scale[at // 16, :, at % 16], ws)
    wc, ws = sref.quantize4(-x.double())
    assert torch.equal(cache.v[at // 16, :, at % 16], wc) and torch.equal(cache.v_scale[at // 16, :, at % 16], ws)
    # without a rotation the 8-bit form is kv_append
    a, b = bs.KVCache.empty(pages, 2, 16, 64), bs.KVCache.empty(pages, 2, 16, 64)
    bs.kv_append(x, -x, i32(slots), a)
    bs.kv_append_rotary(None, x, -x, i32(slots), None, None, b)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("D,page,Hkv", [(64, 16, 3), (128, 64, 8), (128, 128, 1)])
def test_gather(cuda_lib, fp4, D, page, Hkv):
    """Rows in any order, some twice, some left out, into slices of wider tensors."""
    bs = cuda_lib
    gen = torch.Generator(device=DEV).manual_seed(D)
    cache = filled(bs, fp4, 9, Hkv, page, D, gen)
    rng = random.Random(1)
    slots = [rng.randrange(9 * page) for _ in range(301)] + [0, 9 * page - 1, 5, 5]
    for i in (0, 17, 100):
        slots[i] = -1
    T = len(slots)
    wide = torch.full((T, Hkv + 2, 2 * D), 3.0, device=DEV, dtype=torch.bfloat16)
    k, v = wide[:, 1:-1, :D], wide[:, 1:-1, D:]
    bs.clear_device_status()
    assert bs.kv_gather(cache, i32(slots), out=(k, v))[0] is k
    assert bs.device_status()[0] == bs.BS_OK
    for got, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        val = sref.values4(codes, scale) if fp4 else ref.e4m3_table().to(DEV)[codes.long()] * scale.double()[..., None, None]
        at = torch.tensor(slots, device=DEV).clamp(min=0)
        want = val[at // page, :, at % page].to(torch.bfloat16)
        want = torch.where(i32(slots)[:, None, None] >= 0, want, 3.0)
        assert torch.equal(got, want)
    assert bool((wide[:, 0] == 3).all()) and bool((wide[:, -1] == 3).all())
    slots[3] = 9 * page
    bs.kv_gather(cache, i32(slots))
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()
    empty = bs.kv_gather(cache, i32([]))
    assert empty[0].shape == (0, Hkv, D)


@pytest.mark.parametrize("fp4", [False, True])
def test_cache_past_32_bits(cuda_lib, fp4):
    """Pages whose byte offset passes 2^32, written and read back, against the same rows in a small cache."""
    bs = cuda_lib
    page, H, D = 128, 8, 128
    kind = bs.KVCacheFP4 if fp4 else bs.KVCache
    pages = (1 << 32) // (page * H * (D // 2 if fp4 else D)) + 3
    big, small = kind.empty(pages, H, page, D), kind.empty(3, H, page, D)
    gen = torch.Generator(device=DEV).manual_seed(7)
    T = 300
    x = torch.randn((T, 3 * H, D), device=DEV, generator=gen).to(torch.bfloat16)
    q, k, v = x.split(H, 1)
    at = torch.arange(T, device=DEV, dtype=torch.int32)
    angles = bs.rotary_angles(T, D)
    here, there = at + 50, at + 50 + (pages - 3) * page
    a = bs.kv_append_rotary(q, k, v, here, at, angles, small)
    b = bs.kv_append_rotary(q, k, v, there, at, angles, big)
    assert torch.equal(a, b) and all(torch.equal(s, t[-3:]) for s, t in zip(small, big))
    assert all(torch.equal(s, t) for s, t in zip(bs.kv_gather(small, here), bs.kv_gather(big, there)))
    assert all(bool((t[:4] == (0 if t.dtype == torch.uint8 else 1)).all()) for t in big)
    assert bs.device_status()[0] == bs.BS_OK


@pytest.mark.parametrize("fp4", [False, True])
def test_rows_past_32_bits(cuda_lib, fp4):
    """Inputs and outputs whose offsets pass 2^32 bytes."""
    bs = cuda_lib
    cache, want = ((bs.KVCacheFP4 if fp4 else bs.KVCache).empty(2, 1, 16, 64) for _ in range(2))
    wide = torch.zeros(((1 << 31) + (1 << 20),), device=DEV, dtype=torch.bfloat16)      # 4 GiB and more
    gen = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn((3, 1, 64), device=DEV, generator=gen).to(torch.bfloat16)
    far = torch.as_strided(wide, (3, 1, 64), (1 << 30, 64, 1))
    far.copy_(x)
    out = torch.as_strided(wide, (3, 1, 64), (1 << 30, 64, 1), 64)
    slots, pos, angles = i32([0, 1, 2]), i32([4, 5, 6]), bs.rotary_angles(9, 64)
    a = bs.kv_append_rotary(x, x, x, slots, pos, angles, want)
    assert bs.kv_append_rotary(far, far, far, slots, pos, angles, cache, q_out=out) is out
    assert torch.equal(out, a) and all(torch.equal(s, t) for s, t in zip(cache, want))
    assert torch.equal(far, x)
    k, v = (torch.as_strided(wide, (3, 1, 64), (1 << 30, 64, 1), n) for n in (128, 192))
    bs.kv_gather(cache, slots, out=(k, v))
    assert all(torch.equal(s, t) for s, t in zip((k, v), bs.kv_gather(want, slots)))


def test_on_two_streams_and_captured(cuda_lib):
    """Two calls at once on caches of their own, one of them a replayed graph."""
    bs = cuda_lib
    sets = []
    for seed, fp4, T in ((1, True, 700), (2, False, 3000)):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randn((T, 6, 64), device=DEV, generator=gen).to(torch.bfloat16)
        slots, pos, pages = layout(seed, [5, 0], [T // 2, T - T // 2], 64)
        cache = (bs.KVCacheFP4 if fp4 else bs.KVCache).empty(pages, 2, 64, 64)
        args = (*x.split([2, 2, 2], 1), i32(slots), i32(pos), bs.rotary_angles(max(pos) + 1, 32), cache)
        want = bs.kv_append_rotary(*args), *(t.clone() for t in cache)
        sets.append((args, cache, want, torch.cuda.Stream()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bs.kv_append_rotary(*sets[0][0])
    for _ in range(10):
        for args, cache, _, side in sets:
            side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(sets[0][3]):
            g.replay()
        other = bs.kv_append_rotary(*sets[1][0], stream=sets[1][3])
        torch.cuda.synchronize()
        for got, (_, cache, want, _) in zip((out, other), sets):
            assert torch.equal(got, want[0]) and all(torch.equal(s, t) for s, t in zip(cache, want[1:]))
        out.zero_()
        torch.cuda.synchronize()
