"""Block tables and slots from request lengths, pages given back, and the
quantizing append, against plain references; integers and codes are exact."""
import random

import pytest
import torch

from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def requests(rng, B, page, lo, hi, most_new, spare, zero=0.2):
    """Random lengths, a table of owned pages and a free list with `spare`
    pages more than the step needs."""
    seq = [0 if rng.random() < zero else rng.randint(lo, hi) for _ in range(B)]
    new = [0 if rng.random() < zero else rng.randint(1, most_new) for _ in range(B)]
    held = [-(-s // page) for s in seq]
    need = [-(-(s + n) // page) - h for s, n, h in zip(seq, new, held)]
    width = max([h + m for h, m in zip(held, need)] + [1])
    ids = list(range(sum(held) + max(0, sum(need) + spare)))
    rng.shuffle(ids)
    table, at = [[-1] * width for _ in range(B)], 0
    for b in range(B):
        table[b][:held[b]] = ids[at:at + held[b]]
        at += held[b]
    return seq, new, table, ids[at:]


@pytest.mark.parametrize("B,page,lo,hi,most_new,spare", [
    (1, 16, 0, 0, 1, 0), (1, 128, 1, 5000, 3000, 7), (7, 16, 1, 100, 40, 3), (64, 64, 1, 4000, 1, 0),
    (300, 32, 1, 900, 70, 11), (1025, 16, 1, 200, 30, 5), (2500, 64, 1, 300, 4, 1),
    (50, 16, 1, 300, 60, -20), (400, 32, 1, 300, 60, -200), (9, 64, 1, 300, 200, -1000)])
def test_plan(cuda_lib, B, page, lo, hi, most_new, spare):
    bs = cuda_lib
    rng = random.Random(B * page + most_new)
    seq, new, table, free = requests(rng, B, page, lo, hi, most_new, spare)
    T = sum(new) + rng.choice([0, 5])
    n_free = len(free)
    junk = [999] * 3          # entries past n_free are not taken
    want = ref.kv_plan(seq, new, table, free, n_free, page, T)
    # a table that is a slice of a wider one keeps its other columns
    wide = torch.full((B, len(table[0]) + 3), 77, dtype=torch.int32, device=DEV)
    t = wide[:, 1:1 + len(table[0])]
    t.copy_(i32(table))
    bs.clear_device_status()
    cu, kv, slots, left = bs.kv_plan(i32(seq), i32(new), t, i32(free + junk), i32([n_free]), page, T)
    assert t.cpu().tolist() == want[0]
    assert (wide[:, 0] == 77).all() and (wide[:, -2:] == 77).all()
    assert cu.cpu().tolist() == want[1]
    assert kv.cpu().tolist() == want[2]
    assert slots.cpu().tolist() == want[3]
    assert left.cpu().tolist() == [want[4]]
    assert bs.device_status()[0] == (bs.BS_ERR_PAGES if want[5] else bs.BS_OK)
    bs.clear_device_status()


def test_plan_bad_lengths(cuda_lib):
    """Negative lengths and tables too narrow set the status; the request gets nothing, the others are served."""
    bs = cuda_lib
    for seq, new in (([5, -1, 20], [1, 1, 1]), ([5, 40, 20], [1, 100, 1]), ([5, 7, 20], [1, -3, 1])):
        table = i32([[3, -1, -1], [4, -1, -1], [5, 6, -1]])
        bs.clear_device_status()
        cu, kv, slots, left = bs.kv_plan(i32(seq), i32(new), table, i32([9, 8]), i32([2]), 16, 105)
        assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
        assert kv.cpu().tolist() == [6, 0, 21]
        n1 = max(new[1], 0)
        assert slots.cpu().tolist()[:1] == [3 * 16 + 5]
        assert slots.cpu().tolist()[1:2 + n1] == [-1] * n1 + [6 * 16 + 4]
        assert left.item() == 2 and table.cpu().tolist() == [[3, -1, -1], [4, -1, -1], [5, 6, -1]]
    # more rows than slots
    bs.clear_device_status()
    bs.kv_plan(i32([0]), i32([5]), i32([[0]]), i32([9]), i32([1]), 16, 3)
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()


@pytest.mark.parametrize("B,page", [(1, 16), (5, 64), (1300, 32)])
def test_release(cuda_lib, B, page):
    bs = cuda_lib
    rng = random.Random(B)
    seq, _, table, free = requests(rng, B, page, 1, 500, 1, 4)
    done = [rng.randint(0, 1) for _ in range(B)]
    cap = len(free) + sum(-(-s // page) for s in seq)
    t, f, n = i32(table), torch.full((cap,), -5, dtype=torch.int32, device=DEV), i32([len(free)])
    f[:len(free)] = i32(free)
    bs.kv_release(i32(seq), i32(done), t, f, n, page)
    for b in range(B):
        if done[b]:
            held = -(-seq[b] // page)
            free = free + table[b][:held]
            table[b][:held] = [-1] * held
    assert t.cpu().tolist() == table and n.item() == len(free)
    assert f.cpu().tolist()[:len(free)] == free
    assert bs.device_status()[0] == bs.BS_OK


def make_cache(bs, gen, pages, H, page, D, lo=-9, hi=-5):
    c = bs.KVCache.empty(pages, H, page, D)
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = torch.randn(codes.shape, device=DEV, generator=gen) * 100
        codes.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scale.copy_(torch.exp2(torch.randint(lo, hi, scale.shape, device=DEV, generator=gen).float()))
    return c


def check_append(bs, k, v, slots, cache, page):
    table = ref.e4m3_table()
    want = []
    for x, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        val, s = table[codes.cpu().long()], scale.cpu().double()
        ref.kv_append(x.cpu().double(), slots, val, s, page)
        want.append((val, s))
    bs.kv_append(k, v, i32(slots), cache)
    for (val, s), codes, scale in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert torch.equal(scale.cpu().double(), s)
        got = table[codes.cpu().long()]
        assert torch.equal(got, val)
        assert torch.equal(torch.signbit(got), torch.signbit(val))


@pytest.mark.parametrize("H,D,page,dt", [(1, 64, 16, torch.bfloat16), (3, 128, 32, torch.float32),
                                         (8, 128, 64, torch.bfloat16), (2, 64, 128, torch.float32),
                                         (4, 128, 128, torch.bfloat16), (5, 64, 64, torch.bfloat16),
                                         (2, 128, 128, torch.float32)])
@pytest.mark.parametrize("kind", ["decode", "prefill", "mixed"])
def test_append(cuda_lib, H, D, page, dt, kind):
    """Single tokens, long prompts and both; first and later tokens of pages, rows to skip, strided inputs,
    tokens from far below to far above what the pages hold."""
    bs = cuda_lib
    rng = random.Random(H * D + page)
    gen = torch.Generator(device=DEV).manual_seed(H + D + page)
    seq, new = {"decode": ([0, 1, page - 1, page, 3 * page + 5, 7, 2 * page], [1] * 7),
                "prefill": ([0, 3, page], [5 * page + 3, 4 * page, page]),
                "mixed": ([0, 9, 2 * page - 1, 40, page // 2], [1, 2 * page, 2, 0, 3 * page + 1])}[kind]
    B = len(seq)
    pages = [-(-(s + n) // page) for s, n in zip(seq, new)]
    ids = list(range(sum(pages) + 2))
    rng.shuffle(ids)
    slots, at = [], 0
    for b in range(B):
        own = ids[at:at + pages[b]]
        at += pages[b]
        slots += [own[p // page] * page + p % page for p in range(seq[b], seq[b] + new[b])]
        slots += [-1] * (b % 2)
    T = len(slots)
    cache = make_cache(bs, gen, len(ids), H, page, D)
    qkv = torch.randn((T, 3 * H, D), device=DEV, generator=gen)
    qkv *= torch.exp2(torch.randint(-6, 7, (T, 1, 1), device=DEV, generator=gen).float())
    qkv[0] = 0
    qkv[T // 2] *= 1e-6
    qkv = qkv.to(dt)
    check_append(bs, qkv[:, H:2 * H], qkv[:, 2 * H:], slots, cache, page)
    # the same again over what was written, keys and values [H, T, D] in memory
    x = torch.randn((2 * H, T, D), device=DEV, generator=gen).to(dt)
    check_append(bs, x[:H].transpose(0, 1), x[H:].transpose(0, 1), slots, cache, page)
    assert bs.device_status()[0] == bs.BS_OK


@pytest.mark.parametrize("H,D,page,dt", [(1, 128, 128, torch.bfloat16), (3, 64, 128, torch.float32),
                                         (2, 128, 64, torch.float32), (5, 64, 16, torch.bfloat16),
                                         (2, 128, 32, torch.bfloat16), (1, 64, 64, torch.bfloat16)])
def test_append_long(cuda_lib, H, D, page, dt):
    """Calls of thousands of rows: whole pages, pages that begin late and end
    early, single tokens, rows to skip, at every offset to the groups of rows that
    a warp looks at."""
    bs = cuda_lib
    rng = random.Random(page + D)
    gen = torch.Generator(device=DEV).manual_seed(H + D + page)
    slots, pages = [], 0
    kinds = [("whole", 5 * page), ("single", 40), ("part", 12), ("whole", 2 * page + 1), ("skip", 37), ("part", 9)]
    while len(slots) < 2100:
        kind, n = kinds[rng.randrange(len(kinds))]
        if kind == "skip":
            slots += [-1] * rng.randrange(1, n)
        elif kind == "whole":
            first = pages * page + rng.choice([0, 0, 1, page - 1])
            slots += range(first, first + n)
            pages += n // page + 2
        else:
            for _ in range(n):
                m = 1 if kind == "single" else rng.randrange(1, page + 1)
                off = rng.randrange(0, page - m + 1)
                slots += range(pages * page + off, pages * page + off + m)
                pages += 1
    T = len(slots)
    # pages anywhere in the cache; inside a request they follow one another in the rows only
    ids = list(range(pages))
    rng.shuffle(ids)
    slots = [s if s < 0 else ids[s // page] * page + s % page for s in slots]
    cache = make_cache(bs, gen, pages, H, page, D)
    qkv = torch.randn((T, 3 * H, D), device=DEV, generator=gen)
    qkv *= torch.exp2(torch.randint(-6, 7, (T, 1, 1), device=DEV, generator=gen).float())
    qkv = qkv.to(dt)
    check_append(bs, qkv[:, H:2 * H], qkv[:, 2 * H:], slots, cache, page)
    assert bs.device_status()[0] == bs.BS_OK


def test_append_extremes(cuda_lib):
    """Amax exactly at, next to and far from 448 * 2^e; zero rows; the clamped ends of the scale range."""
    bs = cuda_lib
    vals = [448.0, 449.0, 3.5, 3.515625, 3.484375, 0.0, 1e-30, 2.0 ** -24, 448.0 * 2.0 ** -32, 1e20, 3e30, 7.0, 2.0 ** 70]
    T = len(vals)
    x = torch.zeros((T, 1, 64), device=DEV)
    x[:, 0, 5] = torch.tensor(vals, device=DEV)
    x[:, 0, 6] = -x[:, 0, 5] / 3
    cache = make_cache(bs, torch.Generator(device=DEV).manual_seed(1), T, 1, 16, 64)
    for off in (0, 3):
        check_append(bs, x, -x, [16 * i + off for i in range(T)], cache, 16)
    xb = x.to(torch.bfloat16)
    check_append(bs, xb, xb, [16 * i for i in range(T)], cache, 16)


def test_append_skips_slots_past_the_cache(cuda_lib):
    bs = cuda_lib
    cache = make_cache(bs, torch.Generator(device=DEV).manual_seed(2), 3, 2, 16, 64)
    x = torch.randn((4, 2, 64), device=DEV)
    bs.clear_device_status()
    check_append(bs, x, x, [5, 48, -1, 1000], cache, 16)
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()


def test_append_past_32_bits(cuda_lib):
    """Codes of a page whose byte offset passes 2^32."""
    bs = cuda_lib
    page, H, D = 128, 8, 128
    pages = (1 << 32) // (page * H * D) + 3
    k = torch.zeros((pages, H, page, D), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    cache = bs.KVCache(k, v, torch.ones((pages, H), device=DEV), torch.ones((pages, H), device=DEV))
    x = torch.randn((2, H, D), device=DEV, dtype=torch.bfloat16)
    slots = [(pages - 1) * page + 7, (pages - 2) * page]
    bs.kv_append(x, x, i32(slots), cache)
    for i, s in enumerate(slots):
        for codes, scale in ((k, cache.k_scale), (v, cache.v_scale)):
            got = codes[s // page, :, s % page].view(torch.float8_e4m3fn).float() * scale[s // page][:, None]
            assert (got - x[i].float()).abs().max() <= 2.0 ** -4 * x[i].float().abs().max()
    assert int((k.view(-1, H * page * D).amax(1) > 0).sum()) == 2
