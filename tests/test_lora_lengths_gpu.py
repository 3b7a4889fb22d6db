"""Adapters for prompts, single tokens, requests without rows and padding in one call: a
request's tiles follow from its own rows.  Bound of test_lora_gpu."""
import random

import pytest
import torch

from tests.test_lora_gpu import build, check, i32, offsets

pytestmark = pytest.mark.gpu
DEV = "cuda"


def mixed(seed, prompts, singles, empty):
    rng = random.Random(seed)
    lens = list(prompts) + [1] * singles + [0] * empty
    rng.shuffle(lens)
    return lens, [rng.randint(-1, 2) for _ in lens]


CALLS = [([2300], 60, 140), ([2300], 200, 0), ([2400, 31, 32, 33, 500], 90, 100), ([1700, 600, 8, 9], 250, 30),
         ([30] * 100 + [40] * 20, 0, 5), ([700], 69, 0), ([70, 300], 1, 400), ([4100], 2, 60), ([12] * 300, 10, 0)]


@pytest.mark.parametrize("prompts,singles,empty", CALLS)
@pytest.mark.parametrize("r,dt", [(16, torch.bfloat16), (64, torch.float32), (128, torch.bfloat16), (24, torch.float32)])
def test_lengths(cuda_lib, prompts, singles, empty, r, dt):
    """Into an output of its own and in place; rows behind the last request as they were."""
    bs = cuda_lib
    lens, which = mixed(r + singles, prompts, singles, empty)
    T = sum(lens)
    x, y, a, b, s = build(singles, T + 5, 200, 136, r, 3, dt)
    out = torch.full_like(y, 9.0)
    got = check(bs, x, y, a, b, offsets(lens), which, s, out=out)
    assert bool((out[T:] == 9.0).all())
    again = y.clone()
    bs.lora_add(x, again, a, b, i32(offsets(lens)), i32(which), scales=s, out=again)
    assert torch.equal(got[:T], again[:T]) and torch.equal(again[T:], y[T:])
    for i, w in enumerate(which):
        if w < 0:
            lo = sum(lens[:i])
            assert torch.equal(got[lo:lo + lens[i]], y[lo:lo + lens[i]])


@pytest.mark.parametrize("n,r,singles,empty", [(600, 128, 69, 0), (2400, 16, 0, 200), (2400, 16, 199, 0), (1500, 64, 20, 100),
                                               (5000, 64, 120, 0)])
def test_a_prompt_is_what_it_is_alone(cuda_lib, n, r, singles, empty):
    """A prompt's rows, and a single token's, beside other requests and requests without rows have the bits that they
    have alone (K of one slice: no sum depends on how many CTAs share it)."""
    bs = cuda_lib
    lens, _ = mixed(n, [n], singles, empty)
    at = lens.index(n)
    lo = sum(lens[:at])
    x, y, a, b, s = build(r, sum(lens), 64, 136, r, 2, torch.float32)
    which = [1] * len(lens)
    got = check(bs, x, y, a, b, offsets(lens), which, s)
    alone = bs.lora_add(x[lo:lo + n], y[lo:lo + n], a, b, i32([0, n]), i32([1]), scales=s)
    assert torch.equal(got[lo:lo + n], alone)
    row = next((sum(lens[:i]) for i, k in enumerate(lens) if k == 1), None)
    if row is not None:
        assert torch.equal(got[row:row + 1], bs.lora_add(x[row:row + 1], y[row:row + 1], a, b, i32([0, 1]), i32([1]), scales=s))


def test_contract_breaks_in_a_large_call(cuda_lib):
    """Offsets that fall or pass T, among requests of both kinds: the status, and no row outside the call."""
    bs = cuda_lib
    T, B = 2600, 200
    x, y, a, b, s = build(4, T, 72, 136, 16, 3, torch.bfloat16)
    room = torch.full((3 * T, 136), 9.0, device=DEV, dtype=torch.bfloat16)
    good = offsets([1] * (B - 1) + [T - B + 1])
    for place, value in ((5, -7), (100, 3), (B, T + 50), (B, (1 << 31) - 1), (1, T), (0, -1)):
        cu = list(good)
        cu[place] = value
        bs.clear_device_status()
        bs.lora_add(x, y, a, b, i32(cu), i32([i % 3 for i in range(B)]), scales=s, out=room[T:2 * T])
        assert bs.device_status()[0] == bs.BS_ERR_OFFSETS, (place, value)
        assert bool((room[:T] == 9).all()) and bool((room[2 * T:] == 9).all())
    bs.clear_device_status()
    bs.lora_add(x, y, a, b, i32([0, T] * (B // 2) + [0]), i32([0] * B), scales=s, out=room[T:2 * T])   # all claim all
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()
    assert bool((room[:T] == 9).all()) and bool((room[2 * T:] == 9).all())
    check(bs, x, y, a, b, good, [i % 3 for i in range(B)], s)


def test_captured(cuda_lib):
    """A call of both kinds as a graph, whose lengths change between replays."""
    bs = cuda_lib
    lens, which = mixed(1, [1800, 400], 180, 0)
    T = sum(lens)
    x, y, a, b, s = build(2, T, 264, 136, 32, 3, torch.bfloat16)
    cu, w = i32(offsets(lens)), i32(which)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bs.lora_add(x, y, a, b, cu, w, scales=s)
    for seed in (1, 2, 3):
        random.Random(seed).shuffle(lens)
        cu.copy_(i32(offsets(lens)))
        g.replay()
        want = bs.lora_add(x, y, a, b, cu, w, scales=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
