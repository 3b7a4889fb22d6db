"""NaN and infinite keys and values: their own codes, and nothing else's."""
import math

import pytest
import torch

from tests import decode_reference as ref
from tests.test_kv_cache_gpu import i32, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,page,rows", [(2, 64, 16, 40), (1, 128, 64, 300), (3, 128, 128, 2500), (2, 64, 32, 2200)])
def test_nonfinite(cuda_lib, dt, H, D, page, rows):
    """Against the same append with 0 in their places: scales and all other codes,
    those of the pages' earlier tokens among them, are the same; an infinity's code is
    +-448, a NaN's a NaN.  Pages that begin in this call and pages begun before."""
    bs = cuda_lib
    gen = torch.Generator(device=DEV).manual_seed(rows + D)
    off = page // 3
    slots = list(range(off, off + rows))
    pages = -(-(off + rows) // page)
    x = torch.randn((2, rows, H, D), device=DEV, generator=gen).to(dt)
    at = torch.randint(0, x.numel(), (60,), device=DEV, generator=gen)
    at[0], at[1] = 3, x.numel() - 5          # a token of the page begun before; the last row
    x.view(-1)[at] = 0
    x[0, page - off, 0] = 0                  # a page that begins with a row of nothing finite
    clean, dirty = make_cache(bs, gen, pages, H, page, D), None
    dirty = bs.KVCache(*(t.clone() for t in clean))
    bs.kv_append(x[0], x[1], i32(slots), clean)
    kind = torch.tensor([math.inf, -math.inf, math.nan], device=DEV)
    y = x.clone()
    y.view(-1)[at] = kind[torch.arange(60, device=DEV) % 3].to(dt)
    y[0, page - off, 0] = math.inf
    bs.clear_device_status()
    bs.kv_append(y[0], y[1], i32(slots), dirty)
    assert bs.device_status()[0] == bs.BS_OK
    table = ref.e4m3_table().to(DEV)
    s = torch.tensor(slots, device=DEV)
    for which, name in enumerate("kv"):
        assert torch.equal(getattr(clean, name + "_scale"), getattr(dirty, name + "_scale"))
        want, got = (table[getattr(c, name).long()] for c in (clean, dirty))
        v = y[which].double()
        new = want[s // page, :, s % page]
        new = torch.where(v.isnan(), v, torch.where(v.isinf(), 448 * v.sign(), new))
        want[s // page, :, s % page] = new
        assert torch.equal(want.isnan(), got.isnan())
        assert torch.equal(want.nan_to_num(500.0), got.nan_to_num(500.0))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_largest_finite(cuda_lib, dt):
    """Values up to the largest finite one, beside infinities: the scale is 2^64, its largest."""
    bs = cuda_lib
    big = torch.finfo(dt).max
    vals = [2.0 ** 126, 2.0 ** 127, big, -big]
    x = torch.zeros((2 * len(vals), 1, 64), device=DEV, dtype=dt)
    x[::2, 0, 3] = torch.tensor(vals, device=DEV).to(dt)
    x[1::2, 0, 9] = math.inf                 # two rows a page
    x[::2, 0, 4] = 2.0 ** 64
    cache = make_cache(bs, torch.Generator(device=DEV).manual_seed(1), len(vals), 1, 16, 64)
    bs.kv_append(x, x, i32([16 * (i // 2) + i % 2 for i in range(len(x))]), cache)
    v = ref.e4m3_table().to(DEV)[cache.k.long()]
    assert bool((cache.k_scale == 2.0 ** 64).all()) and bool((cache.v_scale == 2.0 ** 64).all())
    assert v[:, 0, 0, 3].tolist() == [448, 448, 448, -448] and bool((v[:, 0, 0, 4] == 1).all())
    assert bool((v[:, 0, 1, 9] == 448).all()) and bool((v[:, 0, 1, 10:] == 0).all())
