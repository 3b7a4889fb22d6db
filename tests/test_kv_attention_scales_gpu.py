"""Attention over pages whose scales lie far apart, each (request, KV head) held to
the scales of its own pages.

A weight below fp16's normal range is off by at most 2^-25, its code by a factor of
at most 448, and the sum of the weights over their scales is at least 1 over the
largest scale s that the row sees, so beside the relative terms of
test_kv_attention_gpu the error is at most  m 2^-25 448 s."""
import math

import pytest
import torch

from tests import decode_reference as ref
from tests.test_kv_attention_gpu import build, i32, values

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(bs, q, cache, table, cu, kv, page):
    T, Hq, D = q.shape
    Hkv = cache.k.shape[1]
    lse = torch.empty((T, Hq), device=DEV)
    bs.clear_device_status()
    out = bs.kv_attention(q, cache, i32(table), i32(cu), i32(kv), 0, lse=lse).double()
    assert bs.device_status()[0] == bs.BS_OK
    want, wlse, A, S = ref.attention(q.double(), values(cache.k, cache.k_scale), values(cache.v, cache.v_scale), table, cu,
                                     kv, page, D ** -0.5)
    floor = torch.zeros((T, Hq, 1), dtype=torch.float64, device=DEV)
    for b, m in enumerate(kv):
        if m:
            s = cache.v_scale[table[b][:-(-m // page)]].amax(0).double()        # [Hkv]
            floor[cu[b]:cu[b + 1], :, 0] = (m * 2.0 ** -25 * 448 * s).repeat_interleave(Hq // Hkv)
    e = (D + 16) * 2.0 ** -24 * S[..., None]
    bound = (2.0 ** -11 + 2 * e) * A + floor + 2.0 ** -8 * want.abs() + 1e-300
    err = (out - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    seen = wlse > -math.inf
    le = (lse.double() - wlse).abs()[seen]
    assert bool((le <= (e[..., 0] + 2.0 ** -20 * (1 + wlse.abs()))[seen]).all())
    # the bound would not let zeros pass, for any request and KV head
    for b, m in enumerate(kv):
        if m and cu[b + 1] > cu[b]:
            w = (want.abs() > bound)[cu[b]:cu[b + 1]].view(-1, Hkv, Hq // Hkv * D)
            assert bool(w.any(2).any(0).all())


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [301, 77, 1]), ([90, 3, 1], [301, 77, 20]),
                                            ([300, 2, 200], [700, 70, 210])])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (24, 4, 128, 64)])
def test_far_apart(cuda_lib, q_lens, kv_lens, Hq, Hkv, D, page):
    bs = cuda_lib
    gen = torch.Generator(device=DEV).manual_seed(sum(q_lens) + D)
    q, cache, table, cu = build(bs, 13, kv_lens, q_lens, Hq, Hkv, D, page)
    shape = cache.v_scale.shape

    def scales(lo, hi):
        return torch.exp2(torch.randint(lo, hi, shape, device=DEV, generator=gen).float())

    cache.v_scale.copy_(scales(-30, 21))
    check(bs, q, cache, table, cu, kv_lens, page)
    cache.k_scale.copy_(scales(-30, -5))
    cache.v_scale.mul_(1.37)                 # any positive scale
    check(bs, q, cache, table, cu, kv_lens, page)
    # one KV head far below the others, and pages near one another
    v = scales(-2, 1)
    v[:, 0] *= 2.0 ** -28
    v[:, 1] *= 2.0 ** 20
    cache.v_scale.copy_(v)
    check(bs, q, cache, table, cu, kv_lens, page)
    # one request far below the others
    v = scales(-2, 1)
    v[[i for i in table[0] if i >= 0]] *= 2.0 ** -28
    cache.v_scale.copy_(v)
    check(bs, q, cache, table, cu, kv_lens, page)
