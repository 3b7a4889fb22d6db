"""Device-side lengths and offsets that break the contract of kv_attention: the
status says so, rows outside the call are not touched, other requests are served."""
import pytest
import torch

from tests import decode_reference as ref
from tests.test_kv_attention_gpu import build, i32, values

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Hq,Hkv,D,T", [(8, 2, 64, 40), (16, 2, 128, 400)])
@pytest.mark.parametrize("kind", ["negative", "descending", "past", "far past", "all past"])
def test_offsets(cuda_lib, Hq, Hkv, D, T, kind):
    bs = cuda_lib
    first, kv = T // 3, [300, 500, 200]
    good = [0, first, 2 * first, T]
    bad = {"negative": [0, first, -7, T], "descending": [0, first, first // 2, T], "past": [0, first, 2 * first, T + 5],
           "far past": [0, first, 2 * first, (1 << 31) - 1], "all past": [0, first, T + 100, T + 5000]}[kind]
    q, cache, table, _ = build(bs, 3, kv, [b - a for a, b in zip(good, good[1:])], Hq, Hkv, D, 64)
    room = torch.zeros((3 * T, Hq, D), dtype=torch.bfloat16, device=DEV)
    room[T:2 * T] = q
    out, lse = torch.full_like(room, 3.0), torch.full((3 * T, Hq), 7.0, device=DEV)
    bs.clear_device_status()
    want = bs.kv_attention(q, cache, i32(table), i32(good), i32(kv), 0)
    assert bs.device_status()[0] == bs.BS_OK
    bs.kv_attention(room[T:2 * T], cache, i32(table), i32(bad), i32(kv), 0, out=out[T:2 * T], lse=lse[T:2 * T])
    assert bs.device_status()[0] == bs.BS_ERR_OFFSETS
    bs.clear_device_status()
    for x, v in ((out, 3.0), (lse, 7.0)):
        assert bool((x[:T] == v).all()) and bool((x[2 * T:] == v).all())
    if kind != "descending":      # there the third request's rows begin among the first's
        o, _, A, S = ref.attention(q[:first].double(), values(cache.k, cache.k_scale), values(cache.v, cache.v_scale),
                                   table, [0, first], kv[:1], 64, D ** -0.5)
        # weights to fp16, scores summed in fp32, output to bf16
        bound = (2.0 ** -11 + (D + 16) * 2.0 ** -23 * S[..., None]) * A + 2.0 ** -8 * o.abs() + kv[0] * 2.0 ** -25 * 448 * 2.0 ** -6
        assert bool(((out[T:T + first].double() - o).abs() <= bound).all())
    # and the workspace is as the next call needs it
    assert torch.equal(bs.kv_attention(q, cache, i32(table), i32(good), i32(kv), 0), want)
    assert bs.device_status()[0] == bs.BS_OK


@pytest.mark.parametrize("q_lens", [[1, 2], [150, 40]])
def test_lengths(cuda_lib, q_lens):
    """A length that the table cannot hold, or a negative one, sets the status (the
    first is cut to the table's, the second counts as 0); the longest it can hold does not."""
    bs = cuda_lib
    q, cache, table, cu = build(bs, 9, [320, 100], q_lens, 16, 2, 64, 64)
    t = i32([r[:5] for r in table])
    for kv, same, status in (([320, 100], None, bs.BS_OK), ([321, 100], [320, 100], bs.BS_ERR_OFFSETS),
                             ([(1 << 31) - 1, 100], [320, 100], bs.BS_ERR_OFFSETS), ([320, -1], [320, 0], bs.BS_ERR_OFFSETS),
                             ([-(1 << 31), 100], [0, 100], bs.BS_ERR_OFFSETS)):
        bs.clear_device_status()
        out = bs.kv_attention(q, cache, t, i32(cu), i32(kv), 0)
        assert bs.device_status()[0] == status, kv
        if same:
            assert torch.equal(out, bs.kv_attention(q, cache, t, i32(cu), i32(same), 0))
    bs.clear_device_status()
