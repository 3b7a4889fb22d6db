"""Sizes and layouts that the binding of the decode-step calls hands on as bare
addresses: what is too small or laid out otherwise is refused (no GPU needed: a
call that went on would reach the stand-ins)."""
import pytest
import torch


@pytest.fixture
def bs(monkeypatch):
    import fp8_quantized_gemm_q4_gb300 as bs

    def reached(*args):
        raise AssertionError("the call went on")

    monkeypatch.setattr(bs, "_stream", reached)
    monkeypatch.setattr(bs, "_not_on_gpu", reached)
    monkeypatch.setattr(bs, "_lib", object())
    return bs


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_sizes_and_layouts(bs):
    w, x = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(2, 64).bfloat16()
    sf = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(AssertionError):
        bs.matvec_fp4(x, w, sf, tensor_scale=torch.ones(1))
    with pytest.raises(ValueError):                       # every second byte
        bs.matvec_fp4(x, w, torch.zeros(1024, dtype=torch.uint8)[::2])
    for ts in (torch.ones(0), torch.ones(2)):
        with pytest.raises(TypeError):
            bs.matvec_fp4(x, w, sf, tensor_scale=ts)
    out = (i32(3), i32(2), i32(4), i32(1))
    with pytest.raises(AssertionError):
        bs.kv_plan(i32(2), i32(2), i32(2, 3), i32(9), i32(1), 16, 4, out=out)
    with pytest.raises(ValueError):
        bs.kv_plan(i32(2), i32(2), i32(2, 3), i32(9), i32(0), 16, 4, out=out)
    with pytest.raises(ValueError):
        bs.kv_plan(i32(2), i32(2), i32(2, 3), i32(9), i32(1), 16, 4, out=(*out[:3], i32(0)))
    with pytest.raises(ValueError):
        bs.kv_release(i32(2), i32(2), i32(2, 3), i32(9), i32(0), 16)


def test_longest_table():
    """Lengths that pass 2^31 when they are rounded up to a tile are refused (host side; nothing is launched)."""
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_gemm_q4_gb300 as bs
    F = 1 << 20

    def call(max_pages, page):
        return bs.load().bs_kv_attention(bs._KV_ATTENTION_ARGS.pack(
            F, 4096, 128, F, 4096, 128, F, F, F, F, F, 100, page, F, max_pages, max_pages, F, F, 0, 4, 32, 8, 128, 1, 0.1, 0,
            0, 0), None)

    for page in (16, 32, 64, 128):
        most = ((1 << 31) - 128) // page
        assert call(most, page) == bs.BS_OK                 # no requests: nothing to do
        assert call(most + 1, page) == bs.BS_ERR_INVALID


def test_arguments_by_position():
    """What calls pass by position stays where it was; later arguments are added at the end."""
    import inspect

    import fp8_quantized_gemm_q4_gb300 as bs
    from fp8_quantized_gemm_q4_gb300 import decode

    def names(f):
        return list(inspect.signature(f).parameters)

    assert names(bs.kv_attention)[:10] == ["q", "cache", "block_table", "cu_q", "kv_lens", "max_q_len", "softmax_scale", "out",
                                           "lse", "stream"]
    assert names(decode.fp4_linear)[:4] == ["x", "codes", "sf", "out"]
    assert names(decode.DecodeAttention)[:9] == ["w_qkv", "w_out", "Hq", "Hkv", "D", "requests", "num_pages", "page_size",
                                                 "max_pages"]


def test_plan_outputs_apart_from_inputs():
    """An output of kv_plan at the address of an input that all its CTAs read is refused (host side)."""
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_gemm_q4_gb300 as bs
    F = 1 << 20
    #        seq  new       B table    ld w free      n_free   cap page T  cu        kv        slots     left
    good = [F, F + 64, 4, F + 128, 8, 8, F + 192, F + 256, 32, 64, 10, F + 320, F + 512, F + 640, F + 1024]
    for out in (11, 12, 13, 14):
        for src in (0, 1, 6, 7):
            a = list(good)
            a[out] = a[src]
            assert bs.load().bs_kv_plan(bs._KV_PLAN_ARGS.pack(*a), None) == bs.BS_ERR_INVALID, (out, src)
