"""Refusals of the decode-step entry points (host side, before any launch) and
checks of the 64-bit reference that the GPU tests compare with (no GPU needed)."""
import ctypes

import pytest
import torch

from tests import decode_reference as ref


@pytest.fixture(scope="module")
def bs():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_gemm_q4_gb300 as bs
    bs.load()
    return bs


P = ctypes.c_void_p
F = 1 << 20          # never dereferenced: validation fails first


def test_plan_refusals(bs):
    f = bs.load().bs_kv_plan
    good = [F, F + 64, 4, F + 128, 8, 8, F, F + 256, 32, 64, 10, F, F + 512, F, F + 1024]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v or 0
        return f(bs._KV_PLAN_ARGS.pack(*a), None)

    assert f(None, None) == bs.BS_ERR_INVALID

    assert call(a2=-1) == bs.BS_ERR_INVALID
    assert call(a2=8193) == bs.BS_ERR_UNSUPPORTED
    assert call(a9=48) == bs.BS_ERR_UNSUPPORTED            # page size
    assert call(a10=-1) == bs.BS_ERR_INVALID
    assert call(a10=1 << 31) == bs.BS_ERR_INVALID
    assert call(a4=7) == bs.BS_ERR_INVALID                 # ld_table < max_pages
    assert call(a4=1 << 26, a5=1 << 26) == bs.BS_ERR_INVALID   # positions pass 2^31
    assert call(a14=F + 256) == bs.BS_ERR_INVALID          # n_free_out is n_free
    assert call(a12=F) == bs.BS_ERR_INVALID                # kv_lens is seq_lens
    for i in (0, 1, 3, 6, 7, 11, 12, 13, 14):
        assert call(**{f"a{i}": None}) == bs.BS_ERR_INVALID, i
        assert call(**{f"a{i}": F + 2}) == bs.BS_ERR_ALIGN, i
    r = bs.load().bs_kv_release
    good = [F, F, 4, F, 8, 8, F, F, 32, 64, None]
    for i, v, want in ((2, -1, 1), (2, 9000, 3), (9, 8, 3), (0, None, 1), (1, None, 1), (3, None, 1), (7, None, 1),
                       (4, 3, 1), (0, F + 1, 2), (2, 0, 0)):
        a = list(good)
        a[i] = v
        assert r(*a) == want, (i, v)


def test_append_refusals(bs):
    lib = bs.load()
    assert lib.bs_kv_append(None, None) == bs.BS_ERR_INVALID

    names = "k v dtype T Hkv D k_token_stride k_head_stride v_token_stride v_head_stride slots k_codes v_codes k_scales " \
            "v_scales num_pages page_size".split()
    good = dict(zip(names, (F, F, 1, 10, 8, 128, 1024, 128, 1024, 128, F, F, F, F, F, 100, 64)))

    def call(**kw):
        a = {k: v or 0 for k, v in {**good, **kw}.items()}
        return lib.bs_kv_append(bs._KV_APPEND_ARGS.pack(*a.values()), None)

    assert call(D=96) == bs.BS_ERR_UNSUPPORTED
    assert call(page_size=24) == bs.BS_ERR_UNSUPPORTED
    assert call(Hkv=0) == bs.BS_ERR_INVALID
    assert call(T=-1) == bs.BS_ERR_INVALID
    assert call(dtype=5) == bs.BS_ERR_INVALID
    assert call(num_pages=1 << 30) == bs.BS_ERR_UNSUPPORTED     # rows pass 2^31
    assert call(Hkv=40000, num_pages=1) == bs.BS_ERR_UNSUPPORTED
    assert call(k_token_stride=1020) == bs.BS_ERR_ALIGN
    assert call(v_head_stride=4) == bs.BS_ERR_ALIGN
    for name in ("k", "v", "slots", "k_codes", "v_codes", "k_scales", "v_scales"):
        assert call(**{name: None}) == bs.BS_ERR_INVALID, name
        assert call(**{name: F + 2}) == bs.BS_ERR_ALIGN, name
    assert call(T=0, k=None) == bs.BS_OK


def test_attention_refusals(bs):
    lib = bs.load()
    assert lib.bs_kv_attention(None, None) == bs.BS_ERR_INVALID

    names = "q q_token_stride q_head_stride out out_token_stride out_head_stride lse k_codes v_codes k_scales v_scales " \
            "num_pages page_size block_table ld_table max_pages cu_q kv_lens B T Hq Hkv D max_q_len softmax_scale " \
            "wait_timeout_us workspace workspace_bytes".split()
    good = dict(zip(names, (F, 4096, 128, F, 4096, 128, F, F, F, F, F, 100, 64, F, 8, 8, F, F, 4, 4, 32, 8, 128, 1, 0.1, 0,
                            0, 0)))

    def call(**kw):
        a = {k: v or 0 for k, v in {**good, **kw}.items()}
        return lib.bs_kv_attention(bs._KV_ATTENTION_ARGS.pack(*a.values()), None)

    assert call(D=256) == bs.BS_ERR_UNSUPPORTED
    assert call(page_size=0) == bs.BS_ERR_UNSUPPORTED
    assert call(Hq=12) == bs.BS_ERR_INVALID                      # not a multiple of Hkv
    assert call(Hq=0) == bs.BS_ERR_INVALID
    assert call(softmax_scale=0.0) == bs.BS_ERR_INVALID
    assert call(softmax_scale=float("nan")) == bs.BS_ERR_INVALID
    assert call(B=-1) == bs.BS_ERR_INVALID
    assert call(T=1 << 40) == bs.BS_ERR_INVALID
    assert call(max_q_len=-1) == bs.BS_ERR_INVALID
    assert call(wait_timeout_us=-1) == bs.BS_ERR_INVALID
    assert call(ld_table=7) == bs.BS_ERR_INVALID
    assert call(q_token_stride=4100) == bs.BS_ERR_ALIGN
    assert call(out_head_stride=4) == bs.BS_ERR_ALIGN
    for name in ("q", "out", "k_codes", "v_codes", "k_scales", "v_scales", "block_table", "cu_q", "kv_lens"):
        assert call(**{name: None}) == bs.BS_ERR_INVALID, name
        assert call(**{name: F + 2}) == bs.BS_ERR_ALIGN, name
    assert call(lse=F + 2) == bs.BS_ERR_ALIGN
    assert call(T=0, q=None) == bs.BS_OK
    assert call(B=0, q=None) == bs.BS_OK


def test_matvec_refusals(bs):
    f = bs.load().bs_fp4_matvec
    good = [F, 256, 4, F, F, 100, 256, 1.0, 0, 0, F, 1, 100]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v or 0
        return f(bs._FP4_MATVEC_ARGS.pack(*a), None)

    assert f(None, None) == bs.BS_ERR_INVALID

    assert call(a2=17) == bs.BS_ERR_UNSUPPORTED
    assert call(a2=-1) == bs.BS_ERR_INVALID
    assert call(a6=96) == bs.BS_ERR_ALIGN
    assert call(a6=0) == bs.BS_ERR_INVALID
    assert call(a5=-5) == bs.BS_ERR_INVALID
    assert call(a11=4) == bs.BS_ERR_INVALID
    assert call(a1=248) == bs.BS_ERR_INVALID               # ldx < K
    assert call(a12=99) == bs.BS_ERR_INVALID               # ldo < N
    assert call(a1=260) == bs.BS_ERR_ALIGN
    for i in (0, 3, 4, 10):
        assert call(**{f"a{i}": None}) == bs.BS_ERR_INVALID, i
    for i in (0, 3, 4):
        assert call(**{f"a{i}": F + 8}) == bs.BS_ERR_ALIGN, i
    assert call(a10=F + 1) == bs.BS_ERR_ALIGN
    assert call(a9=F + 1) == bs.BS_ERR_ALIGN
    assert call(a8=F + 2) == bs.BS_ERR_ALIGN
    assert call(a5=0, a0=None, a12=0) == bs.BS_OK
    assert call(a2=0, a0=None) == bs.BS_OK


def test_binding_refusals(bs):
    """Types, shapes and layouts that the binding turns away before the library sees them."""
    c = bs.KVCache.empty(4, 2, 16, 64, device="cpu")
    x = torch.zeros(3, 2, 64)
    sl = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        bs.kv_append(x[:, :1], x, sl, c)
    with pytest.raises(ValueError):
        bs.kv_append(x, x.to(torch.bfloat16), sl, c)
    with pytest.raises(TypeError):
        bs.kv_append(x, x, sl.long(), c)
    with pytest.raises(ValueError):
        bs.kv_append(x, x, sl, c._replace(k=c.k.transpose(1, 2)))
    with pytest.raises(TypeError):
        bs.kv_append(x, x, sl, c._replace(k=c.k.float()))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    t, cu, kv = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        bs.kv_attention(q.float(), c, t, cu, kv, 1)
    with pytest.raises(ValueError):
        bs.kv_attention(q[..., :32], c, t, cu, kv, 1)
    with pytest.raises(ValueError):
        bs.kv_attention(q, c, t, cu[:1], kv, 1)
    with pytest.raises(ValueError):
        bs.kv_attention(q, c, t, cu, kv, 1, lse=torch.zeros(3, 2))
    with pytest.raises(TypeError):
        bs.kv_attention(q, c, t.long(), cu, kv, 1)
    with pytest.raises(ValueError):
        bs.kv_plan(kv, cu, t, kv, kv, 16, 4)
    with pytest.raises(TypeError):
        bs.kv_plan(kv.long(), kv, t, kv, kv, 16, 4)
    w, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    xb = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bs.matvec_fp4(xb.float(), w, s)
    with pytest.raises(ValueError):
        bs.matvec_fp4(xb[:, :32], w, s)
    with pytest.raises(ValueError):
        bs.matvec_fp4(xb, w, s[:100])
    with pytest.raises(ValueError):
        bs.matvec_fp4(xb, w, s, bias=torch.zeros(8))
    with pytest.raises(ValueError):
        bs.matvec_fp4(xb, w, s, out=torch.zeros(2, 9))


def test_reference_rounding_is_e4m3():
    """The reference's rounding against torch's cast, over every e4m3 midpoint and its neighbours."""
    v = ref.e4m3_table()[:127]
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), torch.tensor([500.0, 1e9], dtype=torch.float64)])
    x = torch.cat([x, -x])
    want = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()
    assert torch.equal(ref.round_e4m3(x), want)


def test_reference_attention_is_softmax():
    """The reference on one page-aligned request against torch's softmax."""
    torch.manual_seed(0)
    k, v = torch.randn(3, 2, 16, 64, dtype=torch.float64), torch.randn(3, 2, 16, 64, dtype=torch.float64)
    q = torch.randn(2, 4, 64, dtype=torch.float64)
    out, lse, _, _ = ref.attention(q, k, v, [[2, 0, 1]], [0, 2], [40], 16, 0.125)
    for i in range(2):
        for h in range(4):
            kk = torch.cat([k[2, h // 2], k[0, h // 2], k[1, h // 2]])[:39 + i]
            vv = torch.cat([v[2, h // 2], v[0, h // 2], v[1, h // 2]])[:39 + i]
            z = kk @ q[i, h] * 0.125
            assert torch.allclose(out[i, h], torch.softmax(z, 0) @ vv, atol=1e-13)
            assert abs(float(lse[i, h] - torch.logsumexp(z, 0))) < 1e-13
