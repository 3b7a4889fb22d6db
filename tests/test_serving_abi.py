"""Refusals of the rotary append, the row gather, attention over the 4-bit cache and the
adapters: the library's before any launch, the binding's before any of the library's; and
checks of the 64-bit references that the GPU tests compare with (no GPU needed)."""
import pytest
import torch

from tests import serving_reference as sref


@pytest.fixture(scope="module")
def bs():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_quantized_gemm_q4_gb300 as bs
    bs.load()
    return bs


F = 1 << 20          # never dereferenced: validation fails first


def caller(f, pack, good, *more):
    def call(**kw):
        assert set(kw) <= set(good)
        return f(pack.pack(*({k: v or 0 for k, v in {**good, **kw}.items()}).values()), *more, None)
    return call


def test_append_rotary_refusals(bs):
    names = "q q_token_stride q_head_stride q_out q_out_token_stride q_out_head_stride k v dtype Hq Hkv D T k_token_stride " \
            "k_head_stride v_token_stride v_head_stride slots positions angles max_positions rotary_dim interleaved " \
            "cache_format page_size k_codes v_codes k_scales v_scales num_pages".split()
    G = 2 * F
    good = dict(zip(names, (F, 1024, 128, G, 1024, 128, F, F, 1, 8, 8, 128, 10, 1024, 128, 1024, 128, F, F, F, 100, 128, 0,
                            bs.FMT_FP4, 64, F, F, F, F, 100)))
    f = bs.load().bs_kv_append_rotary
    assert f(None, None) == bs.BS_ERR_INVALID
    call = caller(f, bs._KV_APPEND_ROTARY_ARGS, good)
    for kw in (dict(D=96), dict(page_size=24), dict(num_pages=1 << 30), dict(Hkv=40000, num_pages=1), dict(Hq=1 << 17),
               dict(T=(1 << 31) - 1)):
        assert call(**kw) == bs.BS_ERR_UNSUPPORTED, kw
    for kw in (dict(Hkv=0), dict(T=-1), dict(T=1 << 31), dict(Hq=-1), dict(dtype=5), dict(cache_format=2), dict(rotary_dim=144),
               dict(rotary_dim=24), dict(rotary_dim=-16), dict(max_positions=0), dict(max_positions=1 << 31), dict(num_pages=-1),
               dict(q_out=F, dtype=0), dict(q_out=F, q_out_token_stride=2048), dict(q_out=F, q_out_head_stride=256)):
        assert call(**kw) == bs.BS_ERR_INVALID, kw
    for name in "k_token_stride k_head_stride v_token_stride v_head_stride q_token_stride q_head_stride q_out_token_stride " \
                "q_out_head_stride".split():
        assert call(**{name: 1020}) == bs.BS_ERR_ALIGN, name
    for name in "q q_out k v slots positions angles k_codes v_codes k_scales v_scales".split():
        assert call(**{name: None}) == bs.BS_ERR_INVALID, name
        assert call(**{name: G + 2}) == bs.BS_ERR_ALIGN, name
    assert call(T=(1 << 30) + 4, Hq=0, Hkv=1, q=None, q_out=None) == bs.BS_ERR_UNSUPPORTED
    assert call(T=0, k=None) == bs.BS_OK


def test_positions_refusals(bs):
    f = bs.load().bs_kv_positions
    for args, want in (((F, F + 64, -1, 3, F + 128), bs.BS_ERR_INVALID), ((F, F + 64, 9000, 3, F + 128), bs.BS_ERR_UNSUPPORTED),
                       ((F, F + 64, 2, -1, F + 128), bs.BS_ERR_INVALID), ((F, F + 64, 2, 1 << 31, F + 128), bs.BS_ERR_INVALID),
                       ((F, F + 64, 2, 3, None), bs.BS_ERR_INVALID), ((None, F + 64, 2, 3, F + 128), bs.BS_ERR_INVALID),
                       ((F, None, 2, 3, F + 128), bs.BS_ERR_INVALID), ((F, F + 2, 2, 3, F + 128), bs.BS_ERR_ALIGN),
                       ((F, F + 64, 2, 3, F), bs.BS_ERR_INVALID), ((F, F + 64, 2, 0, None), bs.BS_OK)):
        assert f(*args, None) == want, args


def test_gather_refusals(bs):
    names = "slots T Hkv D k v k_token_stride k_head_stride v_token_stride v_head_stride cache_format page_size k_codes v_codes " \
            "k_scales v_scales num_pages".split()
    good = dict(zip(names, (F, 10, 8, 128, F, F, 1024, 128, 1024, 128, bs.FMT_FP8, 64, F, F, F, F, 100)))
    f = bs.load().bs_kv_gather
    assert f(None, None) == bs.BS_ERR_INVALID
    call = caller(f, bs._KV_GATHER_ARGS, good)
    for kw, want in ((dict(D=96), bs.BS_ERR_UNSUPPORTED), (dict(page_size=1), bs.BS_ERR_UNSUPPORTED), (dict(T=-1), bs.BS_ERR_INVALID),
                     (dict(cache_format=7), bs.BS_ERR_INVALID), (dict(T=(1 << 31) - 1), bs.BS_ERR_UNSUPPORTED),
                     (dict(Hkv=0), bs.BS_ERR_INVALID), (dict(k_token_stride=1020), bs.BS_ERR_ALIGN),
                     (dict(v_head_stride=4), bs.BS_ERR_ALIGN), (dict(T=0), bs.BS_OK)):
        assert call(**kw) == want, kw
    for name in "slots k v k_codes v_codes k_scales v_scales".split():
        assert call(**{name: None}) == bs.BS_ERR_INVALID, name
        assert call(**{name: F + 2}) == bs.BS_ERR_ALIGN, name


def test_attention_refusals(bs):
    names = "q q_token_stride q_head_stride out out_token_stride out_head_stride lse k_codes v_codes k_scales v_scales num_pages " \
            "page_size block_table ld_table max_pages cu_q kv_lens B T Hq Hkv D max_q_len softmax_scale wait_timeout_us " \
            "workspace workspace_bytes".split()
    good = dict(zip(names, (F, 1024, 128, F, 1024, 128, F, F, F, 0, 0, 100, 64, F, 9, 9, F, F, 3, 10, 8, 2, 128, 4, 0.1, 0, F, 1 << 30)))
    f = bs.load().bs_kv_attention_fp4
    assert f(None, F, F, None) == bs.BS_ERR_INVALID

    def call(ks=F, vs=F, **kw):
        return f(bs._KV_ATTENTION_ARGS.pack(*({k: v or 0 for k, v in {**good, **kw}.items()}).values()), ks, vs, None)

    assert call(ks=None) == bs.BS_ERR_INVALID and call(vs=None) == bs.BS_ERR_INVALID
    assert call(ks=F + 8) == bs.BS_ERR_ALIGN and call(vs=F + 8) == bs.BS_ERR_ALIGN
    for kw, want in ((dict(D=80), bs.BS_ERR_UNSUPPORTED), (dict(Hq=7), bs.BS_ERR_INVALID), (dict(softmax_scale=0.0), bs.BS_ERR_INVALID),
                     (dict(k_codes=F + 8), bs.BS_ERR_ALIGN), (dict(ld_table=3), bs.BS_ERR_INVALID), (dict(T=0), bs.BS_OK)):
        assert call(**kw) == want, kw


def test_lora_refusals(bs):
    names = "x ldx a b scales cu_rows which y ldy out ldo dtype B T K N r adapters".split()
    good = dict(zip(names, (F, 256, F, F, F, F, F, F, 512, 2 * F, 512, 1, 3, 10, 256, 512, 16, 4)))
    lib = bs.load()
    assert lib.bs_lora_add(None, None) == bs.BS_ERR_INVALID
    call = caller(lib.bs_lora_add, bs._LORA_ARGS, good)
    for kw in (dict(T=-1), dict(T=1 << 31), dict(B=-1), dict(K=0), dict(N=-8), dict(adapters=-1), dict(dtype=3), dict(ldx=248),
               dict(ldy=504), dict(ldo=504), dict(out=4 * F, y=4 * F, ldo=1024), dict(out=F, y=4 * F)):
        assert call(**kw) == bs.BS_ERR_INVALID, kw
    for kw in (dict(r=0), dict(r=12), dict(r=136), dict(B=9000), dict(K=1 << 23, ldx=1 << 23)):
        assert call(**kw) == bs.BS_ERR_UNSUPPORTED, kw
    for kw in (dict(K=252), dict(N=508), dict(ldx=260), dict(ldy=516), dict(ldo=516)):
        assert call(**kw) == bs.BS_ERR_ALIGN, kw
    for name in "x a b cu_rows which y out".split():
        assert call(**{name: None}) == bs.BS_ERR_INVALID, name
        assert call(**{name: 4 * F + 2}) == bs.BS_ERR_ALIGN, name
    assert call(scales=F + 2) == bs.BS_ERR_ALIGN
    assert call(T=0) == bs.BS_OK and call(B=0) == bs.BS_OK and call(N=0) == bs.BS_OK


def test_outputs_at_inputs_are_refused(bs):
    """An output at the address of an input that others still read, or of the other output."""
    lib, A = bs.load(), [F << i for i in range(12)]
    q, q_out, k, v, x, y, a, b, out = A[:9]
    pack = bs._KV_APPEND_ROTARY_ARGS.pack
    for o, qq in ((k, q), (v, q), (k, k), (v, v)):
        assert lib.bs_kv_append_rotary(pack(qq, 1024, 128, o, 1024, 128, k, v, bs.DTYPE_BF16, 8, 2, 128, 10, 256, 128, 256, 128, F, F, F,
                                            50, 128, 0, bs.FMT_FP4, 64, F, F, F, F, 100), None) == bs.BS_ERR_INVALID
    assert lib.bs_kv_gather(bs._KV_GATHER_ARGS.pack(F, 10, 8, 128, k, k, 1024, 128, 1024, 128, bs.FMT_FP8, 64, F, F, F, F, 100),
                            None) == bs.BS_ERR_INVALID
    for o in (x, a, b):
        assert lib.bs_lora_add(bs._LORA_ARGS.pack(x, 256, a, b, 0, F, F, y, 512, o, 512, 1, 3, 10, 256, 512, 16, 4), None) == bs.BS_ERR_INVALID


@pytest.fixture
def stopped(bs, monkeypatch):
    """The binding, whose calls must not reach the library."""
    def reached(stream=None):
        raise AssertionError("the call went on to the library")

    monkeypatch.setattr(bs, "_stream", reached)
    monkeypatch.setattr(bs, "_lib", object())
    return bs


def test_binding_refusals(stopped):
    bs = stopped
    bf, i32 = torch.bfloat16, torch.int32
    c4, c8 = bs.KVCacheFP4.empty(4, 2, 16, 64, device="cpu"), bs.KVCache.empty(4, 2, 16, 64, device="cpu")
    q, k, at = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, dtype=i32)
    angles = bs.rotary_angles(5, 32, device="cpu")
    z = lambda *s, dt=i32: torch.zeros(s, dtype=dt)
    app = lambda **kw: bs.kv_append_rotary(**{**dict(q=q, k=k, v=k, slots=at, positions=at, angles=angles, cache=c4), **kw})
    att = lambda cache: bs.kv_attention(q, cache, z(1, 4), z(2), z(1), 3)
    x, y, a, b = z(6, 64, dt=bf), z(6, 32, dt=bf), z(2, 8, 64, dt=bf), z(2, 32, 8, dt=bf)
    lora = lambda **kw: bs.lora_add(**{**dict(x=x, y=y, a=a, b=b, cu_rows=z(3), which=z(2)), **kw})
    values = [lambda: app(k=k[:2]), lambda: app(q=q[:2]), lambda: app(v=k.float()), lambda: app(q=q.float()), lambda: app(q=None, q_out=q),
              lambda: app(k=k[:, :1]), lambda: app(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
              lambda: app(cache=c4._replace(k_scale=c4.k_scale[..., :2])), lambda: app(cache=bs.KVCacheFP4(*c8)),
              lambda: app(cache=c4._replace(k=c4.k.transpose(0, 1).contiguous().transpose(0, 1))),
              lambda: att(bs.KVCacheFP4(*c8)), lambda: att(tuple(c4)), lambda: bs.kv_gather(c4, at, out=(k, k[:2])),
              lambda: lora(y=y[:5]), lambda: lora(b=b[:1]), lambda: lora(a=z(2, 8, 56, dt=bf)), lambda: lora(cu_rows=z(2)),
              lambda: lora(x=x.t().contiguous().t()), lambda: lora(out=y[:, :16]), lambda: lora(b=b.transpose(1, 2)),
              lambda: bs.kv_positions(at, at, 3),
              # the last check of each: nothing is on a GPU
              lambda: bs.kv_positions(at, z(4), 3),
              app, lambda: app(cache=c8), lambda: att(c4), lambda: bs.kv_gather(c4, at), lambda: bs.kv_gather(c8, at), lora,
              lambda: bs.kv_append(k, k, at, c4)]
    types = [lambda: app(slots=at.long()), lambda: app(positions=at.long()), lambda: app(positions=at[:2]), lambda: app(positions=None),
             lambda: app(angles=angles.double()), lambda: app(q_out=q.float()), lambda: app(k=k.half(), v=k.half(), q=q.half()),
             lambda: app(cache=c4._replace(k_scale=c4.k_scale.view(torch.int8))), lambda: bs.kv_gather(c4, at.long()),
             lambda: bs.kv_gather(c4, at, out=(k.float(), k.float())), lambda: lora(x=x.float()), lambda: lora(out=y.float()),
             lambda: lora(which=z(2).long()), lambda: lora(scales=torch.zeros(3)), lambda: lora(scales=torch.zeros(2).double())]
    for i, f in enumerate(values):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
    for i, f in enumerate(types):
        with pytest.raises(TypeError):
            f()
            raise AssertionError(i)


@pytest.mark.gpu
def test_each_tensor_on_the_host(cuda_lib, stopped):
    """Each argument in turn left on the host, the others on the GPU."""
    bs = stopped
    g = lambda t: t.cuda()
    c4, c8 = bs.KVCacheFP4.empty(4, 2, 16, 64), bs.KVCache.empty(4, 2, 16, 64)
    bf = torch.bfloat16
    q, k, at = g(torch.zeros(3, 4, 64, dtype=bf)), g(torch.zeros(3, 2, 64, dtype=bf)), g(torch.zeros(3, dtype=torch.int32))
    n = lambda *s: g(torch.zeros(s, dtype=torch.int32))
    calls = [(lambda q, k, v, s, p, a, o, *c: bs.kv_append_rotary(q, k, v, s, p, a, bs.KVCacheFP4(*c), q_out=o),
              [q, k, k, at, at, bs.rotary_angles(5, 32), q, *c4]),
             (lambda s, k, v, *c: bs.kv_gather(c, s, out=(k, v)), [at, k, k, *c8]),
             (lambda q, t, cu, kv, out, *c: bs.kv_attention(q, bs.KVCacheFP4(*c), t, cu, kv, 3, out=out), [q, n(1, 4), n(2), n(1), q, *c4]),
             (lambda x, y, a, b, cu, w, s, o: bs.lora_add(x, y, a, b, cu, w, scales=s, out=o),
              [q[:, 0], k[:, 0], q.new_zeros(2, 8, 64), q.new_zeros(2, 64, 8), n(3), n(2), torch.zeros(2, device="cuda"), k[:, 1]])]
    for f, args in calls:
        for i in range(len(args)):
            a = list(args)
            a[i] = a[i].cpu()
            with pytest.raises(ValueError, match="GPU"):
                f(*a)


def test_reference_rotation():
    """Position 0 turns nothing, lengths stay, and a turn by a + b is a turn by a and one by b (in 64 bits)."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 2, 64, generator=g)
    pos = torch.tensor([0, 1, 5, 9, 100, 31])
    f = 10000.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    a = torch.arange(101, dtype=torch.float64)[:, None] * f
    angles = torch.cat([a.cos(), a.sin()], 1).float()
    import fp8_quantized_gemm_q4_gb300 as bs
    assert torch.equal(bs.rotary_angles(101, 32, device="cpu"), angles)
    for mixed in (False, True):
        y = sref.rotate(x, pos, angles, mixed)
        assert torch.equal(y[0], x[0].double()) and torch.equal(y[..., 32:], x[..., 32:].double())
        assert torch.allclose(y.norm(dim=-1), x.double().norm(dim=-1), rtol=1e-6)
        i, j = (2, 3) if mixed else (1, 17)          # the second pair by hand
        c, s = a[5, 1].cos(), a[5, 1].sin()
        assert abs(float(y[2, 0, i] - (x[2, 0, i].double() * c - x[2, 0, j].double() * s))) < 1e-6
        assert abs(float(y[2, 0, j] - (x[2, 0, j].double() * c + x[2, 0, i].double() * s))) < 1e-6


def test_reference_quantizer():
    """Against the oracle's FP4 quantizer, which shares no code with it."""
    import numpy as np

    import oracle
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(16, 128, generator=g) * torch.exp2(torch.randint(-14, 12, (16, 1), generator=g).float())).bfloat16()
    codes, sf = oracle.q4_quantize(x)
    c, s = sref.quantize4(x.double())
    assert np.array_equal(codes, c.numpy()) and np.array_equal(np.asarray(sf).reshape(16, 8), s.numpy())
    v = sref.values4(c, s)
    step = s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    # a code is at most one scale off; where the scale is rounded down x passes 6 scales: by 6 * 2^-4 of one at most
    # for normal scales, 6 * 2^-10 for subnormal ones (and 0); at 448 by any distance
    off = (v - x.double()).abs()
    assert bool((off <= torch.where(step < 448, step.clamp(min=6 * 2.0 ** -10), off)).all())


def test_reference_lora():
    x, y = torch.tensor([[1.0, 2.0], [3.0, -1.0]]), torch.ones(2, 3)
    a, b = torch.tensor([[[1.0, 1.0]], [[2.0, 0.0]]]), torch.tensor([[[1.0], [0.0], [-1.0]], [[2.0], [1.0], [0.0]]])
    out, size = sref.lora(x, y, a, b, [0, 1, 2], [0, 1], torch.tensor([0.5, 1.0]))
    assert out.tolist() == [[2.5, 1.0, -0.5], [13.0, 7.0, 1.0]] and size.tolist() == [[1.5, 0.0, 1.5], [12.0, 6.0, 0.0]]
