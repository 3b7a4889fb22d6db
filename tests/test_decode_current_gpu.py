"""Tensors of another GPU than the current one are refused by the binding of the serving
calls: their kernels would run on the current GPU's stream.  The current GPU is stood in for,
so one GPU does."""
import pytest
import torch


class Elsewhere(torch.Tensor):
    """A tensor that says it is on this GPU."""
    @staticmethod
    def of(t, device):
        x = t.as_subclass(Elsewhere)
        x.there = device
        return x

    def get_device(self):
        return self.there

    @property
    def is_cuda(self):
        return self.there >= 0


@pytest.fixture
def bs(monkeypatch):
    import fp8_quantized_gemm_q4_gb300 as bs

    class Library:
        def __getattr__(self, name):
            raise AssertionError("the call went on to the library")

    monkeypatch.setattr(bs, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(bs, "_lib", Library())
    return bs


def calls(bs):
    bf, z = torch.bfloat16, lambda *s: torch.zeros(s, dtype=torch.int32)
    c4, c8 = bs.KVCacheFP4.empty(4, 2, 16, 64, device="cpu"), bs.KVCache.empty(4, 2, 16, 64, device="cpu")
    q, k, a = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf), torch.zeros(9, 32)
    w, sf, x = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.zeros(2, 64, dtype=bf)
    att = lambda kind: (lambda q, t, cu, kv, o, l, w, *c: bs.kv_attention(q, kind(*c), t, cu, kv, 3, out=o, lse=l, workspace=w))
    app = lambda kind: (lambda q, k, v, s, p, a, o, *c: bs.kv_append_rotary(q, k, v, s, p, a, kind(*c), q_out=o))
    return [(lambda *t: bs.kv_plan(*t[:5], 16, 4, out=t[5:]), [z(2), z(2), z(2, 3), z(9), z(1), z(3), z(2), z(4), z(1)]),
            (lambda *t: bs.kv_release(*t, 16), [z(2), z(2), z(2, 3), z(9), z(1)]),
            (lambda k, v, s, *c: bs.kv_append(k, v, s, bs.KVCache(*c)), [k, k, z(3), *c8]),
            (lambda k, v, s, *c: bs.kv_append(k, v, s, bs.KVCacheFP4(*c)), [k, k, z(3), *c4]),
            (att(bs.KVCache), [q, z(1, 4), z(2), z(1), q, torch.zeros(3, 4), w, *c8]),
            (att(bs.KVCacheFP4), [q, z(1, 4), z(2), z(1), q, torch.zeros(3, 4), w, *c4]),
            (app(bs.KVCache), [q, k, k, z(3), z(3), a, q, *c8]), (app(bs.KVCacheFP4), [q, k, k, z(3), z(3), a, q, *c4]),
            (lambda s, k, v, *c: bs.kv_gather(bs.KVCacheFP4(*c), s, out=(k, v)), [z(3), k, k, *c4]),
            (lambda s, cu, o: bs.kv_positions(s, cu, 3, out=o), [z(2), z(3), z(3)]),
            (lambda x, w, s, b, t, o: bs.matvec_fp4(x, w, s, bias=b, tensor_scale=t, out=o),
             [x, w, sf, x[0, :8], torch.ones(1), torch.zeros(2, 8)]),
            (lambda x, y, a, b, cu, w, s, o: bs.lora_add(x, y, a, b, cu, w, scales=s, out=o),
             [q[:, 0], k[:, 0], q.new_zeros(2, 8, 64), q.new_zeros(2, 64, 8), z(3), z(2), torch.zeros(2), k[:, 1]])]


def test_another_gpu(bs, monkeypatch):
    """All tensors on a GPU that is not the current one; each in turn on another than the rest; all where they belong."""
    for f, args in calls(bs):
        monkeypatch.setattr(bs, "_device", lambda: 0)
        with pytest.raises(ValueError, match="GPU"):
            f(*(Elsewhere.of(t, 1) for t in args))
        monkeypatch.setattr(bs, "_device", lambda: 1)
        for i in range(len(args)):
            with pytest.raises(ValueError, match="GPU"):
                f(*(Elsewhere.of(t, int(j != i)) for j, t in enumerate(args)))
        with pytest.raises(AssertionError, match="went on"):
            f(*(Elsewhere.of(t, 1) for t in args))
