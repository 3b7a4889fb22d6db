"""The decode-step calls on a second GPU, and from a second context on the first,
after they ran in the first context of the process."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


class Context:
    """A context of its own on device 0, current inside the block, and zeroed memory in it."""

    def __enter__(self):
        self.cu = ctypes.CDLL("libcuda.so.1")
        self.ctx, self.held = ctypes.c_void_p(), []
        self.ok(self.cu.cuCtxCreate_v2(ctypes.byref(self.ctx), 0, 0))
        return self

    def __exit__(self, *exc):
        self.cu.cuCtxSynchronize()
        for p in self.held:
            self.cu.cuMemFree_v2(p)
        self.cu.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p()))
        self.cu.cuCtxDestroy_v2(self.ctx)

    def ok(self, r):
        assert r == 0, f"driver call failed: {r}"

    def memory(self, n, byte=0):
        p = ctypes.c_uint64()
        self.ok(self.cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(max(n, 16))))
        self.held.append(p)
        self.ok(self.cu.cuMemsetD8_v2(p, ctypes.c_ubyte(byte), ctypes.c_size_t(max(n, 16))))
        return p.value

    def read(self, p, n):
        out = (ctypes.c_ubyte * n)()
        self.ok(self.cu.cuMemcpyDtoH_v2(out, ctypes.c_uint64(p), ctypes.c_size_t(n)))
        return bytes(out)


def calls(bs, memory):
    """(call, address and bytes that it sets to zero) for each kernel that needs more than 48 KB of shared memory."""
    lib = bs.load()
    B, page, Hq, Hkv, D = 8192, 64, 16, 2, 128
    lens, one = memory(4 * B), memory(4 * B)
    kv_lens = memory(4 * B, 0xff)
    a = bs._KV_PLAN_ARGS.pack(lens, one, B, memory(4 * B), 1, 1, memory(64), memory(4), 8, page, 0, memory(4 * B + 4),
                              kv_lens, 0, memory(4))
    yield lambda: lib.bs_kv_plan(a, None), kv_lens, 4 * B
    for T in (1, 300):
        out, most = memory(T * Hq * D * 2, 0xff), T
        ints = [memory(16), memory(16)]     # cu_q 0, 0 and a length of 0: see below
        codes, scales = memory(4 * Hkv * page * D), memory(4 * Hkv * 4, 0x3f)
        head = (memory(T * Hq * D * 2), Hq * D, D, out, Hq * D, D, 0, codes, codes, scales, scales, 4, page, memory(16), 4, 4,
                *ints, 1, T, Hq, Hkv, D, most, 0.1, 0)
        n = int(lib.bs_kv_attention_workspace_bytes(bs._KV_ATTENTION_ARGS.pack(*head, 0, 0)))
        b = bs._KV_ATTENTION_ARGS.pack(*head, memory(n), n)
        yield lambda b=b: lib.bs_kv_attention(b, None), None, 0
    for M, N, K in ((1, 256, 1024), (16, 256, 1024), (1, 256, 8192), (16, 256, 8192)):
        y = memory(M * N * 4, 0xff)
        c = bs._FP4_MATVEC_ARGS.pack(memory(M * K * 2), K, M, memory(N * K // 2), memory(N * K // 16), N, K, 1.0, 0, 0, y, 0, N)
        yield lambda c=c: lib.bs_fp4_matvec(c, None), y, M * N * 4


def run_on(bs, device):
    held = {}

    def memory(n, byte=0):
        t = torch.full((max(n, 16),), byte, dtype=torch.uint8, device="cuda")
        held[t.data_ptr()] = t
        return t.data_ptr()

    with torch.cuda.device(device):
        torch.zeros(1, device="cuda")
        for call, out, n in calls(bs, memory):
            torch.cuda.synchronize()
            assert call() == bs.BS_OK, bs.load().bs_last_error()
            torch.cuda.synchronize()
            assert out is None or not bool(held[out][:n].any())


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one GPU")
def test_second_gpu(cuda_lib):
    run_on(cuda_lib, 0)
    run_on(cuda_lib, 1)
    run_on(cuda_lib, 0)


def test_second_context(cuda_lib):
    bs = cuda_lib
    run_on(bs, 0)
    with Context() as second:
        for call, out, n in calls(bs, second.memory):
            assert call() == bs.BS_OK, bs.load().bs_last_error()
            second.ok(second.cu.cuCtxSynchronize())
            assert out is None or not any(second.read(out, n))
    assert bs.device_status()[0] == bs.BS_OK
    assert float(torch.ones(4, device="cuda").sum()) == 4.0
