"""One layer's attention in serving: FP4 projections around an 8-bit paged cache.

Order of a step, for requests that each bring some new tokens (a prompt, one
token, a few drafted ones, or none):

  1. bs_kv_plan       pages for the new tokens from the free list, their slots
  2. bs_fp4_matvec    q, k and v of the new tokens in one product with the
                      concatenated FP4 weights, x left in bf16 (at most 16
                      tokens; more go through q4_quantize and bs_gemm with the
                      same weights, unless ``activations`` says otherwise)
  3. bs_kv_append     k and v, read where the product left them, to 8 bits in
                      their slots
  4. bs_kv_attention  q over each request's cached tokens, causal
  5. bs_fp4_matvec    the output projection (or q4_quantize and bs_gemm)

bs_kv_release gives the pages of finished requests back.  Lengths, tables and
the free list stay on the device and nothing synchronises the host, so a step of
fixed shape can be captured in a CUDA graph and replayed, between steps of any
other shape: the attention's scratch belongs to the layer.  (A step of 17 to 32
tokens also uses the stream's workspace of bs_gemm: run one such step on the
capture stream first, or each replay zeroes one of its own.)

The kernels are the library's; this module holds the buffers and calls them in
order.  No rotation or normalisation is applied to q and k.
"""
from __future__ import annotations

import torch

from . import (KVCache, gemm_fp4, kv_append, kv_attention, kv_attention_workspace, kv_plan, kv_release, matvec_fp4,
               q4_quantize)

MATVEC_ROWS = 16   # the most rows that bs_fp4_matvec takes


def fp4_linear(x, codes, sf, out=None, tensor_scale=None, activations="auto"):
    """x bf16 [T, K] times FP4 weights (codes [N, K/2] and scales of q4_quantize, or
    with ``tensor_scale`` of q4_quantize_two_level).

    activations  "bf16": x as it is, 16 rows at a time, so that a row's result does
                 not depend on how many are beside it; "fp4": x quantized, whatever
                 their number; "auto": bf16 up to 16 rows, FP4 from 17 on, the
                 faster for each, at the price of x's rounding to FP4 for the
                 rows of a larger call.  bs_gemm takes N in multiples of 128: other
                 weights always meet x in bf16 (and "fp4" is refused)."""
    T, N = x.shape[0], codes.shape[0]
    if activations not in ("auto", "bf16", "fp4"):
        raise ValueError(f"activations are auto, bf16 or fp4, not {activations!r}")
    if activations == "fp4" and N % 128:
        raise ValueError(f"fp4 activations: {N} columns are no multiple of 128")
    if activations == "fp4" or (activations == "auto" and T > MATVEC_ROWS and N % 128 == 0):
        xc, xsf, _ = q4_quantize(x)
        return gemm_fp4(xc, xsf, codes, sf, x.shape[1], out=out, b_tensor_scale=tensor_scale)
    if T <= MATVEC_ROWS:
        return matvec_fp4(x, codes, sf, out=out, tensor_scale=tensor_scale)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=x.device)
    for at in range(0, T, MATVEC_ROWS):
        matvec_fp4(x[at:at + MATVEC_ROWS], codes, sf, out=out[at:at + MATVEC_ROWS], tensor_scale=tensor_scale)
    return out


class DecodeAttention:
    """Attention of one layer over requests 0 .. B - 1.

    w_qkv, w_out    (codes, scales) of q4_quantize, or (codes, scales, tensor scale)
                    of q4_quantize_two_level, for bf16 weights
                    [(Hq + 2 Hkv) D, hidden] (rows of q, then k, then v) and
                    [hidden, Hq D]
    activations     of the two products, as fp4_linear takes them.  With "auto" the
                    same token gets coarser q, k, v and output in a step of 17
                    tokens and more than in a smaller one
    lens            int32 [B], the cached tokens of each request (device)
    n_free          int32 [1], the pages left (device)
    """

    def __init__(self, w_qkv, w_out, Hq: int, Hkv: int, D: int, requests: int, num_pages: int, page_size: int,
                 max_pages: int, activations: str = "auto"):
        rows = (Hq + 2 * Hkv) * D
        if w_qkv[0].shape[0] != rows or w_out[0].shape[1] * 2 != Hq * D:
            raise ValueError(f"DecodeAttention: w_qkv has {rows} rows and w_out {Hq * D} columns")
        if activations not in ("auto", "bf16", "fp4"):
            raise ValueError(f"DecodeAttention: activations are auto, bf16 or fp4, not {activations!r}")
        if activations == "fp4" and (rows % 128 or w_out[0].shape[0] % 128):
            raise ValueError("DecodeAttention: fp4 activations need weights whose rows are multiples of 128")
        dev = w_qkv[0].device
        self.activations = activations
        self.w_qkv, self.w_out = w_qkv, w_out
        self.Hq, self.Hkv, self.D, self.page_size = Hq, Hkv, D, page_size
        self.cache = KVCache.empty(num_pages, Hkv, page_size, D, device=dev)
        self.table = torch.full((requests, max_pages), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(num_pages, dtype=torch.int32, device=dev)
        self.n_free = torch.full((1,), num_pages, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.workspace = kv_attention_workspace(D, dev)

    def _linear(self, x, weight):
        codes, sf, *scale = weight
        return fp4_linear(x, codes, sf, tensor_scale=scale[0] if scale else None, activations=self.activations)

    def step(self, x, new_lens, max_new: int):
        """x bf16 [T, hidden], the new tokens of request 0, then 1, ..;
        new_lens int32 [B] on the device, their sum at most T, each at most
        max_new.  Returns bf16 [T, hidden]; rows past the sum of new_lens hold
        nothing of use.  A request for which the pages do not suffice gets zeros
        and keeps its length (device status BS_ERR_PAGES)."""
        T, q_rows, kv_rows = x.shape[0], self.Hq * self.D, self.Hkv * self.D
        cu, kv_lens, slots, left = kv_plan(self.lens, new_lens, self.table, self.free, self.n_free, self.page_size, T)
        qkv = self._linear(x, self.w_qkv)
        q, k, v = qkv.split([q_rows, kv_rows, kv_rows], 1)
        kv_append(k.view(T, self.Hkv, self.D), v.view(T, self.Hkv, self.D), slots, self.cache)
        att = kv_attention(q.view(T, self.Hq, self.D), self.cache, self.table, cu, kv_lens, max_new,
                           workspace=self.workspace)
        self.n_free.copy_(left)
        torch.maximum(self.lens, kv_lens, out=self.lens)
        return self._linear(att.view(T, q_rows), self.w_out)

    def release(self, done):
        """Give back the pages of the requests with done[b] != 0 (int32 [B])."""
        kv_release(self.lens, done, self.table, self.free, self.n_free, self.page_size)
        self.lens.masked_fill_(done != 0, 0)
