"""Plain 64-bit reference of the decode-step operators, from their definitions
in include/bsgemm.h (no library code)."""
import math

import torch


def e4m3_table():
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if b & 128 else x)
    v[127] = v[255] = math.nan
    return torch.tensor(v, dtype=torch.float64)


def round_e4m3(x):
    """Nearest e4m3 value, ties to the even mantissa, saturating at 448."""
    a = x.abs().clamp(max=512.0)
    e = torch.frexp(a)[1].clamp(min=-5)
    step = torch.ldexp(torch.ones_like(a), e - 4)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def power_scale(amax):
    """Smallest 2^e, -32 <= e <= 64, with amax <= 448 * 2^e (a float)."""
    for e in range(-32, 65):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 64


def kv_plan(seq, new, table, free, n_free, page, T):
    """Python lists in, (table, cu, kv, slots, n_free, refused) out."""
    table = [list(r) for r in table]
    cu, kv, slots, end, refused = [0], [], [-1] * T, 0, []
    left = n_free
    for b in range(len(seq)):
        before, after = -(-seq[b] // page), -(-(seq[b] + new[b]) // page)
        need = after - before
        fits = need == 0 or end + need <= n_free
        if fits:
            for j in range(need):
                table[b][before + j] = free[n_free - 1 - end - j]
            left -= need
            for i in range(new[b]):
                p = seq[b] + i
                slots[cu[-1] + i] = table[b][p // page] * page + p % page
        else:
            refused.append(b)
        end += need
        cu.append(cu[-1] + new[b])
        kv.append(seq[b] + new[b] if fits else 0)
    return table, cu, kv, slots, left, refused


def kv_append(x, slots, values, scales, page):
    """x [T, H, D] float64; values [pages, H, page, D] (codes' values) and
    scales [pages, H] float64, updated in place."""
    T = len(slots)
    r = 0
    while r < T:
        if slots[r] < 0 or slots[r] >= values.shape[0] * page:
            r += 1
            continue
        n = 1
        while r + n < T and slots[r + n] == slots[r] + n and slots[r + n] % page:
            n += 1
        pid, off = slots[r] // page, slots[r] % page
        for h in range(x.shape[1]):
            s = power_scale(float(x[r:r + n, h].abs().max()))
            if off:
                old = float(scales[pid, h])
                s = max(s, old)
                if s > old:
                    values[pid, h, :off] = round_e4m3(values[pid, h, :off] * (old / s))
            values[pid, h, off:off + n] = round_e4m3(x[r:r + n, h] / s)
            scales[pid, h] = s
        r += n


def attention(q, k, v, table, cu, kv_lens, page, scale):
    """q [T, Hq, D]; k, v [pages, Hkv, page, D] float64 with their scales in.
    Returns out, lse, and for the error bound A = sum p |v| / sum p and
    S = the largest sum_d |q_d k_d| * scale of a row."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    dev = q.device
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    A = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    S = torch.zeros((T, Hq), dtype=torch.float64, device=dev)
    for b, m in enumerate(kv_lens):
        n = cu[b + 1] - cu[b]
        if n == 0 or m == 0:
            continue
        ids = torch.tensor(table[b][:-(-m // page)], device=dev)
        kb = k[ids].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :m].repeat_interleave(G, 0)
        vb = v[ids].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :m].repeat_interleave(G, 0)
        qb = q[cu[b]:cu[b + 1]].transpose(0, 1)
        z = qb @ kb.transpose(1, 2) * scale
        seen = torch.arange(m, device=dev)[None] <= (m - n + torch.arange(n, device=dev))[:, None]
        z = z.masked_fill(~seen, -math.inf)
        any_seen = seen.any(1)
        top = z.amax(-1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(z - top)
        tot = p.sum(-1, keepdim=True)
        safe = tot.clamp(min=1e-300)
        rows = slice(cu[b], cu[b + 1])
        out[rows] = ((p @ vb) / safe * any_seen[None, :, None]).transpose(0, 1)
        A[rows] = ((p @ vb.abs()) / safe * any_seen[None, :, None]).transpose(0, 1)
        lse[rows] = (top + torch.log(tot))[..., 0].transpose(0, 1)
        S[rows] = ((qb.abs() @ kb.abs().transpose(1, 2)) * scale).masked_fill(~seen, 0).amax(-1).transpose(0, 1)
    return out, lse, A, S


def fp4_weights(codes, sf, N, K):
    """Weight values [N, K] float64 of packed E2M1 codes and MMA-layout scales."""
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64)
    q = codes.cpu().long()
    w = torch.empty((N, K), dtype=torch.float64)
    for k, nib in ((0, q % 16), (1, q // 16)):
        w[:, k::2] = half[nib % 8] / 2 * (1 - 2 * (nib // 8)).double()
    n = torch.arange(N)[:, None]
    g = torch.arange(K // 16)[None]
    at = ((n // 128) * (K // 64) + g // 4) * 512 + (n % 32) * 16 + (n % 128) // 32 * 4 + g % 4
    s = e4m3_table()[sf.cpu().long()[at]]
    return w * s.repeat_interleave(16, 1)
