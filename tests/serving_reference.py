"""Plain 64-bit references of the rotary append, the 4-bit cache and the adapters, from
their definitions in include/bsgemm.h (no library code).  Steps that the definitions
round to fp32 are computed in 64 bits and rounded: products, sums and quotients of two
fp32 values are then correctly rounded (53 >= 2 * 24 + 2 bits)."""
import torch

from tests import decode_reference as ref


def fl(x):
    return x.float().double()


def rotate(x, positions, angles, interleaved):
    """x [T, H, D] (fp32 or bf16), rotated, as float64 values of fp32 numbers."""
    y = x.double()
    R = angles.shape[1]
    a = angles.double()[positions.long()][:, None]
    c, s = a[..., :R // 2], a[..., R // 2:]
    x1, x2 = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., :R // 2], y[..., R // 2:R])
    y1, y2 = fl(fl(x1 * c) - fl(x2 * s)), fl(fl(x2 * c) + fl(x1 * s))
    y = y.clone()
    if interleaved:
        y[..., 0:R:2], y[..., 1:R:2] = y1, y2
    else:
        y[..., :R // 2], y[..., R // 2:R] = y1, y2
    return y


def round_e4m3(x):
    """Nearest e4m3 value of a non-negative x, ties to the even code, at most 448."""
    powers = torch.tensor([2.0 ** e for e in range(-9, 7)], dtype=torch.float64, device=x.device)
    a = x.clamp(max=512.0)
    step = powers[torch.frexp(a)[1].long().clamp(min=-5) + 5]
    return (torch.round(a / step) * step).clamp(max=448.0)


def e4m3_code(v):
    """Codes of non-negative e4m3 values."""
    table = ref.e4m3_table()[:127].to(v.device)
    code = torch.searchsorted(table, v.contiguous())
    assert bool((table[code] == v).all())
    return code.to(torch.uint8)


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def quantize4(x):
    """x [.., D] float64 of fp32 values -> packed codes [.., D / 2] and scale codes [.., D / 16]."""
    g = x.unflatten(-1, (-1, 16))
    nan = g.isnan().any(-1)
    finite = torch.where(g.isfinite(), g.abs(), 0.0)
    scale = round_e4m3(fl(finite.amax(-1) / 6))
    q = fl(torch.where(scale[..., None] > 0, g.nan_to_num(0.0, 1e300, -1e300) / scale[..., None], 0.0))
    a = q.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = torch.round(a / step) * step
    mag = torch.searchsorted(torch.tensor(E2M1, dtype=torch.float64, device=x.device), a.contiguous())
    code = mag | (torch.signbit(g).long() << 3)
    code = torch.where((scale[..., None] > 0) & ~nan[..., None], code, 0)
    sc = torch.where(nan, torch.full_like(nan, 0x7f, dtype=torch.uint8), e4m3_code(scale))
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return (code[..., 0] | code[..., 1] << 4).to(torch.uint8), sc


def values4(codes, scales):
    """Values [.., D] float64 of packed codes and scale codes."""
    e = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    x = torch.stack([e[(codes & 15).long()], e[(codes >> 4).long()]], -1).flatten(-2)
    return x * ref.e4m3_table().to(codes.device)[scales.long()].repeat_interleave(16, -1)


def lora(x, y, a, b, cu, which, scales):
    """float64 result, and sum |x||A| |B| |scale| for the error bound."""
    out, size = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    for i, w in enumerate(which):
        lo, hi = cu[i], cu[i + 1]
        if w < 0 or hi <= lo:
            continue
        s = 1.0 if scales is None else float(scales[w])
        xd, ad, bd = x[lo:hi].double(), a[w].double(), b[w].double()
        out[lo:hi] += (xd @ ad.T) @ bd.T * s
        size[lo:hi] = (xd.abs() @ ad.abs().T) @ bd.abs().T * abs(s)
    return out, size
