"""Cases, plain forms and 64-bit values of what a serving step on a quantized cache
needs beside the operators of operators.py.

  append      new keys, values and queries with the position rotation applied on the
              way: keys and values into the 8-bit paged cache, queries to bf16
  append4     the same into a 4-bit cache (E2M1 codes, an e4m3 scale for 16 elements
              of a token), and the new rows read back from it
  attention4  causal attention of the new tokens over the 4-bit cache
  adapters    y + scale x A^T B^T with the low-rank adapter (A, B) of each request,
              beside a projection that all requests share

A case is a dict of plain values.  Lengths follow from the case alone (spread
evenly over their logarithm); the seed decides which request has which length,
which pages it owns, which adapter it uses and all values, so that the work of a
case is the same for every seed.
"""
from __future__ import annotations

import math

import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    app, app4, att, ada = dict(op="append"), dict(op="append4"), dict(op="attention4"), dict(op="adapters")
    return [
        # one new token for each of 64 requests, 32 query heads over 8: latency counts
        dict(name="append rotary decode 64", **app, B=64, T=64, Hq=32, Hkv=8, D=128, rot=128, mixed=False, lo=100,
             hi=8000, page=64, x="bf16"),
        # prompts of a prefill batch, most pages written whole
        dict(name="append rotary prefill 16384", **app, B=12, T=16384, Hq=32, Hkv=8, D=128, rot=128, mixed=False,
             lo=30, hi=2000, page=64, x="bf16"),
        # the decode step on the 4-bit cache
        dict(name="append4 decode 64", **app4, B=64, T=64, Hq=32, Hkv=8, D=128, rot=128, mixed=False, lo=100, hi=8000,
             page=64, x="bf16"),
        # short ragged chunks, small pages and heads, half of each head rotated in adjacent pairs, still in fp32
        dict(name="append4 ragged fp32", **app4, B=77, T=1501, Hq=12, Hkv=4, D=64, rot=32, mixed=True, lo=10, hi=3000,
             page=16, x="fp32"),
        dict(name="append4 prefill 16384", **app4, B=12, T=16384, Hq=32, Hkv=8, D=128, rot=128, mixed=False, lo=30,
             hi=2000, page=64, x="bf16"),
        # a single conversation: one token over a short cache
        dict(name="attention4 one request", **att, B=1, T=1, Hq=32, Hkv=8, D=128, lo=1000, hi=1000, page=64),
        # 64 running requests of very different length, grouped heads
        dict(name="attention4 decode 64", **att, B=64, T=64, Hq=32, Hkv=8, D=128, lo=500, hi=16000, page=64),
        # a few drafted tokens for each request to verify, one KV head per query head, small pages
        dict(name="attention4 draft heads", **att, B=16, T=63, Hq=16, Hkv=16, D=64, lo=300, hi=5000, page=16),
        # two chunks of long prompts over what is already cached
        dict(name="attention4 prefill 2048", **att, B=2, T=2048, Hq=32, Hkv=8, D=128, lo=4000, hi=8000, page=128),
        # one token, a small adapter on the output projection
        dict(name="adapters one token", **ada, B=1, T=1, K=4096, N=4096, r=8, n=4, bare=0, y="bf16"),
        # a decode step of 64 requests with 40 adapters among them, some requests without, on q, k and v
        dict(name="adapters decode 64", **ada, B=64, T=64, K=4096, N=6144, r=16, n=40, bare=8, y="bf16"),
        # prompts with adapters of a higher rank
        dict(name="adapters prefill 8190", **ada, B=7, T=8190, K=7168, N=4096, r=64, n=5, bare=1, y="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges; costs no more than the largest listed case of its operator."""
    op = rng.choice(["append", "append4", "append4", "attention4", "attention4", "attention4", "adapters", "adapters"])
    if op in ("append", "append4"):
        B = _log(rng, 1, 128)
        Hkv, G, D = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 3, 4]), rng.choice([64, 128])
        T = rng.choice([B, _log(rng, B, 16384)])
        hi = _log(rng, 10, 4000)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 16, 48]),
                    mixed=rng.random() < 0.4, lo=_log(rng, 1, hi), hi=hi, page=rng.choice([16, 32, 64, 128]),
                    x=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "attention4":
        Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8]), rng.choice([64, 128])
        prefill = rng.random() < 0.3
        B = rng.randint(1, 3) if prefill else _log(rng, 1, 64)
        T = _log(rng, 64, 1500) if prefill else rng.choice([B, B, B * rng.randint(2, 8)])
        hi = _log(rng, 1600, 7000) if prefill else _log(rng, 40, 14000)
        lo = _log(rng, 1500 if prefill else 30, hi)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, lo=max(lo, T // B * 2), hi=max(hi, T // B * 2),
                    page=rng.choice([16, 32, 64, 128]))
    B = _log(rng, 1, 128)
    T = rng.choice([B, _log(rng, B, 6000)])
    return dict(op=op, B=B, T=T, K=64 * _log(rng, 4, 112), N=8 * _log(rng, 16, 900), r=rng.choice([8, 16, 24, 32, 64]),
                n=_log(rng, 1, 64), bare=rng.choice([0, rng.randint(0, B - 1)]), y=rng.choice(["bf16", "bf16", "fp32"]))


def _lengths(c):
    """(tokens cached before, new tokens) of every request, from the case alone."""
    B, T = c["B"], c["T"]
    lo, hi = c.get("lo", 1), c.get("hi", 1)
    old = [int(round(lo * (hi / lo) ** ((i + 1) / B))) for i in range(B)]
    new = [1] * B
    left, total = T - B, B * (B + 1) // 2
    for i in range(B):
        new[i] += left * (i + 1) // total
    new[-1] += T - sum(new)
    if c["op"] == "attention4":  # lo .. hi are the lengths that attention sees
        old = [max(0, n - m) for n, m in zip(old, new)]
    return old, new


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _requests(c, seed):
    """Lengths in the seed's order, and which pages of the pool each request owns (the last of the new tokens included)."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(c["B"], generator=g).tolist()
    old, new = _lengths(c)
    old, new = [old[i] for i in order], [new[i] for i in order]
    ps = c.get("page", 64)
    pages = [-(-(a + b) // ps) for a, b in zip(old, new)]
    pool = torch.randperm(sum(pages) + 8, generator=g).to(torch.int32)
    table = torch.full((c["B"], max(pages) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = pool[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return old, new, cu, table, len(pool)


def _cache8(c, pages, gen):
    """Codes and scales of an 8-bit cache whose values are near N(0, 1); each page and head has a scale of its own."""
    shape = (pages, c["Hkv"], c["page"], c["D"])

    def half():
        scale = torch.exp2(torch.randint(-8, -5, shape[:2], device=DEV, generator=gen).float())
        x = torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16)
        x = (x / scale[:, :, None, None].to(torch.bfloat16)).clamp_(-448, 448)
        return x.to(torch.float8_e4m3fn).view(torch.uint8), scale

    k, ks = half()
    v, vs = half()
    return k, v, ks, vs


def _cache4(c, pages, gen):
    """Codes and scales of a 4-bit cache whose values are near N(0, 1) as it holds them: random codes, scales around 0.4."""
    shape = (pages, c["Hkv"], c["page"])

    def half():
        codes = torch.randint(0, 256, (*shape, c["D"] // 2), device=DEV, generator=gen, dtype=torch.uint8)
        s = torch.rand((*shape, c["D"] // 16), device=DEV, generator=gen, dtype=torch.bfloat16) * 0.4 + 0.15
        return codes, s.to(torch.float8_e4m3fn).view(torch.uint8)

    k, ks = half()
    v, vs = half()
    return k, v, ks, vs


def _angles(rows, rot):
    """cos and sin of position * 10000^(-2 i / rot), i < rot / 2: [rows, rot], as a program lays them out once."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    old, new, cu, table, pages = _requests(c, seed)
    s = dict(c=c, cu=_i32(cu))
    T = c["T"]
    if c["op"] == "adapters":
        K, N, r, n = c["K"], c["N"], c["r"], c["n"]
        g = torch.Generator().manual_seed(seed + 1)
        which = torch.randint(0, n, (c["B"],), generator=g)
        which[torch.randperm(c["B"], generator=g)[:c["bare"]]] = -1
        dt = torch.bfloat16 if c["y"] == "bf16" else torch.float32
        s.update(which=which.to(torch.int32).to(DEV), max_rows=max(new),
                 x=torch.randn((T, K), device=DEV, generator=gen, dtype=torch.bfloat16),
                 y=torch.randn((T, N), device=DEV, generator=gen, dtype=dt),
                 a=torch.randn((n, r, K), device=DEV, generator=gen, dtype=torch.bfloat16) * 0.02,
                 b=torch.randn((n, N, r), device=DEV, generator=gen, dtype=torch.bfloat16) * 0.1,
                 scale=torch.rand(n, device=DEV, generator=gen) + 0.5, out=torch.empty((T, N), device=DEV, dtype=dt))
        return s
    Hq, Hkv, D, ps = c["Hq"], c["Hkv"], c["D"], c["page"]
    if c["op"] == "attention4":
        s.update(cache=_cache4(c, pages, gen), table=table.to(DEV), kv=_i32([a + b for a, b in zip(old, new)]),
                 max_q=max(new), q=torch.randn((T, Hq, D), device=DEV, generator=gen, dtype=torch.bfloat16),
                 out=torch.empty((T, Hq, D), device=DEV, dtype=torch.bfloat16), lse=torch.empty((T, Hq), device=DEV))
        return s
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(old, new)])
    req = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(new))
    # one projection's output, some channels larger than others
    qkv = torch.randn((T, Hq + 2 * Hkv, D), device=DEV, generator=gen,
                      dtype=torch.bfloat16 if c["x"] == "bf16" else torch.float32)
    qkv[:, :, ::31] *= 3
    s.update(cache=(_cache8 if c["op"] == "append" else _cache4)(c, pages, gen),
             slots=(table[req, pos // ps] * ps + pos % ps).to(torch.int32).to(DEV), pos=pos.to(torch.int32).to(DEV),
             angles=_angles(max(a + b for a, b in zip(old, new)), c["rot"]), q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv],
             v=qkv[:, Hq + Hkv:], q_out=torch.empty((T, Hq, D), device=DEV, dtype=torch.bfloat16))
    if c["op"] == "append4":
        s["back"] = [torch.empty((T, Hkv, D), device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["c"]["op"]
    if own:
        return _own(op, state)
    return {"append": _plain_append, "append4": _plain_append4, "attention4": _plain_attention,
            "adapters": _plain_adapters}[op](state)


def _own(op, s):
    import fp8_quantized_gemm_q4_gb300 as bs
    c = s["c"]
    if op == "adapters":
        return bs.lora_add(s["x"], s["y"], s["a"], s["b"], s["cu"], s["which"], scales=s["scale"], out=s["out"])
    if op == "attention4":
        cache = bs.KVCacheFP4(*s["cache"])
        bs.kv_attention(s["q"], cache, s["table"], s["cu"], s["kv"], s["max_q"], out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "append":
        k, v, ks, vs = cache = bs.KVCache(*s["cache"])
        bs.kv_append_rotary(s["q"], s["k"], s["v"], s["slots"], s["pos"], s["angles"], cache, q_out=s["q_out"],
                            interleaved=c["mixed"])
        return s["q_out"], k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs
    cache = bs.KVCacheFP4(*s["cache"])
    bs.kv_append_rotary(s["q"], s["k"], s["v"], s["slots"], s["pos"], s["angles"], cache, q_out=s["q_out"],
                        interleaved=c["mixed"])
    return s["q_out"], *bs.kv_gather(cache, s["slots"], out=s["back"])


def _rotated(s, x):
    """Pairs (x1, x2) of the first rot elements become (x1 cos - x2 sin, x2 cos + x1 sin), products and sums rounded to fp32."""
    rot, x = s["c"]["rot"], x.float()
    a = s["angles"][s["pos"].long()][:, None]
    cos, sin = a[..., :rot // 2], a[..., rot // 2:]
    x1, x2 = (x[..., :rot:2], x[..., 1:rot:2]) if s["c"]["mixed"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack(y, -1).flatten(-2) if s["c"]["mixed"] else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _power_scale(amax):
    """The smallest power of two, 2^-32 at least and 2^64 at most, whose 448-fold holds amax."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), -32).clamp(-32, 64)
    return ((e + 127) << 23).int().view(torch.float32)


def _to_codes(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    """A page's scale grows to what its new tokens need (a page begun anew takes theirs); what it held is rounded to the new scale."""
    k, v, ks, vs = s["cache"]
    page, off = s["slots"].long() // k.shape[2], s["slots"].long() % k.shape[2]
    heads = torch.arange(k.shape[1], device=DEV)[None, :]
    first = torch.full((len(k),), k.shape[2], device=DEV).scatter_reduce(0, page, off, "amin")[:, None]
    begun = page[s["cu"][:-1].long().clamp(max=len(page) - 1)]
    at = torch.arange(k.shape[2], device=DEV)[None, None, :, None]
    outs = []
    for x, codes, scales in ((_rotated(s, s["k"]), k, ks), (s["v"].float(), v, vs)):
        amax = torch.zeros_like(scales).scatter_reduce(0, page[:, None].expand(-1, k.shape[1]), x.abs().amax(-1), "amax")
        need = _power_scale(amax)
        scale = torch.where(first == 0, need, torch.where(first < codes.shape[2], torch.maximum(scales, need), scales))
        held = codes[begun]
        again = _to_codes(held.view(torch.float8_e4m3fn).float() * (scales / scale)[begun][:, :, None, None])
        codes[begun] = torch.where(at < first[begun][:, :, None, None], again, held)
        codes[page[:, None], heads, off[:, None]] = _to_codes(x / scale[page][:, :, None])
        scales.copy_(scale)
        outs.append(codes.view(torch.float8_e4m3fn))
    return _rotated(s, s["q"]).to(torch.bfloat16), outs[0], outs[1], ks, vs


def _values4(codes, scales):
    """What packed E2M1 codes with a scale for 16 elements stand for, fp32."""
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    x = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1)
    x = x.view(*scales.shape, 16) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return x.flatten(-2)


def _plain_append4(s):
    """A group's scale is its largest magnitude / 6 as e4m3, a code the nearest E2M1 value to element / scale, ties to the even code."""
    k, v, ks, vs = s["cache"]
    page, off = (s["slots"].long() // k.shape[2])[:, None], (s["slots"].long() % k.shape[2])[:, None]
    heads = torch.arange(k.shape[1], device=DEV)[None, :]
    back = []
    for x, codes, scales in ((_rotated(s, s["k"]), k, ks), (s["v"].float(), v, vs)):
        x = x.unflatten(-1, (-1, 16))
        sf = (x.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
        scale = sf.float()[..., None]
        x = torch.where(scale > 0, x / scale, 0)
        a = x.abs()
        q = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
             + (a >= 3.5).int() + (a > 5).int()) | (x < 0).int() << 3
        q = q.flatten(-2).unflatten(-1, (-1, 2)).to(torch.uint8)
        codes[page, heads, off] = q[..., 0] | q[..., 1] << 4
        scales[page, heads, off] = sf.view(torch.uint8)
        back.append(_values4(codes[page, heads, off], scales[page, heads, off]).to(torch.bfloat16))
    return _rotated(s, s["q"]).to(torch.bfloat16), back[0], back[1]


def _plain_attention(s):
    """softmax(q K^T / sqrt(D)) V over the pages of each request; new token i of a request sees what was cached and the new tokens up to itself."""
    c = s["c"]
    B, T, Hq, Hkv, D, nq = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], s["max_q"]
    G = Hq // Hkv
    k, v, ks, vs = s["cache"]
    cu, kv = s["cu"].long(), s["kv"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(nq, device=DEV)
    q = s["q"][(cu[:-1, None] + i).clamp(max=T - 1)].float().view(B, nq, Hkv, G, D).permute(0, 2, 1, 3, 4)
    q = q.reshape(B, Hkv, nq * G, D)
    pages = s["table"].long().clamp(min=0)

    def values(codes, scales):
        return _values4(codes[pages], scales[pages]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)

    scores = (q @ values(k, ks).transpose(2, 3)).mul_(D ** -0.5)
    last = (kv - new)[:, None] + i
    seen = torch.arange(scores.shape[3], device=DEV) <= last[..., None]
    seen = seen.repeat_interleave(G, 1)[:, None]
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ values(v, vs)) / total.clamp(min=1e-30)
    lse = top + torch.log(total)
    row = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:], row, right=True)
    at = row - cu[req]

    def back(x):
        return x.view(B, Hkv, nq, G, -1)[req, :, at].reshape(T, Hq, -1)

    return back(out).to(torch.bfloat16), back(lse)[..., 0]


def _plain_adapters(s):
    """Rows of requests side by side, padded to the longest, so that each request is one product with its adapter."""
    T, B = s["c"]["T"], s["c"]["B"]
    cu, which = s["cu"].long(), s["which"].long()
    row = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:], row, right=True)
    x = s["x"][(cu[:-1, None] + torch.arange(s["max_rows"], device=DEV)).clamp(max=T - 1)].float()
    mine = which.clamp(min=0)
    scale = torch.where(which >= 0, s["scale"][mine], 0)
    t = x @ s["a"][mine].float().transpose(1, 2)
    d = (t @ s["b"][mine].float().transpose(1, 2)) * scale[:, None, None]
    return (s["y"].float() + d[req, row - cu[req]]).to(s["y"].dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "adapters":
        # the requests' adapters follow the seed: as many as there are to expect among so many
        used = c["n"] * (1 - (1 - 1 / c["n"]) ** (c["B"] - c["bare"]))
        K, N, r, live = c["K"], c["N"], c["r"], T * (c["B"] - c["bare"]) / c["B"]
        return {"bytes": live * K * 2 + used * r * (K + N) * 2 + T * N * 2 * (2 if c["y"] == "bf16" else 4),
                "flops": 2.0 * live * r * (K + N)}
    old, new = _lengths(c)
    ps, D, Hq, Hkv = c["page"], c["D"], c["Hq"], c["Hkv"]
    if c["op"] in ("append", "append4"):
        places = len({p for a, b in zip(old, new) for p in range(a, a + b)})
        x = T * (Hq + 2 * Hkv) * D
        touched = sum(-(-(a + b) // ps) - a // ps for a, b in zip(old, new))
        b = x * (2 if c["x"] == "bf16" else 4) + 2 * T * Hq * D + 8 * T + 4 * places * c["rot"]
        b += 2 * T * Hkv * D + 16 * touched * Hkv if c["op"] == "append" else 2 * T * Hkv * D * (9 / 16 * 2 + 2) + 4 * T
        return {"bytes": float(b), "flops": 3.0 * T * (Hq + Hkv) * c["rot"] + 4.0 * T * Hkv * D}
    kv = [a + b for a, b in zip(old, new)]
    pairs = sum(n * m - n * (n - 1) / 2 for n, m in zip(new, kv))
    cached = 2.0 * Hkv * sum(kv) * D * 9 / 16
    return {"bytes": cached + 4 * sum(-(-m // ps) for m in kv) + T * Hq * (4 * D + 4), "flops": 4.0 * D * Hq * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_values():
    """The value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if b & 128 else x)
    v[127] = v[255] = math.nan
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _powers(lo, hi):
    return torch.tensor([2.0 ** e for e in range(lo, hi + 1)], dtype=torch.float64, device=DEV)


def _round_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to the even one, held at 448."""
    a = x.abs().clamp(max=512)
    step = _powers(-9, 6)[torch.frexp(a)[1].long().clamp(min=-5) + 5]
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448)


def _round_e2m1(x):
    """x rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, held at 6."""
    a = x.abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.sign(x) * torch.round(a / step) * step


def _turned(s, x):
    """The rotation as a product of complex numbers."""
    c, x = s["c"], x.double()
    rot = c["rot"]
    h = rot // 2
    a = s["angles"].double()[s["pos"].long()]
    turn = torch.complex(a[:, :h], a[:, h:])[:, None]
    z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) if c["mixed"] else torch.complex(x[..., :h], x[..., h:rot])
    z = z * turn
    y = x.clone()
    if c["mixed"]:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        y[..., :h], y[..., h:rot] = z.real, z.imag
    return y


def _pairs4(codes, scales, table):
    """64-bit values of a part of a 4-bit cache."""
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV)
    q = codes.long()
    x = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device=DEV)
    x[..., 0::2] = half[q % 8] / 2 * (1 - 2 * (q // 8 % 2)).double()
    x[..., 1::2] = half[q // 16 % 8] / 2 * (1 - 2 * (q // 128)).double()
    return x * table[scales.long()].repeat_interleave(16, -1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    cu = s["cu"].tolist()
    if c["op"] == "adapters":
        out = s["y"].double()
        for b, w in enumerate(s["which"].tolist()):
            if w >= 0:
                lo, hi = cu[b], cu[b + 1]
                out[lo:hi] += (s["x"][lo:hi].double() @ s["a"][w].double().T) @ s["b"][w].double().T * float(s["scale"][w])
        return out
    table = _e4m3_values()
    k, v, ks, vs = s["cache"]
    ps = c["page"]
    if c["op"] == "append":
        slots, powers = s["slots"].tolist(), _powers(-32, 64)
        outs = []
        for x, codes, scales in ((_turned(s, s["k"]), k, ks), (s["v"].double(), v, vs)):
            val, sc = table[codes.long()], scales.double()
            for b in range(c["B"]):
                lo = cu[b]
                while lo < cu[b + 1]:  # the new tokens of one page
                    page, off = slots[lo] // ps, slots[lo] % ps
                    n = min(cu[b + 1] - lo, ps - off)
                    new = x[lo:lo + n].transpose(0, 1)
                    amax = new.abs().amax((1, 2))
                    scale = powers[torch.searchsorted(448 * powers, amax).clamp(max=96)]
                    if off:
                        scale = torch.maximum(scale, sc[page])
                        val[page, :, :off] = _round_e4m3(val[page, :, :off] * (sc[page] / scale)[:, None, None])
                    val[page, :, off:off + n] = _round_e4m3(new / scale[:, None, None])
                    sc[page] = scale
                    lo += n
            outs.append((val, sc))
        return _turned(s, s["q"]), outs[0][0], outs[1][0], outs[0][1], outs[1][1]
    if c["op"] == "append4":
        back = []
        for x in (_turned(s, s["k"]), s["v"].double()):
            x = x.unflatten(-1, (-1, 16))
            scale = _round_e4m3(x.abs().amax(-1, keepdim=True) / 6)
            back.append((_round_e2m1(torch.where(scale > 0, x / scale, 0)) * scale).flatten(-2))
        return _turned(s, s["q"]), back[0], back[1]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.zeros((c["T"], Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((c["T"], Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, m in enumerate(s["kv"].tolist()):
        n, mine = cu[b + 1] - cu[b], s["table"][b, :-(-m // ps)].long()
        hide = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
        for h in range(Hkv):
            kk = _pairs4(k[mine, h], ks[mine, h], table).reshape(-1, D)[:m]
            vv = _pairs4(v[mine, h], vs[mine, h], table).reshape(-1, D)[:m]
            for g in range(h * G, (h + 1) * G):
                z = s["q"][cu[b]:cu[b + 1], g].double() @ kk.T / math.sqrt(D)
                z[hide] = -math.inf
                lse[cu[b]:cu[b + 1], g] = torch.logsumexp(z, -1)
                out[cu[b]:cu[b + 1], g] = torch.softmax(z, -1) @ vv
    return out, lse
