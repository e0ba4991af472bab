"""Plain fp64 definitions of the serving operators (rotary positions, the 8-bit cache, attention over
it), on the CPU, and the error bounds their tests use."""
from __future__ import annotations

import math

import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
PAGE = 16
U_BF16 = 2.0 ** -8  # half a step of bf16, relative


def rope(x, positions, freqs, layout="half", amplitude=1.0, inverse=False):
    """x [..., rows, d] with positions [..., rows] (broadcast), in fp64, as complex products."""
    x = x.double()
    rot = 2 * freqs.numel()
    a, b = ((x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half"
            else (x[..., 0:rot:2], x[..., 1:rot:2]))
    theta = positions.double()[..., None] * freqs.double()
    w = amplitude * torch.exp(1j * (-theta if inverse else theta))
    y = torch.complex(a, b) * w
    turned = (torch.cat([y.real, y.imag], -1) if layout == "half"
              else torch.stack([y.real, y.imag], -1).flatten(-2))
    return torch.cat([turned, x[..., rot:]], -1)


def rope_bound(x, freqs, layout, amplitude, out_dtype):
    """Elementwise bound on the rotation's error.  The angle's fraction of a turn is rounded to fp32
    (2^-25 turns), sine and cosine are good to 2^-22, the two products and their sum add 2^-23 each:
    below 2^-21 of |a| + |b|; then the output's own rounding."""
    x = x.double().abs()
    rot = 2 * freqs.numel()
    if layout == "half":
        s = x[..., :rot // 2] + x[..., rot // 2:rot]
        s = torch.cat([s, s], -1)
    else:
        s = (x[..., 0:rot:2] + x[..., 1:rot:2]).repeat_interleave(2, -1)
    b = torch.cat([s * abs(amplitude), x[..., rot:] * 0], -1) * 2.0 ** -21
    if out_dtype == torch.bfloat16:
        b = b + U_BF16 * (torch.cat([s * abs(amplitude), x[..., rot:]], -1))
    return b


def quantise(x, dtype):
    """fp32 rows [..., d] -> (codes, scale): fp32 quotients, nearest code, as the cache defines it."""
    x = x.float()
    top = x.abs().amax(-1)
    scale = torch.where(top >= 2.0 ** -100, top / torch.full_like(top, QMAX[dtype]), 0.0)
    y = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    if dtype == torch.int8:
        return y.round().clamp(-127, 127).to(torch.int8), scale
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def make_pool(g, P, H, d, dtype, dev="cuda"):
    """Random 8-bit pool: codes over the whole range, subnormal codes and zero rows among them."""
    x = torch.randn((P, H, PAGE, d), generator=g)
    x = x * torch.exp2(torch.randint(-6, 4, (P, H, PAGE, 1), generator=g).float())
    small = torch.rand((P, H, PAGE, 1), generator=g) < 0.1
    x[..., 1:] = torch.where(small, x[..., 1:] * 2.0 ** -7, x[..., 1:])
    codes, scale = quantise(x, dtype)
    zero = torch.rand((P, H, PAGE), generator=g) < 0.05
    scale = torch.where(zero, 0.0, scale)
    return codes.to(dev), scale.to(dev)


def attention(q, k_pool, v_pool, ks, vs, table, lens, scale, causal=False, tree=None):
    """q [S, Hq, T, d].  Returns (o, lse, o_bound, lse_bound) in fp64.

    Bounds.  Scores: products of bf16 and 8-bit values are exact, and each of the d / 16 tensor-core
    steps aligns and rounds its sum within 2^-23 of the largest partial sum, twice: below 2^-18 of
    e = scale sum |q||K|; scaling adds 2^-23.  A weight is then off by e 2^-18 (times 2 for the
    normaliser) and by exp2's 2^-21.  p vs is rounded to fp16 against a reference that puts the row's
    largest p vs at 1 or above, or its largest p at 2^64 (values of scale 0): half a step is 2^-11 of
    it, or 2^-25 where it is below fp16's normal range, which is 2^-25 max(max w vs, 2^-64) of the
    row's weights, and adds up over the codes.
    With more than 32 rows per key head the value scales are folded into V instead: p, f = vs 2^a / F
    and code * f are rounded to fp16, 2^-11 each.  The largest p is at least 2^6, so below fp16's
    normal range it is off by 2^-31 of the largest weight.  F is at most twice the sequence's largest
    vs.  f is at most 2^6 (e4m3, codes to 448) or 2^8 (int8, codes to 127); where it is below fp16's
    normal range it loses 2^-25, times a code, and so does the product: below 2^-21 of that vs per unit
    of weight.  LSE moves by the scores' error, plus the logarithm's."""
    q = q.double().cpu()
    S, Hq, T, d = q.shape
    Hk = k_pool.shape[1]
    table, lens = table.cpu().long(), lens.cpu().tolist()
    o = torch.zeros(S, Hq, T, d, dtype=torch.float64)
    lse = torch.full((S, Hq, T), -math.inf, dtype=torch.float64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)

    def rows(pool, sc, pages, h, L):
        c = pool[pages.to(pool.device), h].double().cpu().reshape(-1, d)[:L]
        f = sc[pages.to(sc.device), h].double().cpu().reshape(-1, 1)[:L]
        return c * f, c, f

    P = k_pool.shape[0]
    for s, L in enumerate(lens):
        if L <= 0:
            continue
        pages = table[s, :-(-L // PAGE)]
        named = ((pages >= 0) & (pages < P)).repeat_interleave(PAGE)[:L]
        pages = torch.where((pages >= 0) & (pages < P), pages, 0)
        see = named.expand(T, L).clone()
        if tree is not None:
            for t, m in enumerate(tree[s].tolist()):
                see[t, L - T:] &= torch.tensor([(m >> u) & 1 == 1 for u in range(T)])
        elif causal:
            see &= torch.ones(T, L, dtype=torch.bool).tril(L - T)
        for h in range(Hq):
            K = rows(k_pool, ks, pages, h // (Hq // Hk), L)[0]
            V, codes, f = rows(v_pool, vs, pages, h // (Hq // Hk), L)
            z = q[s, h] @ K.T * scale
            z = torch.where(see, z, -math.inf)
            some = see.any(-1)
            e = torch.where(see, q[s, h].abs() @ K.abs().T * scale, 0.0).nan_to_num(0.0).amax(-1)
            lse[s, h] = torch.logsumexp(z, -1)
            w = torch.where(some[:, None], torch.softmax(z, -1), 0.0)
            live = see.any(0)  # a token that no row sees takes no part, whatever it holds
            w, V, codes, f = w[:, live], V[live], codes[live].abs(), f[live]
            o[s, h] = w @ V
            far = torch.log2(f[f > 0]).abs().max() if bool((f > 0).any()) else 0.0
            lb[s, h] = (2.0 ** -18 * e + 2.0 ** -20 * (1.0 + lse[s, h].abs().nan_to_num(0.0, posinf=0.0))
                        + 2.0 ** -24 * (16.0 + far))
            seen = (w > 0).double()
            if Hq // Hk * T <= 32:
                top = (w * f[:, 0]).amax(-1, keepdim=True).clamp(min=2.0 ** -64) if len(f) else 0.0
                floor, steps = 2.0 ** -25 * top * seen @ codes, 1
            else:
                top = w.amax(-1, keepdim=True) if len(f) else 0.0
                largest = vs[pages[named[::PAGE]].to(vs.device), h // (Hq // Hk)].nan_to_num(0.0).max()
                floor, steps = 2.0 ** -31 * top * (seen @ V.abs()) + 2.0 ** -21 * float(largest), 3
            ob[s, h] = (steps * 2.0 ** -11 + 2.0 ** -17 * e + 2.0 ** -18)[:, None] * (w @ V.abs()) + floor
    return o, lse, ob, lb


def check(got, want, bound, what):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN at other places"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), f"{what}: infinities"
    d = (got - want).abs()[fin] - bound.double().cpu().expand_as(want)[fin]
    assert d.numel() == 0 or float(d.max()) <= 0.0, f"{what}: {float(d.max()):.3e} over the bound"
