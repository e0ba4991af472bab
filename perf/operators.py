"""The serving operators around the paged attention: what each is given, its plain form and its cases.

Four operators are covered, each in the form a decoder's inference (and for the rotation, training)
step calls it:

  rope     rotary positions of q and k as the projection leaves them ([B, N, heads, d], strided),
           written head-major as attention reads them; and its gradient, the transposed rotation,
           from head-major dq, dk back to the projection's layout.
  cache    new tokens' keys (rotated on the way) and values written to their slots of the paged
           pool, as bf16 or quantised to 8 bits with one scale per token and head, the step's
           queries rotated beside them; then the rows read back as bf16.
  decode   one query per sequence over an 8-bit paged cache, query heads sharing key/value heads.
  chunk    several queries per sequence over an 8-bit paged cache: a causal chunk, or a tree of
           drafted tokens with a visibility mask per node.

With ``own`` false, ``run`` computes the plain form in elementary torch operations; with ``own``
true it makes the calls a user of the package makes.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 16                      # tokens per physical block of the pool
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}
TINY = 2.0 ** -100             # a row whose largest magnitude is below this is stored as zeros
DEV = "cuda"


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's rotation for 64 sequences: a few hundred kilobytes, so latency counts
        dict(name="rope_step", op="rope", B=64, N=1, Hq=32, Hk=8, d=128, rot=128, layout="half",
             inverse=False, dtype="bf16", far=8000, factor=1.0),
        # the training forward of the package's prefill workload (B8 H16 N2048 d128)
        dict(name="rope_train", op="rope", B=8, N=2048, Hq=16, Hk=16, d=128, rot=128, layout="half",
             inverse=False, dtype="bf16", far=0, factor=1.0),
        # gradients in fp32 of a model that rotates half of each head, interleaved, over an odd
        # length far into a context stretched eightfold
        dict(name="rope_grad", op="rope", B=2, N=4099, Hq=32, Hk=8, d=64, rot=32,
             layout="interleaved", inverse=True, dtype="f32", far=500000, factor=8.0),
        # one decode step of 64 sequences writes one token each, in 8-bit floating point
        dict(name="cache_step", op="cache", T=64, Hq=32, Hk=8, d=128, rot=128, layout="half",
             kind="e4m3", far=8000, pad=3),
        # a long prompt's chunk in 8-bit integers, half of each head rotated, with padding
        dict(name="cache_chunk", op="cache", T=8191, Hq=32, Hk=8, d=128, rot=64,
             layout="interleaved", kind="int8", far=100000, pad=100),
        # an unquantised cache with as many key heads as query heads
        dict(name="cache_bf16", op="cache", T=1000, Hq=16, Hk=16, d=64, rot=64, layout="half",
             kind="bf16", far=1000, pad=0),
        # a single short sequence: the smallest decode call
        dict(name="decode_one", op="decode", S=1, Hq=8, Hk=1, d=64, lo=333, hi=333, kind="int8"),
        # the package's paged-decode workload (64 sequences, H32 d128, 512..8192 tokens) at 8 bits
        dict(name="decode_batch", op="decode", S=64, Hq=32, Hk=32, d=128, lo=512, hi=8192,
             kind="e4m3"),
        # two very long contexts, four query heads to a key head: the context has to be split
        dict(name="decode_long", op="decode", S=2, Hq=32, Hk=8, d=128, lo=100001, hi=131072,
             kind="e4m3"),
        # verification of 13 drafted tokens over short contexts
        dict(name="tree_small", op="chunk", S=3, Hq=16, Hk=2, d=64, T=13, lo=20, hi=700,
             kind="e4m3", tree=True),
        # verification of 48 drafted tokens for 32 sequences
        dict(name="tree_batch", op="chunk", S=32, Hq=32, Hk=8, d=128, T=48, lo=512, hi=4096,
             kind="int8", tree=True),
        # a prompt chunk of 512 tokens for 4 sequences, up to 8192 tokens cached
        dict(name="chunk", op="chunk", S=4, Hq=32, Hk=8, d=128, T=512, lo=1000, hi=8192,
             kind="e4m3", tree=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    hk = rng.choice([h for h in (1, 2, 4, 8, 16, 32) if h <= most])
    return rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * hk <= most]) * hk, hk


def draw(rng):
    """One more case: sizes over the logarithm of their range, capped at the listed cases' work."""
    op = rng.choice(["rope", "cache", "decode", "chunk"])
    d = rng.choice([64, 128])
    if op == "rope":
        hq, hk = _heads(rng, 32)
        B = _log(rng, 1, 64)
        N = _log(rng, 1, max(1, min(8192, (1 << 26) // ((hq + hk) * d * B))))
        return dict(op=op, B=B, N=N, Hq=hq, Hk=hk, d=d, rot=16 * rng.randint(1, d // 16),
                    layout=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]), far=_log(rng, 1, 1000000),
                    factor=rng.choice([1.0, 4.0, 8.0]))
    if op == "cache":
        hq, hk = _heads(rng, 32)
        T = _log(rng, 1, 8191)
        return dict(op=op, T=T, Hq=hq, Hk=hk, d=d, rot=16 * rng.randint(1, d // 16),
                    layout=rng.choice(["half", "interleaved"]),
                    kind=rng.choice(["e4m3", "int8", "bf16"]), far=_log(rng, 1, 1000000),
                    pad=rng.choice([0, T // 50]))
    hq, hk = _heads(rng, 32)
    kind = rng.choice(["e4m3", "int8"])
    if op == "decode":
        S = _log(rng, 1, 64)
        hi = _log(rng, 2, min(131072, (1 << 26) // (S * hk * 4)))
        return dict(op=op, S=S, Hq=hq, Hk=hk, d=d, lo=_log(rng, 1, hi), hi=hi, kind=kind)
    tree = rng.random() < 0.5
    T = rng.randint(2, 64) if tree else _log(rng, 2, 512)
    S = _log(rng, 1, 32)
    hi = _log(rng, T, max(T, min(8192, (1 << 31) // (S * hq * T * 16))))
    return dict(op=op, S=S, Hq=hq, Hk=hk, d=d, T=T, lo=_log(rng, T, hi), hi=hi, kind=kind, tree=tree)


def _lens(c):
    """Context lengths spread over [lo, hi], the same for every seed (so that the work is)."""
    return [c["hi"] if s == 0 else c["lo"] + int((c["hi"] - c["lo"] + 1) * ((s * 0.6180339887) % 1.0))
            for s in range(c["S"])]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hk"])
        e = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * n * c["d"] * e + 4 * c["B"] * c["N"] + 4 * c["rot"],
                    flops=3 * n * c["rot"])
    if c["op"] == "cache":
        live = c["T"] - c["pad"]
        code = 2 if c["kind"] == "bf16" else 1
        scale = 0 if c["kind"] == "bf16" else 4
        row = 2 * c["Hk"] * live  # key and value rows
        # q in and out; k, v in; codes out and in again; k, v out
        return dict(bytes=2 * 2 * c["T"] * c["Hq"] * c["d"] + row * (2 * c["d"] + 2 * (code * c["d"] + scale))
                    + 2 * 2 * c["T"] * c["Hk"] * c["d"] + 16 * c["T"] + 4 * c["rot"],
                    flops=3 * c["T"] * (c["Hq"] + c["Hk"]) * c["rot"] + 4 * row * c["d"])
    lens = _lens(c)
    T = c.get("T", 1)
    tokens = sum(lens)
    if c["op"] == "decode":
        pairs = tokens
    elif c["tree"]:  # the context for every node, and about half of each node's path
        pairs = sum(T * (L - T) + T * 4 for L in lens)
    else:
        pairs = sum(T * (L - T) + T * (T + 1) // 2 for L in lens)
    return dict(bytes=tokens * c["Hk"] * 2 * (c["d"] + 4) + c["S"] * c["Hq"] * T * (4 * c["d"] + 4)
                + 4 * sum(-(-L // PAGE) for L in lens) + 4 * c["S"],
                flops=4 * c["d"] * c["Hq"] * pairs)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _freqs(rot, factor):
    """Radians per position of each rotated pair, in 64 bits; for a context stretched by `factor`
    pairs that turn less than once in 4096 positions are slowed by it, those that turn more than 32
    times are kept, with a linear ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep)


def _quantise(x, kind):
    """[..., d] in 32 bits -> codes and one scale per row (0 for rows that count as zeros)."""
    top = x.abs().amax(-1)
    # (a tensor as the divisor: a quotient, where a plain number may become a reciprocal's product)
    scale = torch.where(top >= TINY, top / torch.full_like(top, QMAX[kind]), 0.0)
    y = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    if kind == "int8":
        return y.round().clamp(-127, 127).to(torch.int8), scale
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    st = dict(c)
    if c["op"] == "rope":
        B, N, Hq, Hk, d = c["B"], c["N"], c["Hq"], c["Hk"], c["d"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st["freqs"] = _freqs(c["rot"], c["factor"]).to(DEV)
        st["amplitude"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
        start = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        st["positions"] = start + torch.arange(N, device=DEV, dtype=torch.int32)
        if c["inverse"]:
            st["q"], st["k"] = normal(B, Hq, N, d, dtype=dt), normal(B, Hk, N, d, dtype=dt)
        else:  # the fused projection's output: q, k and v heads of a token side by side
            x = normal(B, N, Hq + 2 * Hk, d, dtype=dt)
            st["q"], st["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
        return st
    Hq, Hk, d = c["Hq"], c["Hk"], c["d"]
    if c["op"] == "cache":
        T = c["T"]
        x = normal(T, Hq + 2 * Hk, d)
        # a few tokens carry much larger keys and values, as the first tokens of a context do
        loud = torch.rand((T, 1, 1), generator=g, device=DEV) < 0.05
        x = torch.where(loud, x * 16, x)
        st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        blocks = -(-T // PAGE) + 7
        st["slots"] = torch.randperm(blocks * PAGE, generator=g, device=DEV)[:T]
        if c["pad"]:
            st["slots"][-c["pad"]:] = -1
        st["positions"] = (torch.randint(0, c["far"] + 1, (1,), generator=g, device=DEV)
                           + torch.arange(T, device=DEV)).to(torch.int32)
        st["freqs"] = _freqs(c["rot"], 1.0).to(DEV)
        shape = (blocks, Hk, PAGE, d)
        st["k_pool"] = torch.zeros(shape, dtype=CODE[c["kind"]], device=DEV)
        st["v_pool"] = torch.zeros(shape, dtype=CODE[c["kind"]], device=DEV)
        st["k_scale"] = st["v_scale"] = None
        if c["kind"] != "bf16":
            st["k_scale"] = torch.zeros(shape[:3], device=DEV)
            st["v_scale"] = torch.zeros(shape[:3], device=DEV)
        return st
    lens = _lens(c)
    pages = [-(-L // PAGE) for L in lens]
    P, most, T = sum(pages), max(pages), c.get("T", 1)
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["S"], most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    for n in ("k", "v"):
        x = normal(P, Hk, PAGE, d, dtype=torch.float32)
        st[n + "_pool"], st[n + "_scale"] = _quantise(x, c["kind"])
        del x
        # the slots past a sequence's end were never written: what is there is not a number
        for s, L in enumerate(lens):
            if L % PAGE:
                st[n + "_scale"][table[s, pages[s] - 1].long(), :, L % PAGE:] = math.nan
    st["table"], st["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["q"] = normal(c["S"], Hq, d) if c["op"] == "decode" else normal(c["S"], Hq, T, d)
    st["sm_scale"] = 1.0 / math.sqrt(d)
    if c["op"] == "chunk" and c["tree"]:
        h = torch.Generator()
        h.manual_seed(seed)
        draws = torch.rand((c["S"], T), generator=h).tolist()
        masks = []
        for row in draws:
            bits = []
            for t, u in enumerate(row):
                parent = int(u * (t + 1)) - 1
                bits.append((1 << t) | (bits[parent] if parent >= 0 else 0))
            masks.append([m - (1 << 64) if m >= 1 << 63 else m for m in bits])
        st["mask"] = torch.tensor(masks, dtype=torch.int64).to(DEV)
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def _rotate(x, positions, freqs, rot, layout, amplitude, inverse):
    """x [..., d] in 32 bits, positions broadcastable to x's leading dimensions."""
    angle = positions[..., None].double() * freqs
    cos, sin = (angle.cos() * amplitude).float(), (angle.sin() * amplitude).float()
    if inverse:
        sin = -sin
    head, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _rope_plain(s):
    def one(x):
        y = _rotate(x.float(), s["positions"][:, None], s["freqs"], s["rot"], s["layout"],
                    s["amplitude"], s["inverse"]).to(x.dtype)
        return y.transpose(1, 2).contiguous() if s["inverse"] else y.contiguous()
    return one(s["q"]), one(s["k"])


def _cache_plain(s):
    rot = lambda x: _rotate(x.float(), s["positions"][:, None], s["freqs"], s["rot"], s["layout"],  # noqa: E731
                            1.0, False)
    live = s["T"] - s["pad"]
    blk, row = s["slots"][:live] // PAGE, s["slots"][:live] % PAGE
    back = []
    for n, x in (("k", rot(s["k"])), ("v", s["v"].float())):
        pool = s[n + "_pool"]
        y = torch.zeros_like(x)
        if s["kind"] == "bf16":
            pool[blk, :, row] = x[:live].to(torch.bfloat16)
            y[:live] = pool[blk, :, row].float()
        else:
            codes, scale = _quantise(x[:live], s["kind"])
            pool.view(torch.uint8)[blk, :, row] = codes.view(torch.uint8)
            s[n + "_scale"][blk, :, row] = scale
            y[:live] = (pool.view(torch.uint8)[blk, :, row].view(pool.dtype).float()
                        * s[n + "_scale"][blk, :, row][..., None])
        back.append(y.to(torch.bfloat16))
    return rot(s["q"]).to(torch.bfloat16), back[0], back[1]


def _gathered(s, n, seen):
    """The sequences' keys or values [S, Hk, L, d] in 32 bits, zero past their lengths."""
    pages = s["table"].clamp(min=0).long()
    S, most = pages.shape
    codes = s[n + "_pool"].view(torch.uint8)[pages].view(s[n + "_pool"].dtype)
    x = codes.float() * s[n + "_scale"][pages][..., None]
    x = x.permute(0, 2, 1, 3, 4).reshape(S, s["Hk"], most * PAGE, s["d"])
    return torch.where(seen[:, None, :, None], x, 0.0)


def _attend_plain(s):
    S, Hk, d, group = s["S"], s["Hk"], s["d"], s["Hq"] // s["Hk"]
    T = s.get("T", 1)
    at = torch.arange(s["table"].shape[1] * PAGE, device=DEV)
    lens = s["lens"].long()
    inside = at < lens[:, None]
    q = s["q"].float().reshape(S, Hk, group, T, d)
    if s["op"] == "decode":
        seen = inside[:, None, :]
    else:
        first = (lens - T)[:, None, None]  # the cached position of the first query
        t = torch.arange(T, device=DEV)[None, :, None]
        if s["tree"]:
            u = (at - first)  # [S, 1, L]: which node a cached token is
            bit = (s["mask"][:, :, None] >> u.clamp(0, 63)) & 1
            seen = (u < 0) | ((u < T) & (bit == 1))
        else:
            seen = at <= first + t
        seen = seen & inside[:, None, :]
    score = torch.einsum("shgtd,shld->shgtl", q, _gathered(s, "k", inside)) * s["sm_scale"]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("shgtl,shld->shgtd", p, _gathered(s, "v", inside))
    o = torch.where(total > 0, o / total, 0.0)
    lse = (total.log() + top)[..., 0]
    if s["op"] == "decode":
        return o.reshape(S, s["Hq"], d).to(torch.bfloat16), lse.reshape(S, s["Hq"])
    return o.reshape(S, s["Hq"], T, d).to(torch.bfloat16), lse.reshape(S, s["Hq"], T)


def run(state):
    s = state
    if own:
        import exact_attention_158_b200 as fa
        if s["op"] == "rope":
            if s["inverse"]:
                dx = torch.empty((s["B"], s["N"], s["Hq"], s["d"]), dtype=s["q"].dtype, device=DEV)
                dy = torch.empty((s["B"], s["N"], s["Hk"], s["d"]), dtype=s["q"].dtype, device=DEV)
                fa.fa_rope(s["q"], s["k"], s["positions"], s["freqs"], layout=s["layout"],
                           amplitude=s["amplitude"], inverse=True, q_out=dx.transpose(1, 2),
                           k_out=dy.transpose(1, 2))
                return dx, dy
            return fa.fa_rope(s["q"], s["k"], s["positions"], s["freqs"], layout=s["layout"],
                              amplitude=s["amplitude"])
        if s["op"] == "cache":
            q = fa.fa_cache_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   positions=s["positions"], freqs=s["freqs"], layout=s["layout"],
                                   q=s["q"])
            k, v = fa.fa_cache_read(s["k_pool"], s["v_pool"], s["slots"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"])
            return q, k, v
        a = (s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["lens"])
        if s["op"] == "decode":
            return fa.fa_decode_paged_q8(*a, scale=s["sm_scale"])
        if s["tree"]:
            return fa.fa_tree_attention_q8(*a, s["mask"], scale=s["sm_scale"])
        return fa.fa_prefill_paged_q8(*a, causal=True, scale=s["sm_scale"])
    if s["op"] == "rope":
        return _rope_plain(s)
    if s["op"] == "cache":
        return _cache_plain(s)
    return _attend_plain(s)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain form
# ------------------------------------------------------------------------------------------------

def _turn64(x, pos, freqs, layout, amplitude, sign):
    """Rotation as a complex product: pair j of the row at position p times a e^(i sign p f_j)."""
    rot = 2 * freqs.numel()
    z = x[..., :rot].double()
    if layout == "half":
        z = torch.stack([z[..., :rot // 2], z[..., rot // 2:]], -1)
    else:
        z = z.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_complex(z.contiguous())
    w = torch.polar(torch.full_like(freqs, amplitude).expand(*pos.shape, -1).contiguous(),
                    sign * pos.double()[..., None] * freqs)
    y = torch.view_as_real(z * w)
    y = torch.cat([y[..., 0], y[..., 1]], -1) if layout == "half" else y.flatten(-2)
    return torch.cat([y, x[..., rot:].double()], -1)


def _stored64(x, kind):
    """What a cache of this kind gives back for rows x in 64 bits."""
    if kind == "bf16":
        return x.to(torch.bfloat16).double()
    top = x.abs().max(-1, keepdim=True).values
    # the scale that is stored is a 32-bit number, and the code is the one nearest to the 32-bit
    # quotient: 16-bit inputs lie on the border between two codes often enough for that to matter
    step = (top / QMAX[kind]).float().double()
    y = (x / torch.where(top > 0, step, 1.0)).float().double()
    if kind == "int8":
        return torch.round(y) * step
    # nearest of the 8-bit floating-point values: 3 fraction bits, exponents from -6
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    return torch.round(y * 2.0 ** (3 - e)) * 2.0 ** (e - 3) * step


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        sign = -1.0 if s["inverse"] else 1.0
        out = []
        for x in (s["q"], s["k"]):
            y = torch.stack([_turn64(x[b], s["positions"][b].expand(x.shape[1], -1), s["freqs"],
                                     s["layout"], s["amplitude"], sign) for b in range(s["B"])])
            out.append(y.transpose(1, 2).contiguous() if s["inverse"] else y)
        return tuple(out)
    if s["op"] == "cache":
        live = s["T"] - s["pad"]
        turn = lambda x: _turn64(x, s["positions"][:, None].expand(-1, x.shape[1]), s["freqs"],  # noqa: E731
                                 s["layout"], 1.0, 1.0)
        k, v = _stored64(turn(s["k"]), s["kind"]), _stored64(s["v"].double(), s["kind"])
        k[live:], v[live:] = 0.0, 0.0
        return turn(s["q"]), k, v
    T, group = s.get("T", 1), s["Hq"] // s["Hk"]
    o_all, l_all = [], []
    for i, L in enumerate(_lens(s)):
        pages = s["table"][i, :-(-L // PAGE)].long()
        kv = []
        for n in ("k", "v"):
            x = (s[n + "_pool"].view(torch.uint8)[pages].view(s[n + "_pool"].dtype).double()
                 * s[n + "_scale"][pages].double()[..., None])
            kv.append(x.transpose(0, 1).reshape(s["Hk"], -1, s["d"])[:, :L])
        see = torch.ones((T, L), dtype=torch.bool, device=DEV)
        if s["op"] == "chunk" and s["tree"]:
            for t, m in enumerate(s["mask"][i].tolist()):
                see[t, L - T:] = torch.tensor([(m >> u) & 1 == 1 for u in range(T)], device=DEV)
        elif s["op"] == "chunk":
            see = torch.tril(see, diagonal=L - T)
        q = s["q"][i].double().view(s["Hq"], T, s["d"])
        o, l = [], []
        for h in range(s["Hq"]):
            z = q[h] @ kv[0][h // group].T * s["sm_scale"]
            z = torch.where(see, z, -math.inf)
            l.append(torch.logsumexp(z, -1))
            o.append(torch.softmax(z, -1) @ kv[1][h // group])
        o_all.append(torch.stack(o))
        l_all.append(torch.stack(l))
    o, l = torch.stack(o_all), torch.stack(l_all)
    return (o[:, :, 0], l[:, :, 0]) if s["op"] == "decode" else (o, l)
