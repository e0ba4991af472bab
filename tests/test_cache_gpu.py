"""fa_cache_append and fa_cache_read: what is stored, against the definition; slots, padding, strides,
rows that hold nothing finite."""
import math

import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float8_e4m3fn, torch.int8]


def pools(P, H, d, dtype, fill=0):
    kp, vp = (torch.full((P, H, 16, d), fill, dtype=torch.float32).to(dtype).cuda() for _ in range(2))
    if dtype == torch.bfloat16:
        return kp, vp, None, None
    return kp, vp, *(torch.full((P, H, 16), float(fill), device="cuda") for _ in range(2))


def at(pool, slots):
    """The rows at slots: [T, H, ...]."""
    s = slots.to(pool.device)
    return (pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool)[s // 16, :, s % 16]


def stored_bound(x, dtype):
    """Half a code step of each value: e4m3 steps are 2^-3 of the binade below x (at most 2^-4 of |x|
    to a side) down to the subnormals' 2^-9 of the scale, int8 steps are the scale; with the fp32
    quotients' 2^-23.  bf16: 2^-8."""
    if dtype == torch.bfloat16:
        return x.abs() * R.U_BF16
    scale = x.abs().amax(-1, keepdim=True) / R.QMAX[dtype]
    if dtype == torch.int8:
        return 0.5001 * scale + x.abs() * 2.0 ** -21
    return torch.maximum(x.abs() * (2.0 ** -4 + 2.0 ** -20), scale * 2.0 ** -10 * 1.001)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,rot,layout", [(64, 64, "half"), (128, 64, "interleaved"), (128, 0, "half"),
                                          (128, 96, "half")])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 8, 1), (33, 6, 3), (700, 1, 2)])
def test_write_and_read(dtype, d, rot, layout, T, Hq, Hk):
    import exact_attention_158_b200 as fa
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn((T, Hq + 2 * Hk, d), generator=g)
    x = (x * torch.exp2(torch.randint(-9, 9, (T, Hq + 2 * Hk, 1), generator=g).float())).to(torch.bfloat16).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    P = T // 16 + 3
    slots = torch.randperm(P * 16, generator=g)[:T].cuda()
    if T > 3:
        slots[2] = -1
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32).cuda()
    freqs, amp = fa.rope_frequencies(rot, scaling="ramp", factor=4.0) if rot else (None, 1.0)
    kp, vp, ks, vs = pools(P, Hk, d, dtype, fill=3)
    before = [None if t is None else t.clone() for t in (kp, vp, ks, vs)]
    yq = fa.fa_cache_append(k, v, kp, vp, slots, ks, vs, pos if rot else None, freqs, layout, amp, q=q)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    f = torch.zeros(0, dtype=torch.float64) if freqs is None else freqs.cpu()
    p = pos.cpu()[:, None]
    R.check(yq, R.rope(q.cpu(), p, f, layout, amp), R.rope_bound(q.cpu(), f, layout, amp, torch.bfloat16), "q")
    live = slots >= 0
    kw = R.rope(k.cpu(), p, f, layout, amp)
    k32 = R.rope_bound(k.cpu(), f, layout, amp, torch.float32)
    back_k, back_v = fa.fa_cache_read(kp, vp, slots, ks, vs)
    for name, back, want, more, pool, sc in (("k", back_k, kw, k32, kp, ks),
                                             ("v", back_v, v.cpu().double(), 0 * k32, vp, vs)):
        assert torch.equal(back[~live], torch.zeros_like(back[~live]))
        want, more, got = want[live.cpu()], more[live.cpu()], back[live]
        if dtype == torch.bfloat16:
            R.check(got, want, stored_bound(want, dtype) + more, name)
            continue
        # the reader: code * scale rounded to bf16
        codes = at(pool, slots[live])
        codes = codes.view(dtype).float() if dtype != torch.int8 else codes.float()
        exact = codes * at(sc, slots[live])[..., None]
        assert torch.equal(got, exact.to(torch.bfloat16)), name
        R.check(exact, want, stored_bound(want, dtype) + 2 * more, name)
    if dtype != torch.bfloat16:  # values are not rotated: codes and scales to the bit
        codes, scale = R.quantise(v[live].float().cpu(), dtype)
        assert torch.equal(at(vs, slots[live]).cpu(), scale)
        got = at(vp, slots[live]).cpu()
        assert torch.equal(got, codes.view(torch.uint8) if dtype != torch.int8 else codes)
    # slots that no token names are left as they were
    other = torch.ones(P * 16, dtype=torch.bool)
    other[slots[live].cpu()] = False
    rest = torch.arange(P * 16)[other]
    for t, b in zip((kp, vp, ks, vs), before):
        if t is not None:
            assert torch.equal(at(t, rest), at(b, rest))


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
def test_rows_of_nothing_and_of_no_number(dtype):
    import exact_attention_158_b200 as fa
    d = 128
    k = torch.ones((7, 1, d), dtype=torch.bfloat16, device="cuda")
    k[0] = 0.0
    k[1] = 2.0 ** -120           # counts as zeros
    k[2, 0, 5] = math.inf
    k[3, 0, 127] = math.nan
    k[4] = 3.0e38                # the largest magnitudes still have a finite scale
    k[5] = 0.0
    k[5, 0, 64] = -1.0           # one value alone is its own maximum
    k[6] = 2.0 ** -99
    kp, vp, ks, vs = pools(1, 1, d, dtype, fill=1)
    slots = torch.arange(7, device="cuda")
    fa.fa_cache_append(k, -k, kp, vp, slots, ks, vs)
    rk, rv = fa.fa_cache_read(kp, vp, slots, ks, vs)
    assert fa.device_status() == 0
    assert torch.equal(rk[:2], torch.zeros_like(rk[:2])) and torch.equal(ks[0, 0, :2], torch.zeros(2, device="cuda"))
    assert torch.isnan(rk[2:4]).all() and torch.isnan(rv[2:4]).all() and torch.isnan(ks[0, 0, 2:4]).all()
    for i in (4, 5, 6):
        assert torch.allclose(rk[i].float(), k[i].float(), rtol=2.0 ** -7, atol=0) and torch.equal(rv[i], -rk[i])


@pytest.mark.parametrize("dtype", TYPES)
def test_slots_past_the_pool_are_reported(dtype):
    import exact_attention_158_b200 as fa
    kp, vp, ks, vs = pools(2, 2, 64, dtype, fill=1)
    before = kp.clone()
    k = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([32, 2 ** 40, -7], device="cuda")
    fa.fa_cache_append(k, k, kp, vp, slots, ks, vs)
    assert fa.device_status() == 1 and torch.equal(kp.view(torch.uint8), before.view(torch.uint8))
    rk, _ = fa.fa_cache_read(kp, vp, slots, ks, vs)
    assert fa.device_status() == 1 and torch.equal(rk, torch.zeros_like(rk))


def test_empty_step_and_capture():
    import exact_attention_158_b200 as fa
    kp, vp, ks, vs = pools(2, 1, 64, torch.int8)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert fa.fa_cache_append(e, e, kp, vp, none, ks, vs) is None
    assert fa.fa_cache_read(kp, vp, none, ks, vs)[0].shape == (0, 1, 64)
    k = torch.randn((4, 1, 64), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([0, 1, 2, 3], device="cuda")
    fa.fa_cache_append(k, k, kp, vp, slots, ks, vs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_cache_append(k, k, kp, vp, slots, ks, vs)
    slots += 20
    k.mul_(2)
    graph.replay()
    want, scale = R.quantise(k.float().cpu(), torch.int8)
    assert torch.equal(at(vp, slots).cpu(), want) and torch.equal(at(vs, slots).cpu(), scale)


def test_offsets_past_32_bits():
    import exact_attention_158_b200 as fa
    P, H, d = 140_000, 8, 128  # 2.3 GB of codes per pool
    kp, vp = (torch.empty((P, H, 16, d), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((P, H, 16), device="cuda") for _ in range(2))
    k = torch.randn((2, H, d), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([16 * P - 1, 16 * (P - 3) + 2], device="cuda")
    fa.fa_cache_append(k, k, kp, vp, slots, ks, vs)
    rk, rv = fa.fa_cache_read(kp, vp, slots, ks, vs)
    codes, scale = R.quantise(k.float().cpu(), torch.int8)
    want = (codes.float() * scale[..., None]).to(torch.bfloat16)
    assert torch.equal(rk.cpu(), want) and torch.equal(rv.cpu(), want)
