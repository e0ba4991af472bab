"""fa_cache_append and fa_cache_read where a thread walks many heads of its token (prompt chunks):
groups of heads that start and end inside q, k and v, heads that do not fill the rows on their way
at once, and padding."""
import pytest
import torch

from tests import serving_ref as R
from tests.test_cache_gpu import TYPES, at, pools, stored_bound

pytestmark = pytest.mark.gpu


def heads_per_thread(tokens, heads, d):
    """As the library splits them: groups enough for 12 warps per SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    warps = max(1, tokens * (d // 16) // 32)
    groups = min(heads, -(-12 * sms // warps))
    return -(-heads // groups)


# (T, Hq, Hk): all 15 heads of a token in a thread (d = 128), or 8 and 7; groups of 14 (d = 128) and 8
# (d = 64), which cross from q to k and from k to v; 48 heads in three and five groups
@pytest.mark.parametrize("T,Hq,Hk", [(8191, 5, 5), (3000, 26, 7), (3000, 32, 8)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,rot,layout", [(64, 48, "half"), (128, 128, "half"), (128, 32, "interleaved")])
def test_write_and_read(dtype, d, rot, layout, T, Hq, Hk):
    import exact_attention_158_b200 as fa
    assert heads_per_thread(T, Hq + 2 * Hk, d) > 4
    assert heads_per_thread(T, 2 * Hk, d) > 4 or T < 8191  # the reader's, of k and v
    g = torch.Generator(device="cuda").manual_seed(T + d + Hq)
    x = torch.randn((T, Hq + 2 * Hk, d), generator=g, device="cuda")
    x = (x * torch.exp2(torch.randint(-9, 9, (T, Hq + 2 * Hk, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    P = T // 16 + 5
    slots = torch.randperm(P * 16, generator=g, device="cuda")[:T]
    slots[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    slots[-20:] = -3
    pos = torch.randint(0, 200000, (T,), generator=g, device="cuda", dtype=torch.int32)
    freqs, amp = fa.rope_frequencies(rot, scaling="ramp", factor=4.0)
    kp, vp, ks, vs = pools(P, Hk, d, dtype, fill=3)
    before = [None if t is None else t.clone() for t in (kp, vp, ks, vs)]
    yq = fa.fa_cache_append(k, v, kp, vp, slots, ks, vs, pos, freqs, layout, amp, q=q)
    back = fa.fa_cache_read(kp, vp, slots, ks, vs)
    assert fa.device_status() == 0
    p = pos[:, None]
    R.check(yq, R.rope(q, p, freqs, layout, amp), R.rope_bound(q, freqs, layout, amp, torch.bfloat16), "q")
    live = slots >= 0
    sources = (("k", R.rope(k, p, freqs, layout, amp), R.rope_bound(k, freqs, layout, amp, torch.float32), kp, ks),
               ("v", v.double(), 0.0 * v.double(), vp, vs))
    for (name, want, more, pool, sc), got in zip(sources, back):
        assert torch.equal(got[~live], torch.zeros_like(got[~live])), name
        want, more, got = want[live], more[live], got[live]
        if dtype == torch.bfloat16:
            R.check(got, want, stored_bound(want, dtype) + more, name)
            continue
        codes = at(pool, slots[live])
        codes = codes.view(dtype).float() if dtype != torch.int8 else codes.float()
        stored = codes * at(sc, slots[live])[..., None]
        assert torch.equal(got, stored.to(torch.bfloat16)), name
        R.check(stored, want, stored_bound(want, dtype) + 2 * more, name)
    if dtype != torch.bfloat16:  # values are not rotated: codes and scales to the bit
        codes, scale = R.quantise(v[live].float().cpu(), dtype)
        assert torch.equal(at(vs, slots[live]).cpu(), scale)
        assert torch.equal(at(vp, slots[live]).cpu(), codes.view(torch.uint8) if dtype != torch.int8 else codes)
    else:
        assert torch.equal(back[1][live], v[live])
    other = torch.ones(P * 16, dtype=torch.bool, device="cuda")
    other[slots[live]] = False
    rest = torch.arange(P * 16, device="cuda")[other]
    for t, b in zip((kp, vp, ks, vs), before):
        if t is not None:
            assert torch.equal(at(t, rest), at(b, rest))


@pytest.mark.parametrize("dtype", TYPES)
def test_nothing_but_padding(dtype):
    import exact_attention_158_b200 as fa
    T, Hq, Hk, d = 5000, 6, 2, 64
    x = torch.randn((T, Hq + 2 * Hk, d), device="cuda").to(torch.bfloat16)
    kp, vp, ks, vs = pools(4, Hk, d, dtype, fill=3)
    before = kp.clone()
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    y = fa.fa_cache_append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], kp, vp, slots, ks, vs, q=x[:, :Hq])
    assert torch.equal(y, x[:, :Hq])  # no frequencies: q as it is
    assert torch.equal(kp.view(torch.uint8), before.view(torch.uint8)) and fa.device_status() == 0


@pytest.mark.parametrize("H,d,lens", [(4, 128, [1, 16, 700, 2049]), (3, 64, [33, 1500])])
def test_a_bf16_cache_is_what_the_16_bit_decode_reads(H, d, lens):
    import exact_attention_158_b200 as fa
    import workloads as W
    from oracle import oracle as orc
    from tests import parity
    g = torch.Generator(device="cuda").manual_seed(d)
    pages = [-(-n // 16) for n in lens]
    P = sum(pages) + 2
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
    first = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[first:first + n]
        first += n
    kp, vp = (torch.zeros((P, H, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    freqs, amp = fa.rope_frequencies(d)
    last = []
    for s, n in enumerate(lens):
        x = torch.randn((n, 3 * H, d), generator=g, device="cuda").to(torch.bfloat16)
        t = torch.arange(n, device="cuda")
        slots = table[s, t // 16].long() * 16 + t % 16
        y = fa.fa_cache_append(x[:, H:2 * H], x[:, 2 * H:], kp, vp, slots, positions=t.to(torch.int32),
                               freqs=freqs, amplitude=amp, q=x[:, :H])
        want = R.rope(x[:, H:2 * H], t[:, None], freqs)
        got = at(kp, slots)
        R.check(got, want, stored_bound(want, torch.bfloat16) + R.rope_bound(x[:, H:2 * H], freqs, "half", amp, torch.float32), "k")
        assert torch.equal(at(vp, slots), x[:, 2 * H:])
        last.append(y[-1])
    q, seq_lens = torch.stack(last), torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.fa_decode_paged(q, kp, vp, table, seq_lens, out_dtype=torch.float32)
    assert fa.device_status() == 0
    o_ref, lse_ref = orc.decode_paged(W.bf16_bits(q), W.bf16_bits(kp), W.bf16_bits(vp), table.cpu().numpy(),
                                      seq_lens.cpu().numpy(), 1.0 / d ** 0.5)
    parity.assert_close(o.cpu().numpy(), lse.cpu().numpy(), o_ref, lse_ref, "bf16 cache")
