"""Attention over the 8-bit cache where many sequences share the GPU (taken by length), tiles run long,
tables are wider than the contexts, and workspaces hold anything; and a serving step against the codes
that its own tokens left."""
import math

import pytest
import torch

from tests import serving_ref as R
from tests.test_q8_gpu import E4M3, INT8, call, make, masks, verify

pytestmark = pytest.mark.gpu


def sorted_by_length(S, Hq, Hk, Lq, max_blocks, d):
    """Whether the kernel of many rows takes the sequences by length, as the library decides it."""
    import exact_attention_158_b200 as fa
    rows = Hq // Hk * Lq
    tiles = -(-rows // (256 if rows > 128 else 128))
    whole = fa.fa_q8_workspace_size(S, Hq, Hk, Lq, d, max_blocks) == 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return rows > 32 and 1 < S <= 128 and whole and S * Hk * tiles > sms


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", [(8, 4, 20), (16, 4, 48)])  # 40 and 192 rows: one row tile, two
@pytest.mark.parametrize("tree", [False, True])
def test_many_sequences_taken_by_length(dtype, Hq, Hk, T, tree):
    g = torch.Generator().manual_seed(T)
    lens = [int(x) for x in torch.randint(T, 900, (40,), generator=g)]
    lens[3], lens[17] = 3000, 2950              # 47 tiles of tokens: every ring goes round
    lens[8] = lens[9] = lens[30] = 640          # ties
    lens[0] = lens[21] = lens[39] = 0           # empty slots
    lens[5] = T
    a = make(80 + T, 40, Hq, Hk, 128, lens, dtype, T)
    assert sorted_by_length(40, Hq, Hk, T, a[5].shape[1], 128)
    if tree:
        m = masks(T, 40, T)
        o, lse = call("fa_tree_attention_q8", a, m.cuda(), out_dtype=torch.float32)
        verify(a, o, lse, tree=m, what="by length")
    else:
        o, lse = call("fa_prefill_paged_q8", a, out_dtype=torch.float32)
        verify(a, o, lse, causal=True, what="by length")
    for _ in range(3):  # and the same bits again
        again = (call("fa_tree_attention_q8", a, m.cuda(), out_dtype=torch.float32) if tree
                 else call("fa_prefill_paged_q8", a, out_dtype=torch.float32))
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("S", [128, 129])
@pytest.mark.parametrize("d", [64, 128])
def test_as_many_sequences_as_are_ranked_and_one_more(S, d):
    T, Hq, Hk = 9, 8, 2
    lens = [T + (53 * s) % 400 for s in range(S)]
    lens[1:4] = [0, 300, 300]
    a = make(S, S, Hq, Hk, d, lens, INT8, T)
    assert sorted_by_length(S, Hq, Hk, T, a[5].shape[1], d) == (S == 128)
    o, lse = call("fa_prefill_paged_q8", a)
    verify(a, o, lse, causal=True, what="ranked")


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,T", [(4, 10), (4, 48), (1, 300)])  # 40, 192 and 300 rows
def test_long_runs_of_tiles(dtype, Hq, T):
    # enough sequences that the longest is not split: 63 tiles of tokens in one CTA
    lens = [4000] + [T + 3 * s for s in range(159)]
    a = make(90, 160, Hq, 1, 128, lens, dtype, T)
    import exact_attention_158_b200 as fa
    assert fa.fa_q8_workspace_size(160, Hq, 1, T, 128, a[5].shape[1]) == 0
    o, lse = call("fa_prefill_paged_q8", a, out_dtype=torch.float32)
    verify(a, o, lse, causal=True, what="long run")


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", [(8, 2, None), (6, 2, 6), (8, 2, 10), (8, 2, 60)])
@pytest.mark.parametrize("width", [300, 8192])
def test_tables_wider_than_any_context(dtype, Hq, Hk, T, width):
    # as a loop keeps them that is captured once; what lies past a sequence's pages is not looked at
    lens = [T or 1, 0, 700, 2100]
    a = list(make(95, 4, Hq, Hk, 128, lens, dtype, T))
    wide = torch.full((4, width), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, :a[5].shape[1]] = a[5]
    tight, a[5] = a[5], wide
    for s, L in enumerate(lens):
        wide[s, -(-L // 16):] = 10 ** 9
    fn = "fa_decode_paged_q8" if T is None else "fa_prefill_paged_q8"
    o, lse = call(fn, a, out_dtype=torch.float32)
    a[5] = tight
    verify(a, o, lse, causal=T is not None, what="wide table")


@pytest.mark.parametrize("T,Hq", [(None, 8), (6, 8), (10, 8), (60, 8)])
def test_the_same_bits_whatever_the_workspace_held(T, Hq):
    import exact_attention_158_b200 as fa
    lens = [3000, 0, 17 + (T or 0), 1250]
    a = make(97, 4, Hq, 2, 128, lens, E4M3, T)
    f = fa.fa_decode_paged_q8 if T is None else fa.fa_prefill_paged_q8
    need = fa.fa_q8_workspace_size(4, Hq, 2, T or 1, 128, a[5].shape[1])
    assert need > 0
    room = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
    want = None
    for fill in (0, 255, 127, 66):
        room.fill_(fill)
        got = f(*a, out_dtype=torch.float32, workspace=room[:need])
        torch.cuda.synchronize()
        assert bool((room[need:] == fill).all())
        want = want or [t.clone() for t in got]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    verify(a, *got, causal=T is not None, what="workspace")


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("d,rot,layout", [(64, 48, "half"), (128, 128, "interleaved")])
def test_a_serving_step_against_its_own_codes(dtype, d, rot, layout):
    """Prompts, decode steps and a drafted tree.  Each new token's rotated query, and what the cache
    gives back for it, against the definition within a rounding or half a code step; then the attention
    against the stored codes, within its own bounds."""
    import exact_attention_158_b200 as fa
    from tests.test_cache_gpu import stored_bound
    g = torch.Generator(device="cuda").manual_seed(51)
    S, Hq, Hk, n0 = 3, 8, 2, [40, 17, 64]
    freqs, amp = fa.rope_frequencies(rot, scaling="ramp", factor=4.0)
    maxb = 10
    table = torch.randperm(S * maxb, generator=g, device="cuda").to(torch.int32).view(S, maxb)
    kp, vp = (torch.zeros((S * maxb, Hk, 16, d), dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((S * maxb, Hk, 16), device="cuda") for _ in range(2))
    kept = {}

    def add(s_of, places):
        x = torch.randn((len(s_of), Hq + 2 * Hk, d), generator=g, device="cuda").to(torch.bfloat16)
        s_t, a_t = torch.tensor(s_of, device="cuda"), torch.tensor(places, device="cuda")
        slots = table[s_t, a_t // 16].long() * 16 + a_t % 16
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        y = fa.fa_cache_append(k, v, kp, vp, slots, ks, vs, a_t.to(torch.int32), freqs, layout, amp, q=q)
        p = a_t[:, None]
        R.check(y, R.rope(q, p, freqs, layout, amp), R.rope_bound(q, freqs, layout, amp, torch.bfloat16), "q")
        more = 2 * R.rope_bound(k, freqs, layout, amp, torch.float32)
        for i, slot in enumerate(slots.tolist()):
            kept[slot] = (R.rope(k, p, freqs, layout, amp)[i], more[i], v[i].double())
        return y

    def step(fn, q, lens, *rest, **how):
        # everything in the cache, not the newest tokens alone
        slots = torch.tensor(list(kept), device="cuda")
        back = fa.fa_cache_read(kp, vp, slots, ks, vs)
        want_k, more, want_v = (torch.stack([t[i] for t in kept.values()]) for i in range(3))
        for got, want, extra in ((back[0], want_k, more), (back[1], want_v, 0.0)):
            bound = stored_bound(want, dtype) + extra
            R.check(got, want, bound + R.U_BF16 * (want.abs() + bound), "cache")
        a = (q, kp, vp, ks, vs, table, lens)
        o, lse = call(fn, a, *rest, out_dtype=torch.float32)
        verify(a, o, lse, what=fn, **how)
        # the outputs are far from zero by the bounds' measure
        assert float(o.abs().mean()) > 0.05

    q = add([s for s in range(S) for _ in range(n0[s])], [t for s in range(S) for t in range(n0[s])])
    lens = torch.tensor(n0, dtype=torch.int32, device="cuda")
    first = 0
    for s in range(S):  # the prompts, one sequence at a time
        qs = q[first:first + n0[s]].transpose(0, 1).contiguous()[None]
        first += n0[s]
        a = (qs, kp, vp, ks, vs, table[s:s + 1].contiguous(), lens[s:s + 1].contiguous())
        o, lse = call("fa_prefill_paged_q8", a, out_dtype=torch.float32)
        verify(a, o, lse, causal=True, what="prompt")
    for _ in range(3):
        q = add(list(range(S)), lens.tolist())
        lens = lens + 1
        step("fa_decode_paged_q8", q, lens)
    for T in (5, 11):  # 20 and 44 rows per key head: either kernel
        m = masks(T, S, T)
        q = add([s for s in range(S) for _ in range(T)], [int(n) + t for n in lens for t in range(T)])
        lens = lens + T
        step("fa_tree_attention_q8", q.view(S, T, Hq, d).transpose(1, 2).contiguous(), lens, m.cuda(), tree=m)
