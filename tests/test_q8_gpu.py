"""Attention over the 8-bit paged cache (decode, chunk, tree; shared key heads) against fp64."""
import math

import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def make(seed, S, Hq, Hk, d, lens, dtype, T=None, spare=3):
    """A call's inputs: a shuffled table over a pool with spare pages, unused table entries -1, and
    slots past the sequences' ends that hold no numbers."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-max(L, 0) // 16) for L in lens]
    P = sum(pages) + spare
    kp, ks = R.make_pool(g, P, Hk, d, dtype)
    vp, vs = R.make_pool(g, P, Hk, d, dtype)
    perm = torch.randperm(P, generator=g)
    table = torch.full((S, max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n].to(torch.int32)
        at += n
        if lens[s] % 16 and n:
            last = int(table[s, n - 1])
            for t in (ks, vs):
                t[last, :, lens[s] % 16:] = math.nan
            for t in (kp, vp):
                t.view(torch.uint8)[last, :, lens[s] % 16:] = 0x7f
    q = torch.randn((S, Hq, d) if T is None else (S, Hq, T, d), generator=g).to(torch.bfloat16).cuda()
    return q, kp, vp, ks, vs, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def verify(a, o, lse, causal=False, tree=None, what=""):
    import exact_attention_158_b200 as fa
    torch.cuda.synchronize()
    q, kp, vp, ks, vs, table, lens = a
    four = q if q.dim() == 4 else q[:, :, None]
    wo, wl, ob, lb = R.attention(four, kp, vp, ks, vs, table, lens, 1.0 / math.sqrt(q.shape[-1]), causal, tree)
    if o.dtype == torch.bfloat16:
        ob = ob + R.U_BF16 * (wo.abs() + ob)
    R.check(o.reshape(wo.shape), wo, ob, what + " O")
    if lse is not None:
        R.check(lse.reshape(wl.shape), wl, lb, what + " LSE")


def call(fn, a, *rest, **kw):
    import exact_attention_158_b200 as fa
    out = getattr(fa, fn)(*a, *rest, **kw)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    return out


LENS = [1, 0, 15, 16, 17, 333, 64, 1030]


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (6, 2), (8, 1), (9, 1), (16, 1), (20, 1), (32, 32)])
def test_decode(dtype, d, Hq, Hk):
    a = make(Hq + d, len(LENS), Hq, Hk, d, LENS, dtype)
    o, lse = call("fa_decode_paged_q8", a, out_dtype=torch.float32)
    verify(a, o, lse, what="decode")


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_decode_long_context_is_split(dtype):
    a = make(11, 2, 8, 2, 128, [20011, 7000], dtype)
    import exact_attention_158_b200 as fa
    assert fa.fa_q8_workspace_size(2, 8, 2, 1, 128, a[5].shape[1]) > 0
    o, lse = call("fa_decode_paged_q8", a)
    verify(a, o, lse, what="split")


def test_decode_one_chunk_needs_no_workspace():
    import exact_attention_158_b200 as fa
    assert fa.fa_q8_workspace_size(64, 8, 8, 1, 64, 1) == 0
    a = make(12, 64, 8, 8, 64, [1 + s % 16 for s in range(64)], INT8)
    o, lse = call("fa_decode_paged_q8", a, return_lse=False)
    assert lse is None
    verify(a, o, None, what="one chunk")


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,T", [(1, 1, 2), (4, 2, 5), (8, 1, 64), (3, 3, 33), (6, 2, 50), (16, 2, 17)])
def test_chunk_causal(dtype, d, Hq, Hk, T):
    lens = [T, T + 1, T + 15, 300, T + 128, 0]
    a = make(T + d, len(lens), Hq, Hk, d, lens, dtype, T)
    o, lse = call("fa_prefill_paged_q8", a, out_dtype=torch.float32)
    verify(a, o, lse, causal=True, what="chunk")


@pytest.mark.parametrize("Lq,lens", [(200, [200, 1000, 333]), (129, [129, 4000]), (1, [1, 40])])
@pytest.mark.parametrize("causal", [False, True])
def test_chunk_long(Lq, lens, causal):
    a = make(Lq, len(lens), 8, 2, 128, lens, E4M3, Lq)
    o, lse = call("fa_prefill_paged_q8", a, causal=causal)
    verify(a, o, lse, causal=causal, what="long chunk")


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,T", [(2, 10), (2, 17), (2, 64), (4, 50)])  # 20, 34, 128 and 200 rows
def test_many_tiles_of_tokens_in_one_range(dtype, Hq, T):
    # enough (sequence, head) pairs that contexts are not split: dozens of tiles follow one another,
    # of ragged numbers, and the roles of a CTA run at their own pace
    lens = [T + (37 * s) % 1900 for s in range(150)]
    lens[7] = 3000
    a = make(60 + T, 150, Hq, 1, 64, lens, dtype, T)
    for _ in range(3):
        o, lse = call("fa_prefill_paged_q8", a)
    verify(a, o, lse, causal=True, what="many tiles")


def masks(seed, S, T, dev="cuda"):
    import workloads as W
    rows = [W.tree_visibility(p) for p in W.random_tree_parents(seed, S, T)]
    signed = [[m - (1 << 64) if m >= 1 << 63 else m for m in r] for r in rows]
    return torch.tensor(signed, dtype=torch.int64)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,T", [(2, 2, 1), (4, 1, 13), (8, 2, 64), (3, 1, 31)])
def test_tree(dtype, d, Hq, Hk, T):
    lens = [T, T + 1, 700, T + 127, T + 16]
    a = make(T, len(lens), Hq, Hk, d, lens, dtype, T)
    m = masks(T, len(lens), T)
    m[0, T // 2] = 0            # with no context, this node sees nothing
    o, lse = call("fa_tree_attention_q8", a, m.cuda(), out_dtype=torch.float32)
    verify(a, o, lse, tree=m, what="tree")
    assert torch.equal(o[0, :, T // 2], torch.zeros_like(o[0, :, T // 2]))
    assert (lse[0, :, T // 2] == -math.inf).all()


@pytest.mark.parametrize("T,Hq", [(None, 4), (40, 8)])
def test_no_number_stays_where_it_is_seen(T, Hq):
    # a token whose scales are NaN makes the rows that see it NaN and no other
    n = T or 1
    a = make(21, 2, Hq, 2, 64, [100, 60], E4M3, T)
    q, kp, vp, ks, vs, table, lens = a
    blk, row = int(table[0, (100 - n) // 16]), (100 - n) % 16  # the first of the queries' own tokens
    ks[blk, 1, row] = math.nan
    if T is None:
        o, lse = call("fa_decode_paged_q8", a)
        assert torch.isnan(o[0, Hq // 2:]).all() and torch.isnan(lse[0, Hq // 2:]).all()
        assert torch.isfinite(o[0, :Hq // 2]).all() and torch.isfinite(o[1]).all()
        ks[blk, 1, row], vs[blk, 1, row] = 1.0, math.nan
        o, lse = call("fa_decode_paged_q8", a)
        assert torch.isnan(o[0, Hq // 2:]).all() and torch.isfinite(lse).all()
        return
    m = masks(3, 2, T)
    m &= ~1                     # no node sees node 0 but itself
    m[:, 0] = 1
    vs[blk, 1, row] = math.nan
    o, lse = call("fa_tree_attention_q8", a, m.cuda())
    assert torch.isnan(o[0, Hq // 2:, 0]).all()
    assert torch.isfinite(o[0, Hq // 2:, 1:]).all() and torch.isfinite(o[0, :Hq // 2]).all()
    assert torch.isfinite(o[1]).all()


def test_scales_far_apart():
    # one token's values are 2^20 times the others': both it and they keep their precision
    a = make(22, 1, 4, 1, 128, [400], E4M3)
    q, kp, vp, ks, vs, table, lens = a
    vs[int(table[0, 3]), 0, 4] *= 2.0 ** 20
    vs[int(table[0, 9]), 0, 7] *= 2.0 ** -20
    ks[int(table[0, 3]), 0, 4] *= 2.0 ** -12
    o, lse = call("fa_decode_paged_q8", a, out_dtype=torch.float32)
    verify(a, o, lse, what="far apart")


def test_peaked_and_rising_scores():
    for T in (None, 30):
        a = make(23, 2, 8, 2, 128, [900, 1500], INT8, T)
        q, kp, vp, ks, vs, table, lens = a
        for s in range(2):  # keys grow along the context: the reference maximum keeps moving
            for i in range(-(-int(lens[s]) // 16)):
                ks[int(table[s, i])] *= 2.0 ** (i / 8)
        fn = "fa_decode_paged_q8" if T is None else "fa_prefill_paged_q8"
        o, lse = call(fn, a, out_dtype=torch.float32)
        verify(a, o, lse, causal=T is not None, what="rising")


@pytest.mark.parametrize("T", [None, 48])
def test_bad_table_entries_and_lengths_are_reported(T):
    import exact_attention_158_b200 as fa
    a = make(24, 3, 8, 2, 64, [200, 300, 100], E4M3, T)
    q, kp, vp, ks, vs, table, lens = a
    table[0, 2] = kp.shape[0] + 5
    table[1, 0] = -3
    f = fa.fa_decode_paged_q8 if T is None else fa.fa_prefill_paged_q8
    o, lse = f(*a, out_dtype=torch.float32)
    assert fa.device_status() == 1
    verify(a, o, lse, causal=T is not None, what="left out")
    lens[2] = 10 ** 6
    o, lse = f(*a)
    assert fa.device_status() == 1
    assert torch.isfinite(o[:2].float()).all()


@pytest.mark.parametrize("T", [None, 48])
def test_captured_and_replayed_on_other_inputs(T):
    import exact_attention_158_b200 as fa
    f = fa.fa_decode_paged_q8 if T is None else fa.fa_prefill_paged_q8
    a = make(25, 2, 8, 2, 128, [2000, 900], E4M3, T)
    q, kp, vp, ks, vs, table, lens = a
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], device="cuda")
    f(*a, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(*a, out=out, lse=lse)
    lens -= 77
    q.copy_(torch.randn(q.shape, device="cuda").to(torch.bfloat16))
    graph.replay()
    verify(a, out, lse, causal=T is not None, what="replayed")


def test_two_calls_at_once_with_their_own_workspaces():
    import exact_attention_158_b200 as fa
    calls = [make(30 + i, 2, 8, 2, 128, [3000, 1200], E4M3) for i in range(2)]
    want = [fa.fa_decode_paged_q8(*a) for a in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [None, None]
    for _ in range(20):
        for i, (a, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i] = fa.fa_decode_paged_q8(*a)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])  # no atomics: the same bits


def test_pool_past_32_bits():
    import exact_attention_158_b200 as fa
    P, Hk, d = 140_000, 8, 128
    g = torch.Generator().manual_seed(40)
    small_k, sk = R.make_pool(g, 4, Hk, d, INT8)
    small_v, sv = R.make_pool(g, 4, Hk, d, INT8)
    kp, vp = (torch.empty((P, Hk, 16, d), dtype=INT8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((P, Hk, 16), device="cuda") for _ in range(2))
    where = torch.tensor([P - 1, P - 2, 3, P // 2], device="cuda")
    for big, s in ((kp, small_k), (vp, small_v), (ks, sk), (vs, sv)):
        big[where] = s
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    for T in (None, 20):
        q = torch.randn((1, 16, d) if T is None else (1, 16, T, d), device="cuda").to(torch.bfloat16)
        f = fa.fa_decode_paged_q8 if T is None else fa.fa_prefill_paged_q8
        big = f(q, kp, vp, ks, vs, where[None].to(torch.int32), lens)
        few = f(q, small_k, small_v, sk, sv, torch.arange(4, dtype=torch.int32, device="cuda")[None], lens)
        torch.cuda.synchronize()
        assert torch.equal(big[0], few[0]) and torch.equal(big[1], few[1])


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_a_serving_step(dtype):
    """Prompt, then decode steps, then a drafted tree, each token through fa_cache_append: the 8-bit
    path against 16-bit attention over the rotated tokens, within what the codes lose."""
    import exact_attention_158_b200 as fa
    g = torch.Generator(device="cuda").manual_seed(50)
    S, Hq, Hk, d, n0 = 3, 8, 2, 64, [40, 17, 64]
    freqs, amp = fa.rope_frequencies(48)
    maxb = 10
    table = torch.randperm(S * maxb, generator=g, device="cuda").to(torch.int32).view(S, maxb)
    kp, vp = (torch.zeros((S * maxb, Hk, 16, d), dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((S * maxb, Hk, 16), device="cuda") for _ in range(2))
    kept = [[], [], []]

    def add(s_of, at):
        """Tokens of sequences s_of at cache places `at`; returns their rotated queries."""
        T = len(s_of)
        x = torch.randn((T, Hq + 2 * Hk, d), generator=g, device="cuda").to(torch.bfloat16)
        s_t, a_t = torch.tensor(s_of, device="cuda"), torch.tensor(at, device="cuda")
        slots = table[s_t, a_t // 16].long() * 16 + a_t % 16
        q = fa.fa_cache_append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], kp, vp, slots, ks, vs,
                               a_t.to(torch.int32), freqs, "half", amp, q=x[:, :Hq])
        k = R.rope(x[:, Hq:Hq + Hk].cpu(), a_t.cpu()[:, None], freqs.cpu())
        for i, s in enumerate(s_of):
            kept[s].append((k[i], x[i, Hq + Hk:].double().cpu()))
        return q

    def reference(s, q, see):
        """q [Hq, T, d] against the kept tokens in fp64; see [T, L]."""
        K, V = (torch.stack([t[i] for t in kept[s]], 1) for i in (0, 1))  # [Hk, L, d]
        K, V = (t.repeat_interleave(Hq // Hk, 0) for t in (K, V))
        z = (q.double().cpu() @ K.transpose(1, 2)) / math.sqrt(d)
        w = torch.softmax(torch.where(see, z, -math.inf), -1)
        # a code is off by up to 2^-4 of its value (int8: 1/254 of the row's largest): a score by
        # that of scale sum |q||k|, a weight by twice that relative, and the values likewise
        c = 2.0 ** -4
        e = c * (q.double().cpu().abs() @ K.abs().transpose(1, 2) / math.sqrt(d)).amax(-1, keepdim=True)
        return w @ V, (torch.expm1(2 * e) + c + 4 * R.U_BF16) * (w @ V.abs()) + 0.03

    def compare(o, s, q, see, what):
        want, bound = reference(s, q, see)
        R.check(o, want, bound, what)

    q = add([s for s in range(S) for _ in range(n0[s])], [t for s in range(S) for t in range(n0[s])])
    lens = torch.tensor(n0, dtype=torch.int32, device="cuda")
    first = 0
    for s in range(S):  # the prompts, one sequence at a time
        qs = q[first:first + n0[s]].transpose(0, 1).contiguous()[None]
        first += n0[s]
        o, _ = call("fa_prefill_paged_q8", (qs, kp, vp, ks, vs, table[s:s + 1].contiguous(), lens[s:s + 1]))
        compare(o[0], s, qs[0], torch.ones(n0[s], n0[s], dtype=torch.bool).tril(), "prompt")
    for step in range(3):
        q = add(list(range(S)), [int(x) for x in lens])
        lens = lens + 1
        o, _ = call("fa_decode_paged_q8", (q, kp, vp, ks, vs, table, lens))
        for s in range(S):
            compare(o[s][:, None], s, q[s][:, None], torch.ones(1, int(lens[s]), dtype=torch.bool), "step")
    T = 5
    m = masks(9, S, T)
    q = add([s for s in range(S) for _ in range(T)], [int(lens[s]) + t for s in range(S) for t in range(T)])
    lens = lens + T
    q = q.view(S, T, Hq, d).transpose(1, 2).contiguous()
    o, _ = call("fa_tree_attention_q8", (q, kp, vp, ks, vs, table, lens), m.cuda())
    for s in range(S):
        see = torch.ones(T, int(lens[s]), dtype=torch.bool)
        for t in range(T):
            see[t, -T:] = torch.tensor([(int(m[s, t]) >> u) & 1 == 1 for u in range(T)])
        compare(o[s], s, q[s], see, "tree")


def test_new_tensors_belong_to_the_given_stream():
    # the current stream has freed memory that it still writes to; a call on another stream whose
    # results or workspace lay there would lose them
    import exact_attention_158_b200 as fa
    a = make(70, 2, 8, 2, 128, [3000, 700], E4M3)
    kp, vp, ks, vs = a[1:5]
    slots = (a[5][0, :4].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
    x = torch.randn((2, 8, 32, 128), device="cuda").to(torch.bfloat16)
    pos = torch.arange(32, dtype=torch.int32, device="cuda")
    freqs = fa.rope_frequencies(128)[0].cuda()
    side = torch.cuda.Stream()
    calls = [lambda **kw: fa.fa_decode_paged_q8(*a, **kw),
             lambda **kw: fa.fa_rope(x, x, pos, freqs, **kw),
             lambda **kw: fa.fa_cache_read(kp, vp, slots, ks, vs, **kw)]
    for f in calls:
        want = f()
        torch.cuda.synchronize()
        late = [torch.empty_like(t) for t in want for _ in range(2)]
        if f is calls[0]:
            need = fa.fa_q8_workspace_size(2, 8, 2, 1, 128, a[5].shape[1])
            assert need > 0
            late.append(torch.empty(need, dtype=torch.uint8, device="cuda"))
        torch.cuda._sleep(40_000_000)
        for t in late:
            t.fill_(7)
        del late, t
        got = f(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
