"""Scales of the 8-bit cache far apart, very small or zero, against fp64 with bounds that hold only
what a row sees: both kernels, every length and mask."""
import math

import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def make(seed, S, Hq, Hk, d, L, dtype, T=None):
    """S sequences of L tokens, each in pages of its own in order; values and keys of the same size."""
    g = torch.Generator().manual_seed(seed)
    n = -(-L // 16)
    pools = [R.quantise(torch.randn((S * n, Hk, 16, d), generator=g), dtype) for _ in range(2)]
    (kp, ks), (vp, vs) = ((c.cuda(), s.cuda()) for c, s in pools)
    q = torch.randn((S, Hq, d) if T is None else (S, Hq, T, d), generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(S * n, dtype=torch.int32).view(S, n).cuda()
    return [q, kp, vp, ks, vs, table, torch.full((S,), L, dtype=torch.int32).cuda()]


def tokens(x, a, s):
    """Sequence s's part of a pool or of its scales, by token: a view [tokens, Hk, ...]."""
    n = a[5].shape[1]
    return x.view(a[5].shape[0], n, *x.shape[1:])[s].transpose(1, 2).flatten(0, 1)


def scale_by(x, a, s, at, factor):
    """Multiplies the scales of sequence s's tokens `at` (all heads)."""
    n = a[5].shape[1]
    for t in range(*at.indices(n * 16)) if isinstance(at, slice) else [at]:
        x[s * n + t // 16, :, t % 16] *= factor


def see_of(T, L, causal, mask):
    see = torch.ones(T, L, dtype=torch.bool)
    if mask is not None:
        for t, m in enumerate(mask):
            see[t, L - T:] = torch.tensor([(m >> u) & 1 == 1 for u in range(T)])
    elif causal:
        see = see.tril(L - T)
    return see


def reference(a, causal, masks):
    """(o, lse, o_bound, lse_bound) in fp64, [S, Hq, T, ...].

    With w a row's weights and e its largest scale sum |q||K|: the scores are off by less than 2^-18 e
    (products are exact; each of the d / 16 steps of a tensor-core sum rounds within 2^-23 of its
    largest term, twice) and 2^-23 for scaling; a weight by twice that and exp2's 2^-21.  The weight,
    the value's scale and their product with the code are rounded to fp16, 2^-11 each at most.
    Where p times the values' power of two lies below fp16's normal range it is off by 2^-25, and the
    row's largest is at least 2^6, with a fraction of 2^-9 at least left to V (or at least 1 with
    the whole scale in it): 2^-22 of the row's largest w vs, times a code.  No term holds a
    scale that the row does not see.
    LSE: the scores' error, 2^-20 for exponentials, sum and logarithm, and the rounding of scores that are
    held against a reference as far away as the values' log2 (or 64, for values of scale 0)."""
    q, kp, vp, ks, vs, table, lens = a
    q4 = (q if q.dim() == 4 else q[:, :, None]).double().cpu()
    S, Hq, T, d = q4.shape
    Hk = kp.shape[1]
    out = [torch.zeros(S, Hq, T, d, dtype=torch.float64), torch.full((S, Hq, T), -math.inf, dtype=torch.float64)]
    bounds = [torch.zeros_like(x) for x in out]
    for s, L in enumerate(lens.tolist()):
        if L <= 0:
            continue
        see = see_of(T, L, causal, None if masks is None else masks[s])
        cv = [tokens(x.float(), a, s)[:L].double().cpu() for x in (kp, vp)]
        sc = [tokens(x, a, s)[:L].double().cpu() for x in (ks, vs)]
        for h in range(Hq):
            kh = h // (Hq // Hk)
            K, f, code = cv[0][:, kh] * sc[0][:, kh, None], sc[1][:, kh], cv[1][:, kh]
            z = torch.where(see, q4[s, h] @ K.T / math.sqrt(d), -math.inf)
            w = torch.softmax(z, -1).nan_to_num(0.0)
            V = code * f[:, None]
            out[0][s, h], out[1][s, h] = w @ V, torch.logsumexp(z, -1)
            e = torch.where(see, q4[s, h].abs() @ K.abs().T / math.sqrt(d), 0.0).amax(-1)
            top = (w * f).amax(-1)
            bounds[0][s, h] = ((3 * 2.0 ** -11 + 2.0 ** -17 * e + 2.0 ** -18)[:, None] * (w @ V.abs())
                               + 2.0 ** -22 * top[:, None] * (see.double() @ (code.abs() * (f > 0)[:, None])))
            far = torch.where(see & (f > 0), f.clamp(min=1e-300).log2().abs(), 0.0).amax(-1)
            far = torch.where((see & (f == 0)).any(-1), far.clamp(min=64.0), far)
            bounds[1][s, h] = (2.0 ** -18 * e + 2.0 ** -20 * (1.0 + out[1][s, h].abs().nan_to_num(0.0, posinf=0.0))
                               + 2.0 ** -24 * (16.0 + far))
    return out, bounds


def verify(a, what, causal=False, masks=None):
    import exact_attention_158_b200 as fa
    if a[0].dim() == 3:
        got = fa.fa_decode_paged_q8(*a, out_dtype=torch.float32)
    elif masks is not None:
        signed = [[m - (1 << 64) if m >= 1 << 63 else m for m in r] for r in masks]
        got = fa.fa_tree_attention_q8(*a, torch.tensor(signed, dtype=torch.int64, device="cuda"),
                                      out_dtype=torch.float32)
    else:
        got = fa.fa_prefill_paged_q8(*a, causal=causal, out_dtype=torch.float32)
    assert fa.device_status() == 0
    want, bounds = reference(a, causal, masks)
    for g, w, b, n in zip(got, want, bounds, ("O", "LSE")):
        R.check(g.reshape(w.shape), w, b, f"{what} {n}")
    return got


# rows per key head: 4 and 18 take the kernel of few rows; 40 and 120 one row tile of the kernel of many
# rows, 200 and 328 two (a whole and a ragged one, then a third)
FEW = [(4, 1, None), (6, 1, 3)]
MANY = [(8, 1, 5), (6, 2, 40), (5, 1, 40), (8, 1, 41)]


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", FEW + MANY)
@pytest.mark.parametrize("S,L", [(2, 333), (1, 2500)])
def test_values_of_a_few_binades_above_the_smallest_kept(dtype, Hq, Hk, T, S, L):
    a = make(1, S, Hq, Hk, 128, L, dtype, T)
    a[4] *= 2.0 ** -88          # scales of about 2^-95 (e4m3) and 2^-93
    verify(a, "tiny values", causal=T is not None)


@pytest.mark.parametrize("Hq,Hk,T", FEW + MANY)
@pytest.mark.parametrize("S,L", [(2, 333), (1, 2500)])
@pytest.mark.parametrize("up", [20, 70, 110])
def test_a_loud_token_among_values_of_zero(Hq, Hk, T, S, L, up):
    # zeros set no reference, so theirs lies far below the loud token's: their weights still count
    for first in (5, L // 2, L - 9):
        a = make(2, S, Hq, Hk, 64, L, INT8, T)
        a[4] *= 0
        scale = a[4][:, :, 0].clone().fill_(2.0 ** up)
        n = a[5].shape[1]
        for s in range(S):
            a[4][s * n + first // 16, :, first % 16] = scale[0]
        a[0] *= 0.25
        verify(a, f"loud at {first}", causal=T is not None)


@pytest.mark.parametrize("Hq,Hk,T", FEW + MANY)
def test_values_of_zero_alone(Hq, Hk, T):
    a = make(3, 2, Hq, Hk, 64, 700, E4M3, T)
    a[4] *= 0
    verify(a, "zeros", causal=T is not None)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", FEW[1:] + MANY)
@pytest.mark.parametrize("up", [9, 24, 31, 60, 110])
def test_a_loud_token_that_other_rows_do_not_see(dtype, Hq, Hk, T, up):
    # one of the queries' own tokens: the rows before it (causal), the nodes off its branch (tree)
    L, mid = 230, T // 2
    a = make(4, 2, Hq, Hk, 128, L, dtype, T)
    for s in range(2):
        scale_by(a[4], a, s, L - T + mid, 2.0 ** up)
    verify(a, "hidden", causal=True)
    masks = [[(1 << t) | (1 << (t // 2)) | 1 for t in range(T)] for _ in range(2)]  # few see the middle node
    verify(a, "off the branch", masks=masks)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", FEW + MANY)
@pytest.mark.parametrize("up", [24, 40])
def test_a_loud_token_of_next_to_no_weight(dtype, Hq, Hk, T, up):
    L = 500
    a = make(5, 1, Hq, Hk, 128, L, dtype, T)
    u = torch.randn(128, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    a[0][:] = u.cuda()
    codes, scale = R.quantise(-4.0 * u.float()[None], dtype)  # a score of about -45
    for at in (3, 200, 450):
        a[1][at // 16, :, at % 16] = codes[0].cuda()
        a[3][at // 16, :, at % 16] = scale[0].cuda()
        scale_by(a[4], a, 0, at, 2.0 ** up)
    verify(a, "weightless", causal=T is not None)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", FEW + MANY)
@pytest.mark.parametrize("spread", [4, 7, 8, 9, 30])
def test_scales_rise_and_fall_along_the_context(dtype, Hq, Hk, T, spread):
    # by `spread` binades up and down again within 50 tokens, and by 40 over the whole context
    L = 1100
    a = make(7, 2, Hq, Hk, 64, L, dtype, T)
    at = torch.arange(a[5].shape[1] * 16)
    wave = torch.exp2(spread * (1 - (at % 50 - 25).abs() / 25) + 40 * (at % 700) / 700).float().cuda()
    n = a[5].shape[1]
    a[4] *= wave.view(1, n, 1, 16).expand(2, -1, -1, -1).reshape(2 * n, 1, 16)
    verify(a, "wave", causal=T is not None)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", FEW + MANY)
def test_scales_alike(dtype, Hq, Hk, T):
    a = make(8, 2, Hq, Hk, 128, 1500, dtype, T)
    verify(a, "alike", causal=T is not None)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("Hq,Hk,T", FEW[1:] + MANY)
@pytest.mark.parametrize("up", [10, 13, 30, 60, 125])
def test_queries_of_any_size_side_by_side(dtype, Hq, Hk, T, up):
    # rows of one key head whose queries are 2^up times the others', as padding that holds anything
    # may be: each row keeps the precision that it has alone
    a = make(9, 2, Hq, Hk, 128, 300, dtype, T)
    loud = torch.zeros(2, Hq, T, dtype=torch.bool)
    loud[:, :, T // 3] = True
    loud[1, Hq // 2, ::2] = True
    a[0][loud] *= 2.0 ** up
    a[0][0, 0, T - 1] = 0.0
    got = verify_rows(a, ~loud)
    assert torch.isfinite(got[0][~loud]).all()


def verify_rows(a, rows):
    """As verify (causal), of the rows given; the others' scores may be of any size."""
    import exact_attention_158_b200 as fa
    got = fa.fa_prefill_paged_q8(*a, out_dtype=torch.float32)
    assert fa.device_status() == 0
    want, bounds = reference(a, True, None)
    for g, w, b, n in zip(got, want, bounds, ("O", "LSE")):
        R.check(g.cpu()[rows], w[rows], b[rows], f"rows {n}")
    return got
