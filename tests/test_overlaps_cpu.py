"""Outputs that share memory with what is read, or with themselves, are refused; layouts that only
alternate in one buffer are not (no GPU needed: the accepted calls fail a later check)."""
import ctypes
import itertools
import random

import pytest
import torch

import exact_attention_158_b200 as fa
from exact_attention_158_b200 import build as fab

A = 1 << 24  # a fake device address, never dereferenced
D = 64
INVALID, MISALIGNED = 1, 3


@pytest.fixture(scope="module")
def lib():
    fab.build()
    return fa.load_library()


def st(v):
    return (ctypes.c_longlong * len(v))(*v)


def rope(lib, q, qs, qo, qos, k=None, ks=(0, 0, 0), ko=None, kos=(0, 0, 0), B=1, Hq=1, Hk=0, N=1, idt=0,
         odt=0, pos=1 << 40, pos_stride=0, fr=1 << 41, rot=16):
    """A call that is refused in any case: its frequencies are misaligned, which is looked at after the
    overlaps."""
    return lib.fa_rope(q, st(qs), qo, st(qos), k, st(ks), ko, st(kos), idt, odt, pos, pos_stride, fr + 4,
                       rot, 0, 1.0, 0, B, Hq, Hk, N, D, None)


def test_rope_shifted_and_crossed(lib):
    dense = dict(qs=(0, 512, 64), qos=(0, 512, 64), Hq=4, N=8)
    assert rope(lib, A, qo=A, **dense) == MISALIGNED                       # in place
    assert rope(lib, A, qo=A + 2 * 64, **dense) == INVALID                 # a row further on
    assert rope(lib, A, qo=A + 2 * 8 * 4 * 64, **dense) == MISALIGNED      # just behind
    assert rope(lib, A, qo=A - 2 * 8 * 4 * 64, **dense) == MISALIGNED      # just before
    assert rope(lib, A, qo=A + 2 * 8 * 4 * 64 - 16, **dense) == INVALID
    kv = dict(dense, k=2 * A, ks=(0, 512, 64), ko=3 * A, kos=(0, 512, 64), Hk=4)
    assert rope(lib, A, qo=4 * A, **kv) == MISALIGNED
    assert rope(lib, A, qo=2 * A, **kv) == INVALID                         # q_out over k
    assert rope(lib, A, qo=3 * A, **kv) == INVALID                         # q_out over k_out
    assert rope(lib, A, qo=4 * A, **dict(kv, ko=A)) == INVALID             # k_out over q
    assert rope(lib, A, qo=1 << 40, **dense) == INVALID                    # q_out over the positions
    assert rope(lib, A, qo=1 << 41, **dense) == INVALID                    # q_out over the frequencies


def test_rope_outputs_on_themselves(lib):
    for qos in ((64, 64, 64), (0, 64, 64), (512, 64, 32), (1024, 1024, 64)):
        assert rope(lib, A, (2048, 512, 64), 2 * A, qos, B=2, Hq=4, N=8) == INVALID, qos
    # rows that fill one another's gaps share nothing
    assert rope(lib, A, (0, 512, 64), 2 * A, (0, 64, 4 * 64), Hq=4, N=8) == MISALIGNED
    assert rope(lib, A, (0, 512, 64), 2 * A, (0, 3 * 64, 2 * 64), Hq=2, N=3) == MISALIGNED


def test_rope_fused_projection_in_place(lib):
    B, N, Hq, Hk = 3, 50, 8, 2
    W = (Hq + 2 * Hk) * D
    s = (N * W, D, W)
    k = A + 2 * Hq * D
    both = dict(B=B, N=N, Hq=Hq, Hk=Hk)
    assert rope(lib, A, s, A, s, k, s, k, s, **both) == MISALIGNED
    assert rope(lib, A, s, A, s, k, s, 2 * A, s, **both) == MISALIGNED       # q in place, k elsewhere
    assert rope(lib, A, s, k + 2 * Hk * D, s, k, s, k, s, **both) == INVALID  # q_out past the v heads
    assert rope(lib, A, s, A, s, k - 2 * D, s, k - 2 * D, s, **both) == INVALID


def test_rope_strides_of_any_size(lib):
    far = 1 << 59
    assert rope(lib, A, (0, 512, 64), 2 * A, (far, far, far), B=1, Hq=1, N=1) == MISALIGNED
    assert rope(lib, A, (-far, 512, 64), 2 * A, (-far, 512, 64), B=4, Hq=4, N=8) == MISALIGNED
    assert rope(lib, A, (0, 512, 64), 1 << 30, (0, -512, -64), Hq=4, N=8) == MISALIGNED
    assert rope(lib, A, (0, 512, 64), A, (0, 512, 64), Hq=4, N=8, odt=1) == INVALID


def rows(p, s, n, size):
    return [p + sum(i * x * size for i, x in zip(idx, s)) for idx in itertools.product(*map(range, n))]


def test_rope_against_every_pair_of_rows(lib):
    rng = random.Random(1)
    seen = {INVALID: 0, MISALIGNED: 0}
    for _ in range(4000):
        B, H, N = (rng.randint(1, 3) for _ in range(3))
        idt, odt = rng.randint(0, 1), rng.randint(0, 1)
        size = (2, 4)
        strides = [tuple(rng.choice([-1, 1]) * 8 * rng.choice([0, 4, 8, 12, 16, 24, 32, 48, 72, 96])
                         for _ in range(3)) for _ in range(2)]
        p, y = A, A + 16 * rng.randint(-150, 150)
        got = rope(lib, p, strides[0], y, strides[1], B=B, Hq=H, N=N, idt=idt, odt=odt)
        ins = rows(p, strides[0], (B, H, N), size[idt])
        outs = rows(y, strides[1], (B, H, N), size[odt])
        w, r = D * size[odt], D * size[idt]
        on = [a == 0 or b == c for a, b, c in zip((B - 1, H - 1, N - 1), *strides)]
        same = p == y and idt == odt and all(on)
        meet = any(-w < a - b < w for a, b in itertools.combinations(outs, 2))
        meet |= not same and any(-w < a - b < r for a in outs for b in ins)
        assert got == (INVALID if meet or (p == y and not same) else MISALIGNED), (B, H, N, strides, y - p)
        seen[got] += 1
    assert min(seen.values()) > 300


def append(lib, k, ks, v, vs, q=None, qs=(0, 0), qo=None, qos=(0, 0), T=4, Hq=0, Hk=2, pos=1 << 41,
           fr=1 << 42, slots=1 << 43, rot=16, vp=1 << 45, kp=1 << 44):
    return lib.fa_cache_append(k, st(ks), v, st(vs), kp, vp, 1 << 46, 1 << 47, 1, slots, 8, q, st(qs), qo,
                               st(qos), pos, fr, rot, 0, 1.0, T, Hq, Hk, D, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would be launched")
def test_append_queries_over_what_is_read(lib):
    T, Hq, Hk = 4, 6, 2
    W = (Hq + 2 * Hk) * D
    k, v, q = A + 2 * Hq * D, A + 2 * (Hq + Hk) * D, A
    s = (W, D)
    a = dict(k=k, ks=s, v=v, vs=s, q=q, qs=s, T=T, Hq=Hq, Hk=Hk)
    dense = (Hq * D, D)
    assert append(lib, qo=k, qos=dense, **a) == INVALID          # over k
    assert append(lib, qo=v, qos=dense, **a) == INVALID          # over v
    assert append(lib, qo=q + 2 * D, qos=s, **a) == INVALID      # q, one head further on
    assert append(lib, qo=q + 2 * W, qos=s, **a) == INVALID      # q, one token further on
    assert append(lib, qo=2 * A, qos=(D, D), **a) == INVALID     # over itself
    assert append(lib, qo=2 * A, qos=(2 * D, 3 * D), **dict(a, T=4)) == INVALID  # rows 0, 3 and 2, 1 meet
    for name in ("slots", "pos", "fr"):
        assert append(lib, qo=2 * A, qos=dense, **dict(a, **{name: 2 * A + 64})) == INVALID, name
    assert append(lib, qo=2 * A, qos=dense, **dict(a, fr=(1 << 44) + 64)) == INVALID  # the pool over freqs


def test_strides_of_single_elements_are_not_looked_at(lib):
    # a misaligned stride that matters is told before the amplitude, which is refused in any case
    def status(qs, qos, B, Hq, N):
        return lib.fa_rope(A, st(qs), 2 * A, st(qos), None, None, None, None, 0, 0, 1 << 40, 0, 1 << 41, 16, 0,
                           float("nan"), 0, B, Hq, 0, N, D, None)

    for a in range(3):
        n = [4, 4, 4]
        n[a] = 1
        s = [[4096, 1024, 64], [4096, 1024, 64]]
        for i in range(2):
            odd = [list(x) for x in s]
            odd[i][a] = 1001
            assert status(*odd, *n) == INVALID
            assert status(*odd, 4, 4, 4) == MISALIGNED
