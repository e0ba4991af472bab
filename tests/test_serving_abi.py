"""Host-side refusals of the rotary, cache and 8-bit attention entry points (no GPU needed), the
frequency tables, and the workspace sizes."""
import ctypes
import math

import pytest
import torch

import exact_attention_158_b200 as fa
from exact_attention_158_b200 import build as fab


@pytest.fixture(scope="module")
def lib():
    fab.build()
    return fa.load_library()


A = 1 << 24  # fake device addresses, far enough apart not to overlap; never dereferenced


def st(*v):
    return (ctypes.c_longlong * len(v))(*v)


def rope(lib, q=A, qs=(4096, 512, 64), qo=2 * A, qos=(4096, 512, 64), k=3 * A, ko=4 * A, idt=0, odt=0,
         pos=5 * A, fr=6 * A, rot=64, layout=0, amp=1.0, inv=0, B=2, Hq=8, Hk=8, N=8, d=64):
    return lib.fa_rope(q, st(*qs), qo, st(*qos), k, st(*qs), ko, st(*qos), idt, odt, pos, 0, fr, rot,
                       layout, amp, inv, B, Hq, Hk, N, d, None)


def test_rope_refusals(lib):
    assert rope(lib, q=None) == 1 and rope(lib, qo=None) == 1 and rope(lib, k=None) == 1
    assert rope(lib, pos=None) == 1 and rope(lib, fr=None) == 1
    assert rope(lib, rot=24) == 1 and rope(lib, rot=80) == 1 and rope(lib, rot=-16) == 1
    assert rope(lib, layout=2) == 1 and rope(lib, inv=3) == 1 and rope(lib, idt=5) == 1 and rope(lib, odt=5) == 1
    assert rope(lib, amp=math.nan) == 1 and rope(lib, amp=math.inf) == 1
    assert rope(lib, Hq=0) == 1 and rope(lib, B=-1) == 1 and rope(lib, N=-1) == 1
    assert rope(lib, d=96) == 2
    assert rope(lib, q=A + 8) == 3 and rope(lib, ko=4 * A + 2) == 3 and rope(lib, pos=5 * A + 2) == 3
    assert rope(lib, qs=(4096, 512, 68)) == 3 and rope(lib, qos=(4096, 516, 64)) == 3
    assert rope(lib, idt=1, odt=1, qs=(4096, 512, 66)) == 3
    assert rope(lib, qos=(4096, 0, 64)) == 1  # the output's heads would lie on one another
    assert rope(lib, B=1 << 16, N=1 << 16) == 1
    assert rope(lib, N=0) == 0 and rope(lib, B=0) == 0  # nothing to do


def test_rope_in_place_is_the_same_tensor(lib):
    assert rope(lib, qo=A, odt=1) == 1                       # written wider than read
    assert rope(lib, qo=A, qos=(4096, 64, 512)) == 1         # written elsewhere
    assert rope(lib, ko=3 * A, qos=(8192, 512, 64)) == 1
    assert rope(lib, qo=A, ko=3 * A, N=0) == 0


def append(lib, k=A, ks=(512, 64), v=2 * A, kp=16 * A, vp=18 * A, ksc=20 * A, vsc=22 * A, ty=1, slots=3 * A,
           P=8, q=4 * A, qo=5 * A, qos=(512, 64), pos=6 * A, fr=7 * A, rot=64, layout=0, amp=1.0, T=4, Hq=8,
           Hk=8, d=64):
    return lib.fa_cache_append(k, st(*ks), v, st(*ks), kp, vp, ksc, vsc, ty, slots, P, q, st(*ks), qo,
                               st(*qos), pos, fr, rot, layout, amp, T, Hq, Hk, d, None)


def test_append_refusals(lib):
    assert append(lib, k=None) == 1 and append(lib, slots=None) == 1 and append(lib, kp=None) == 1
    assert append(lib, ksc=None) == 1 and append(lib, vsc=None, ty=2) == 1
    assert append(lib, q=None) == 1 and append(lib, qo=None) == 1
    assert append(lib, ty=3) == 1 and append(lib, T=-1) == 1 and append(lib, Hk=0) == 1 and append(lib, Hq=-1) == 1
    assert append(lib, P=0) == 1 and append(lib, P=2 ** 30, Hk=2) == 1
    assert append(lib, rot=8) == 1 and append(lib, pos=None) == 1 and append(lib, layout=-1) == 1
    assert append(lib, d=32) == 2
    assert append(lib, kp=16 * A + 8) == 3 and append(lib, ksc=20 * A + 4) == 3 and append(lib, slots=3 * A + 4) == 3
    assert append(lib, ks=(516, 64)) == 3 and append(lib, q=4 * A + 8) == 3
    assert append(lib, qos=(0, 64)) == 1
    assert append(lib, vp=16 * A + 1024) == 1      # the pools overlap
    assert append(lib, vsc=20 * A + 64) == 1       # the scales overlap
    assert append(lib, slots=16 * A + 64) == 1     # slots inside the pool
    assert append(lib, T=0) == 0


def read(lib, kp=16 * A, vp=18 * A, ksc=20 * A, vsc=22 * A, ty=1, slots=3 * A, P=8, k=A, v=2 * A, T=4, H=8, d=64):
    return lib.fa_cache_read(kp, vp, ksc, vsc, ty, slots, P, k, v, T, H, d, None)


def test_append_overlaps(lib):
    far = A // 64  # T = 4 rows of 64 features this far apart (in elements) span 3 A / 32 bytes
    for over in (16 * A - A // 16, 18 * A - A // 16):
        assert append(lib, k=over, ks=(far, 64)) == 1 and append(lib, v=over, ks=(far, 64)) == 1
        assert append(lib, qo=over, qos=(far, 64)) == 1 and append(lib, q=over, ks=(far, 64)) == 1
    assert append(lib, k=22 * A + A // 16, ks=(-far, 64)) == 1  # backwards into a scale
    assert append(lib, qo=20 * A) == 1 and append(lib, qo=3 * A) == 1 and append(lib, qo=6 * A) == 1
    assert append(lib, qo=4 * A, qos=(512, 128)) == 1           # in place with other strides


def test_read_refusals(lib):
    assert read(lib, k=None) == 1 and read(lib, slots=None) == 1 and read(lib, vp=None) == 1
    assert read(lib, ksc=None) == 1 and read(lib, ty=-1) == 1 and read(lib, T=-2) == 1 and read(lib, H=0) == 1
    assert read(lib, d=256) == 2 and read(lib, k=A + 2) == 3 and read(lib, slots=3 * A + 1) == 3
    assert read(lib, k=16 * A) == 1 and read(lib, v=A + 64) == 1
    assert read(lib, T=0) == 0


def q8(lib, fn="decode", q=A, kp=16 * A, vp=18 * A, ksc=20 * A, vsc=22 * A, ty=1, table=3 * A, maxb=4, lens=4 * A,
       P=8, o=5 * A, odt=0, lse=None, S=2, Hq=8, Hk=2, Lq=16, d=64, causal=1, scale=0.0, ws=6 * A, wsb=1 << 20,
       mask=7 * A):
    head = (q, kp, vp, ksc, vsc, ty, table, maxb, lens, P)
    if fn == "decode":
        return lib.fa_decode_paged_q8(*head, o, odt, lse, S, Hq, Hk, d, scale, ws, wsb, None)
    if fn == "tree":
        return lib.fa_tree_attention_q8(*head, mask, o, odt, lse, S, Hq, Hk, Lq, d, scale, ws, wsb, None)
    return lib.fa_prefill_paged_q8(*head, o, odt, lse, S, Hq, Hk, Lq, d, causal, scale, ws, wsb, None)


@pytest.mark.parametrize("fn", ["decode", "chunk", "tree"])
def test_q8_refusals(lib, fn):
    c = lambda **k: q8(lib, fn, **k)  # noqa: E731
    assert c(q=None) == 1 and c(kp=None) == 1 and c(ksc=None) == 1 and c(table=None) == 1 and c(o=None) == 1
    assert c(ty=0) == 1 and c(ty=3) == 1 and c(odt=2) == 1
    assert c(S=0) == 1 and c(Hq=0) == 1 and c(Hk=0) == 1 and c(Hk=3) == 1 and c(maxb=0) == 1 and c(P=0) == 1
    assert c(scale=math.nan) == 1 and c(scale=math.inf) == 1
    assert c(d=80) == 2
    assert c(q=A + 4) == 3 and c(vp=18 * A + 8) == 3 and c(vsc=22 * A + 8) == 3 and c(table=3 * A + 2) == 3
    assert c(lse=8 * A + 2) == 3
    assert c(o=A) == 1 and c(o=16 * A + 16) == 1 and c(lse=5 * A + 4) == 1 and c(lse=20 * A) == 1
    assert c(P=2 ** 30, Hk=2) == 1 and c(S=1 << 16, Hq=1 << 14, Hk=1) == 1
    assert c(maxb=4000, ws=None) == 6 and c(maxb=4000, wsb=16) == 6 and c(maxb=4000, ws=6 * A + 4, wsb=1 << 30) == 3
    assert c(maxb=4000, ws=5 * A, wsb=1 << 30) == 1  # the workspace overlaps the output
    if fn != "decode":
        assert c(Lq=0) == 1 and c(Lq=65) == 1  # a table row maps 64 tokens
    if fn == "chunk":
        assert c(causal=2) == 1
    if fn == "tree":
        assert c(mask=None) == 1 and c(Lq=65, maxb=100) == 1 and c(mask=7 * A + 4) == 3 and c(o=7 * A) == 1


def test_workspace_sizes(lib):
    assert fa.fa_q8_workspace_size(1, 8, 3, 1, 64, 4) == 0      # heads do not divide
    assert fa.fa_q8_workspace_size(1, 8, 2, 1, 96, 4) == 0
    assert fa.fa_q8_workspace_size(64, 32, 32, 1, 128, 8) == 0  # short contexts are not split
    long = fa.fa_q8_workspace_size(1, 8, 1, 1, 128, 4096)
    assert long > 0 and long % (8 * (128 + 2) * 4) == 0         # whole partials of the 8 rows


def test_python_refusals():
    t = torch.zeros(2, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_rope(t, None, None, None)  # not on the GPU
    with pytest.raises(ValueError):
        fa.fa_cache_append(t[0], t[0], t, t, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        fa.fa_decode_paged_q8(t[0], t, t, None, None, None, None)


def test_frequencies():
    f, a = fa.rope_frequencies(64, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    want = torch.tensor([10000.0 ** (-2 * j / 64) for j in range(32)], dtype=torch.float64)
    assert torch.allclose(f, want, rtol=1e-14, atol=0)
    lin, _ = fa.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin * 4, want, rtol=1e-14, atol=0)
    base, _ = fa.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert base[0] == 1.0 and math.isclose(float(base[-1]) * 4, float(want[-1]), rel_tol=1e-12)
    ramp, amp = fa.rope_frequencies(64, scaling="ramp", factor=4.0, device="cpu")
    turns = 4096 * want / (2 * math.pi)
    assert torch.equal(ramp[turns >= 32], want[turns >= 32])
    assert torch.allclose(ramp[turns <= 1] * 4, want[turns <= 1], rtol=1e-14, atol=0)
    assert (ramp[1:] < ramp[:-1]).all() and math.isclose(amp, 0.1 * math.log(4) + 1)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=64, scaling="other"), dict(rot=64, factor=0.5),
                dict(rot=2, scaling="base"), dict(rot=64, scaling="ramp", fast=1.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**bad, device="cpu")
