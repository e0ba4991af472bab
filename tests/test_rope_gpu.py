"""fa_rope against the rotation in fp64: layouts, partial heads, strides, types, far positions, and
the transposed rotation as its gradient."""
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu


def rotate(q, k, pos, freqs, layout, amp=1.0, inverse=False, out_dtype=None, **kw):
    import exact_attention_158_b200 as fa
    out = fa.fa_rope(q, k, pos, freqs, layout=layout, amplitude=amp, inverse=inverse,
                     out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    return out


def verify(x, y, pos, freqs, layout, amp, inverse, out_dtype, what):
    x, f = x.cpu(), freqs.cpu()
    p = pos.cpu()
    p = p[:, None] if p.dim() == 2 else p
    want = R.rope(x, p, f, layout, amp, inverse)
    R.check(y, want, R.rope_bound(x, f, layout, amp, out_dtype), what)


def freqs_of(rot, **kw):
    import exact_attention_158_b200 as fa
    return fa.rope_frequencies(rot, **kw)


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 96), (128, 128), (128, 0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
def test_layouts(d, rot, layout, inverse):
    g = torch.Generator().manual_seed(d + rot)
    B, N, Hq, Hk = 3, 37, 5, 2
    x = torch.randn((B, N, Hq + 2 * Hk, d), generator=g).to(torch.bfloat16).cuda()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    pos = torch.randint(0, 5000, (B, N), generator=g, dtype=torch.int32).cuda()
    freqs = freqs_of(rot)[0] if rot else torch.zeros(0, dtype=torch.float64, device="cuda")
    yq, yk = rotate(q, k, pos, freqs, layout, 1.25, inverse)
    assert yq.is_contiguous() and yk.is_contiguous()
    verify(q, yq, pos, freqs, layout, 1.25, inverse, torch.bfloat16, "q")
    verify(k, yk, pos, freqs, layout, 1.25, inverse, torch.bfloat16, "k")


@pytest.mark.parametrize("src,dst", [(a, b) for a in (torch.bfloat16, torch.float32)
                                     for b in (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_types_and_far_positions(src, dst, layout):
    g = torch.Generator().manual_seed(7)
    q = torch.randn((2, 3, 9, 128), generator=g).to(src).cuda()
    pos = torch.tensor([0, 1, -5, 4095, 131071, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31],
                       dtype=torch.int32).cuda()
    freqs, amp = freqs_of(64, scaling="ramp", factor=8.0)
    y, none = rotate(q, None, pos, freqs, layout, amp, out_dtype=dst)
    assert none is None and y.dtype == dst
    verify(q, y, pos, freqs, layout, amp, False, dst, f"{src} -> {dst}")


@pytest.mark.parametrize("B,N,Hq,Hk", [(1, 1, 1, 1), (64, 1, 32, 8), (1, 2049, 1, 1), (700, 3, 7, 1),
                                       (2, 1031, 16, 16)])
def test_sizes(B, N, Hq, Hk):
    g = torch.Generator(device="cuda").manual_seed(N)
    q = torch.randn((B, Hq, N, 64), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((B, Hk, N, 64), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") + 100
    freqs, amp = freqs_of(64)
    yq, yk = rotate(q, k, pos, freqs, "half")
    verify(q, yq, pos, freqs, "half", 1.0, False, torch.bfloat16, "q")
    verify(k, yk, pos, freqs, "half", 1.0, False, torch.bfloat16, "k")


def test_gradient_of_a_projection():
    # head-major gradients back to the projection's layout: <rope(x), g> = <x, rope^T(g)>
    g = torch.Generator().manual_seed(3)
    B, N, Hq, Hk, d = 2, 65, 4, 2, 64
    x = torch.randn((B, N, Hq + 2 * Hk, d), generator=g).cuda()
    pos = torch.randint(0, 100000, (B, N), generator=g, dtype=torch.int32).cuda()
    freqs, amp = freqs_of(32, scaling="linear", factor=4.0)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    gq, gk = (torch.randn(t.shape, generator=g).cuda() for t in (q, k))
    dx = torch.full_like(x, 7.0)
    dq, dk = dx[:, :, :Hq].transpose(1, 2), dx[:, :, Hq:Hq + Hk].transpose(1, 2)
    rotate(gq, gk, pos, freqs, "interleaved", 1.5, True, q_out=dq, k_out=dk)
    verify(gq, dq, pos, freqs, "interleaved", 1.5, True, torch.float32, "dq")
    verify(gk, dk, pos, freqs, "interleaved", 1.5, True, torch.float32, "dk")
    assert torch.equal(dx[:, :, Hq + Hk:], torch.full_like(dx[:, :, Hq + Hk:], 7.0)), "v's part is left alone"
    # differences of L = sum(g * rope(x)): linear in x, so any step gives the derivative.  The fp32
    # outputs are off by 2^-21 of amplitude (|a| + |b|) each, on both sides of the difference.
    yq, _ = rotate(q, None, pos, freqs, "interleaved", 1.5)
    step = torch.randn(q.shape, generator=g).cuda()
    y2, _ = rotate(q + step, None, pos, freqs, "interleaved", 1.5)
    lhs = ((y2.double() - yq.double()) * gq.double()).sum()
    rhs = (((q + step).double() - q.double()) * dq.double()).sum()
    f = freqs.cpu()
    err = sum((R.rope_bound(a.cpu(), f, "interleaved", 1.5, torch.float32) * b.double().abs().cpu()).sum()
              for a, b in ((q, gq), (q + step, gq), (gq, step)))
    assert abs(float(lhs - rhs)) <= float(err)


def test_in_place_broadcast_and_other_stream():
    g = torch.Generator().manual_seed(5)
    freqs, _ = freqs_of(128)
    pos = torch.arange(33, dtype=torch.int32).cuda()
    q = torch.randn((2, 4, 33, 128), generator=g).to(torch.bfloat16).cuda()
    want, _ = rotate(q, None, pos, freqs, "half")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mine = q.clone()
    torch.cuda.synchronize()
    rotate(mine, None, pos, freqs, "half", q_out=mine, stream=s)
    s.synchronize()
    assert torch.equal(mine, want)
    one = q[:1].expand(3, -1, -1, -1)  # stride 0 over b
    y, _ = rotate(one, None, pos, freqs, "half")
    assert torch.equal(y, want[:1].expand(3, -1, -1, -1))


def test_empty_and_captured():
    import exact_attention_158_b200 as fa
    freqs, _ = freqs_of(64)
    e = torch.empty((2, 3, 0, 64), dtype=torch.bfloat16, device="cuda")
    y, _ = rotate(e, None, torch.empty(0, dtype=torch.int32, device="cuda"), freqs, "half")
    assert y.shape == e.shape
    q = torch.randn((1, 2, 5, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    fa.fa_rope(q, None, pos, freqs, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(q, None, pos, freqs, q_out=out)
    pos += 1000
    graph.replay()
    verify(q, out, pos, freqs, "half", 1.0, False, torch.bfloat16, "replayed")
