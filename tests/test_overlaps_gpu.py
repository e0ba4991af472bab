"""Layouts that alternate in one buffer, or fill one another's gaps, are taken and give what separate
tensors give."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotating_a_fused_projection_in_place(dtype, layout):
    import exact_attention_158_b200 as fa
    B, N, Hq, Hk, d = 3, 50, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, N, Hq + 2 * Hk, d), generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 9000, (B, N), generator=g, device="cuda", dtype=torch.int32)
    freqs, amp = fa.rope_frequencies(96)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    v = x[:, :, Hq + Hk:].clone()
    want_q, want_k = fa.fa_rope(q, k, pos, freqs, layout)
    fa.fa_rope(q, k, pos, freqs, layout, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(x[:, :, Hq + Hk:], v)
    with pytest.raises(fa.FaError):  # k's rows would land on heads of q that others still read
        fa.fa_rope(q, k, pos, freqs, layout, q_out=q, k_out=x[:, :, 1:1 + Hk].transpose(1, 2))
    with pytest.raises(fa.FaError):
        fa.fa_rope(q[:, :, 1:], None, pos[:, 1:].contiguous(), freqs, layout, q_out=q[:, :, :-1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn, torch.int8])
def test_queries_of_a_fused_projection_in_place(dtype):
    import exact_attention_158_b200 as fa
    T, Hq, Hk, d = 37, 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, Hq + 2 * Hk, d), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 900
    slots = torch.randperm(64, generator=g, device="cuda")[:T]
    freqs, amp = fa.rope_frequencies(64)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    kv = x[:, Hq:].clone()

    def call(**kw):
        pools = [torch.zeros((4, Hk, 16, d), device="cuda").to(dtype) for _ in range(2)]
        scales = [None if dtype == torch.bfloat16 else torch.zeros((4, Hk, 16), device="cuda") for _ in range(2)]
        y = fa.fa_cache_append(k, v, *pools, slots, *scales, pos, freqs, q=q, **kw)
        return y, fa.fa_cache_read(*pools, slots, *scales)

    # head-major beside token-major: the rows alternate, and share nothing
    room = torch.zeros((Hq, 2 * T, d), dtype=torch.bfloat16, device="cuda")
    want, want_kv = call()
    got, _ = call(q_out=room[:, ::2].transpose(0, 1))
    assert torch.equal(got, want) and torch.equal(room[:, 1::2], torch.zeros_like(room[:, 1::2]))
    for q_out in (x[:, 1:1 + Hq], x[:, Hk * 2:Hk * 2 + Hq], want[:1].expand(T, -1, -1)):
        with pytest.raises(fa.FaError):
            call(q_out=q_out)
    got, got_kv = call(q_out=q)
    assert torch.equal(q, want) and torch.equal(x[:, Hq:], kv)
    assert all(torch.equal(a, b) for a, b in zip(got_kv, want_kv))


def test_a_batch_of_one_with_any_stride():
    import exact_attention_158_b200 as fa
    N, H, d = 9, 2, 64
    room = torch.randn(2 * N * H * d + 10, device="cuda").to(torch.bfloat16)
    x = room.as_strided((1, H, N, d), (N * H * d + 5, d, H * d, 1))  # a batch's odd stride, one element
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freqs, _ = fa.rope_frequencies(64)
    got, _ = fa.fa_rope(x, None, pos, freqs)
    want, _ = fa.fa_rope(x.contiguous(), None, pos, freqs)
    assert torch.equal(got, want)
    one = room.as_strided((1, H, d), (77, d, 1))  # one token
    pools = [torch.zeros((1, H, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.fa_cache_append(one, one, *pools, torch.tensor([3], device="cuda"))
    assert torch.equal(pools[0][0, :, 3], one[0]) and torch.equal(pools[1][0, :, 3], one[0])
