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
