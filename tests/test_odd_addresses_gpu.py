"""Scales and offsets that start 4 bytes past a 16-byte boundary, as the header allows, give the same results."""
import pytest

pytestmark = pytest.mark.gpu


def odd(t):
    """The same values 4 bytes past a 16-byte boundary."""
    import torch
    out = torch.empty(t.numel() + 4, dtype=t.dtype, device="cuda")[1:1 + t.numel()].view(t.shape)
    assert out.data_ptr() % 16 == 4
    return out.copy_(t)


# one kernel, few tokens (split and whole), CTA pairs
@pytest.mark.parametrize("M,N,K", [(1, 264, 1040), (16, 5120, 272), (37, 264, 1040), (130, 520, 144), (300, 9736, 144), (2000, 2056, 2064)])
def test_scales(M, N, K):
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(M)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    x, dy = new(M, K), new(M, N)
    wc, ws = wa.int8_quantize_rows(new(N, K))
    y, codes, scales = wa.int8_linear(x, wc, ws, return_checkpoint=True)
    at = odd(torch.zeros(M, device="cuda"))
    assert torch.equal(wa.int8_quantize_rows(x, scales=at)[1], scales)
    assert torch.equal(wa.int8_linear(x, wc, odd(ws)), y) and torch.equal(wa.int8_gemm(codes, at, wc, odd(ws)), y)
    assert torch.equal(wa.int8_dequantize_rows(codes, at), wa.int8_dequantize_rows(codes, scales))
    assert torch.equal(wa.int8_grad_weight(dy, codes, at), wa.int8_grad_weight(dy, codes, scales))
    assert torch.equal(wa.int8_grad_input(dy, wc, odd(ws)), wa.int8_grad_input(dy, wc, ws))
    wa.check_status()


@pytest.mark.parametrize("lens_q,lens_k", [([5, 200], [5, 200]), ([1, 1, 1], [4000, 17, 900])])
def test_offsets(lens_q, lens_k):
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    cu = [torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() for lens in (lens_q, lens_k)]
    q, k, v = new(sum(lens_q), 4, 128), new(sum(lens_k), 2, 128), new(sum(lens_k), 2, 128)
    o, lse = wa.varlen_fwd(q, k, v, *cu, causal=True)
    o1, lse1 = wa.varlen_fwd(q, k, v, odd(cu[0]), odd(cu[1]), causal=True)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    a, b = (wa.varlen_bwd(q, k, v, o, q, lse, *c, causal=True) for c in (cu, [odd(c) for c in cu]))
    # dQ, and dK, dV of split key tiles, are summed in no fixed order: two bf16 half steps, and the fp32 sums'
    for s, t in zip(a, b):
        assert ((s.float() - t.float()).abs() <= 2.0 ** -7 * t.float().abs() + 2.0 ** -12 * t.float().abs().max()).all()
    wa.check_status()
