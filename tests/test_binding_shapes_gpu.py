"""Tensors of the right number of elements in another order are refused by the packed and int8 calls; the same
order with axes joined or split is taken and gives the same results."""
import pytest

pytestmark = pytest.mark.gpu

T, H, HKV, D = 40, 4, 2, 128


def packed():
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    cu = torch.tensor([0, 31, T], dtype=torch.int32, device="cuda")
    q, k, v, do = new(T, H, D), new(T, HKV, D), new(T, HKV, D), new(T, H, D)
    return q, k, v, do, cu, *wa.varlen_fwd(q, k, v, cu, cu, causal=True)


def swapped(t):
    return t.transpose(0, 1).contiguous()


def test_backward_refuses_another_order():
    import video_dit_full_b200 as wa
    q, k, v, do, cu, o, lse = packed()
    wa.varlen_bwd(q, k, v, o, do, lse, cu, cu, causal=True)
    for args in ((swapped(o), do, lse), (o, swapped(do), lse), (o, do, swapped(lse)),
                 (o.view(T, D, H), do, lse), (o, do.view(T // 2, H, 2 * D), lse)):
        with pytest.raises(ValueError):
            wa.varlen_bwd(q, k, v, *args, cu, cu, causal=True)


def test_given_outputs_of_another_order_are_refused():
    import torch
    import video_dit_full_b200 as wa
    q, k, v, do, cu, o, lse = packed()
    x = torch.randn(10, 64, device="cuda").to(torch.bfloat16)
    dy = torch.randn(10, 24, device="cuda").to(torch.bfloat16)
    wc, ws = wa.int8_quantize_rows(torch.randn(24, 64, device="cuda").to(torch.bfloat16))
    codes, scales = wa.int8_quantize_rows(x)
    new = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")                # noqa: E731
    for call, out in ((lambda t: wa.varlen_fwd(q, k, v, cu, cu, o=t), new(H, T, D)),
                      (lambda t: wa.varlen_fwd(q, k, v, cu, cu, lse=t), new(T, H).float()),
                      (lambda t: wa.int8_quantize_rows(x, codes=t), torch.full((64, 10), 7, dtype=torch.int8, device="cuda")),
                      (lambda t: wa.int8_dequantize_rows(codes, scales, x=t), new(64, 10)),
                      (lambda t: wa.int8_gemm(codes, scales, wc, ws, y=t), new(24, 10)),
                      (lambda t: wa.int8_grad_weight(dy, codes, scales, dw=t), new(64, 24)),
                      (lambda t: wa.int8_grad_input(dy, wc, ws, dx=t), new(64, 10))):
        with pytest.raises(ValueError):
            call(out)
        assert (out == 7).all()


def test_joined_and_split_axes_are_taken():
    import torch
    import video_dit_full_b200 as wa
    q, k, v, do, cu, o, lse = packed()
    want = wa.varlen_bwd(q, k, v, o, do, lse, cu, cu, causal=True)
    for shapes in (((T, H * D), (T, H * D), (H * T,)), ((T * H, D), (T * H * D,), (1, H, T)), ((5, 8, H, D), (T, H, 2, 64), (H, 5, 8))):
        got = wa.varlen_bwd(q, k, v, *(t.view(*s) for t, s in zip((o, do, lse), shapes)), cu, cu, causal=True)
        # dK, dV of unsplit key tiles are summed in a fixed order
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    out = torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
    got, _ = wa.varlen_fwd(q, k, v, cu, cu, causal=True, o=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out.view(T, H, D), o)
    x = torch.randn(10, 64, device="cuda").to(torch.bfloat16)
    codes, scales = wa.int8_quantize_rows(x, scales=torch.empty(10, 1, device="cuda"))
    again, flat = wa.int8_quantize_rows(x, codes=torch.empty(2, 5, 64, dtype=torch.int8, device="cuda"))
    assert scales.shape == (10, 1) and torch.equal(scales[:, 0], flat) and torch.equal(again.view(10, 64), codes)
    assert torch.equal(wa.int8_dequantize_rows(codes, scales), wa.int8_dequantize_rows(codes, flat))
    wa.check_status()
