"""The int8 linear layer, its 8-bit checkpoints and its backward against the oracle
(oracle/int8_linear.py).

Bars.  Codes, scales and the values read back are exact.  y: the int32 sums are exact, so
|dy| <= 2^-8 |y| (bf16's half step) + 2^-21 (|y before bias| + |bias|) (four fp32 roundings).
dW, dX: every code times its scale is rounded to bf16 and summed in fp32 over n terms:
(2^-8 + n 2^-24) sum |a b| + 2^-8 |result|; the relative Frobenius error stays below 5e-3.
"""
import numpy as np
import pytest

from oracle import int8_linear as il

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def bf16(shape, seed, outliers=False):
    import torch
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=gen)
    if outliers:
        x[:, ::37] *= 20
    return x.to(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def weight(N, K, seed):
    import torch
    codes, scales = il.quant_rows((bf16((N, K), seed).float() / K ** 0.5).numpy())
    return codes, scales, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()


def within(got, want, bound, frob=5e-3):
    got = f64(got)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= bound + 1e-30).all(), float((err / (bound + 1e-30)).max())
    assert np.linalg.norm(err) <= frob * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (130, 144), (37, 5120), (5, 16400)])
def test_rows_exact(M, K):
    import torch
    import video_dit_full_b200 as wa
    x = bf16((M, K), M + K, outliers=True)
    if M > 2:
        x[1] = 0
        x[2] = x[2, :1] * torch.linspace(-1, 1, K).to(torch.bfloat16)
        x[2, : K // 2] = x[2].abs().max() / 2                       # ties at 63.5
    codes, scales = wa.int8_quantize_rows(x.cuda())
    back = wa.int8_dequantize_rows(codes, scales)
    wa.check_status()
    want, want_s = il.quant_rows(x.float().numpy())
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    want_x = (torch.from_numpy(want).float() * torch.from_numpy(want_s)[:, None]).to(torch.bfloat16)
    assert torch.equal(back.cpu(), want_x)


@pytest.mark.parametrize("power", [-126, -133, -64, 60, 120])
def test_rows_of_extreme_magnitude(power):
    import torch
    import video_dit_full_b200 as wa
    x = (bf16((4, 272), 3).double() * 2.0 ** power).to(torch.bfloat16)
    codes, scales = wa.int8_quantize_rows(x.cuda())
    want, want_s = il.quant_rows(x.float().numpy())
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)


def test_non_finite_rows_show():
    import torch
    import video_dit_full_b200 as wa
    x = bf16((5, 64), 1)
    x[1, 3], x[2, 63], x[4, 0] = float("inf"), float("nan"), float("-inf")
    codes, scales = wa.int8_quantize_rows(x.cuda())
    assert torch.isnan(scales).tolist() == [False, True, True, False, True]
    assert not codes[[1, 2, 4]].any()
    _, _, wc, ws = weight(24, 64, 2)
    y = wa.int8_linear(x.cuda(), wc, ws)
    wa.check_status()
    assert torch.isnan(y).all(1).tolist() == [False, True, True, False, True]
    assert torch.isfinite(y[[0, 3]]).all()


def test_strided_rows():
    import torch
    import video_dit_full_b200 as wa
    wide = bf16((70, 3 * 64), 5).cuda()
    x = wide[:, 64:128]
    _, _, wc, ws = weight(40, 64, 3)
    y, codes, scales = wa.int8_linear(x, wc, ws, return_checkpoint=True)
    y2, codes2, scales2 = wa.int8_linear(x.contiguous(), wc, ws, return_checkpoint=True)
    wa.check_status()
    assert torch.equal(y, y2) and torch.equal(codes, codes2) and torch.equal(scales, scales2)


LAYERS = [(1, 8, 16), (1, 5120, 1536), (2, 1000, 272), (7, 264, 1040), (16, 128, 128), (17, 136, 2048), (33, 520, 144),
          (64, 1536, 8960), (65, 256, 256), (100, 264, 5120), (128, 256, 512), (129, 256, 512), (257, 1032, 2064), (300, 8, 16),
          (515, 1536, 1536), (1000, 520, 1040)]


@pytest.mark.parametrize("M,N,K", LAYERS)
@pytest.mark.parametrize("with_bias", [False, True])
def test_layer(M, N, K, with_bias):
    import torch
    import video_dit_full_b200 as wa
    x = bf16((M, K), M, outliers=True)
    wc, ws, wcd, wsd = weight(N, K, N)
    bias = bf16((N,), 9) if with_bias else None
    bd = None if bias is None else bias.cuda()
    y, codes, scales = wa.int8_linear(x.cuda(), wcd, wsd, bias=bd, return_checkpoint=True)
    y2 = wa.int8_gemm(codes, scales, wcd, wsd, bias=bd)
    wa.check_status()
    assert torch.equal(y, y2)                                     # the same sums, exactly
    c, s = il.quant_rows(x.float().numpy())
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    b = 0.0 if bias is None else f64(bias)
    want, mag = il.linear(c, s, wc, ws, b)
    within(y, want, U * np.abs(want) + 2.0 ** -21 * (mag + np.abs(b)))


def test_largest_sums():
    """K = 131072 codes of 127: the int32 sum 127^2 * 131072 < 2^31."""
    import torch
    import video_dit_full_b200 as wa
    for M in (1, 200):
        x = torch.ones(M, 131072, dtype=torch.bfloat16, device="cuda")
        w = torch.full((8, 131072), 127, dtype=torch.int8, device="cuda")
        y = wa.int8_linear(x, w, torch.full((8,), 2.0 ** -17, device="cuda"))
        wa.check_status()
        want = 127.0
        assert ((y.float() - want).abs() <= 2 * U * want).all()


@pytest.mark.parametrize("M,N,K", LAYERS)
def test_gradients(M, N, K):
    import torch
    import video_dit_full_b200 as wa
    x, dy = bf16((M, K), M, outliers=True), bf16((M, N), M + 1)
    wc, ws, wcd, wsd = weight(N, K, N)
    c, s = il.quant_rows(x.float().numpy())
    dw = wa.int8_grad_weight(dy.cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda())
    dx = wa.int8_grad_input(dy.cuda(), wcd, wsd)
    wa.check_status()
    g = f64(dy)
    want, mag = il.grad_weight(g, c, s)
    within(dw, want, (U + M * 2.0 ** -24) * mag + U * np.abs(want))
    want, mag = il.grad_input(g, wc, ws)
    within(dx, want, (U + N * 2.0 ** -24) * mag + U * np.abs(want))


def test_gradient_of_many_tokens():
    """A contraction long enough to be split, deterministic all the same."""
    import torch
    import video_dit_full_b200 as wa
    M, N, K = 20011, 136, 272
    x, dy = bf16((M, K), 1), bf16((M, N), 2)
    codes, scales = wa.int8_quantize_rows(x.cuda())
    dw = wa.int8_grad_weight(dy.cuda(), codes, scales)
    again = wa.int8_grad_weight(dy.cuda(), codes, scales)
    wa.check_status()
    assert torch.equal(dw, again)
    want, mag = il.grad_weight(f64(dy), codes.cpu().numpy(), scales.cpu().numpy())
    within(dw, want, (U + M * 2.0 ** -24) * mag + U * np.abs(want))


def test_no_rows():
    import torch
    import video_dit_full_b200 as wa
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    _, _, wc, ws = weight(24, 64, 2)
    y, codes, scales = wa.int8_linear(x, wc, ws, return_checkpoint=True)
    dy = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    assert y.shape == (0, 24) and wa.int8_grad_input(dy, wc, ws).shape == (0, 64)
    dw = torch.full((24, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wa.int8_grad_weight(dy, codes, scales, dw=dw)
    assert (dw == 0).all() and wa.int8_dequantize_rows(codes, scales).shape == (0, 64)


@pytest.mark.parametrize("M,N,K", [(3, 264, 1040), (130, 264, 144)])
def test_guards_around_outputs(M, N, K):
    """Nothing is written past the ends of y, codes, scales, dw, dx."""
    import torch
    import video_dit_full_b200 as wa

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        whole = torch.full((n + 4096,), 7, dtype=dtype, device="cuda")
        return whole, whole[2048:2048 + n].view(*shape)
    x, dy = bf16((M, K), 1).cuda(), bf16((M, N), 2).cuda()
    _, _, wc, ws = weight(N, K, 3)
    buffers = [guarded((M, K), torch.int8), guarded((M,), torch.float32), guarded((M, N), torch.bfloat16),
               guarded((N, K), torch.bfloat16), guarded((M, K), torch.bfloat16), guarded((M, K), torch.bfloat16)]
    (_, codes), (_, scales), (_, y), (_, dw), (_, dx), (_, back) = buffers
    wa.int8_quantize_rows(x, codes, scales)
    wa.int8_gemm(codes, scales, wc, ws, y=y)
    wa.int8_grad_weight(dy, codes, scales, dw=dw)
    wa.int8_grad_input(dy, wc, ws, dx=dx)
    wa.int8_dequantize_rows(codes, scales, x=back)
    wa.check_status()
    for whole, part in buffers:
        n = part.numel()
        assert (whole[:2048] == 7).all() and (whole[2048 + n:] == 7).all()


def test_weight_quantised_just_before_the_layer():
    """The layer must wait for whatever the stream did to its weight."""
    import torch
    import video_dit_full_b200 as wa
    N, K = 5120, 5120
    w, x = (bf16((N, K), 1) / 64).cuda(), bf16((4, K), 2).cuda()
    wc = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    ws = torch.zeros(N, device="cuda")
    wa.int8_quantize_rows(w, wc, ws)
    torch.cuda.synchronize()
    want = wa.int8_linear(x, wc, ws)
    for _ in range(20):
        wc.zero_()
        ws.zero_()
        wa.int8_quantize_rows(w, wc, ws)
        y = wa.int8_linear(x, wc, ws)
        assert torch.equal(y, want)
    wa.check_status()


@pytest.mark.parametrize("M", [1, 300])
def test_captured_and_replayed(M):
    import torch
    import video_dit_full_b200 as wa
    N, K = 264, 1040
    _, _, wc, ws = weight(N, K, 3)
    x, dy = bf16((M, K), 1).cuda(), bf16((M, N), 2).cuda()

    def step():
        y, codes, scales = wa.int8_linear(x, wc, ws, return_checkpoint=True)
        return y, wa.int8_grad_weight(dy, codes, scales), wa.int8_grad_input(dy, wc, ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    x.copy_(bf16((M, K), 5))
    dy.copy_(bf16((M, N), 6))
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)
    wa.check_status()


def test_stream_argument():
    import torch
    import video_dit_full_b200 as wa
    _, _, wc, ws = weight(264, 1040, 3)
    for M in (3, 300):
        x, dy = bf16((M, 1040), 1).cuda(), bf16((M, 264), 2).cuda()
        want = wa.int8_linear(x, wc, ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y, codes, scales = wa.int8_linear(x, wc, ws, return_checkpoint=True, stream=s)
        again = [wa.int8_linear(x, wc, ws, stream=s) for _ in range(5)]        # scratch reused in stream order
        dw = wa.int8_grad_weight(dy, codes, scales, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want) and all(torch.equal(a, want) for a in again)
        assert torch.equal(dw, wa.int8_grad_weight(dy, codes, scales))
    wa.check_status()


def test_refused_tensors():
    import torch
    import video_dit_full_b200 as wa
    x, dy = bf16((10, 64), 1).cuda(), bf16((10, 24), 2).cuda()
    _, _, wc, ws = weight(24, 64, 3)
    codes, scales = wa.int8_quantize_rows(x)
    bad = [(lambda: wa.int8_linear(x.float(), wc, ws), TypeError), (lambda: wa.int8_linear(x[:, :48], wc, ws), ValueError),
           (lambda: wa.int8_linear(x, wc, ws[:-1]), (TypeError, ValueError)), (lambda: wa.int8_linear(x.t(), wc, ws), ValueError),
           (lambda: wa.int8_linear(x, wc.float(), ws), TypeError), (lambda: wa.int8_linear(x, wc, ws, bias=ws), TypeError),
           (lambda: wa.int8_linear(x, wc[:20].contiguous(), ws[:20].contiguous()), wa.WanAttnError),       # N % 8
           (lambda: wa.int8_quantize_rows(x[:, :40].contiguous()), wa.WanAttnError),                       # K % 16
           (lambda: wa.int8_quantize_rows(x[0]), ValueError), (lambda: wa.int8_dequantize_rows(codes, scales[:-1]), (TypeError, ValueError)),
           (lambda: wa.int8_grad_weight(dy[:-1], codes, scales), ValueError), (lambda: wa.int8_grad_input(dy, codes, scales), ValueError),
           (lambda: wa.int8_grad_weight(dy, codes, scales, dw=dy), (TypeError, ValueError)),
           (lambda: wa.int8_gemm(codes, scales, wc, ws, y=x), ValueError)]
    for call, error in bad:
        with pytest.raises(error):
            call()


def test_rows_without_a_finite_scale_show_in_the_gradients():
    import torch
    import video_dit_full_b200 as wa
    x, dy = bf16((40, 64), 1), bf16((40, 24), 2).cuda()
    x[7, 3] = float("inf")
    codes, scales = wa.int8_quantize_rows(x.cuda())
    assert torch.isnan(wa.int8_grad_weight(dy, codes, scales)).all()
    wa.check_status()


@pytest.mark.parametrize("M,N,K,one_kernel", [(1, 5120, 5120, True), (16, 136, 2048, True), (5, 24, 8208, True), (5, 24, 20480, False),
                                             (17, 136, 272, False)])
def test_layer_without_a_checkpoint(M, N, K, one_kernel):
    """Null codes and scales are taken where the layer is one kernel, and refused where they are its scratch."""
    import torch
    from video_dit_full_b200 import wan_attn
    x = bf16((M, K), 3, outliers=True).cuda()
    _, _, wc, ws = weight(N, K, 4)
    want, codes, scales = wan_attn.int8_linear(x, wc, ws, return_checkpoint=True)
    assert torch.equal(wan_attn.int8_linear(x, wc, ws), want)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = wan_attn.lib().wan_int8_linear(x.data_ptr(), wc.data_ptr(), ws.data_ptr(), None, y.data_ptr(), None, None, M, N,
                                            K, K, torch.cuda.current_stream().cuda_stream)
    if one_kernel:
        assert status == 0 and torch.equal(y, want)
    else:
        assert status == wan_attn.WORKSPACE and (y == 7).all()
    only = torch.empty(M, device="cuda")
    if one_kernel:
        wan_attn.lib().wan_int8_linear(x.data_ptr(), wc.data_ptr(), ws.data_ptr(), None, y.data_ptr(), None, only.data_ptr(), M, N,
                                       K, K, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(only, scales)
    wan_attn.check_status()
