"""The int8 layer's kernels of large sizes: the CTA-pair product, the pair kernels of dW and dX with more stages
than their rings hold and several tiles to a pair, and every form of the row quantiser.  Ragged in all sizes;
which kernel a size takes is asserted by the dispatch rules, restated here.

Reference: the definitions in fp64 on the GPU.  Codes: the exact quotient 127 x / absmax is a tie or more than
2^-16 away from one (1/64768 at the least, over all pairs of 8-bit significands and exponents), so fp64's
rounding decides none.  Products of codes are exact in fp64 (below 2^53).
Bars: as in test_int8_gpu.py.
"""
import numpy as np
import pytest

from oracle import int8_linear as il
from test_int8_gpu import U, bf16

pytestmark = pytest.mark.gpu


def up(a, b):
    return (a + b - 1) // b


def takes_pair_product(M, N):
    return M > 128 and 2 * up(M, 256) * up(N, 256) >= 74


def takes_pair_gradient(rows, cols):
    return up(up(rows, 256) * up(cols, 256), 74) < up(up(rows, 128) * up(cols, 128), 148)


def quantised(x):
    """(codes, scales) of bf16 rows on the GPU, fp64."""
    import torch
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, x * 127 / top, x).round()
    # the fp32 scale from an fp64 quotient: a / 127 repeats every 7 bits and lies near no tie of fp32
    return codes, torch.where(top > 0, top / 127, torch.ones_like(top))[:, 0].float()


def within(got, want, bound):
    import torch
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= bound + 1e-30).all(), float((err / (bound + 1e-30)).max())
    assert err.norm() <= 5e-3 * want.norm()


def guarded(*shape):
    """A bf16 tensor inside a buffer of 7s; the check that the 7s are still there."""
    import torch
    n = int(np.prod(shape))
    whole = torch.full((n + 8192,), 7.0, dtype=torch.bfloat16, device="cuda")
    return whole[4096:4096 + n].view(*shape), lambda: (whole[:4096] == 7).all() and (whole[4096 + n:] == 7).all()


@pytest.mark.parametrize("M", [149, 333])
@pytest.mark.parametrize("K", [16, 1024, 1040, 2048, 2064, 4096, 4112, 5120, 8192, 8208, 16384, 16400, 20480])
def test_rows(M, K):
    import torch
    import video_dit_full_b200 as wa
    x = bf16((M, K), M + K, outliers=True)
    x[3] = 0
    x[4, : K // 2] = x[4].abs().max() / 2                              # ties at 63.5
    x[5, 7] = float("inf")
    x = x.cuda()
    codes, scales = wa.int8_quantize_rows(x)
    back = wa.int8_dequantize_rows(codes, scales)
    wa.check_status()
    good = torch.arange(M, device="cuda") != 5
    want, want_s = quantised(x[good])
    assert torch.equal(codes[good].double(), want) and torch.equal(scales[good], want_s)
    assert scales[5].isnan() and not codes[5].any()
    assert torch.equal(back[good], (codes[good].float() * want_s[:, None]).to(torch.bfloat16))
    c, s = il.quant_rows(x[:5].float().cpu().numpy())                   # and by integer arithmetic
    np.testing.assert_array_equal(codes[:5].cpu().numpy(), c)
    np.testing.assert_array_equal(scales[:5].cpu().numpy(), s)


# one tile a pair; rings that wrap; two accumulators in turn; one stage; the last tiles ragged in every way
LAYERS = [(1500, 2056, 2064), (5000, 5128, 1040), (3001, 4104, 48), (300, 9736, 5120), (1024, 5120, 5120), (9001, 264, 400),
          (2560, 4864, 128)]


@pytest.mark.parametrize("M,N,K", LAYERS)
@pytest.mark.parametrize("with_bias", [False, True])
def test_pair_product(M, N, K, with_bias):
    import torch
    import video_dit_full_b200 as wa
    assert takes_pair_product(M, N)
    x, w = bf16((M, K), M, outliers=True).cuda(), (bf16((N, K), N) / K ** 0.5).cuda()
    bias = bf16((N,), 9).cuda() if with_bias else None
    wc, ws = wa.int8_quantize_rows(w)
    y, codes, scales = wa.int8_linear(x, wc, ws, bias=bias, return_checkpoint=True)
    out, whole = guarded(M, N)
    wa.int8_gemm(codes, scales, wc, ws, bias=bias, y=out)
    wa.check_status()
    assert torch.equal(y, out) and whole()
    c, s = quantised(x)
    assert torch.equal(codes.double(), c) and torch.equal(scales, s)
    want = (c @ wc.double().T) * s.double()[:, None] * ws.double()
    b = 0.0 if bias is None else bias.double()
    bound = 2.0 ** -21 * (want.abs() + (0.0 if bias is None else b.abs()))
    want = want + b
    within(y, want, U * want.abs() + bound)


# rows, cols, terms of the result: dW has N, K, M of them and dX has M, K, N
GRADIENTS = [(2000, 2064, 1504), (2000, 2064, 40), (2056, 2048, 1104), (5000, 5136, 704), (5120, 5120, 1024), (9600, 784, 512),
             (3848, 4112, 64), (3848, 4112, 520)]


@pytest.mark.parametrize("rows,cols,terms", GRADIENTS)
@pytest.mark.parametrize("which", ["weight", "input"])
def test_pair_gradients(rows, cols, terms, which):
    import torch
    import video_dit_full_b200 as wa
    assert takes_pair_gradient(rows, cols)
    codes, scales = wa.int8_quantize_rows(bf16((terms, cols), rows, outliers=True).cuda())
    out, whole = guarded(rows, cols)
    if which == "weight":
        dy = bf16((terms, rows), 5).cuda()
        call, left = (lambda **kw: wa.int8_grad_weight(dy, codes, scales, **kw)), dy.double().T
    else:
        dy = bf16((rows, terms), 5).cuda()
        call, left = (lambda **kw: wa.int8_grad_input(dy, codes, scales, **kw)), dy.double()
    call(dw=out) if which == "weight" else call(dx=out)
    assert whole() and torch.equal(call(), out)                          # a fixed order
    wa.check_status()
    right = codes.double() * scales.double()[:, None]
    want = left @ right
    within(out, want, (U + terms * 2.0 ** -24) * (left.abs() @ right.abs()) + U * want.abs())


def test_both_products_agree():
    """Sizes on both sides of the product's rule give the same results: the int32 sums are exact."""
    import torch
    import video_dit_full_b200 as wa
    M, N, K = 1001, 2304, 528
    assert takes_pair_product(2 * M, N) and not takes_pair_product(M, N)
    x = bf16((2 * M, K), 1).cuda()
    wc, ws = wa.int8_quantize_rows(bf16((N, K), 2).cuda())
    y = wa.int8_linear(x, wc, ws)
    assert torch.equal(y[:M], wa.int8_linear(x[:M], wc, ws)) and torch.equal(y[M:], wa.int8_linear(x[M:], wc, ws))
    wa.check_status()
