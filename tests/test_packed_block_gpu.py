"""The operators together, as a packed block uses them: fused int8 q-k-v projection, causal packed
attention on its slices, int8 output projection; backward from the 8-bit checkpoints of both layers'
inputs, with q, k, v themselves read back from 8 bits.

Reference: the same block in fp64 on the values that the codes stand for, differentiated by torch's
autograd straight through the quantisers.  Every stage rounds its inputs and its result to bf16 (half
step 2^-8 each, relative in norm): the forward has 4 such steps and the backward 8 more, so
12 * 2^-8 bounds the relative error of the norm.
"""
import pytest

pytestmark = pytest.mark.gpu


def test_block_step_with_8_bit_checkpoints():
    import torch
    import video_dit_full_b200 as wa
    H, Hkv, E, lens = 4, 2, 512, [130, 1, 257, 64]
    T, F = sum(lens), (H + 2 * Hkv) * 128
    gen = torch.Generator(device="cuda").manual_seed(0)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen)                     # noqa: E731
    x, dy = new(T, E).bfloat16(), new(T, E).bfloat16()
    w1 = wa.int8_quantize_rows((new(F, E) / E ** 0.5).bfloat16())
    w2 = wa.int8_quantize_rows((new(E, H * 128) / (H * 128) ** 0.5).bfloat16())
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    heads = lambda t: t.view(T, H + 2 * Hkv, 128).split([H, Hkv, Hkv], 1)              # noqa: E731

    # forward: what is kept is 8-bit (x's codes, qkv's codes, o's codes) but for o and lse
    qkv, cx, sx = wa.int8_linear(x, *w1, return_checkpoint=True)
    kept = wa.int8_quantize_rows(qkv.view(-1, 128))                # a scale per token and head
    back = wa.int8_dequantize_rows(*kept).view(T, F)
    q, k, v = heads(back)
    o, lse = wa.varlen_fwd(q, k, v, cu, cu, causal=True)
    y, co, so = wa.int8_linear(o.view(T, H * 128), *w2, return_checkpoint=True)
    # backward
    dw2 = wa.int8_grad_weight(dy, co, so)
    do = wa.int8_grad_input(dy, *w2)
    q, k, v = heads(wa.int8_dequantize_rows(*kept).view(T, F))
    dqkv = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    wa.varlen_bwd(q, k, v, o, do.view(T, H, 128), lse, cu, cu, True, *heads(dqkv))
    dw1 = wa.int8_grad_weight(dqkv, cx, sx)
    dx = wa.int8_grad_input(dqkv, *w1)
    wa.check_status()

    values = lambda c, s: c.double() * s.double()[:, None]                             # noqa: E731
    X, W1, W2 = (values(*t).requires_grad_() for t in ((cx, sx), w1, w2))
    QKV = X @ W1.T
    # straight through: the values kept in 8 bits, the gradient of the product
    QKV = QKV + (values(*kept).view(T, F) - QKV).detach()
    Q, K, V = heads(QKV)
    outs, a = [], 0
    for n in lens:
        s = torch.einsum("ihd,jhd->hij", Q[a:a + n], K[a:a + n].repeat_interleave(H // Hkv, 1)) / 128 ** 0.5
        s = s.masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), float("-inf"))
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), V[a:a + n].repeat_interleave(H // Hkv, 1)))
        a += n
    O = torch.cat(outs).reshape(T, H * 128)                                            # noqa: E741
    Oq = O + (values(co, so) - O).detach()
    Y = Oq @ W2.T
    Y.backward(dy.double())
    for name, got, want in (("o", o.view(T, -1), O), ("y", y, Y), ("dw2", dw2, W2.grad), ("dw1", dw1, W1.grad),
                            ("dx", dx, X.grad)):
        rel = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert rel <= 12 * 2.0 ** -8, (name, rel)
