"""Rows past 2^31 elements: packed queries, 8-bit rows, results of the int8 product and its backward.  The far
rows give what the same rows give by themselves."""
import pytest

from test_varlen_gpu import compare, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
def test_far_queries(causal):
    import torch
    import video_dit_full_b200 as wa
    x, cu_q, cu_k = make([1, 40, 300], [300, 129, 300], 40, 8, seed=2)
    d, cq, ck = dev(x, cu_q, cu_k)
    T = 430_000                                                   # x 40 x 128 > 2^31
    far = T - cu_q[-1]
    q, do = (torch.empty(T, 40, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[far:], do[far:] = d["q"], d["do"]
    cq = cq + far
    o, lse = wa.varlen_fwd(q, d["k"], d["v"], cq, ck, causal=causal)
    dq, dk, dv = wa.varlen_bwd(q, d["k"], d["v"], o, do, lse, cq, ck, causal)
    wa.check_status()
    compare(x, cu_q, cu_k, causal, o[far:], lse[:, far:], (dq[far:], dk, dv))


def test_far_rows_of_8_bits():
    import torch
    import video_dit_full_b200 as wa
    M, K, N, n = 430_000, 5120, 264, 1000                         # M x K > 2^31
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, dtype=torch.bfloat16, device="cuda", generator=gen)
    wc, ws = wa.int8_quantize_rows((torch.randn(N, K, device="cuda", generator=gen) / 64).to(torch.bfloat16))
    y, codes, scales = wa.int8_linear(x, wc, ws, return_checkpoint=True)
    y1, codes1, scales1 = wa.int8_linear(x[-n:], wc, ws, return_checkpoint=True)
    assert torch.equal(y[-n:], y1) and torch.equal(codes[-n:], codes1) and torch.equal(scales[-n:], scales1)
    assert torch.equal(wa.int8_dequantize_rows(codes, scales)[-n:], (codes1.float() * scales1[:, None]).to(torch.bfloat16))
    # dY is zero but for the last rows: dW is theirs, dX zero elsewhere
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dy[-n:] = torch.randn(n, N, device="cuda", generator=gen).to(torch.bfloat16)
    for got, a, b in ((wa.int8_grad_weight(dy, codes, scales), dy[-n:].double().T, codes1.double() * scales1.double()[:, None]),
                      (wa.int8_grad_input(dy, wc, ws)[-n:], dy[-n:].double(), wc.double() * ws.double()[:, None])):
        terms, want = a.shape[1], a @ b
        bound = (2.0 ** -8 + terms * 2.0 ** -24) * (a.abs() @ b.abs()) + 2.0 ** -8 * want.abs()
        assert ((got.double() - want).abs() <= bound).all()
    assert (wa.int8_grad_input(dy, wc, ws)[:-n] == 0).all()
    wa.check_status()


def test_far_results():
    import torch
    import video_dit_full_b200 as wa
    M, K, N, n = 140_000, 128, 16384, 1000                        # M x N > 2^31
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, K, dtype=torch.bfloat16, device="cuda", generator=gen)
    wc, ws = wa.int8_quantize_rows(torch.randn(N, K, device="cuda", generator=gen).to(torch.bfloat16))
    assert torch.equal(wa.int8_linear(x, wc, ws)[-n:], wa.int8_linear(x[-n:], wc, ws))
    wa.check_status()
