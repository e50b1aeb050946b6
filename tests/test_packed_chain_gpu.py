"""Packed and int8 calls one behind the other, each reading what the last one wrote into buffers that every
round uses again: a kernel that starts under the one before it must neither read nor write too early.
The same calls with a synchronisation after each give the results to the bit."""
import pytest

pytestmark = pytest.mark.gpu


def rounds(wait, lens, width, heads):
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    T = sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    x, w = new(T, width), [new(3 * width, width) * width ** -0.5 for _ in range(3)]
    w_out = [new(width, width) * width ** -0.5 for _ in range(3)]
    codes, scales = torch.empty(3 * width, width, dtype=torch.int8, device="cuda"), torch.empty(3 * width, device="cuda")
    o, lse = torch.zeros(T, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(heads, T, device="cuda")
    back = torch.empty_like(x)
    out = []

    def step(result):
        if wait:
            torch.cuda.synchronize()
        return result

    torch.cuda.synchronize()
    for i in range(12):
        step(wa.int8_quantize_rows(w[i % 3], codes, scales))                    # the weight of the very next call
        y = step(wa.int8_linear(x, codes, scales)).view(T, 3 * heads, 128)
        step(wa.varlen_fwd(y[:, :heads], y[:, heads:2 * heads], y[:, 2 * heads:], cu, cu, True, o, lse))
        a = step(wa.int8_quantize_rows(o.view(T, width)))
        step(wa.int8_dequantize_rows(*a, back))
        wc, ws = step(wa.int8_quantize_rows(w_out[i % 3], codes[:width], scales[:width]))
        x = step(wa.int8_gemm(*a, wc, ws))
        dw = step(wa.int8_grad_weight(back, *a))
        dx = step(wa.int8_grad_input(back, wc, ws))
        out += [lse.clone(), o.clone(), x, back.clone(), dw, dx]
    torch.cuda.synchronize()
    wa.check_status()
    return out


@pytest.mark.parametrize("lens", [[1], [3, 8], [1, 7, 33, 64, 130, 2], [700, 1, 300]])
def test_calls_behind_one_another(lens):
    import torch
    want = rounds(True, lens, 768, 6)
    for _ in range(3):
        for a, b in zip(rounds(False, lens, 768, 6), want):
            assert torch.equal(a, b)


def test_backward_behind_its_forward():
    """dQ is summed in no fixed order: against the waited-for run within two bf16 half steps and the sum's 2^-12."""
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(6)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    lens = [5, 200, 64, 1]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    q, do = new(sum(lens), 4, 128), new(sum(lens), 4, 128)
    k, v = new(sum(lens), 2, 128), new(sum(lens), 2, 128)
    need = wa.varlen_bwd_workspace_size(len(lens), sum(lens), sum(lens), 4, 2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(scale, wait):
        o, lse = wa.varlen_fwd(q * scale, k, v, cu, cu, causal=True)
        if wait:
            torch.cuda.synchronize()
        grads = wa.varlen_bwd(q * scale, k, v, o, do, lse, cu, cu, causal=True, workspace=ws)
        if wait:
            torch.cuda.synchronize()
        return grads

    scales = [1.0, 0.25, 0.5, 1.0, 0.125] * 4
    want = [step(s, True) for s in scales]
    got = [step(s, False) for s in scales]
    wa.check_status()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            bar = b.abs().float() * 2 ** -7 + b.float().abs().max() * 2 ** -12
            assert ((a.float() - b.float()).abs() <= bar).all()


def small():
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(9)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    cu = torch.tensor([0, 3, 200]).to(torch.int32).cuda()
    q, kv = new(200, 4, 128), new(200, 2, 128)
    wc, ws = wa.int8_quantize_rows(new(256, 512))

    def call():
        o, lse = wa.varlen_fwd(q, kv, kv, cu, cu, causal=True)
        y, codes, scales = wa.int8_linear(o.view(200, 512), wc, ws, return_checkpoint=True)
        return o, lse, y, codes, scales, wa.int8_grad_weight(y, codes, scales), wa.int8_linear(o.view(200, 512)[:9], wc, ws)

    want = call()
    torch.cuda.synchronize()
    return call, want


def test_threads():
    """Calls from several threads, each on a stream of its own, at once."""
    import threading

    import torch
    call, want = small()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(100):
                got = call()
            torch.cuda.current_stream().synchronize()
            bad.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_modes_and_memory():
    """Inference mode and parameters as arguments; what a call allocates is given back."""
    import torch
    import video_dit_full_b200 as wa
    call, want = small()
    with torch.inference_mode():
        got = call()
    assert got[0].is_inference() and all(torch.equal(a, b) for a, b in zip(got, want))
    w = torch.nn.Parameter(torch.randn(64, 64, device="cuda").to(torch.bfloat16))
    codes, scales = wa.int8_quantize_rows(w)
    assert not codes.requires_grad and torch.equal(codes, wa.int8_quantize_rows(w.detach())[0])
    del got
    before = torch.cuda.memory_allocated()
    for _ in range(50):
        call()
        for wrong in (lambda: wa.int8_linear(w, codes, scales[:-1]), lambda: wa.int8_quantize_rows(w[:, :40].contiguous())):
            with pytest.raises((ValueError, wa.WanAttnError)):
                wrong()
    assert torch.cuda.memory_allocated() == before
