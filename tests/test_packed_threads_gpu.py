"""Packed and int8 calls from several threads at once, each on a stream of its own: every round's results, and
every exception."""
import pytest

pytestmark = pytest.mark.gpu

THREADS, ROUNDS = 4, 60


def calls():
    import torch
    import video_dit_full_b200 as wa
    gen = torch.Generator(device="cuda").manual_seed(31)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)       # noqa: E731
    cu = torch.tensor([0, 3, 200], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, 700, 1500], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    q, kv, cache, last = new(200, 4, 128), new(200, 2, 128), new(1500, 2, 128), new(2, 4, 128)
    wc, ws = wa.int8_quantize_rows(new(256, 512))

    def call():
        o, lse = wa.varlen_fwd(q, kv, kv, cu, cu, causal=True)
        y, codes, scales = wa.int8_linear(o.view(200, 512), wc, ws, return_checkpoint=True)
        _, dk, dv = wa.varlen_bwd(q, kv, kv, o, q, lse, cu, cu, causal=True)      # dQ is summed in no fixed order
        return (o, lse, y, codes, scales, dk, dv, wa.int8_grad_weight(y, codes, scales), wa.int8_grad_input(y, wc, ws),
                wa.int8_linear(o.view(200, 512)[:9], wc, ws), wa.int8_dequantize_rows(codes, scales),
                *wa.varlen_fwd(last, cache, cache, one, ck, causal=True))         # keys split: a join kernel

    return call


def test_every_round_of_every_thread():
    import threading

    import torch
    import video_dit_full_b200 as wa
    call = calls()
    want = call()
    torch.cuda.synchronize()
    finished, raised, wrong = [], [], []
    start = threading.Barrier(THREADS)

    def work(me):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                differ = torch.zeros(len(want), dtype=torch.int64, device="cuda")
                start.wait(60)
                for _ in range(ROUNDS):
                    differ += torch.stack([(a != b).sum() for a, b in zip(call(), want)])
                wrong.extend((me, i, int(n)) for i, n in enumerate(differ.tolist()) if n)
            finished.append(me)
        except BaseException as e:          # noqa: BLE001  (a thread's exception would go unseen)
            raised.append((me, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not raised and sorted(finished) == list(range(THREADS)) and not wrong
    wa.check_status()


def test_a_refused_call_raises_in_its_thread():
    import threading

    import torch
    import video_dit_full_b200 as wa
    x = torch.zeros(4, 40, dtype=torch.bfloat16, device="cuda")       # K is no multiple of 16
    seen = []

    def work():
        try:
            wa.int8_quantize_rows(x)
        except wa.WanAttnError as e:
            seen.append(e.status)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert seen == [1]
