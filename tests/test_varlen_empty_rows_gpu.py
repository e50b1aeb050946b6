"""Packed attention, causal with more queries than keys: the first queries see no key, and whatever they hold (a
gradient taken at o = 0 is often NaN) leaves no trace in anything else; their own dQ is zero.  Bars: as in
test_varlen_gpu.py."""
import pytest

from test_varlen_gpu import compare, dev, make

pytestmark = pytest.mark.gpu

# lens_q, lens_k, H, Hkv; the empty rows end inside a tile, at its edge, in the sequence's first and last tile
CASES = {
    "inside": ([200, 5, 260], [70, 0, 131], 4, 4),
    "edge": ([256, 300], [128, 44], 2, 2),
    "grouped": ([90, 7, 333], [40, 3, 200], 8, 2),
    "group_of_3": ([150, 64], [1, 63], 6, 2),
    "group_of_16": ([40, 9], [13, 8], 16, 1),
    "few_key_tiles": ([3000], [100], 4, 1),
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_without_keys_leave_no_trace(case, bad):
    import torch
    import video_dit_full_b200 as wa
    lens_q, lens_k, H, Hkv = CASES[case]
    x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=21)
    empty = [i for n, (a, b) in enumerate(zip(lens_q, lens_k)) for i in range(cu_q[n], cu_q[n] + a - min(a, b))]
    clean = {n: t.clone() for n, t in x.items()}
    for name in ("q", "do"):
        clean[name][empty] = 0
        x[name][empty] = bad
    d, cq, ck = dev(x, cu_q, cu_k)
    o, lse = wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal=True)
    assert (o[empty] == 0).all() and (lse[:, empty] == -float("inf")).all()
    grads = wa.varlen_bwd(d["q"], d["k"], d["v"], o, d["do"], lse, cq, ck, causal=True)
    wa.check_status()
    assert (grads[0][empty] == 0).all() and all(torch.isfinite(g).all() for g in grads)
    compare(clean, cu_q, cu_k, True, o, lse, grads)


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 70, 200, 1]])
def test_cache_with_room_to_grow(new):
    """Slack rows behind each sequence's keys are sequences without queries; NaN in them leaves no trace."""
    import torch
    import video_dit_full_b200 as wa
    cached, room = [300, 70, 4096, 129], [100, 58, 513, 0]
    lens_q, lens_k = [], []
    for a, b, c in zip(new, cached, room):
        lens_q += [a, 0]
        lens_k += [b, c]
    x, cu_q, cu_k = make(lens_q, lens_k, 8, 2, seed=22)
    d, cq, ck = dev(x, cu_q, cu_k)
    slack = torch.cat([torch.arange(cu_k[n], cu_k[n + 1]) for n in range(1, len(lens_k), 2)])
    for name in ("k", "v"):
        d[name][slack.cuda()] = float("nan")
    o, lse = wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal=True)
    grads = wa.varlen_bwd(d["q"], d["k"], d["v"], o, d["do"], lse, cq, ck, causal=True)
    wa.check_status()
    compare(x, cu_q, cu_k, True, o, lse, grads)
    assert (grads[1][slack.cuda()] == 0).all() and (grads[2][slack.cuda()] == 0).all()


@pytest.mark.parametrize("lens_q,H", [([12000], 1), ([3000, 4097], 2), ([700, 0, 1], 40)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_queries_and_no_key_at_all(lens_q, H, causal):
    import video_dit_full_b200 as wa
    x, cu_q, cu_k = make(lens_q, [0] * len(lens_q), H, 1, seed=23)
    d, cq, ck = dev(x, cu_q, cu_k)
    o, lse = wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal=causal)
    dq, dk, dv = wa.varlen_bwd(d["q"], d["k"], d["v"], o, d["do"], lse, cq, ck, causal=causal)
    wa.check_status()
    assert (o == 0).all() and (lse == -float("inf")).all() and (dq == 0).all() and dk.shape == dv.shape == (0, 1, 128)
