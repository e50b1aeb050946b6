"""Packed attention (varlen_fwd, varlen_bwd) against the fp64 oracle (oracle/packed.py).

Bars.  Element by element the bound that ``attn_packed`` derives from bf16's half step (2^-8:
P, dS, o and the results are rounded) and fp32's.  Its fp32 part eta = 2^-11 covers an
exponential's relative error: a score of |q_d k_d| terms summing to m / scale is off by at most
(128 + 2) 2^-24 m, twice that between two scores, and 2^-22 from exp2; the inputs here keep
m <= 60, so 2 * 130 * 2^-24 * 60 + 2^-22 < 2^-10 / 1.04 in the worst case and far less in the
sum.  As a statistical check the relative Frobenius error stays below the framework's 5e-3
(forward) and 2e-2 (backward).  lse: 130 * 2^-24 * m plus 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

from oracle.packed import attn_packed

pytestmark = pytest.mark.gpu

# lens_q, lens_k, H, Hkv, causal
CASES = {
    "one": ([1], [1], 1, 1, True),
    "ragged_causal": ([1, 7, 0, 33, 64, 130, 2], [1, 7, 0, 33, 64, 130, 2], 3, 3, True),
    "edges_full": ([127, 128, 129, 255, 256, 257], [127, 128, 129, 255, 256, 257], 2, 2, False),
    "edges_causal": ([127, 128, 129, 255, 256, 257], [127, 128, 129, 255, 256, 257], 4, 2, True),
    "grouped": ([300, 1, 515], [300, 1, 515], 8, 2, True),
    "group_of_5": ([70, 33], [70, 33], 10, 2, True),
    "group_of_3": ([90, 141], [140, 141], 6, 2, True),
    "group_of_16": ([21, 40], [21, 300], 16, 1, True),
    "group_of_12_full": ([21, 40], [210, 3], 12, 1, False),
    "more_queries_than_keys": ([200, 5, 260], [70, 0, 131], 4, 4, True),
    "other_keys_full": ([200, 5, 0], [70, 0, 131], 4, 2, False),
    "continued": ([100, 300, 1], [500, 300, 257], 4, 1, True),
    "single_tokens": ([1] * 6, [1, 2, 127, 128, 300, 1000], 8, 2, True),
    "single_token_long": ([1], [20011], 8, 1, True),
    "few_tokens_long": ([3, 17], [9000, 4097], 4, 4, True),
    "long": ([2049, 517], [2049, 517], 4, 2, True),
    "no_queries": ([0, 0], [40, 200], 2, 1, True),
    "no_keys": ([40, 3], [0, 0], 2, 1, False),
}


def make(lens_q, lens_k, H, Hkv, seed, before=0, after=0, q_mul=1.0):
    """bf16 CPU tensors with `before` and `after` rows outside every sequence, and the offsets."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    cu_q, cu_k = ([before + int(a) for a in np.cumsum([0] + lens)] for lens in (lens_q, lens_k))
    new = lambda cu, h: torch.randn(cu[-1] + after, h, 128, generator=gen)       # noqa: E731
    x = {"q": (new(cu_q, H) * q_mul), "k": new(cu_k, Hkv), "v": new(cu_k, Hkv), "do": new(cu_q, H)}
    return {n: t.to(torch.bfloat16) for n, t in x.items()}, cu_q, cu_k


def dev(x, cu_q, cu_k):
    import torch
    return ({n: t.cuda() for n, t in x.items()}, torch.tensor(cu_q, dtype=torch.int32).cuda(),
            torch.tensor(cu_k, dtype=torch.int32).cuda())


def within(name, got, want, bound, frob):
    got = got.float().cpu().numpy().astype(np.float64)
    real = ~np.isnan(want)
    err = np.abs(got - want)[real]
    assert np.isfinite(got[real]).all(), name
    assert (err <= bound[real] * (1 + 1e-6) + 1e-30).all(), (name, float((err / (bound[real] + 1e-30)).max()))
    # 2^-6 bound: where dP and D cancel (one key: dS = 0 exactly) their fp32 rounding is left, up to
    # (128 + 2) 2^-24 (sum |do v| + |D|) P < 2^-6 eta (...) P, and eta (...) P is one of the bound's terms
    allowed = frob * np.linalg.norm(want[real]) + 2.0 ** -6 * np.linalg.norm(bound[real])
    assert np.linalg.norm(err) <= allowed + 1e-30, (name, np.linalg.norm(err), allowed)


def within_lse(got, want, x):
    got = got.cpu().numpy().astype(np.float64)
    real = ~np.isnan(want)
    empty = real & np.isinf(want)
    assert (got[empty] == -np.inf).all()
    some = real & ~empty
    m = float(np.abs(x["q"].float().numpy()).max() * np.abs(x["k"].float().numpy()).max()) * 128 ** 0.5 if some.any() else 0
    assert (np.abs(got - np.where(some, want, 0))[some] <= 130 * 2.0 ** -24 * m + 2.0 ** -20 * (1 + np.abs(want[some]))).all()


def compare(x, cu_q, cu_k, causal, o, lse, grads=None):
    f = {n: t.float().numpy().astype(np.float64) for n, t in x.items()}
    want, bound = attn_packed(f["q"], f["k"], f["v"], cu_q, cu_k, causal, f["do"] if grads else None)
    within("o", o, want["o"], bound["o"], 5e-3)
    within_lse(lse, want["lse"], x)
    for name, g in zip(("dq", "dk", "dv"), grads or ()):
        within(name, g, want[name], bound[name], 2e-2)
    return want


def run(d, cu_q, cu_k, causal, **kw):
    import video_dit_full_b200 as wa
    o, lse = wa.varlen_fwd(d["q"], d["k"], d["v"], cu_q, cu_k, causal=causal, **kw)
    grads = wa.varlen_bwd(d["q"], d["k"], d["v"], o, d["do"], lse, cu_q, cu_k, causal=causal, **kw)
    return o, lse, grads


@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(case):
    import video_dit_full_b200 as wa
    lens_q, lens_k, H, Hkv, causal = CASES[case]
    x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=len(case))
    o, lse, grads = run(*dev(x, cu_q, cu_k), causal)
    wa.check_status()
    compare(x, cu_q, cu_k, causal, o, lse, grads)


@pytest.mark.parametrize("causal", [True, False])
def test_peaked_scores(causal):
    import video_dit_full_b200 as wa
    x, cu_q, cu_k = make([300, 17], [300, 17], 2, 1, seed=5, q_mul=4.0)
    o, lse, grads = run(*dev(x, cu_q, cu_k), causal)
    wa.check_status()
    compare(x, cu_q, cu_k, causal, o, lse, grads)


@pytest.mark.parametrize("case", ["ragged_causal", "edges_full", "group_of_5", "single_tokens", "more_queries_than_keys"])
def test_rows_outside_every_sequence(case):
    """They hold NaN and infinities in the inputs, and their outputs keep what they held."""
    import torch
    import video_dit_full_b200 as wa
    lens_q, lens_k, H, Hkv, causal = CASES[case]
    x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=7, before=3, after=150)
    for name, cu in (("q", cu_q), ("k", cu_k), ("v", cu_k), ("do", cu_q)):
        x[name][:cu[0]] = float("nan")
        x[name][cu[-1]:] = float("inf") if name == "v" else float("nan")
    d, dq_, dk_ = dev(x, cu_q, cu_k)
    Tq, Tk = len(x["q"]), len(x["k"])
    o = torch.full((Tq, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, Tq), 7.0, device="cuda")
    wa.varlen_fwd(d["q"], d["k"], d["v"], dq_, dk_, causal=causal, o=o, lse=lse)
    # the backward's o and lse hold NaN there
    ob, lb = o.clone(), lse.clone()
    ob[:cu_q[0]], ob[cu_q[-1]:] = float("nan"), float("nan")
    lb[:, :cu_q[0]], lb[:, cu_q[-1]:] = float("nan"), float("nan")
    grads = [torch.full_like(d[n], 7.0) for n in ("q", "k", "v")]
    wa.varlen_bwd(d["q"], d["k"], d["v"], ob, d["do"], lb, dq_, dk_, causal, *grads)
    wa.check_status()
    for t, cu in ((o, cu_q), (lse.T, cu_q), (grads[0], cu_q), (grads[1], cu_k), (grads[2], cu_k)):
        assert (t[:cu[0]] == 7).all() and (t[cu[-1]:] == 7).all()
    for name, cu in (("q", cu_q), ("k", cu_k), ("v", cu_k), ("do", cu_q)):
        x[name][:cu[0]] = 0
        x[name][cu[-1]:] = 0
    compare(x, cu_q, cu_k, causal, o, lse, grads)


def test_neighbours_do_not_mix():
    """A sequence's non-finite values stay in its own results."""
    import torch
    import video_dit_full_b200 as wa
    lens = [100, 77, 140]
    x, cu, _ = make(lens, lens, 4, 2, seed=9)
    clean = {n: t.clone() for n, t in x.items()}
    for name in ("q", "k", "v", "do"):
        x[name][cu[1]:cu[2]] = float("nan")
    for causal in (True, False):
        o, lse, grads = run(*dev(x, cu, cu), causal)
        wa.check_status()
        co, clse, cgrads = run(*dev(clean, cu, cu), causal)
        for a, b in ((o, co), (lse.T, clse.T), (grads[1], cgrads[1]), (grads[2], cgrads[2])):
            for i in (0, 2):
                assert torch.equal(a[cu[i]:cu[i + 1]], b[cu[i]:cu[i + 1]])
        for i in (0, 2):      # dq: summed in no fixed order
            a, b = (g[0][cu[i]:cu[i + 1]].float() for g in (grads, cgrads))
            assert torch.isfinite(a).all() and (a - b).norm() <= 2.0 ** -8 * b.norm()


def test_strided_tokens():
    """q, k, v as slices of a fused projection's output, their gradients into slices of one buffer."""
    import torch
    import video_dit_full_b200 as wa
    H, Hkv, lens = 4, 2, [130, 61, 257]
    x, cu, _ = make(lens, lens, H, Hkv, seed=3)
    d, c, _ = dev(x, cu, cu)
    fused = torch.cat([d["q"], d["k"], d["v"]], 1)
    q, k, v = fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]
    o, lse = wa.varlen_fwd(q, k, v, c, c, causal=True)
    out = torch.full_like(fused, 7.0)
    wa.varlen_bwd(q, k, v, o, d["do"], lse, c, c, True, out[:, :H], out[:, H:H + Hkv], out[:, H + Hkv:])
    wa.check_status()
    compare(x, cu, cu, True, o, lse, (out[:, :H], out[:, H:H + Hkv], out[:, H + Hkv:]))


def test_offsets_past_32_bits():
    """Sequences at the far end of a cache of more than 2^32 bytes and 2^31 elements."""
    import torch
    import video_dit_full_b200 as wa
    lens_q, lens_k, Hkv = [1, 40], [300, 129], 8
    x, cu_q, cu_k = make(lens_q, lens_k, 8, Hkv, seed=2)
    Tk = 2_200_000
    far = Tk - cu_k[-1]
    d, cq, ck = dev(x, cu_q, cu_k)
    k, v, dk, dv = (torch.empty(Tk, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    k[far:], v[far:] = d["k"], d["v"]
    ck = ck + far
    o, lse = wa.varlen_fwd(d["q"], k, v, cq, ck, causal=True)
    dq, _, _ = wa.varlen_bwd(d["q"], k, v, o, d["do"], lse, cq, ck, True, None, dk, dv)
    wa.check_status()
    compare(x, cu_q, cu_k, True, o, lse, (dq, dk[far:], dv[far:]))


def test_bad_offsets_stay_in_bounds():
    """Decreasing or out-of-range offsets are clipped: guarded buffers around the outputs stay whole."""
    import torch
    import video_dit_full_b200 as wa
    T, H = 200, 2
    x, _, _ = make([T], [T], H, H, seed=1)
    d = {n: t.cuda() for n, t in x.items()}
    for cu in ([0, 500], [-70, 90], [150, 20], [100, 50, 300], [-5, -1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        guard = {n: torch.full((T + 400, H, 128), 7.0, dtype=torch.bfloat16, device="cuda") for n in ("o", "q", "k", "v")}
        part = {n: t[200:200 + T] for n, t in guard.items()}
        lse = torch.zeros(H, T, device="cuda")
        wa.varlen_fwd(d["q"], d["k"], d["v"], c, c, causal=True, o=part["o"], lse=lse)
        wa.varlen_bwd(d["q"], d["k"], d["v"], part["o"], d["do"], lse, c, c, True, part["q"], part["k"], part["v"])
        wa.check_status()
        for t in guard.values():
            assert (t[:200] == 7).all() and (t[200 + T:] == 7).all()


def test_decreasing_offsets_of_many_sequences():
    """Offsets that name 300,000 overlapping sequences of 8192 key tiles: their sum passes 2^31, the call's bounds hold."""
    import torch
    import video_dit_full_b200 as wa
    T, N = 1 << 20, 600_001
    k = torch.ones(T, 1, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(4, 1, 128, dtype=torch.bfloat16, device="cuda")
    cu_k = (torch.arange(N + 1, device="cuda") % 2 * T).to(torch.int32)
    cu_q = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    need = wa.varlen_bwd_workspace_size(N, 4, T, 1, 1)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    grads = [torch.full((T + 256, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    dq = torch.full_like(q, 7.0)
    wa.varlen_bwd(q, k, k, q, q, torch.zeros(1, 4, device="cuda"), cu_q, cu_k, True, dq, grads[0][:T], grads[1][:T],
                  workspace=ws[:need])
    wa.check_status()
    assert (ws[need:] == 77).all() and (dq == 7).all()
    for g in grads:
        assert (g[:128] == 0).all() and (g[T:] == 7).all()


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv", [([40, 300], [40, 300], 2, 2), ([1, 3], [700, 260], 8, 2),
                                                 ([1], [20011], 8, 1), ([200, 5], [70, 0], 4, 4)])
def test_nan_shows(lens_q, lens_k, H, Hkv):
    """A NaN (or +inf) score shows in the rows that see it and in no other: a NaN query, a NaN key, scores of +inf."""
    import torch
    import video_dit_full_b200 as wa
    x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=8)
    d, cq, ck = dev(x, cu_q, cu_k)
    want, _ = wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal=True)
    q = d["q"].clone()
    row = lens_q[0] - 1                                         # its last row sees every key
    q[row, H - 1] = float("nan")
    o, lse = wa.varlen_fwd(q, d["k"], d["v"], cq, ck, causal=True)
    assert o[row, H - 1].isnan().all() and lse[H - 1, row].isnan()
    o[row, H - 1] = want[row, H - 1]
    assert torch.equal(o, want)
    for bad in (float("nan"), 3e38):                            # 3e38 times a positive query: +inf
        k, q = d["k"].clone(), d["q"].abs()
        plain, _ = wa.varlen_fwd(q, k, d["v"], cq, ck, causal=True)
        k[lens_k[0] - 1] = bad                                  # the last key: only the last row of sequence 0 sees it
        o, lse = wa.varlen_fwd(q, k, d["v"], cq, ck, causal=True)
        assert o[row].isnan().all() and lse[:, row].isnan().all()
        o[row] = plain[row]
        assert torch.equal(o, plain)
    wa.check_status()


SPLIT = {
    "mixed": ([1] * 9, [9000, 20, 0, 300, 4000, 17, 800, 128, 1], 8, 2, True),
    "most_parts": ([1], [40000], 2, 1, True),
    "more_items_than_estimated": ([300, 0, 0], [20000, 5, 0], 1, 1, True),
    "more_items_than_estimated_full": ([300, 0, 0], [20000, 5, 0], 1, 1, False),
    "few_rows_full": ([5, 40, 1], [3000, 9000, 1], 4, 4, False),
    "more_queries_than_keys": ([40, 30], [20, 7000], 4, 2, True),
    "sixty": ([1] * 60, [(37 * i * i) % 1500 for i in range(60)], 6, 2, True),
}


@pytest.mark.parametrize("case", SPLIT)
def test_split_keys(case):
    """Calls whose keys go to several work items: rows before and behind the sequences stay as they were."""
    import torch
    import video_dit_full_b200 as wa
    lens_q, lens_k, H, Hkv, causal = SPLIT[case]
    x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=12, before=3, after=5)
    d, cq, ck = dev(x, cu_q, cu_k)
    T = d["q"].shape[0]
    assert wa.varlen_fwd_workspace_size(len(lens_q), T, d["k"].shape[0], H, Hkv) > 0
    o = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, T), 7.0, device="cuda")
    wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal=causal, o=o, lse=lse)
    wa.check_status()
    for n in range(T):
        if n < 3 or n >= T - 5:
            assert (o[n] == 7).all() and (lse[:, n] == 7).all()
    again = wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal=causal)[0]
    assert torch.equal(again[3:T - 5], o[3:T - 5])
    _, _, grads = run(d, cq, ck, causal)
    compare(x, cu_q, cu_k, causal, o, lse, grads)


def test_many_sequences():
    import video_dit_full_b200 as wa
    rng = np.random.default_rng(0)
    lens = [int(a) for a in rng.integers(0, 5, 700)]
    x, cu_q, cu_k = make(lens, lens, 2, 1, seed=4)
    o, lse, grads = run(*dev(x, cu_q, cu_k), True)
    wa.check_status()
    compare(x, cu_q, cu_k, True, o, lse, grads)


def test_side_stream_and_two_calls_at_once():
    import torch
    import video_dit_full_b200 as wa
    xs = [make([200, 31], [200, 31], 4, 2, seed=s) for s in (1, 2)]
    ds = [dev(*x) for x in xs]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    outs = []
    for d, s in zip(ds, streams):
        with torch.cuda.stream(s):
            outs.append(run(*d, True))
    torch.cuda.synchronize()
    wa.check_status()
    for x, (o, lse, grads) in zip(xs, outs):
        compare(*x, True, o, lse, grads)


@pytest.mark.parametrize("case", ["grouped", "single_token_long"])
def test_captured_and_replayed(case):
    """Two graphs with workspaces of their own, replayed on new inputs."""
    import torch
    import video_dit_full_b200 as wa
    lens_q, lens_k, H, Hkv, causal = CASES[case]
    graphs = []
    for seed in (1, 2):
        x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=seed)
        d, cq, ck = dev(x, cu_q, cu_k)
        run(d, cq, ck, causal)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(d, cq, ck, causal)
        graphs.append((g, d, out, cq, ck))                  # the offsets live as long as the graph
    for seed, (_, d, *_) in zip((3, 4), graphs):
        x, _, _ = make(lens_q, lens_k, H, Hkv, seed=seed)
        for n in d:
            d[n].copy_(x[n])
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    wa.check_status()
    for seed, (_, _, (o, lse, grads), *_) in zip((3, 4), graphs):
        x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=seed)
        compare(x, cu_q, cu_k, causal, o, lse, grads)


def test_stream_argument():
    """A call given a stream runs, and allocates what it needs, there."""
    import torch
    import video_dit_full_b200 as wa
    for case in ("grouped", "single_token_long"):
        lens_q, lens_k, H, Hkv, causal = CASES[case]
        x, cu_q, cu_k = make(lens_q, lens_k, H, Hkv, seed=11)
        d, cq, ck = dev(x, cu_q, cu_k)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        o, lse, grads = run(d, cq, ck, causal, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        wa.check_status()
        compare(x, cu_q, cu_k, causal, o, lse, grads)


def test_the_rest_of_the_batch_does_not_matter():
    """A sequence's forward is the same alone, in a batch, and at another place of it."""
    import torch
    import video_dit_full_b200 as wa
    lens = [300, 77, 513]
    x, cu, _ = make(lens, lens, 6, 2, seed=13)
    d, c, _ = dev(x, cu, cu)
    o, lse = wa.varlen_fwd(d["q"], d["k"], d["v"], c, c, causal=True)
    for i, n in enumerate(lens):
        part = [d[name][cu[i]:cu[i + 1]] for name in ("q", "k", "v")]
        one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        o1, lse1 = wa.varlen_fwd(*part, one, one, causal=True)
        assert torch.equal(o1, o[cu[i]:cu[i + 1]]) and torch.equal(lse1, lse[:, cu[i]:cu[i + 1]])
    wa.check_status()


def test_refused_tensors():
    import torch
    import video_dit_full_b200 as wa
    x, cu, _ = make([40, 9], [40, 9], 4, 2, seed=1)
    d, c, _ = dev(x, cu, cu)
    q, k, v = d["q"], d["k"], d["v"]
    bad = [((q.float(), k, v, c, c), TypeError), ((q, k[:-1], v, c, c), ValueError), ((q, k, v, c.long(), c), TypeError),
           ((q, k, v, c[:2], c), ValueError), ((q, k[:, :1].expand(-1, 3, -1), v[:, :1].expand(-1, 3, -1), c, c), ValueError),
           ((q.transpose(0, 1), k, v, c, c), ValueError), ((q[..., :64], k[..., :64], v[..., :64], c, c), ValueError),
           ((q[..., :64].contiguous(), k[..., :64].contiguous(), v[..., :64].contiguous(), c, c), wa.WanAttnError),
           ((q, k, v, c[:1], c[:1]), ValueError)]
    for args, error in bad:
        with pytest.raises(error):
            wa.varlen_fwd(*args)
    o, lse = wa.varlen_fwd(q, k, v, c, c)
    with pytest.raises(ValueError):
        wa.varlen_bwd(q, k, v, o, d["do"], lse[:, :-1].contiguous(), c, c)
    with pytest.raises(wa.WanAttnError):                    # a gradient over an input
        wa.varlen_bwd(q, k, v, o, d["do"], lse, c, c, dq=q)
    with pytest.raises(wa.WanAttnError):
        wa.varlen_bwd(q, k, v, o, d["do"], lse, c, c, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
