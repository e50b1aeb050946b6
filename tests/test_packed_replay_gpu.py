"""Graphs of the packed calls replayed with other offsets than the captured ones (the lengths are read on the
device), on workspaces that hold NaN.  Bars: as in test_varlen_gpu.py."""
import random

import numpy as np
import pytest

from test_varlen_gpu import compare, make

pytestmark = pytest.mark.gpu


def lengths(rng, total, n):
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


@pytest.mark.parametrize("Tq,Tk,n,H,Hkv,causal", [(500, 500, 6, 8, 2, True), (6, 3010, 6, 8, 2, True), (300, 2500, 4, 4, 4, False),
                                                  (40, 5000, 40, 10, 2, True), (1000, 900, 3, 6, 2, True)])
def test_replayed_with_other_lengths(Tq, Tk, n, H, Hkv, causal):
    import torch
    import video_dit_full_b200 as wa
    rng = random.Random(Tq)
    x, _, _ = make([Tq], [Tk], H, Hkv, seed=1)
    d = {name: t.cuda() for name, t in x.items()}
    cq, ck = (torch.zeros(n + 1, dtype=torch.int32, device="cuda") for _ in range(2))
    full = lambda size: torch.full((size,), 255, dtype=torch.uint8, device="cuda")          # noqa: E731
    ws = full(max(256, wa.varlen_fwd_workspace_size(n, Tq, Tk, H, Hkv)))
    wsb = full(wa.varlen_bwd_workspace_size(n, Tq, Tk, H, Hkv))
    o, lse = torch.zeros_like(d["q"]), torch.zeros(H, Tq, device="cuda")

    def step():
        wa.varlen_fwd(d["q"], d["k"], d["v"], cq, ck, causal, o, lse, workspace=ws)
        return wa.varlen_bwd(d["q"], d["k"], d["v"], o, d["do"], lse, cq, ck, causal, workspace=wsb)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = step()
    for _ in range(4):
        cu_q, cu_k = ([int(a) for a in np.cumsum([0] + lengths(rng, t, n))] for t in (Tq, Tk))
        cq.copy_(torch.tensor(cu_q))
        ck.copy_(torch.tensor(cu_k))
        ws.fill_(255)
        wsb.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        wa.check_status()
        compare(x, cu_q, cu_k, causal, o, lse, grads)
