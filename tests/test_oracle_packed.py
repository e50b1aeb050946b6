"""Pins of the packed-attention oracle (oracle/packed.py), CPU only: pure-Python brute force with
math.fsum, the dense oracle on each sequence, and gradients against central differences."""
import itertools
import math

import numpy as np
import pytest

import oracle
from oracle.packed import attn_packed


def rand(shape, seed, scale=0.7):
    return np.random.default_rng(seed).standard_normal(shape) * scale


CASES = [([0, 3, 3, 8], [0, 5, 6, 9], 4, 2, True),      # an empty query run, Lq > Lk leaves rows empty
         ([0, 3, 4], [0, 0, 7], 2, 1, True),            # no keys at all
         ([1, 5, 6], [0, 4, 6], 3, 3, False)]           # a row before the first sequence


@pytest.mark.parametrize("cu_q,cu_k,H,Hkv,causal", CASES)
def test_brute_force(cu_q, cu_k, H, Hkv, causal):
    D = 4
    q, k, v = rand((cu_q[-1] + 1, H, D), 1), rand((cu_k[-1] + 1, Hkv, D), 2), rand((cu_k[-1] + 1, Hkv, D), 3)
    out, _ = attn_packed(q, k, v, cu_q, cu_k, causal)
    done = np.zeros(len(q), bool)
    for n in range(len(cu_q) - 1):
        lq, lk = cu_q[n + 1] - cu_q[n], cu_k[n + 1] - cu_k[n]
        for i, h in itertools.product(range(lq), range(H)):
            row, g = cu_q[n] + i, h // (H // Hkv)
            done[row] = True
            keys = [cu_k[n] + j for j in range(lk) if not causal or j <= i + lk - lq]
            if not keys:
                assert (out["o"][row, h] == 0).all() and out["lse"][h, row] == -np.inf
                continue
            w = [math.exp(math.fsum(q[row, h] * k[j, g]) / math.sqrt(D)) for j in keys]
            z = math.fsum(w)
            assert out["lse"][h, row] == pytest.approx(math.log(z), abs=1e-12)
            for d in range(D):
                want = math.fsum(a * v[j, g, d] for a, j in zip(w, keys)) / z
                assert out["o"][row, h, d] == pytest.approx(want, abs=1e-12)
    assert np.isnan(out["o"][~done]).all()


def test_dense_oracle_per_sequence():
    cu = [0, 5, 12]
    q, k, v, do = (rand((12, 3, 8), s) for s in range(4))
    out, _ = attn_packed(q, k, v, cu, cu, False, do)
    for a, b in zip(cu, cu[1:]):
        part = [t[None, a:b] for t in (q, k, v, do)]
        o, lse = oracle.attn_fwd(*part[:3])
        np.testing.assert_allclose(out["o"][a:b], o[0], atol=1e-13)
        np.testing.assert_allclose(out["lse"][:, a:b], lse[0], atol=1e-13)
        g = oracle.attn_bwd(*part)
        for n in ("dq", "dk", "dv"):
            np.testing.assert_allclose(out[n][a:b], g[n][0], atol=1e-13)


@pytest.mark.parametrize("cu_q,cu_k,H,Hkv,causal", CASES)
def test_gradients_against_differences(cu_q, cu_k, H, Hkv, causal):
    D, e = 4, 1e-5
    x = {"q": rand((cu_q[-1], H, D), 4), "k": rand((cu_k[-1], Hkv, D), 5), "v": rand((cu_k[-1], Hkv, D), 6)}
    do = rand((cu_q[-1], H, D), 7)
    out, _ = attn_packed(x["q"], x["k"], x["v"], cu_q, cu_k, causal, do)
    loss = lambda y: np.nansum(attn_packed(y["q"], y["k"], y["v"], cu_q, cu_k, causal)[0]["o"] * do)   # noqa: E731
    rng = np.random.default_rng(0)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        for flat in rng.choice(x[name].size, 12, replace=False):
            at = np.unravel_index(flat, x[name].shape)
            up, down = ({m: t.copy() for m, t in x.items()} for _ in range(2))
            up[name][at] += e
            down[name][at] -= e
            diff = (loss(up) - loss(down)) / (2 * e)
            assert np.nan_to_num(out[grad][at]) == pytest.approx(diff, abs=1e-8)
