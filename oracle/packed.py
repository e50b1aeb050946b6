"""Packed attention (sequences of different lengths on one token axis): the oracle.

TEST INFRASTRUCTURE ONLY (same rule as ``oracle.attention``).

Sequence n owns rows cu_q[n]..cu_q[n+1] of q [Tq, H, D] and cu_k[n]..cu_k[n+1] of k, v
[Tk, Hkv, D]; query head h reads kv head h // (H // Hkv).  With lengths Lq, Lk, query i sees
key j of its own sequence when not causal or j <= i + (Lk - Lq):
    lse_i = ln sum_j exp(q_i . k_j / sqrt(D)),  o_i = sum_j exp(s_ij - lse_i) v_j
    D_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - D_i)
    dq_i = sum_j dS_ij k_j / sqrt(D),  dk_j = sum_i dS_ij q_i / sqrt(D),  dv_j = sum_i P_ij do_i
(dk, dv summed over the heads of the group).  A row that sees no key has o = 0, lse = -inf.
Rows outside every sequence come back as NaN.

``attn_packed`` also returns, element by element, how far a computation may be off that rounds
P, dS, o and its results to a type of half step ``u`` and does the rest in fp32 (relative error
``eta`` of an exponential, from the scores' and the sums' fp32 rounding):
    |do_| <= (u + eta) sum_j P_ij |v_j| + u |o|
    |ddelta_i| <= sum_d |do_id| |do_id error|
    |ddS| <= P (ddelta_i + eta (sum_d |do_id v_jd| + |D_i|)) + (u + eta) |dS|
    |ddq| <= sum_j |ddS| |k_j| / sqrt(D) + u |dq|, and so on.
"""
from __future__ import annotations

import numpy as np

U_BF16, ETA = 2.0 ** -8, 2.0 ** -11


def attn_packed(q, k, v, cu_q, cu_k, causal, do=None, u=U_BF16, eta=ETA):
    """fp64 arrays in; {"o", "lse"[, "dq", "dk", "dv"]} and {name: bound} out."""
    (Tq, H, D), (Tk, Hkv, _) = q.shape, k.shape
    group, scale = H // Hkv, 1 / np.sqrt(D)
    new = lambda *shape: np.full(shape, np.nan)                       # noqa: E731
    out = {"o": new(Tq, H, D), "lse": new(H, Tq)}
    bound = {"o": new(Tq, H, D)}
    if do is not None:
        for name, shape in (("dq", q.shape), ("dk", k.shape), ("dv", k.shape)):
            out[name], bound[name] = new(*shape), new(*shape)
    for n in range(len(cu_q) - 1):
        a, b, c, d = cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]
        lq, lk = b - a, d - c
        sees = np.ones((lq, lk), bool)
        if causal:
            sees = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)
        if do is not None:
            for name in ("dk", "dv"):
                out[name][c:d] = 0
                bound[name][c:d] = 0
        for h in range(H):
            g = h // group
            qh, kh, vh = q[a:b, h], k[c:d, g], v[c:d, g]
            s = np.where(sees, qh @ kh.T * scale, -np.inf)
            top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(top), top, 0))
            p[~sees] = 0
            total = p.sum(1, keepdims=True)
            p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
            with np.errstate(divide="ignore"):
                out["lse"][h, a:b] = (np.where(np.isfinite(top), top, 0) + np.log(total))[:, 0]
            o = p @ vh
            do_err = (u + eta) * (p @ np.abs(vh)) + u * np.abs(o)
            out["o"][a:b, h], bound["o"][a:b, h] = o, do_err
            if do is None:
                continue
            gh = do[a:b, h]
            delta = (gh * o).sum(1, keepdims=True)
            ds = p * (gh @ vh.T - delta)
            ds_err = p * ((np.abs(gh) * do_err).sum(1, keepdims=True)
                          + eta * (np.abs(gh) @ np.abs(vh).T + np.abs(delta))) + (u + eta) * np.abs(ds)
            out["dq"][a:b, h] = ds @ kh * scale
            bound["dq"][a:b, h] = ds_err @ np.abs(kh) * scale + u * np.abs(out["dq"][a:b, h])
            out["dk"][c:d, g] += ds.T @ qh * scale
            bound["dk"][c:d, g] += ds_err.T @ np.abs(qh) * scale
            out["dv"][c:d, g] += p.T @ gh
            bound["dv"][c:d, g] += (u + eta) * (p.T @ np.abs(gh))
        if do is not None:
            for name in ("dk", "dv"):
                bound[name][c:d] += u * np.abs(out[name][c:d])
    return out, bound
