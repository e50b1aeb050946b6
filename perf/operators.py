"""Measured cases of packed attention, the int8 linear layer and 8-bit activation checkpoints.

``run`` makes one pass in the plain form (elementary torch operations in fp32, rounded once at
the end) or, with ``own`` set, through this package's calls; ``exact`` restates each operator in
fp64 from its definition.

Kinds of case:
  attn    packed attention.  q [Tq, H, 128], k and v [Tk, Hkv, 128]; sequence n owns rows
          cu_q[n]..cu_q[n+1] of q and cu_k[n]..cu_k[n+1] of k and v.  causal: query i of a
          sequence sees key j when j <= i + (Lk - Lq).  train: the forward, then the backward.
  linear  y = x w^T + bias with x and w in 8-bit integers, a scale per token and per output
          channel.  train: the forward keeping the codes of x, then dW from those codes and dX
          from the weight's codes.
  ckpt    activations to 8-bit codes with a scale per token, and the values they stand for.
"""
import math

import torch

own = False

D = 128                       # head dimension
ROWS = 1 << 30                # largest padded score matrix that the plain form makes at once


# ------------------------------------------------------------------------------------ cases
def _attn(name, lens_q, lens_k, heads, kv_heads, causal, train):
    case = {"kind": "attn", "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)),
            "heads": heads, "kv_heads": kv_heads, "causal": causal, "train": train}
    return {"name": name, **case} if name else case


def _linear(name, tokens, k, n, bias, train):
    case = {"kind": "linear", "tokens": tokens, "k": k, "n": n, "bias": bias, "train": train}
    return {"name": name, **case} if name else case


def _ckpt(name, tokens, k):
    case = {"kind": "ckpt", "tokens": tokens, "k": k}
    return {"name": name, **case} if name else case


def listed():
    prompts = [4501, 3333, 2048, 1999, 1024, 1001, 777, 512, 387, 128, 63, 1]
    cached = [17 + 251 * i for i in range(40)]
    train = [2049, 1536, 1281, 1024, 517, 255, 130, 5]
    return [
        # a handful of short prompts at once: launch latency
        _attn("prompts_short", [1, 7, 33, 64, 130, 2], [1, 7, 33, 64, 130, 2], 12, 12, True, False),
        # a serving step's prompts, grouped heads
        _attn("prompts_grouped", prompts, prompts, 40, 8, True, False),
        # clips of different lengths packed into one sequence axis (17 frames of 256 x 256 are 1280
        # tokens, 81 frames of 480 x 832 are 32760), every token of a clip sees the whole clip
        _attn("clips_full", [32760, 1280, 7801], [32760, 1280, 7801], 12, 12, False, False),
        # one new token for each of 40 sequences against 17 to 9806 cached ones
        _attn("single_tokens", [1] * 40, cached, 40, 8, True, False),
        # a training step's attention over packed documents, grouped heads
        _attn("train_prompts", train, train, 40, 8, True, True),
        # a training step's attention over packed clips
        _attn("train_clips", [7800, 1280, 5001], [7800, 1280, 5001], 12, 12, False, True),
        # one token through a 5120-wide layer: the weight's bytes and latency
        _linear("linear_one_token", 1, 5120, 5120, True, False),
        # a few tokens, an uneven number
        _linear("linear_few_tokens", 37, 1536, 8960, False, False),
        # the fused query-key-value projection of a 480p clip
        _linear("linear_clip", 32760, 5120, 15360, True, False),
        # a small layer's training step
        _linear("train_linear_small", 515, 1536, 1536, True, True),
        # a layer's training step on a 480p clip
        _linear("train_linear_clip", 32760, 5120, 5120, False, True),
        # a 480p clip's activations kept in 8 bits and read back
        _ckpt("checkpoint_clip", 32760, 5120),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "attn", "linear", "linear", "linear", "ckpt"])
    if kind == "ckpt":
        return _ckpt(None, _log(rng, 1, 32760), 16 * _log(rng, 8, 320))
    if kind == "linear":
        tokens, k, n = _log(rng, 1, 16000), 16 * _log(rng, 20, 480), 8 * _log(rng, 40, 1100)
        return _linear(None, tokens, k, n, rng.random() < 0.5, rng.random() < 0.5)
    heads, kv_heads = rng.choice([(12, 12), (12, 4), (40, 40), (40, 8), (16, 1), (6, 2), (32, 4)])
    form = rng.choice(["prompts", "clips", "tokens", "continued"])
    if form == "tokens":
        n = _log(rng, 1, 60)
        return _attn(None, [1] * n, [_log(rng, 1, 9000) for _ in range(n)], heads, kv_heads, True, False)
    n = _log(rng, 1, 24)
    lens = [_log(rng, 1, 5000) for _ in range(n)]
    while sum(lens) > 16000:
        lens.pop()
    lens = lens or [4999]
    if form == "continued":      # new tokens behind a cached prefix
        return _attn(None, lens, [a + _log(rng, 1, 3000) for a in lens], heads, kv_heads, True, rng.random() < 0.5)
    return _attn(None, lens, lens, heads, kv_heads, form == "prompts", rng.random() < 0.5)


def _lens(case):
    return [int(a) for a in case["lens_q"].split(",")], [int(a) for a in case["lens_k"].split(",")]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    total = 0
    for a, b in zip(*_lens(case)):
        total += a * b - a * (a - 1) // 2 if case["causal"] else a * b      # cases here have Lk >= Lq
    return total


def work(case):
    if case["kind"] == "attn":
        lens_q, lens_k = _lens(case)
        q, kv = sum(lens_q) * case["heads"], sum(lens_k) * case["kv_heads"]
        flops = 4 * D * case["heads"] * _pairs(case)
        nbytes = 2 * D * (2 * q + 2 * kv) + 4 * q
        if case["train"]:
            flops = flops * 7 // 2
            nbytes += 2 * D * (4 * q + 4 * kv) + 4 * q
        return {"bytes": nbytes, "flops": flops}
    m, k = case["tokens"], case["k"]
    if case["kind"] == "ckpt":
        return {"bytes": 2 * m * k + 2 * (m * k + 4 * m) + 2 * m * k, "flops": 2 * m * k}
    n = case["n"]
    nbytes, flops = 2 * m * k + n * k + 4 * n + 2 * m * n, 2 * m * n * k
    if case["train"]:
        nbytes += 2 * (m * k + 4 * m) + 2 * 2 * m * n + n * k + 4 * n + 2 * n * k + 2 * m * k
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)

    if case["kind"] == "attn":
        lens_q, lens_k = _lens(case)
        tq, tk, h, hk = sum(lens_q), sum(lens_k), case["heads"], case["kv_heads"]
        state = {"q": normal(tq, h, D, scale=1.5), "k": normal(tk, hk, D), "v": normal(tk, hk, D)}
        if case["train"]:
            state["do"] = normal(tq, h, D)
        for name, lens in (("cu_q", lens_q), ("cu_k", lens_k)):
            ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
            state[name] = ends.to(torch.int32).cuda()
        # sequences that the plain form takes at once, padded to their longest
        groups, first = [], 0
        for i in range(1, len(lens_q) + 1):
            pad = lambda a, b: (b - a) * max(lens_q[a:b]) * max(lens_k[a:b]) * h       # noqa: E731
            if i == len(lens_q) or pad(first, i + 1) > ROWS:
                groups.append((first, i, max(lens_q[first:i]), max(lens_k[first:i])))
                first = i
        state.update(kind="attn", causal=case["causal"], train=case["train"], groups=groups)
        return state
    m, k = case["tokens"], case["k"]
    # activations with a few channels far larger than the rest, tokens of different magnitude
    channel = torch.where(torch.rand(k, device="cuda", generator=gen) < 0.005, 12.0, 1.0)
    token = torch.exp(0.5 * torch.randn(m, 1, device="cuda", generator=gen))
    x = (torch.randn(m, k, device="cuda", generator=gen) * channel * token).to(torch.bfloat16)
    if case["kind"] == "ckpt":
        return {"kind": "ckpt", "x": x}
    n = case["n"]
    w = normal(n, k, scale=1.0 / math.sqrt(k))
    w_codes, w_scales = _quantize(w)
    state = {"kind": "linear", "x": x, "w_codes": w_codes, "w_scales": w_scales, "train": case["train"],
             "bias": normal(n, scale=0.5) if case["bias"] else None}
    if case["train"]:
        state["dy"] = normal(m, n)
    return state


# ------------------------------------------------------------------------------- plain forms
def _quantize(x):
    """int8 codes rint(127 x / absmax) of each row and its scale absmax / 127 (1 for a zero row)."""
    x = x.float()
    top = x.abs().amax(dim=1, keepdim=True)
    scales = torch.where(top > 0, top / 127, torch.ones_like(top))
    codes = torch.round(x * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    return codes.to(torch.int8), scales[:, 0]


def _rows(cu, first, last, longest):
    """Packed rows of sequences first..last-1, padded: indexes [n, longest] and which are real."""
    begin, end = cu[first:last, None].long(), cu[first + 1:last + 1, None].long()
    at = begin + torch.arange(longest, device=cu.device)
    return torch.where(at < end, at, 0), at < end


def _scores(state, group, heads):
    """Padded fp32 q [n, kv head, group head x row, D], k, v [n, kv head, row, D], scaled scores
    [n, kv head, group head x row, key], which pairs are visible, and the packed rows."""
    first, last, long_q, long_k = group
    iq, real_q = _rows(state["cu_q"], first, last, long_q)
    ik, real_k = _rows(state["cu_k"], first, last, long_k)
    hk = state["k"].shape[1]
    q = _by_head(state["q"], hk, heads, iq)
    k = state["k"][:, heads][ik].float().permute(0, 2, 1, 3)
    v = state["v"][:, heads][ik].float().permute(0, 2, 1, 3)
    sees = real_q[:, :, None] & real_k[:, None, :]
    if state["causal"]:
        shift = real_k.sum(1) - real_q.sum(1)
        i = torch.arange(long_q, device=iq.device)[None, :, None] + shift[:, None, None]
        sees = sees & (torch.arange(long_k, device=iq.device) <= i)
    sees = sees[:, None].repeat(1, 1, q.shape[2] // long_q, 1)
    s = torch.where(sees, (q @ k.transpose(-1, -2)) / math.sqrt(D), -math.inf)
    return q, k, v, s, sees, iq, real_q, ik, real_k


def _by_head(x, kv_heads, heads, rows):
    """Rows of packed x [T, H, D] as fp32 [n, kv head, group head x row, D]."""
    return x.unflatten(1, (kv_heads, -1))[:, heads][rows].float().permute(0, 2, 3, 1, 4).flatten(2, 3)


def _by_row(x, real):
    """[n, kv head, group head x row, ...] back to packed rows [T, kv head, group head, ...]."""
    return x.unflatten(2, (-1, real.shape[1])).movedim(3, 1)[real]


def _parts(state):
    """(group of sequences, slice of kv heads) whose padded scores stay below ROWS."""
    h, hk = state["q"].shape[1], state["k"].shape[1]
    for group in state["groups"]:
        first, last, long_q, long_k = group
        step = max(1, ROWS // max(1, (last - first) * long_q * long_k * (h // hk)))
        for a in range(0, hk, step):
            yield group, slice(a, min(a + step, hk))


def _plain_attention(state):
    q, k, v = state["q"], state["k"], state["v"]
    hk = k.shape[1]
    o, lse = torch.zeros_like(q), torch.empty(q.shape[1], q.shape[0], device=q.device)
    o5, lse4 = o.unflatten(1, (hk, -1)), lse.unflatten(0, (hk, -1))
    for group, heads in _parts(state):
        _, _, vv, s, sees, iq, real_q, _, _ = _scores(state, group, heads)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top > -math.inf, top, 0.0)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        out = torch.where(total > 0, (p @ vv) / total, 0.0)
        o5[iq[real_q], heads] = _by_row(out, real_q).to(torch.bfloat16)
        lse4[heads, :, iq[real_q]] = _by_row((top + torch.log(total))[..., 0], real_q).permute(1, 2, 0)
    if not state["train"]:
        return o, lse
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dq5 = dq.unflatten(1, (hk, -1))
    for group, heads in _parts(state):
        qq, kk, vv, s, sees, iq, real_q, ik, real_k = _scores(state, group, heads)
        row = lse4[heads][:, :, iq].permute(2, 0, 1, 3).flatten(2, 3)[..., None]
        p = torch.where(sees, torch.exp(s - torch.where(row > -math.inf, row, 0.0)), 0.0)
        do = _by_head(state["do"], hk, heads, iq)
        oo = _by_head(o, hk, heads, iq)
        ds = p * (do @ vv.transpose(-1, -2) - (do * oo).sum(-1, keepdim=True))
        dq5[iq[real_q], heads] = _by_row((ds @ kk) / math.sqrt(D), real_q).to(torch.bfloat16)
        dk[ik[real_k], heads] = ((ds.transpose(-1, -2) @ qq) / math.sqrt(D)).permute(0, 2, 1, 3)[real_k].to(torch.bfloat16)
        dv[ik[real_k], heads] = (p.transpose(-1, -2) @ do).permute(0, 2, 1, 3)[real_k].to(torch.bfloat16)
    return o, lse, dq, dk, dv


def _plain_linear(state):
    codes, scales = _quantize(state["x"])
    w = state["w_codes"].float()
    y = (codes.float() @ w.T) * scales[:, None] * state["w_scales"][None, :]
    if state["bias"] is not None:
        y = y + state["bias"].float()
    y = y.to(torch.bfloat16)
    if not state["train"]:
        return y
    dy = state["dy"].float()
    dw = dy.T @ (codes.float() * scales[:, None])
    dx = dy @ (w * state["w_scales"][:, None])
    return y, dw.to(torch.bfloat16), dx.to(torch.bfloat16)


def run(state):
    if own:
        return _own(state)
    if state["kind"] == "attn":
        return _plain_attention(state)
    if state["kind"] == "linear":
        return _plain_linear(state)
    codes, scales = _quantize(state["x"])
    return (codes.float() * scales[:, None]).to(torch.bfloat16)


# --------------------------------------------------------------------- this package's calls
def _own(state):
    import video_dit_full_b200 as wa
    if state["kind"] == "attn":
        q, k, v, cu_q, cu_k = (state[n] for n in ("q", "k", "v", "cu_q", "cu_k"))
        o, lse = wa.varlen_fwd(q, k, v, cu_q, cu_k, causal=state["causal"])
        if not state["train"]:
            return o, lse
        return (o, lse, *wa.varlen_bwd(q, k, v, o, state["do"], lse, cu_q, cu_k, causal=state["causal"]))
    if state["kind"] == "ckpt":
        return wa.int8_dequantize_rows(*wa.int8_quantize_rows(state["x"]))
    if not state["train"]:
        return wa.int8_linear(state["x"], state["w_codes"], state["w_scales"], bias=state["bias"])
    y, codes, scales = wa.int8_linear(state["x"], state["w_codes"], state["w_scales"], bias=state["bias"],
                                      return_checkpoint=True)
    return (y, wa.int8_grad_weight(state["dy"], codes, scales),
            wa.int8_grad_input(state["dy"], state["w_codes"], state["w_scales"]))


# ---------------------------------------------------------------------- definitions in fp64
def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "attn":
        return _exact_attention(case, state)
    x = state["x"].double()
    top = x.abs().max(dim=1, keepdim=True).values
    codes = torch.where(top > 0, x * 127 / top, x).round()
    scales = torch.where(top > 0, top / 127, torch.ones_like(top))
    if case["kind"] == "ckpt":
        return codes * scales
    w = state["w_codes"].double() * state["w_scales"].double()[:, None]
    y = torch.addmm(torch.zeros(case["n"], device="cuda", dtype=torch.float64) if state["bias"] is None
                    else state["bias"].double(), codes * scales, w.T)
    if not case["train"]:
        return y
    dy = state["dy"].double()
    return y, dy.T @ (codes * scales), dy @ w


def _exact_attention(case, state):
    q, k, v = (state[n].double() for n in ("q", "k", "v"))
    group = case["heads"] // case["kv_heads"]
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], device="cuda", dtype=torch.float64)
    grads = [torch.zeros_like(t) for t in (q, k, v)] if case["train"] else []
    a = b = 0
    for lq, lk in zip(*_lens(case)):
        for h in range(case["heads"]):
            kh, vh = k[b:b + lk, h // group], v[b:b + lk, h // group]
            for r in range(0, lq, 4096):
                rows = min(4096, lq - r)
                qh = q[a + r:a + r + rows, h]
                s = qh @ kh.T * D ** -0.5
                if case["causal"]:
                    s.masked_fill_(torch.ones(rows, lk, device="cuda", dtype=torch.bool).triu_(lk - lq + r + 1), -math.inf)
                lse[h, a + r:a + r + rows] = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                o[a + r:a + r + rows, h] = oh = p @ vh
                if case["train"]:
                    g = state["do"][a + r:a + r + rows, h].double()
                    ds = p * (g @ vh.T - (g * oh).sum(1, keepdim=True)) * D ** -0.5
                    grads[0][a + r:a + r + rows, h] += ds @ kh
                    grads[1][b:b + lk, h // group] += ds.T @ qh
                    grads[2][b:b + lk, h // group] += p.T @ g
        a, b = a + lq, b + lk
    return (o, lse, *grads)
