"""The framework's stand-alone operators over the range of calls that serving makes: their inputs, plain forms,
exact values and the work each call cannot do without.

Operators: attention over a prefix that the whole batch shares, the filtered draw of the next token, the short
causal convolution and the selective scan. ``run`` computes a case in its plain form (elementary torch
operations), or where ``own`` is true with the framework's kernels."""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"


def _dt(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _bytes(name):
    return 2 if name == BF16 else 4


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # a few continuations of a short prompt in fp32, one verify block each: the smallest call, latency counts
        dict(name="attn_block_f32", op="attn", dtype=F32, batch=4, cand=1, block=7, heads=4, kv_heads=4, dh=16,
             prefix=256, own=40),
        # one token for each of 8 continuations of an 8K prompt, 1024 wide
        dict(name="attn_step_8k", op="attn", dtype=BF16, batch=8, cand=1, block=1, heads=8, kv_heads=8, dh=128,
             prefix=8192, own=511),
        # a verify block of 4 sequences x 4 candidates that share a 32K prompt, 4096 wide: 208 query rows a head
        dict(name="attn_candidates_32k", op="attn", dtype=BF16, batch=4, cand=4, block=13, heads=32, kv_heads=32,
             dh=128, prefix=32768, own=700),
        # one token for each request of a large batch behind one system prompt of ragged length, grouped heads
        dict(name="attn_batch_grouped", op="attn", dtype=BF16, batch=64, cand=1, block=1, heads=32, kv_heads=8,
             dh=128, prefix=30001, own=2048),
        # the draw of a byte-vocabulary decode step, every filter in use and one greedy request
        dict(name="sample_bytes", op="sample", dtype=F32, rows=4, vocab=512, top_k=40, top_p=0.95, min_p=0.02,
             probs=False),
        # a drafter's proposals: filtered draws together with the distribution they were drawn from
        dict(name="sample_draft_probs", op="sample", dtype=F32, rows=208, vocab=4096, top_k=0, top_p=0.9, min_p=0.0,
             probs=True),
        # a word-piece vocabulary of odd size, a batch of requests with top-k and top-p
        dict(name="sample_odd_vocab", op="sample", dtype=BF16, rows=64, vocab=50021, top_k=50, top_p=0.9, min_p=0.0,
             probs=False),
        # the largest vocabulary and batch, nucleus and min-p only, so that thousands of tokens stay
        dict(name="sample_large", op="sample", dtype=F32, rows=256, vocab=131072, top_k=0, top_p=0.98, min_p=1e-4,
             probs=False),
        # single tokens of 64 requests: the convolution's tail is most of the traffic
        dict(name="conv_step", op="conv", dtype=BF16, batch=64, tokens=1, width=4096, taps=4, ragged=False),
        # two ragged prompts through the convolution
        dict(name="conv_prompt", op="conv", dtype=BF16, batch=2, tokens=8191, width=4096, taps=4, ragged=True),
        # single tokens of 64 requests: the carried state is the traffic
        dict(name="scan_step", op="scan", dtype=BF16, batch=64, tokens=1, width=4096, states=16, ragged=False),
        # two ragged prompts through the scan
        dict(name="scan_prompt", op="scan", dtype=BF16, batch=2, tokens=4096, width=4096, states=16, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "sample", "sample", "conv", "scan"])
    if op == "attn":
        dtype = rng.choice([BF16, BF16, BF16, F32])
        group = rng.choice([1, 1, 2, 4, 8])
        if dtype == F32:
            dh = rng.choice([16, 32, 64, 128])
            kvh, P, batch = rng.choice([1, 2, 4]), _log(rng, 16, 2048), _log(rng, 1, 8)
            group = min(group, 4)
        else:
            dh = rng.choice([64, 128])
            kvh, P, batch = rng.choice([1, 2, 4, 8]), _log(rng, 64, 49152), _log(rng, 1, 64)
        block, cand = _log(rng, 1, 16), rng.choice([1, 1, 2, 4])
        if batch * cand * block > 512:
            cand = 1
            block = max(1, 512 // batch)
        rows = batch * cand * block * kvh * group
        P = max(16, min(P, int(1.7e8 / rows)))       # at most the largest listed case's products
        return dict(op=op, dtype=dtype, batch=batch, cand=cand, block=block, heads=kvh * group, kv_heads=kvh, dh=dh,
                    prefix=P, own=_log(rng, 16, 1024))
    if op == "sample":
        vocab = _log(rng, 256, 131072)
        rows = max(1, min(_log(rng, 1, 512), 256 * 131072 // vocab))
        return dict(op=op, dtype=rng.choice([BF16, F32]), rows=rows, vocab=vocab,
                    top_k=rng.choice([0, 1, 20, 50, 1000]), top_p=rng.choice([1.0, 0.99, 0.95, 0.8]),
                    min_p=rng.choice([0.0, 0.0, 0.001, 0.05]), probs=rng.random() < 0.4)
    width = 64 * _log(rng, 1, 64)
    dtype = rng.choice([BF16, BF16, F32])
    if op == "conv":
        tokens = rng.choice([1, _log(rng, 2, 16), _log(rng, 17, 8192)])
        batch = max(1, min(_log(rng, 1, 64), 2 * 8191 * 4096 // (tokens * width * (2 if dtype == F32 else 1))))
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, width=width, taps=rng.choice([2, 3, 4, 7, 16]),
                    ragged=tokens > 1)
    states = rng.choice([4, 8, 16, 32])
    tokens = rng.choice([1, _log(rng, 2, 16), _log(rng, 17, 4096)])
    batch = max(1, min(_log(rng, 1, 64), 2 * 4096 * 4096 * 16 // (tokens * width * states)))
    return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, width=width, states=states, ragged=tokens > 1)


# ---- inputs -----------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def prepare(case, seed):
    g = _gen(seed)
    c = case
    dev = "cuda"

    def randn(*shape, dtype=torch.float32, scale=1.0):
        t = torch.randn(*shape, device=dev, generator=g, dtype=dtype if dtype != torch.float64 else torch.float32)
        return t.mul_(scale) if scale != 1.0 else t

    st = {"case": c}
    if c["op"] == "attn":
        dt = _dt(c["dtype"])
        B, C, T, H, G, dh, P = (c[k] for k in ("batch", "cand", "block", "heads", "kv_heads", "dh", "prefix"))
        S = c["own"]
        # queries a little larger than unit variance, so that the softmax has a shape; one sequence has only just
        # left the prompt and one has filled its own rows
        own_len = torch.randint(1, S + 1, (B,), device=dev, generator=g, dtype=torch.int32)
        own_len[0] = 0
        own_len[B - 1] = S
        st.update(q=randn(B, C, T, H, dh, dtype=dt, scale=1.5), k_prefix=randn(G, P, dh, dtype=dt),
                  v_prefix=randn(G, P, dh, dtype=dt), k_own=randn(B, G, S, dh, dtype=dt),
                  v_own=randn(B, G, S, dh, dtype=dt), own_len=own_len, k_block=randn(B, C, G, T, dh, dtype=dt),
                  v_block=randn(B, C, G, T, dh, dtype=dt))
    elif c["op"] == "sample":
        R, V = c["rows"], c["vocab"]
        # a Zipf-like body with Gaussian scatter, its ids shuffled; a tenth of the tokens ruled out by a grammar
        base = -1.1 * torch.log1p(torch.rand(R, V, device=dev, generator=g) * V)
        logits = base.add_(torch.randn(R, V, device=dev, generator=g), alpha=1.2)
        logits.masked_fill_(torch.rand(R, V, device=dev, generator=g) < 0.1, -math.inf)
        t = torch.rand(R, device=dev, generator=g) * 0.8 + 0.6
        if R > 3:
            t[R // 3] = 0.0                          # a greedy request in the batch
        full = lambda v, d: torch.full((R,), v, device=dev, dtype=d)  # noqa: E731
        st.update(logits=logits.to(_dt(c["dtype"])), temperature=t,
                  uniforms=torch.rand(R, device=dev, generator=g),
                  top_k=full(c["top_k"], torch.int32) if c["top_k"] else None,
                  top_p=full(c["top_p"], torch.float32) if c["top_p"] < 1.0 else None,
                  min_p=full(c["min_p"], torch.float32) if c["min_p"] > 0.0 else None)
    else:
        dt = _dt(c["dtype"])
        B, T, D = c["batch"], c["tokens"], c["width"]
        lens = None
        if c["ragged"]:
            lens = torch.randint(max(1, T // 2), T + 1, (B,), device=dev, generator=g, dtype=torch.int32)
            lens[0] = T
        st.update(lens=lens, x=randn(B, T, D).to(dt), y=torch.zeros(B, T, D, device=dev, dtype=dt))
        if c["op"] == "conv":
            L = c["taps"]
            st.update(weight=randn(D, L, scale=L ** -0.5), bias=randn(D, scale=0.1), tail=randn(B, L - 1, D),
                      tail_out=torch.empty(B, L - 1, D, device=dev))
        else:
            N = c["states"]
            # step sizes between 0.001 and 0.1 in the logarithm, decay rates 1..N with some scatter
            step = torch.exp(torch.rand(D, device=dev, generator=g) * math.log(100.0) + math.log(1e-3))
            rate = torch.arange(1, N + 1, device=dev, dtype=torch.float32) * \
                (0.5 + torch.rand(D, N, device=dev, generator=g))
            st.update(dt=randn(B, T, D).to(dt), dt_bias=torch.log(torch.expm1(step)), A=-rate,
                      B=randn(B, T, N).to(dt), C=randn(B, T, N).to(dt), D=1.0 + randn(D, scale=0.1),
                      z=randn(B, T, D).to(dt), state=randn(B, D, N), state_out=torch.empty(B, D, N, device=dev))
    return st


# ---- plain forms ------------------------------------------------------------------------------
def _plain_attn(s):
    c = s["case"]
    B, C, T, H, G, dh, P = (c[k] for k in ("batch", "cand", "block", "heads", "kv_heads", "dh", "prefix"))
    S, n = c["own"], H // G
    q = s["q"].float() * dh ** -0.5
    q = q.view(B, C, T, G, n, dh).permute(3, 0, 1, 2, 4, 5)                       # [G, B, C, T, n, dh]
    sp = q.reshape(G, -1, dh) @ s["k_prefix"].float().transpose(1, 2)
    so = q.permute(1, 0, 2, 3, 4, 5).reshape(B, G, C * T * n, dh) @ s["k_own"].float().transpose(2, 3)
    so.masked_fill_((torch.arange(S, device=so.device) >= s["own_len"][:, None])[:, None, None], -math.inf)
    qb = q.permute(1, 2, 0, 3, 4, 5).reshape(B, C, G, T * n, dh)
    sb = (qb @ s["k_block"].float().transpose(3, 4)).view(B, C, G, T, n, T)
    j = torch.arange(T, device=sb.device)
    sb = sb.masked_fill((j[None, :] > j[:, None])[:, None], -math.inf)
    sp = sp.view(G, B, C, T, n, P)
    so = so.view(B, G, C, T, n, S).permute(1, 0, 2, 3, 4, 5)
    sb = sb.permute(2, 0, 1, 3, 4, 5)
    m = torch.maximum(torch.maximum(sp.amax(-1), so.amax(-1)), sb.amax(-1))[..., None]
    sp, so, sb = torch.exp(sp - m), torch.exp(so - m), torch.exp(sb - m)
    total = sp.sum(-1) + so.sum(-1) + sb.sum(-1)
    o = (sp.view(G, -1, P) @ s["v_prefix"].float()).view(G, B, C, T, n, dh)
    o = o + (so.permute(1, 0, 2, 3, 4, 5).reshape(B, G, C * T * n, S) @ s["v_own"].float()).view(
        B, G, C, T, n, dh).permute(1, 0, 2, 3, 4, 5)
    o = o + (sb.permute(1, 2, 0, 3, 4, 5).reshape(B, C, G, T * n, T) @ s["v_block"].float()).view(
        B, C, G, T, n, dh).permute(2, 0, 1, 3, 4, 5)
    o = (o / total[..., None]).permute(1, 2, 3, 0, 4, 5).reshape(B, C, T, H, dh).to(s["q"].dtype)
    lse = (m[..., 0] + torch.log(total)).permute(1, 2, 3, 0, 4).reshape(B, C, T, H)
    return [o, lse]


def _plain_sample(s):
    c = s["case"]
    V = c["vocab"]
    l = s["logits"].double()
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    k = s["top_k"][:, None].long() if s["top_k"] is not None else torch.full_like(greedy, V, dtype=torch.long)
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    l, ids = torch.sort(l, dim=-1, descending=True, stable=True)      # equal logits in the order of their ids
    w = torch.exp((l - l[:, :1]) / torch.where(greedy, 1.0, t))
    w = torch.where(torch.arange(V, device=w.device) < k, w, 0.0)
    if s["top_p"] is not None:
        before = torch.cumsum(w, -1) - w
        before[:, 0] = -1.0
        w = torch.where(before < s["top_p"].double()[:, None] * w.sum(-1, keepdim=True), w, 0.0)
    if s["min_p"] is not None:
        w = torch.where(w >= s["min_p"].double()[:, None], w, 0.0)
    w = torch.zeros_like(w).scatter_(-1, ids, w)                       # back to ascending ids
    cum = torch.cumsum(w, -1)
    total = cum[:, -1:]
    token = (cum <= s["uniforms"].double()[:, None] * total).sum(-1)
    last = V - 1 - torch.argmax((w > 0).flip(-1).to(torch.uint8), -1)
    token = torch.minimum(token, last)
    p = w / total
    logprob = torch.log(p.gather(-1, token[:, None])[:, 0])
    return [token.int(), logprob.float()] + ([p.float()] if c["probs"] else [])


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_conv(s):
    x, tail, w, lens = s["x"].float(), s["tail"], s["weight"], s["lens"]
    T, L = x.shape[1], w.shape[1]
    full = torch.cat([tail, x], 1)
    y = s["bias"].expand_as(x)
    for j in range(L):
        y = y + w[:, j] * full[:, L - 1 - j:L - 1 - j + T]
    y = _silu(y)
    if lens is None:
        return [y.to(s["x"].dtype), full[:, T:].clone()]
    y = torch.where(torch.arange(T, device=x.device)[None, :, None] < lens[:, None, None], y, 0.0)
    rows = (lens.long()[:, None] + torch.arange(L - 1, device=x.device))[:, :, None].expand(-1, -1, x.shape[2])
    return [y.to(s["x"].dtype), full.gather(1, rows)]


def _plain_scan(s):
    x, lens, A = s["x"].float(), s["lens"], s["A"]
    T = x.shape[1]
    v = s["dt"].float() + s["dt_bias"]
    dl = torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))
    a = torch.exp(dl[..., None] * A)
    b = (dl * x)[..., None] * s["B"].float()[:, :, None, :]
    b[:, 0] += a[:, 0] * s["state"]
    step = 1
    while step < T:                                                   # doubling: (a, b) composed over 2^i steps
        b[:, step:] = b[:, step:] + a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    y = (b * s["C"].float()[:, :, None, :]).sum(-1) + s["D"] * x
    y = y * _silu(s["z"].float())
    if lens is None:
        return [y.to(s["x"].dtype), b[:, -1].clone()]
    y = torch.where(torch.arange(T, device=x.device)[None, :, None] < lens[:, None, None], y, 0.0)
    last = (lens.long() - 1)[:, None, None, None].expand(-1, 1, b.shape[2], b.shape[3])
    return [y.to(s["x"].dtype), b.gather(1, last)[:, 0]]


def _own(s):
    import lossless_speculative_verify_gb300 as evs
    op = s["case"]["op"]
    if op == "attn":
        return evs.shared_prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k_own"], s["v_own"], s["own_len"],
                                           s["k_block"], s["v_block"], return_lse=True)
    if op == "sample":
        return evs.sample(s["logits"], s["uniforms"], temperature=s["temperature"], top_k=s["top_k"],
                          top_p=s["top_p"], min_p=s["min_p"], return_logprob=True,
                          return_probs=s["case"]["probs"])
    if op == "conv":
        evs.causal_conv(s["x"], s["weight"], s["bias"], tail=s["tail"], tail_out=s["tail_out"], lens=s["lens"],
                        out=s["y"])
        return [s["y"], s["tail_out"]]
    evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                       state=s["state"], state_out=s["state_out"], lens=s["lens"], out=s["y"])
    return [s["y"], s["state_out"]]


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "sample": _plain_sample, "conv": _plain_conv, "scan": _plain_scan}[
        state["case"]["op"]](state)


# ---- exact values -----------------------------------------------------------------------------
def _exact_attn(s):
    B, C, T, H, dh = s["q"].shape
    G = s["k_prefix"].shape[0]
    n = H // G
    o = torch.zeros(B, C, T, H, dh, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, C, T, H, dtype=torch.float64, device="cuda")
    lens = s["own_len"].tolist()
    for g in range(G):
        kp, vp = s["k_prefix"][g].double(), s["v_prefix"][g].double()
        for b in range(B):
            ko, vo = s["k_own"][b, g, :lens[b]].double(), s["v_own"][b, g, :lens[b]].double()
            for c in range(C):
                k = torch.cat([kp, ko, s["k_block"][b, c, g].double()])
                v = torch.cat([vp, vo, s["v_block"][b, c, g].double()])
                q = s["q"][b, c, :, g * n:(g + 1) * n].double()               # [T, n, dh]
                sc = torch.einsum("tnd,kd->tnk", q, k) / math.sqrt(dh)
                first = k.shape[0] - T
                for i in range(T - 1):
                    sc[i, :, first + i + 1:] = -math.inf
                z = torch.logsumexp(sc, -1)
                lse[b, c, :, g * n:(g + 1) * n] = z
                o[b, c, :, g * n:(g + 1) * n] = torch.einsum("tnk,kd->tnd", torch.exp(sc - z[..., None]), v)
    return [o, lse]


def _exact_sample(s):
    host = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    l, t, u = host(s["logits"]), host(s["temperature"]), host(s["uniforms"])
    ks, ps, ms = host(s["top_k"]), host(s["top_p"]), host(s["min_p"])
    R, V = l.shape
    token, logprob, probs = np.zeros(R, np.int32), np.zeros(R), np.zeros((R, V))
    for r in range(R):
        fine = np.flatnonzero(np.isfinite(l[r]))
        order = fine[np.argsort(-l[r, fine], kind="stable")]
        if t[r] <= 0:
            order, temp = order[:1], 1.0
        else:
            temp = t[r]
            if ks is not None and ks[r] > 0:
                order = order[:int(ks[r])]
        w = np.exp((l[r, order] - l[r, order[0]]) / temp)
        if ps is not None:
            reach = np.cumsum(w)
            order = order[:1 + int(np.sum(reach[:-1] < ps[r] * reach[-1]))]
            w = w[:len(order)]
        if ms is not None:
            order = order[w >= ms[r]]
            w = w[w >= ms[r]]
        ids = np.sort(order)
        w = np.exp((l[r, ids] - l[r, order[0]]) / temp)
        reach = np.cumsum(w)
        at = min(int(np.searchsorted(reach, u[r] * reach[-1], side="right")), len(ids) - 1)
        token[r], logprob[r] = ids[at], math.log(w[at] / reach[-1])
        probs[r, ids] = w / reach[-1]
    out = [torch.from_numpy(token), torch.from_numpy(logprob)]
    return out + [torch.from_numpy(probs)] if s["case"]["probs"] else out


def _exact_conv(s):
    x, w = s["x"].double(), s["weight"].double()
    B, T, D = x.shape
    L = w.shape[1]
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    y, tail = torch.zeros_like(x), torch.zeros(B, L - 1, D, dtype=torch.float64, device=x.device)
    for b in range(B):
        seq = torch.cat([s["tail"][b].double(), x[b, :lens[b]]])
        win = seq.unfold(0, L, 1)                                      # [len, D, L], oldest first
        v = s["bias"].double() + (win * w.flip(1)).sum(-1)
        y[b, :lens[b]] = v * torch.sigmoid(v)
        tail[b] = seq[lens[b]:]
    return [y, tail]


def _exact_scan(s):
    c = s["case"]
    x, Bm, Cm, z = (s[k].double() for k in ("x", "B", "C", "z"))
    Bn, T, D = x.shape
    dl = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=50)
    A, h = s["A"].double(), s["state"].double()
    y = torch.zeros_like(x)
    lens = torch.full((Bn,), T, device=x.device) if s["lens"] is None else s["lens"]
    for t in range(T):
        live = (t < lens)[:, None]
        new = torch.exp(dl[:, t, :, None] * A) * h + (dl[:, t] * x[:, t])[..., None] * Bm[:, t, None, :]
        h = torch.where(live[..., None], new, h)
        out = ((h * Cm[:, t, None, :]).sum(-1) + s["D"].double() * x[:, t]) * z[:, t] * torch.sigmoid(z[:, t])
        y[:, t] = torch.where(live, out, 0.0)
    return [y, h]


def exact(case, seed):
    c = case
    # fp64 products of the longest cases on the device stay within seconds; longer ones have no exact value
    if c["op"] == "attn" and c["batch"] * c["cand"] * c["kv_heads"] > 4096:
        return None
    s = prepare(case, seed)
    return {"attn": _exact_attn, "sample": _exact_sample, "conv": _exact_conv, "scan": _exact_scan}[c["op"]](s)


# ---- work -------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "attn":
        B, C, T, H, G, dh, P = (c[k] for k in ("batch", "cand", "block", "heads", "kv_heads", "dh", "prefix"))
        es = _bytes(c["dtype"])
        own_rows = (B - 1) * (c["own"] + 1) / 2 if B == 1 else c["own"] + (B - 2) * (c["own"] + 1) / 2
        kv = 2 * es * G * dh * (P + own_rows + B * C * T)
        qo = 2 * es * B * C * T * H * dh + 4 * B * C * T * H
        flops = 4 * dh * H * C * T * (B * P + own_rows + B * (T + 1) / 2)
        return {"bytes": kv + qo + 4 * B, "flops": flops}
    if c["op"] == "sample":
        R, V = c["rows"], c["vocab"]
        return {"bytes": R * V * _bytes(c["dtype"]) + R * 28 + (4 * R * V if c["probs"] else 0), "flops": 4 * R * V}
    B, T, D = c["batch"], c["tokens"], c["width"]
    es = _bytes(c["dtype"])
    live = B * T if not c["ragged"] else T + (B - 1) * 0.75 * T
    if c["op"] == "conv":
        L = c["taps"]
        return {"bytes": 2 * es * live * D + 8 * B * (L - 1) * D + 4 * D * (L + 1), "flops": (2 * L + 6) * live * D}
    N = c["states"]
    return {"bytes": 4 * es * live * D + 2 * es * live * N + 8 * B * D * N + 4 * D * (N + 2),
            "flops": (6 * N + 12) * live * D}
