"""Operators of verifying a tree of drafted tokens, over the range of calls that serving makes: their inputs, plain
forms, exact values and the work each call cannot do without.

Operators: causal attention over whole packed prompts (which fills the cache), attention of a tree of drafted tokens
over that cache (a tree of one node is a decode step), and the log probabilities of the drafted tokens with the
entropy and the top alternatives of each row (what accepts drafts and grows the next tree). ``run`` computes a case
in its plain form (elementary torch operations), or where ``own`` is true with the framework's kernels."""
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
        # four short prompts of a byte model in fp32, 64 wide: the smallest call, latency counts
        dict(name="prompt_bytes_f32", op="prompt", dtype=F32, batch=4, tokens=613, heads=4, kv_heads=4, dh=16),
        # one prompt of 8192 tokens, 1024 wide
        dict(name="prompt_8k", op="prompt", dtype=BF16, batch=1, tokens=8192, heads=8, kv_heads=8, dh=128),
        # the prompts of thirteen requests packed behind each other, 4096 wide with grouped heads
        dict(name="prompt_packed", op="prompt", dtype=BF16, batch=13, tokens=16381, heads=32, kv_heads=8, dh=128),
        # one long prompt
        dict(name="prompt_32k", op="prompt", dtype=BF16, batch=1, tokens=32768, heads=8, kv_heads=8, dh=128),
        # a few small trees over a short cache in fp32: the smallest call, latency counts
        dict(name="tree_bytes_f32", op="tree", dtype=F32, batch=4, nodes=7, heads=4, kv_heads=4, dh=16, cache=256,
             ragged=False),
        # a decode step: one token for each of 64 requests, grouped heads
        dict(name="tree_step", op="tree", dtype=BF16, batch=64, nodes=1, heads=32, kv_heads=8, dh=128, cache=4096,
             ragged=False),
        # the trees of 4 sequences whose candidate blocks share what they agree on, 32K of cache each, 4096 wide
        dict(name="tree_candidates_32k", op="tree", dtype=BF16, batch=4, nodes=41, heads=32, kv_heads=32, dh=128,
             cache=32768, ragged=True),
        # larger trees of a batch with grouped heads: 240 query rows for each K/V head
        dict(name="tree_grouped", op="tree", dtype=BF16, batch=16, nodes=60, heads=32, kv_heads=8, dh=128,
             cache=8192, ragged=False),
        # the rows of a small byte-vocabulary verify: the drafts' log probabilities alone
        dict(name="logprob_bytes", op="logprob", dtype=F32, rows=13, vocab=512, tokens=1, top=0, entropy=False,
             temperature=False),
        # every node of four trees, the log probabilities of its children and the alternatives for the next tree
        dict(name="logprob_tree", op="logprob", dtype=F32, rows=208, vocab=4096, tokens=4, top=8, entropy=True,
             temperature=True),
        # a word-piece vocabulary of odd size in bf16
        dict(name="logprob_odd_vocab", op="logprob", dtype=BF16, rows=64, vocab=50021, tokens=1, top=20, entropy=True,
             temperature=True),
        # scoring: the prompt's own tokens under a large vocabulary
        dict(name="logprob_large", op="logprob", dtype=F32, rows=512, vocab=131072, tokens=1, top=5, entropy=True,
             temperature=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "logprob"])
    if op == "logprob":
        vocab = _log(rng, 256, 262144)
        rows = max(1, min(_log(rng, 1, 4096), 512 * 131072 // vocab))
        return dict(op=op, dtype=rng.choice([BF16, F32]), rows=rows, vocab=vocab, tokens=rng.choice([1, 1, 2, 5, 8]),
                    top=rng.choice([0, 1, 5, 8, 20, 32, 64]), entropy=rng.random() < 0.6,
                    temperature=rng.random() < 0.5)
    dtype = rng.choice([BF16, BF16, BF16, F32])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 4, 8])
    dh = rng.choice([64, 128, 128]) if dtype == BF16 else rng.choice([16, 32, 64, 128])
    if dtype == F32:
        kv_heads, group = min(kv_heads, 4), min(group, 2)
    heads = kv_heads * group
    if op == "prompt":
        batch = rng.choice([1, 1, _log(rng, 2, 32)])
        # at most the longest listed prompt's products, in fp32 a thirtieth of them
        most = math.sqrt((32768 ** 2 * 8 * 128 if dtype == BF16 else 6500 ** 2 * 8 * 128) / (heads * dh))
        tokens = min(_log(rng, 17, 32768 if dtype == BF16 else 6500), int(most))
        return dict(op=op, dtype=dtype, batch=min(batch, tokens), tokens=tokens, heads=heads, kv_heads=kv_heads, dh=dh)
    batch, nodes = _log(rng, 1, 64), rng.choice([1, _log(rng, 2, 128)])
    cache = _log(rng, 16, 49152 if dtype == BF16 else 4096)
    # at most the largest listed case's products, in fp32 a twentieth of them, and 4 GB of cache
    most = (2.4e8 if dtype == BF16 else 1.2e7) / (batch * nodes * heads)
    cache = max(16, min(cache, int(most), int(4e9 / (batch * kv_heads * dh * 2 * _bytes(dtype)))))
    return dict(op=op, dtype=dtype, batch=batch, nodes=nodes, heads=heads, kv_heads=kv_heads, dh=dh, cache=cache,
                ragged=nodes > 1 and rng.random() < 0.4)


def _spread(n, total):
    """n whole lengths that add up to total, a few times the shortest to the longest."""
    weight = [0.25 + (0.6180339887 * (i + 1)) % 1.0 for i in range(n)]
    ends, run = [0], 0.0
    for w in weight:
        run += w
        ends.append(int(round(total * run / sum(weight))))
    return [b - a for a, b in zip(ends, ends[1:])]


def _caches(c):
    """Cached rows of each sequence: from a quarter of the capacity to all of it, one full and one just begun."""
    B, S = c["batch"], c["cache"]
    lens = [max(1, int(S * (0.25 + 0.75 * (0.6180339887 * (i + 1)) % 0.75))) for i in range(B)]
    lens[0] = S
    if B > 2:
        lens[1] = 3
    return lens


def _trees(c):
    """Nodes of each sequence's tree."""
    B, T = c["batch"], c["nodes"]
    if not c["ragged"]:
        return [T] * B
    return [T if i == 0 else max(1, T - (7 * i) % (T // 2 + 1)) for i in range(B)]


# ---- inputs -----------------------------------------------------------------------------------
def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32, scale=1.0):
        t = torch.randn(*shape, device=dev, generator=g, dtype=dtype)
        return t.mul_(scale) if scale != 1.0 else t

    def shuffled(lens):
        return [lens[i] for i in torch.randperm(len(lens), generator=host).tolist()]

    st = {"case": c}
    if c["op"] == "prompt":
        N, H, G, dh = c["tokens"], c["heads"], c["kv_heads"], c["dh"]
        lens = shuffled(_spread(c["batch"], N))
        # one projection's output holds q, k and v of a token; queries a little larger than unit variance, so that
        # the softmax has a shape
        qkv = randn(N, H + 2 * G, dh, dtype=_dt(c["dtype"]))
        qkv[:, :H] *= 1.5
        starts = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32)
        st.update(q=qkv[:, :H], k=qkv[:, H:H + G], v=qkv[:, H + G:], lens=lens, starts=starts.to(dev))
    elif c["op"] == "tree":
        dt = _dt(c["dtype"])
        B, T, H, G, dh, S = (c[k] for k in ("batch", "nodes", "heads", "kv_heads", "dh", "cache"))
        cached, sizes = shuffled(_caches(c)), shuffled(_trees(c))
        # each node hangs below one of the eight before it, or below the last cached token
        parents = torch.zeros(B, T, dtype=torch.int32)
        for i in range(T):
            parents[:, i] = torch.randint(max(-1, i - 8), i, (B,), generator=host) if i else -1
        st.update(q=randn(B, T, H, dh, dtype=dt, scale=1.5), k_cache=randn(B, G, S, dh, dtype=dt),
                  v_cache=randn(B, G, S, dh, dtype=dt), k_nodes=randn(B, G, T, dh, dtype=dt),
                  v_nodes=randn(B, G, T, dh, dtype=dt), parents=parents.to(dev), sizes=sizes,
                  cache_len=torch.tensor(cached, dtype=torch.int32).to(dev),
                  lens=torch.tensor(sizes, dtype=torch.int32).to(dev) if c["ragged"] else None)
    else:
        R, V, n = c["rows"], c["vocab"], c["tokens"]
        # a Zipf-like body with Gaussian scatter, its ids shuffled; a tenth of the tokens ruled out by a grammar
        logits = torch.rand(R, V, device=dev, generator=g).mul_(V).log1p_().mul_(-1.1)
        logits += torch.randn(R, V, device=dev, generator=g).mul_(1.2)
        logits.masked_fill_(torch.rand(R, V, device=dev, generator=g) < 0.1, -math.inf)
        # drafts: what a drafter that scatters around the same logits would propose
        guess = torch.rand(R, min(V, 4096), device=dev, generator=g) + logits[:, :min(V, 4096)]
        st.update(tokens=guess.topk(n).indices.int(), logits=logits.to(_dt(c["dtype"])),
                  temperature=torch.rand(R, device=dev, generator=g) * 0.8 + 0.6 if c["temperature"] else None)
    return st


# ---- plain forms ------------------------------------------------------------------------------
def _plain_prompt(s):
    c = s["case"]
    N, H, G, dh = c["tokens"], c["heads"], c["kv_heads"], c["dh"]
    n, dev = H // G, s["q"].device
    o = torch.empty(N, H, dh, dtype=s["q"].dtype, device=dev)
    lse = torch.empty(N, H, device=dev)
    at = 0
    for size in s["lens"]:
        k = s["k"][at:at + size].float().permute(1, 2, 0)                          # [G, dh, size]
        v = s["v"][at:at + size].float().transpose(0, 1)                           # [G, size, dh]
        rows = 2048
        for r0 in range(0, size, rows):
            r1 = min(size, r0 + rows)
            q = (s["q"][at + r0:at + r1].float() * dh ** -0.5).view(r1 - r0, G, n, dh).permute(1, 2, 0, 3)
            sc = (q.reshape(G, -1, dh) @ k[:, :, :r1]).view(G, n, r1 - r0, r1)
            ahead = torch.arange(r1, device=dev) > torch.arange(r0, r1, device=dev)[:, None]
            sc.masked_fill_(ahead, -math.inf)
            m = sc.amax(-1, keepdim=True)
            sc.sub_(m).exp_()
            total = sc.sum(-1, keepdim=True)
            out = (sc.view(G, -1, r1) @ v[:, :r1]).view(G, n, r1 - r0, dh) / total
            o[at + r0:at + r1] = out.permute(2, 0, 1, 3).reshape(r1 - r0, H, dh)
            lse[at + r0:at + r1] = (m + torch.log(total))[..., 0].permute(2, 0, 1).reshape(r1 - r0, H)
        at += size
    return [o, lse]


def _plain_tree(s):
    c = s["case"]
    B, T, H, G, dh, S = (c[k] for k in ("batch", "nodes", "heads", "kv_heads", "dh", "cache"))
    n, dev = H // G, s["q"].device
    ids = torch.arange(T, device=dev)
    parents = s["parents"].long()
    sees = torch.zeros(B, T, T, dtype=torch.bool, device=dev)                      # node i sees node j
    for i in range(T):
        above = sees.gather(1, parents[:, i].clamp(min=0)[:, None, None].expand(B, 1, T))[:, 0]
        sees[:, i] = (above & (parents[:, i] >= 0)[:, None]) | (ids == i)
    q = (s["q"].float() * dh ** -0.5).view(B, T, G, n, dh).permute(0, 2, 1, 3, 4)  # [B, G, T, n, dh]
    o = torch.empty(B, G, T, n, dh, device=dev)
    lse = torch.empty(B, G, T, n, device=dev)
    live = None if s["lens"] is None else ids[None, :] < s["lens"][:, None]
    step = max(1, int(4e9 / (G * T * n * S * 4)))                                  # sequences at once
    for b in range(0, B, step):
        e = min(B, b + step)
        qq = q[b:e].reshape(e - b, G, T * n, dh)
        sc = qq @ s["k_cache"][b:e].float().transpose(2, 3)
        sc.masked_fill_((torch.arange(S, device=dev) >= s["cache_len"][b:e, None])[:, None, None], -math.inf)
        st = (qq @ s["k_nodes"][b:e].float().transpose(2, 3)).view(e - b, G, T, n, T)
        st = st.masked_fill(~sees[b:e, None, :, None], -math.inf).view(e - b, G, T * n, T)
        m = torch.maximum(sc.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
        sc.sub_(m).exp_()
        st = torch.exp(st - m)
        total = sc.sum(-1, keepdim=True) + st.sum(-1, keepdim=True)
        out = sc @ s["v_cache"][b:e].float() + st @ s["v_nodes"][b:e].float()
        o[b:e] = (out / total).view(e - b, G, T, n, dh)
        lse[b:e] = (m + torch.log(total)).view(e - b, G, T, n)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H, dh)
    if live is not None:                     # nodes past a tree's size are zero
        return [torch.where(live[:, :, None, None], o, 0.0).to(s["q"].dtype)]
    return [o.to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(B, T, H)]


def _plain_logprob(s):
    c = s["case"]
    l = s["logits"].float()
    top = l.amax(-1, keepdim=True)
    x = l - top
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None]
    w = torch.exp(x)
    total = w.sum(-1, keepdim=True, dtype=torch.float64)
    norm = torch.log(total)
    out = [(x.gather(-1, s["tokens"].long()) - norm).float()]
    if c["entropy"]:
        mean = torch.where(w > 0, w * x, 0.0).sum(-1, dtype=torch.float64)
        out.append((norm[:, 0] - mean / total[:, 0]).float())
    if c["top"]:
        ids = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :c["top"]]   # ties: the lowest id
        out += [(x.gather(-1, ids) - norm).float(), ids.int()]
    return out


def _own(s):
    import lossless_speculative_verify_gb300 as evs
    c = s["case"]
    if c["op"] == "prompt":
        return evs.prompt_attention(s["q"], s["k"], s["v"], s["starts"], return_lse=True)
    if c["op"] == "tree":
        got = evs.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["cache_len"], s["parents"], s["k_nodes"],
                                 s["v_nodes"], lens=s["lens"], return_lse=not c["ragged"])
        return [got] if c["ragged"] else got
    got = evs.token_logprobs(s["logits"], s["tokens"], temperature=s["temperature"], top=c["top"],
                             return_entropy=c["entropy"])
    return got if isinstance(got, list) else [got]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "logprob": _plain_logprob}[state["case"]["op"]](state)


# ---- exact values -----------------------------------------------------------------------------
def _exact_prompt(s):
    N, H, dh = s["q"].shape
    n = H // s["k"].shape[1]
    o = torch.empty(N, H, dh, dtype=torch.float64, device="cuda")
    lse = torch.empty(N, H, dtype=torch.float64, device="cuda")
    first = 0
    for size in s["lens"]:
        for h in range(H):
            k, v = s["k"][first:first + size, h // n].double(), s["v"][first:first + size, h // n].double()
            for i in range(0, size, 4096):
                q = s["q"][first + i:first + i + min(4096, size - i), h].double()
                hi = i + q.shape[0]
                sc = torch.einsum("id,jd->ij", q, k[:hi]) / math.sqrt(dh)
                sc = sc + torch.full_like(sc, -math.inf).triu_(i + 1)
                z = torch.logsumexp(sc, 1)
                lse[first + i:first + hi, h] = z
                o[first + i:first + hi, h] = torch.einsum("ij,jd->id", torch.exp(sc - z[:, None]), v[:hi])
        first += size
    return [o, lse]


def _exact_tree(s):
    c = s["case"]
    B, T, H, dh = s["q"].shape
    G = s["k_cache"].shape[1]
    n = H // G
    o = torch.zeros(B, T, H, dh, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, H, dtype=torch.float64, device="cuda")
    cached, parents = s["cache_len"].tolist(), s["parents"].tolist()
    for b in range(B):
        m, size = cached[b], s["sizes"][b]
        hidden = np.full((size, size), -math.inf)
        for i in range(size):
            j = i
            while j >= 0:                                        # up to the last cached token
                hidden[i, j] = 0.0
                j = parents[b][j]
        hidden = torch.from_numpy(hidden).cuda()
        for g in range(G):
            k = torch.cat([s["k_cache"][b, g, :m], s["k_nodes"][b, g, :size]]).double()
            v = torch.cat([s["v_cache"][b, g, :m], s["v_nodes"][b, g, :size]]).double()
            for h in range(g * n, g * n + n):
                sc = torch.einsum("id,jd->ij", s["q"][b, :size, h].double(), k) / math.sqrt(dh)
                sc[:, m:] += hidden
                z = torch.logsumexp(sc, 1)
                lse[b, :size, h] = z
                o[b, :size, h] = torch.einsum("ij,jd->id", torch.exp(sc - z[:, None]), v)
    return [o] if c["ragged"] else [o, lse]


def _exact_logprob(s):
    c = s["case"]
    R, V = s["logits"].shape
    logprob = torch.empty(R, c["tokens"], dtype=torch.float64)
    entropy = torch.empty(R, dtype=torch.float64)
    top, top_id = torch.empty(R, c["top"], dtype=torch.float64), torch.empty(R, c["top"], dtype=torch.int32)
    for r in range(R):
        raw = s["logits"][r].double()
        y = raw if s["temperature"] is None else raw / s["temperature"][r].double()
        y = y - torch.logsumexp(y, 0)
        logprob[r] = y[s["tokens"][r].long()]
        alive = y[torch.isfinite(y)]
        entropy[r] = -(alive.exp() * alive).sum()
        if c["top"]:
            row = raw.cpu().numpy()
            border = np.partition(row, V - c["top"])[V - c["top"]]
            best = np.flatnonzero(row >= border)
            best = best[np.argsort(-row[best], kind="stable")][:c["top"]]
            top_id[r], top[r] = torch.from_numpy(best), y[torch.from_numpy(best).to(y.device)]
    return [logprob] + ([entropy] if c["entropy"] else []) + ([top, top_id] if c["top"] else [])


def exact(case, seed):
    c = case
    if c["op"] == "prompt" and c["heads"] * c["dh"] * c["tokens"] ** 2 / c["batch"] > 1.2e12:
        return None                                              # minutes in 64 bits
    return {"prompt": _exact_prompt, "tree": _exact_tree, "logprob": _exact_logprob}[c["op"]](prepare(case, seed))


# ---- work -------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "prompt":
        N, H, G, dh, es = c["tokens"], c["heads"], c["kv_heads"], c["dh"], _bytes(c["dtype"])
        pairs = sum(n * (n + 1) // 2 for n in _spread(c["batch"], N))
        return {"bytes": es * N * dh * 2 * (H + G) + 4 * N * H + 4 * (c["batch"] + 1), "flops": 4 * dh * H * pairs}
    if c["op"] == "tree":
        B, T, H, G, dh = (c[k] for k in ("batch", "nodes", "heads", "kv_heads", "dh"))
        es, cached, nodes = _bytes(c["dtype"]), _caches(c), _trees(c)
        live = sum(nodes)
        # sequences and trees are paired at random: the mean over the pairings; a node sees some ancestors
        pairs = sum(cached) * live / B + 5 * live
        return {"bytes": 2 * es * G * dh * (sum(cached) + live) + 2 * es * live * H * dh + 4 * B * (T + 1) +
                (0 if c["ragged"] else 4 * live * H), "flops": int(4 * dh * H * pairs)}
    R, V = c["rows"], c["vocab"]
    return {"bytes": R * V * _bytes(c["dtype"]) + 8 * R * c["tokens"] + 8 * R * c["top"] +
            4 * R * (int(c["entropy"]) + int(c["temperature"])), "flops": (6 if c["entropy"] else 4) * R * V}
