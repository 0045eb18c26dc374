"""Plain 64-bit definitions of the operators of verifying a tree of drafts, for their tests. Each returns, beside the
value, what a tolerance is derived from (sums of magnitudes)."""
from __future__ import annotations

import math

import torch


def _one(q, k, v, sees, scale):
    """o, lse, sum p|v| and the largest scale * sum |q||k| of q [n, dh] over k, v [m, dh]; sees [n, m]."""
    s = torch.einsum("nd,md->nm", q, k) * scale
    s = s.masked_fill(~sees, -math.inf)
    z = torch.logsumexp(s, -1) if k.shape[0] else torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(torch.isneginf(z)[:, None] | ~sees, 0.0, torch.exp(s - z[:, None]))
    # a key of weight 0 adds nothing, whatever its value
    v = torch.where(sees.any(0)[:, None], v, 0.0)
    qk = float((torch.einsum("nd,md->nm", q.abs(), k.abs()) * scale)[sees].max()) if bool(sees.any()) else 0.0
    return p @ v, z, p @ v.abs(), qk


def prompt(q, k, v, starts, scale=None):
    N, H, dh = q.shape
    n = H // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    o = torch.zeros(N, H, dh, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(o)
    lse = torch.full((N, H), -math.inf, dtype=torch.float64, device=q.device)
    qk = 0.0
    for a, e in zip(starts, starts[1:]):
        sees = torch.ones(e - a, e - a, dtype=torch.bool, device=q.device).tril()
        for h in range(H):
            if e > a:
                r = _one(q[a:e, h].double(), k[a:e, h // n].double(), v[a:e, h // n].double(), sees, scale)
                o[a:e, h], lse[a:e, h], mag[a:e, h], qk = r[0], r[1], r[2], max(qk, r[3])
    return o, lse, mag, qk


def ancestry(parents, n):
    """[n][n]: node i sees node j; a parent that is no earlier node is the root."""
    sees = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        p = parents[i]
        if 0 <= p < i:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def tree(q, kc, vc, cached, parents, kn=None, vn=None, lens=None, scale=None):
    """cached, lens: lists; parents: list of lists."""
    B, T, H, dh = q.shape
    G, S = kc.shape[1:3]
    n = H // G
    scale = dh ** -0.5 if scale is None else scale
    o = torch.zeros(B, T, H, dh, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(o)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=q.device)
    qk = 0.0
    for b in range(B):
        m = max(0, min(cached[b], S))
        size = T if lens is None else max(0, min(lens[b], T))
        if size == 0:
            continue
        keys = size if kn is not None else min(size, S - m)
        sees = torch.ones(size, m + keys, dtype=torch.bool)
        sees[:, m:] = ancestry(parents[b], size)[:, :keys]
        sees = sees.to(q.device)
        for g in range(G):
            tail_k, tail_v = (kn[b, g, :keys], vn[b, g, :keys]) if kn is not None else (kc[b, g, m:m + keys], vc[b, g, m:m + keys])
            k, v = torch.cat([kc[b, g, :m], tail_k]).double(), torch.cat([vc[b, g, :m], tail_v]).double()
            for h in range(g * n, (g + 1) * n):
                r = _one(q[b, :size, h].double(), k, v, sees, scale)
                o[b, :size, h], lse[b, :size, h], mag[b, :size, h], qk = r[0], r[1], r[2], max(qk, r[3])
    return o, lse, mag, qk


def logprobs(logits, tokens, temperature=None, top=0):
    """logprob, entropy, top_logprob, top_token, and the tolerances' parts: sum p|y|, sum p y^2, y of the tokens
    and of the top. fp64, rows one at a time."""
    R, V = logits.shape
    out = [[] for _ in range(8)]
    for r in range(R):
        l = logits[r].double().clone()
        l[torch.isnan(l)] = -math.inf
        t = 1.0 if temperature is None else float(temperature[r])
        order = sorted(range(V), key=lambda i: (-float(l[i]), i)) if V <= 64 else torch.sort(l, descending=True, stable=True).indices.tolist()
        best = float(l[order[0]])
        if best == -math.inf:
            y = torch.full_like(l, -math.inf)
            z = 0.0
        elif not t > 0:
            y = torch.full_like(l, -math.inf)
            y[order[0]] = 0.0
            z = 0.0
        elif best == math.inf:
            y = torch.where(l == math.inf, 0.0, -math.inf).double()
            z = math.log(float((l == math.inf).sum()))
        else:
            y = (l - best) / min(t, 1e30)
            y[torch.isneginf(l)] = -math.inf
            z = float(torch.logsumexp(y, 0))
        lp = y - z
        p = torch.exp(lp)
        ok = p > 0
        out[0].append([float(lp[i]) if 0 <= i < V else -math.inf for i in tokens[r]])
        out[1].append(float(-(p[ok] * lp[ok]).sum()))
        ids = [i if float(l[i]) > -math.inf else -1 for i in order[:top]]
        out[2].append([float(lp[i]) if i >= 0 else -math.inf for i in ids])
        out[3].append(ids)
        out[4].append(float((p[ok] * y[ok].abs()).sum()))
        out[5].append(float((p[ok] * y[ok] ** 2).sum()))
        fin = lambda i: abs(float(y[i])) if 0 <= i < V and float(y[i]) > -math.inf else 0.0  # noqa: E731
        out[6].append([fin(i) for i in tokens[r]])
        out[7].append([fin(i) for i in ids])
    return out
