"""Plain 64-bit definitions of the stand-alone operators, for their tests. Each returns, beside
the value, what a tolerance is derived from (sums of magnitudes)."""
from __future__ import annotations

import math

import numpy as np
import torch


def attention(q, kp, vp, ko, vo, own, kb=None, vb=None, scale=None):
    """o, lse, sum p|v| and the largest scale * sum |q||k|, all fp64, by one softmax per query over the
    concatenated readable rows. Without kb the block rows are own rows own[b] + j."""
    B, C, T, H, dh = q.shape
    G = kp.shape[0]
    n = H // G
    S = ko.shape[2]
    scale = dh ** -0.5 if scale is None else scale
    dev = q.device
    o = torch.zeros(B, C, T, H, dh, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(o)
    lse = torch.full((B, C, T, H), -math.inf, dtype=torch.float64, device=dev)
    qk = 0.0
    for b in range(B):
        m = max(0, min(int(own[b]), S))
        for g in range(G):
            for c in range(C):
                if kb is None:
                    e = min(m + T, S)
                    bk, bv = ko[b, g, m:e], vo[b, g, m:e]
                else:
                    bk, bv = kb[b, c, g], vb[b, c, g]
                k = torch.cat([kp[g], ko[b, g, :m], bk]).double()
                v = torch.cat([vp[g], vo[b, g, :m], bv]).double()
                first = k.shape[0] - bk.shape[0]
                qq = q[b, c, :, g * n:(g + 1) * n].double()
                s = torch.einsum("tnd,kd->tnk", qq, k) * scale
                pos = torch.arange(k.shape[0], device=dev)
                for i in range(T):
                    s[i, :, pos > first + i] = -math.inf
                if k.shape[0] == 0:
                    continue
                qk = max(qk, float((torch.einsum("tnd,kd->tnk", qq.abs(), k.abs()) * scale).max()))
                z = torch.logsumexp(s, -1)
                p = torch.where(torch.isneginf(z)[..., None], 0.0, torch.exp(s - z[..., None]))
                lse[b, c, :, g * n:(g + 1) * n] = z
                o[b, c, :, g * n:(g + 1) * n] = torch.einsum("tnk,kd->tnd", p, v)
                mag[b, c, :, g * n:(g + 1) * n] = torch.einsum("tnk,kd->tnd", p, v.abs())
    return o, lse, mag, qk


def draw_row(l, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, probs) of one row in fp64; token -1 where everything is ruled out."""
    l = np.array(l, np.float64)
    V = l.shape[0]
    l[np.isnan(l)] = -np.inf
    probs = np.zeros(V)
    fine = np.flatnonzero(l > -np.inf)
    if fine.size == 0:
        return -1, -math.inf, probs
    order = fine[np.argsort(-l[fine], kind="stable")]
    top = l[order[0]]
    if not temperature > 0:
        order, temperature = order[:1], 1.0
    elif 0 < top_k < V:
        order = order[:top_k]
    greedy = len(order) == 1 and not temperature > 0

    def weights(ids):
        with np.errstate(invalid="ignore"):
            return np.where(l[ids] == top, 1.0, np.exp((l[ids] - top) / temperature))

    w = weights(order)
    if len(order) > 1 and top_p < 1:
        reach = np.cumsum(w)
        keep = np.concatenate([[True], reach[:-1] < top_p * reach[-1]])
        order, w = order[keep], w[keep]
    if min_p > 0 and not greedy:
        keep = w >= min(min_p, 1.0)
        order, w = order[keep], w[keep]
    ids = np.sort(order)
    w = weights(ids)
    reach = np.cumsum(w)
    at = int(np.searchsorted(reach, min(max(u, 0.0), 1.0) * reach[-1], side="right"))
    if at >= len(ids):
        at = int(np.flatnonzero(w > 0)[-1])
    probs[ids] = w / reach[-1]
    return int(ids[at]), math.log(w[at] / reach[-1]), probs


def conv(x, w, bias, tail, lens, silu=True):
    """y, tail, and the sum of magnitudes before the activation; fp64 torch, lens a list."""
    B, T, D = x.shape
    L = w.shape[1]
    y = torch.zeros(B, T, D, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    tails = torch.zeros(B, L - 1, D, dtype=torch.float64, device=x.device)
    for b in range(B):
        old = torch.zeros(L - 1, D, dtype=torch.float64, device=x.device) if tail is None else tail[b].double()
        seq = torch.cat([old, x[b, :lens[b]].double()])
        tails[b] = seq[lens[b]:]
        for t in range(lens[b]):
            terms = [w[:, j].double() * seq[L - 1 + t - j] for j in range(L)]
            if bias is not None:
                terms.append(bias.double())
            v = sum(terms)
            mag[b, t] = sum(z.abs() for z in terms)
            y[b, t] = v * torch.sigmoid(v) if silu else v
    return y, tails, mag


def scan(x, dt, A, B, C, D, z, dt_bias, state, lens, softplus=True):
    """y, state, and bounds of their fp32 errors; fp64 torch, lens a list.

    Errors, with u = 2^-24: softplus to 12u relative (the exponential 5u, its quotient 4u and a half, the series,
    the product and the sum one each; its own argument's rounding apart); A log2(e) and its product with the
    step 2u, ex2.approx 4u: so a decay exp(-r) is off by (12 + 2) u r + 4u relative, the input term by 16u, and
    each step's multiply-add rounds once more (2u of the magnitudes)."""
    Bn, T, W = x.shape
    N = A.shape[1]
    u = 2.0 ** -24
    dev = x.device
    f = lambda t: None if t is None else t.double()  # noqa: E731
    x, dt, A, B, C, D, z, dt_bias = map(f, (x, dt, A, B, C, D, z, dt_bias))
    y = torch.zeros(Bn, T, W, dtype=torch.float64, device=dev)
    ye = torch.zeros_like(y)
    out = torch.zeros(Bn, W, N, dtype=torch.float64, device=dev)
    oe = torch.zeros_like(out)
    for b in range(Bn):
        h = torch.zeros(W, N, dtype=torch.float64, device=dev) if state is None else state[b].double()
        mag, err = h.abs(), torch.zeros_like(h)
        for t in range(lens[b]):
            v = dt[b, t] + (0.0 if dt_bias is None else dt_bias)
            dl = torch.nn.functional.softplus(v, threshold=50) if softplus else v
            r = dl[:, None] * A
            a = torch.exp(r)
            inp = (dl * x[b, t])[:, None] * B[b, t]
            # v rounds by u |v| before the softplus, whose slope there is at most dl
            err = a * err + a * mag * u * (14.0 * r.abs() + v.abs()[:, None] * r.abs() + 6.0) + \
                inp.abs() * u * (18.0 + v.abs()[:, None])
            mag = a * mag + inp.abs()
            h = a * h + inp
            s = (h * C[b, t]).sum(-1)
            se = ((err + mag * u * (N + 2)) * C[b, t].abs()).sum(-1)
            if D is not None:
                s = s + D * x[b, t]
                se = se + 2 * u * (D * x[b, t]).abs()
            if z is not None:
                g = z[b, t] * torch.sigmoid(z[b, t])
                se = se * g.abs() + (s * g).abs() * u * (16.0 + 2 * z[b, t].abs())
                s = s * g
            y[b, t], ye[b, t] = s, se + 4 * u * s.abs()
        out[b], oe[b] = h, err
    return y, ye, out, oe
