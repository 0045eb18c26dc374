"""Prompt attention, tree attention and token log probabilities at the far ends of the ranges that they take.

Tolerances count roundings, as in the tests of the same operators at small sizes."""
import ctypes
import math

import pytest
import torch

import tree_reference as ref
from test_gpu_tree_ops import BF16, F32, NAN, RUNS, U, check, evs, gen, i32, make_prompt, make_tree, randn  # noqa: F401
from test_gpu_tree_ops import run_prompt, run_tree, same, shape_of, want_tree

pytestmark = pytest.mark.gpu
FAR = 1 << 31


def offset_of(t, *at):
    """Elements from the tensor's first to the one at these indices."""
    return sum(i * s for i, s in zip(at, t.stride()))


# ---- offsets -----------------------------------------------------------------------------------
def test_tree_tensor_maps_past_32_bits(evs):  # noqa: F811
    """The ninth sequence of a cache begins 2^31 elements into it."""
    B, G, S, dh, T, H = 9, 2, 1 << 20, 128, 3, 4
    kc, vc = (torch.empty(B, G, S, dh, dtype=BF16, device="cuda") for _ in range(2))     # 4.8 GB each
    assert offset_of(kc, 8, 0, 0, 0) >= FAR
    small = make_tree(1, BF16, T, H, G, dh, 500, [500], nodes=False)
    small["cached"], small["parents"] = [500 - T], [[-1, 0, 0]]
    kc[8, :, :500], vc[8, :, :500] = small["kc"][0], small["vc"][0]
    kc[:8, :, 0], vc[:8, :, 0] = 0.0, 0.0
    q = torch.zeros(B, T, H, dh, dtype=BF16, device="cuda")
    q[8] = small["q"][0]
    lens, cached, parents = i32([1] * 8 + [T]), i32([0] * 8 + [500 - T]), i32([-1, 0, 0])

    def last(kn=None, vn=None):
        o, lse = evs.tree_attention(q, kc, vc, cached, parents, kn, vn, lens=lens, return_lse=True)
        assert (o[:8] == 0).all()
        return o[8:], lse[8:]

    want = want_tree(small)
    in_cache = last()
    check(in_cache, want, BF16, dh, 500)
    # the nodes' own K/V: rows of the same tensors, as far apart
    kn, vn = (t[:, :, 500 - T:500] for t in (kc, vc))
    kn[:8], vn[:8] = 0.0, 0.0
    assert same(last(kn, vn), in_cache)
    # values that are not finite are added where they belong by the kernel's own addresses
    vc[8, 1, 500 - T + 1, 7] = NAN
    for o, lse in (last(), last(kn, vn)):
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[0, 1, 2:, 7] = True
        assert torch.equal(torch.isnan(o), hit) and torch.equal(o[~hit], in_cache[0][~hit]) and torch.equal(lse, in_cache[1])


@pytest.mark.parametrize("dtype,dh", [(F32, 16), (BF16, 32), (BF16, 128)])
@pytest.mark.parametrize("T", [1, 20])
def test_tree_cuda_cores_past_32_bits(evs, dtype, dh, T):  # noqa: F811
    """Rows of 2^18 elements, where what is behind row 8191 is past 2^31; sequences of 2^30 elements. Rows off 16 bytes
    keep heads of 128 on the CUDA cores."""
    H, G, S = 4, 2, 8700
    odd = 1 if dh == 128 else 0
    buf = torch.empty(S << 18, dtype=dtype, device="cuda")

    def view(at, B, s, row, head, seq):
        return buf[at:].as_strided((B, G, s, dh), (seq, head, row, 1))

    d = make_tree(T, dtype, T, H, G, dh, S, [S - T], nodes=False)
    kc, vc = (view(at, 1, S, 1 << 18, 512, 1 << 30) for at in (odd, 2048 + odd))
    assert offset_of(kc, 0, 0, S - T, 0) > FAR
    kc.copy_(d["kc"])
    vc.copy_(d["vc"])
    far = dict(d, kc=kc, vc=vc)
    check(run_tree(evs, far), want_tree(d), dtype, dh, S)
    # and the nodes' own rows there
    own = dict(d, kn=d["kc"][:, :, S - T:], vn=d["vc"][:, :, S - T:])
    check(run_tree(evs, dict(far, kn=kc[:, :, S - T:], vn=vc[:, :, S - T:])), want_tree(own), dtype, dh, S)
    # sequences
    d = make_tree(T + 1, dtype, T, H, G, dh, 130 + T, [77, 0, 130], nodes=False)
    kc, vc = (view(at, 3, 130 + T, 1 << 10, 512, 1 << 30) for at in (odd, (1 << 20) + odd))
    assert offset_of(kc, 2, 0, 0, 0) >= FAR
    kc.copy_(d["kc"])
    vc.copy_(d["vc"])
    check(run_tree(evs, dict(d, kc=kc, vc=vc)), want_tree(d), dtype, dh, 130 + T)


@pytest.mark.parametrize("dtype,dh,odd", [(F32, 16, 0), (BF16, 16, 0), (BF16, 128, 1), (BF16, 128, 0), (BF16, 64, 0)])
@pytest.mark.parametrize("empty", [0, 63])
def test_prompt_past_32_bits(evs, dtype, dh, odd, empty):  # noqa: F811
    """Rows of 2^18 elements of q, k, v and out, read and written behind 2^31; on CUDA cores, in whole items (with empty
    sequences before it) and in runs of tiles. Values that are not finite among the last rows."""
    N, H, G, n = 9000, 2, 1, 300
    d = make_prompt(dh, dtype, [n], H, G, dh)
    big = torch.empty(N, 1 << 18, dtype=dtype, device="cuda")
    part = lambda at, heads: big[:, at + odd:at + odd + heads * dh].unflatten(1, (heads, dh))  # noqa: E731
    q, k, v, out = part(0, H), part(512, G), part(1024, G), part(2048, H)
    at = N - n
    assert offset_of(q, at, 0, 0) > FAR and offset_of(out, at, 0, 0) > FAR
    q[at:], k[at:], v[at:] = d["q"], d["k"], d["v"]
    starts = i32([at] * (empty + 1) + [N])
    o, lse = evs.prompt_attention(q, k, v, starts, out=out, return_lse=True)
    clean = o[at:].clone()
    check((clean, lse[at:]), ref.prompt(d["q"], d["k"], d["v"], d["starts"]), dtype, dh, n)
    v[N - 5, 0, 3], v[at + 40, 0, dh - 1] = math.inf, NAN
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[n - 5:, :, 3] = hit[40:, :, dh - 1] = True
    again, _ = evs.prompt_attention(q, k, v, starts, out=out, return_lse=True)
    again = again[at:]
    assert torch.equal(~torch.isfinite(again), hit) and torch.equal(again[~hit], clean[~hit])


# ---- scales ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 16)])
def test_scales(evs, dtype, dh):  # noqa: F811
    """From 1e-30 to 1e30, where queries of zeros still weigh all keys alike; others are refused, also those that are no
    value of the struct's type."""
    d = make_prompt(dh, dtype, [150], 2, 1, dh)
    d["q"][:] = 0.0
    t = make_tree(dh, dtype, 5, 2, 1, dh, 150, [150])
    t["q"][:] = 0.0
    for scale in (1e-30, 1.0, 1e30):
        check(run_prompt(evs, d, scale=scale), ref.prompt(d["q"], d["k"], d["v"], d["starts"], scale), dtype, dh, 150)
        check(run_tree(evs, t, scale=scale), want_tree(t, scale), dtype, dh, 155)
    for scale in (3e38, 1e39, 1e300, 1e-31, math.inf, -1.0, 0.0, NAN):
        with pytest.raises(ValueError):
            run_prompt(evs, d, scale=scale)
        with pytest.raises(ValueError):
            run_tree(evs, t, scale=scale)


def test_outputs_are_no_keys_or_values(evs):  # noqa: F811
    """Rows of K and V are read after others of the output are written."""
    d = make_prompt(3, BF16, [100], 2, 2, 64)
    q, k, v, s = d["q"], d["k"].contiguous(), d["v"].contiguous(), i32(d["starts"])
    t = make_tree(4, BF16, 6, 2, 2, 64, 6, [3, 2])
    tree = lambda out, own=True: evs.tree_attention(  # noqa: E731
        t["q"], t["kc"], t["vc"], i32(t["cached"]), i32(t["parents"]), *((t["kn"], t["vn"]) if own else ()), out=out)
    for call in (lambda: evs.prompt_attention(q, k, v, s, out=k), lambda: evs.prompt_attention(q, k, v, s, out=v),
                 lambda: tree(t["kn"].view_as(t["q"])), lambda: tree(t["vn"].view_as(t["q"])),
                 lambda: tree(t["kc"].view_as(t["q"]), False), lambda: tree(t["vc"].view_as(t["q"]), False)):
        with pytest.raises(ValueError, match="may not be k or v"):
            call()
    assert evs.prompt_attention(q, k, v, s, out=torch.empty_like(v)).shape == v.shape


# ---- values that are not finite ----------------------------------------------------------------
def comb(n):
    """Two chains in turn: no node's parent is the node before it."""
    return [i - 2 if i > 1 else -1 for i in range(n)]


@pytest.mark.parametrize("kind", ["chain", "star", "binary", "comb"])
@pytest.mark.parametrize("dtype,dh,T,H,G,own", [(BF16, 128, 128, 8, 2, True), (BF16, 64, 127, 4, 4, True), (BF16, 128, 100, 4, 2, False),
                                                (BF16, 64, 90, 8, 1, False), (F32, 32, 40, 2, 1, True)])
def test_tree_of_values_that_are_not_finite(evs, kind, dtype, dh, T, H, G, own):  # noqa: F811
    """An infinity in every node's V, each in a column of its own: a row has those of the nodes on its path."""
    cached = [300, 0, 77]
    d = make_tree(80, dtype, T, H, G, dh, 300 + T, cached)
    d["parents"] = [comb(T) if kind == "comb" else shape_of(kind, T, None)] * 3
    vn = d["vn"]
    if not own:
        for b, m in enumerate(cached):
            d["kc"][b, :, m:m + T], d["vc"][b, :, m:m + T] = d["kn"][b], d["vn"][b]
        d["kn"] = d["vn"] = None
    clean = run_tree(evs, d)
    at = torch.arange(T, device="cuda")
    column = (at * 5) % dh
    for b, m in enumerate(cached):
        (vn[b] if own else d["vc"][b, :, m:m + T])[:, at, column] = math.inf
    hit = (ref.ancestry(d["parents"][0], T).double() @ torch.nn.functional.one_hot(column.cpu(), dh).double()).cuda() > 0
    o, lse = run_tree(evs, d)
    assert torch.equal(lse, clean[1])
    assert torch.equal(torch.isposinf(o), hit[None, :, None].expand_as(o))
    assert torch.equal(o[:, ~hit.any(1)], clean[0][:, ~hit.any(1)]) and torch.equal(torch.where(hit[:, None], 0, o), torch.where(hit[:, None], 0, clean[0]))


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 32)])
@pytest.mark.parametrize("lens,H", [([700, 33, 300], 2), ([3000], 1), ([257] * 3, 40)], ids=str)
def test_prompt_of_values_that_are_not_finite(evs, dtype, dh, lens, H):  # noqa: F811
    d = make_prompt(81, dtype, lens, H, 1, dh)
    d["v"] = d["v"].contiguous()
    d["q"], d["k"] = d["q"].contiguous(), d["k"].contiguous()
    N = sum(lens)
    # a few columns: the ones that begin to be infinite in the middle of a tile, of a lane, of an item, and late
    begins = {1: 0, 2: 5, 4: 100, 5: 128, 7: 200, 8: 255, 10: 256, 11: 300, 13: 690, 14: 2990}
    d["v"][:, 0, list(begins)] = 1.0
    clean = run_prompt(evs, dict(d, v=d["v"].expand(N, 1, dh)))
    hit = torch.zeros(N, dh, dtype=torch.bool, device="cuda")
    for s, n in zip(d["starts"], lens):
        for c, j in begins.items():
            d["v"][s + j:s + n, 0, c] = math.inf
            hit[s + min(j, n):s + n, c] = True
    o, lse = run_prompt(evs, d)
    assert torch.equal(lse, clean[1])
    assert torch.equal(torch.isposinf(o), hit[:, None].expand_as(o))
    assert torch.equal(torch.where(hit[:, None], 0, o), torch.where(hit[:, None], 0, clean[0]))


def test_no_finite_value_at_all(evs):  # noqa: F811
    """What a model that has diverged gives: NaN everywhere, in about the time of a call (a walk for each key and row took
    75 and 40 ms here)."""
    d = make_tree(82, BF16, 128, 8, 8, 128, 500, [500] * 4, "chain")
    p = make_prompt(83, BF16, [1260] * 13, 32, 8, 128)
    d["vn"][:] = NAN
    p["v"][:] = NAN

    def timed(call):
        best = math.inf
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            o, lse = call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        assert torch.isnan(o).all() and torch.isfinite(lse).all()
        return best

    assert timed(lambda: run_tree(evs, d)) < 5.0
    assert timed(lambda: run_prompt(evs, p)) < 8.0


# ---- many keys ---------------------------------------------------------------------------------
def measures(n, dh, dtype):
    """V [n, dh] whose column c is 1 for the c-th part of the keys: an output is the weights that such a part has, all of
    one sign, so that a tile or a partial that is left out, or taken twice, shows in a column by far more than its
    tolerance."""
    j = torch.arange(n, device="cuda")
    v = torch.zeros(n, dh, device="cuda", dtype=dtype)
    v[j, j * dh // n] = 1.0
    return v


LONG = [
    (BF16, 1, 32, 8, 128, 50000, [50000, 20011, 3]), (BF16, 1, 8, 8, 64, 20480, [20480, 20479]), (BF16, 1, 2, 1, 128, 49999, [49999]),
    (BF16, 41, 8, 8, 128, 32768, [32768, 20001]), (BF16, 60, 16, 4, 128, 24000, [24000, 23999, 77]), (BF16, 100, 8, 1, 64, 20001, [20001]),
    (BF16, 5, 4, 2, 32, 20000, [20000, 7]), (F32, 1, 4, 2, 64, 20000, [20000, 19937]), (F32, 9, 4, 4, 128, 20000, [20000]),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: ("b" if c[0] == BF16 else "f") + "-" + "-".join(map(str, c[1:6])))
def test_tree_over_long_caches(evs, case):  # noqa: F811
    dtype, T, H, G, dh, S, cached = case
    d = make_tree(S + T, dtype, T, H, G, dh, S, cached)
    a = run_tree(evs, d)
    check(a, want_tree(d), dtype, dh, S + T)
    assert same(a, run_tree(evs, d))
    for b, m in enumerate(cached):
        d["vc"][b, :, :m] = measures(m, dh, dtype)
    d["vn"][:] = measures(T, dh, dtype)
    check(run_tree(evs, d), want_tree(d), dtype, dh, S + T)


PACKED = [
    # one long prompt beside short requests, before and behind; whole items and runs of tiles
    ([16384] + [24] * 7, 2, 1, 128), ([24] * 15 + [16384], 2, 2, 128), ([8192, 512, 512, 512, 512], 4, 2, 128), ([20001], 1, 1, 128),
    ([9000, 300, 5000], 16, 4, 128), ([33, 7000, 1, 0, 6000], 12, 4, 64), ([16385], 2, 1, 64), ([24] * 40 + [12000], 3, 3, 64),
    ([3000, 40], 4, 2, 32),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: "_".join(map(str, c[0][:3])) + f"-{len(c[0])}-{c[1]}-{c[3]}")
def test_prompt_over_many_rows(evs, case):  # noqa: F811
    lens, H, G, dh = case
    d = make_prompt(sum(lens) + dh, BF16, lens, H, G, dh)
    a = run_prompt(evs, d)
    check(a, ref.prompt(d["q"], d["k"], d["v"], d["starts"]), BF16, dh, max(lens))
    assert same(a, run_prompt(evs, d))
    for s, n in zip(d["starts"], lens):
        if n:
            d["v"][s:s + n] = measures(n, dh, BF16)[:, None]
    check(run_prompt(evs, d), ref.prompt(d["q"], d["k"], d["v"], d["starts"]), BF16, dh, max(lens))


# ---- a prompt's workspace ----------------------------------------------------------------------
IN_RUNS = [c for c in RUNS if len(c[0]) < 6] + [([0, 6000, 0, 1, 0, 5999], 1, 1, 128), ([300] * 5 + [9000], 1, 1, 64)]
STARTS = {
    "as given": lambda s, N: s,
    "one sequence": lambda s, N: [0] * (len(s) - 1) + [N],
    "the first": lambda s, N: [0] + [N] * (len(s) - 1),
    "empty": lambda s, N: [N // 2] * len(s),
    "out of order": lambda s, N: [N // 3] + [N + 7, -5, 0, N // 2] * len(s),
}


@pytest.mark.parametrize("how", STARTS)
@pytest.mark.parametrize("case", IN_RUNS, ids=lambda c: "_".join(map(str, c[0][:4])) + f"-{c[1]}-{c[3]}")
def test_prompt_keeps_to_its_workspace(evs, case, how):  # noqa: F811
    """The bytes asked for and no others, whatever the lengths on the device are."""
    from lossless_speculative_verify_gb300 import _lib
    lens, H, G, dh = case
    d = make_prompt(sum(lens) + H, BF16, lens, H, G, dh, before=3, behind=5)
    N, B, lib = d["q"].shape[0], len(lens), evs.load()
    at = STARTS[how](d["starts"], N)[:B + 1]
    starts, p = i32(at), lambda t: t.data_ptr()  # noqa: E731
    q, k, v = d["q"], d["k"], d["v"]
    o, lse = torch.full((N, H, dh), 5.0, dtype=BF16, device="cuda"), torch.empty(N, H, device="cuda")
    a = _lib.PromptAttnArgs(tokens=N, batch=B, heads=H, kv_heads=G, head_dim=dh, dtype=1, zero_rest=1, q=p(q),
                            q_row=q.stride(0), q_head=q.stride(1), k=p(k), v=p(v), kv_row=k.stride(0), kv_head=k.stride(1),
                            starts=p(starts), o=p(o), o_row=H * dh, lse=p(lse))
    n = lib.evs_prompt_attention_workspace(ctypes.byref(a))
    assert n > 0
    ws = torch.full((n + 65536,), 0xff, dtype=torch.uint8, device="cuda")        # NaN, if it is read before it is written
    a.workspace, a.ws_bytes = p(ws), n
    assert lib.evs_prompt_attention(ctypes.byref(a), None) == 0
    torch.cuda.synchronize()
    assert (ws[n:] == 0xff).all()
    read, run = [], 0
    for x in at:
        run = max(run, min(max(x, 0), N))
        read.append(run)
    want = ref.prompt(q, k, v, read)
    check((o, lse), want, BF16, dh, N)
    rest = torch.ones(N, dtype=torch.bool)
    rest[read[0]:read[-1]] = False
    assert (o[rest] == 0).all() and torch.isneginf(lse[rest]).all()


# ---- large vocabularies ------------------------------------------------------------------------
@pytest.mark.parametrize("R,V,dtype,kind", [
    # eight CTAs a row; one CTA a row, whose threads have 65536 tokens each (and rows further than 2^31 elements apart)
    (1, 1 << 24, F32, "flat"), (304, 1 << 24, BF16, "flat"), (304, 1 << 22, F32, "flat"), (3, (1 << 24) - 5, BF16, "normal"),
    (2, 1 << 24, F32, "normal"), (304, (1 << 20) + 1, F32, "rising"), (5, 1 << 19, BF16, "flat")], ids=str)
def test_logprob_of_many_tokens(evs, R, V, dtype, kind):  # noqa: F811
    """Sums whose every addition rounds the same way, of tokens that are alike; of scattered ones; with a maximum that
    grows as the row goes on."""
    g = gen(V + R)
    logits = torch.empty(R, V, dtype=dtype, device="cuda")
    for r in range(R):
        if kind == "flat":
            # every thread sees the maximum first: then all of its terms are the same fraction of it
            logits[r] = -0.3 - 1.2 * (r % 7)
            logits[r].view(8, V // 8)[:, :8192] = 0.0
        elif kind == "normal":
            logits[r] = torch.randn(V, device="cuda", generator=g) * 2
        else:
            logits[r] = torch.linspace(-20.0 - r, 3.0, V, device="cuda")
    rows = sorted({0, 1 % R, R // 2, R - 1})
    if R == 304 and V == 1 << 24:
        assert offset_of(logits, rows[-1], 0) > FAR
    tok = torch.randint(0, V, (R, 2), device="cuda", generator=g).int()
    lp, ent, tlp, tid = evs.token_logprobs(logits, tok, top=3, return_entropy=True)
    for r in rows:
        l = logits[r].double()
        y = l - l.max()
        z = float(torch.logsumexp(y, 0))
        p = torch.exp(y - z)
        py, pyy = float((p * -y).sum()), float((p * y * y).sum())
        # a weight: the exponent's three roundings and the exponential's four; 32 at most added up one after another; those
        # sums added with what each addition lost carried along, two roundings; the tree of threads, warps and CTAs. A
        # sum that is moved to a larger maximum is rounded and scaled by such a weight, six roundings: a few times, or where
        # the row rises once for 16 tokens of a thread, after which what was before weighs less by what it rose
        moves = 6 * 16 if kind != "rising" else 6 / (float(l[-1] - l[0]) / (V / (256 * 16)))
        soft = U * (3 * py + 4 + 32 + 2 + 64 + moves)
        order = torch.sort(l, descending=True, stable=True).indices[:3]
        assert torch.equal(tid[r].long(), order)
        for got, ids in ((lp[r], tok[r].long()), (tlp[r], order)):
            for a, i in zip(got.tolist(), ids.tolist()):
                b = float(y[i]) - z
                assert abs(a - b) <= soft + U * (4 * abs(float(y[i])) + abs(b)), (r, a, b)
        h = z + py
        assert abs(float(ent[r]) - h) <= 2 * soft * (1 + py) + U * (8 * pyy + 4), (r, float(ent[r]), h)
