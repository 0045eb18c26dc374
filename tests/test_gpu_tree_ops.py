"""Prompt attention, tree attention and token log probabilities against their 64-bit definitions
(tests/tree_reference.py): sizes at tile edges, ragged and empty lengths, trees of every shape, masks, infinities and
NaN where nothing may read them, strides, streams, captured graphs, and a run of all of them as a verify uses them.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of fp32 u = 2^-24."""
import math
import threading

import pytest
import torch

import tree_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def evs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from lossless_speculative_verify_gb300.build import build
    build()
    import lossless_speculative_verify_gb300 as pkg
    return pkg


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(got, want, dtype, dh, keys, rows=None):
    """rows: a mask of those that are compared."""
    (o, lse), (ro, rl, mag, qk) = got, want
    # scores: a dot product of dh terms in fp32; the exponential's argument and value; sums of all keys (in tiles, so
    # the count is far above what is reached)
    soft = U * ((dh + 4) * qk + keys + 128)
    tol = 2 * soft * mag
    if dtype == BF16:                # weights and the output rounded to bf16
        tol = tol + BF * mag + BF * ro.abs()
    assert torch.isfinite(o.float()).all()
    worst = float(((o.double() - ro).abs() / (tol + 1e-30)).max())
    assert worst <= 1.0, f"o: {worst:.2f} of the tolerance"
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    if bool((~empty).any()):
        assert float((lse.double() - rl)[~empty].abs().max()) <= 2 * soft + 4 * U * 16


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# ---- prompts -----------------------------------------------------------------------------------
def make_prompt(seed, dtype, lens, H, G, dh, before=0, behind=0):
    g = gen(seed)
    N = before + sum(lens) + behind
    starts = [before]
    for n in lens:
        starts.append(starts[-1] + n)
    qkv = randn(g, N, H + 2 * G, dh, dtype=dtype)
    qkv[:, :H] *= 1.5
    return dict(q=qkv[:, :H], k=qkv[:, H:H + G], v=qkv[:, H + G:], starts=starts)


def run_prompt(evs, d, **kw):
    return evs.prompt_attention(d["q"], d["k"], d["v"], i32(d["starts"]), return_lse=True, **kw)


PROMPT = [
    (BF16, [1], 1, 1, 128), (BF16, [2, 1, 3], 4, 4, 128), (BF16, [127, 128, 129], 2, 1, 128),
    (BF16, [255, 256, 257, 1], 2, 2, 64), (BF16, [15, 16, 17, 143, 144, 145], 3, 1, 128),
    (BF16, [385, 0, 511, 0, 640], 2, 2, 128), (BF16, [1153], 8, 1, 64), (BF16, [2100], 4, 2, 128),
    (BF16, [1] * 40 + [33] * 7, 2, 1, 64), (BF16, [700, 1, 900, 300, 2, 1300], 16, 4, 128),
    (BF16, [0, 0, 5], 1, 1, 64),
    (F32, [1], 1, 1, 16), (F32, [63, 64, 65, 1], 2, 2, 16), (F32, [200, 0, 7], 4, 2, 32), (F32, [130, 61], 2, 1, 64),
    (F32, [257], 2, 2, 128), (BF16, [100, 77], 2, 1, 16), (BF16, [65, 1], 2, 2, 32),
]


def pid(c):
    return ("b" if c[0] == BF16 else "f") + "-" + "_".join(map(str, c[1][:6])) + f"-{c[2]}-{c[3]}-{c[4]}"


@pytest.mark.parametrize("case", PROMPT, ids=pid)
def test_prompt_matches_definition(evs, case):
    dtype, lens, H, G, dh = case
    d = make_prompt(sum(lens), dtype, lens, H, G, dh)
    a, b = run_prompt(evs, d), run_prompt(evs, d)
    check(a, ref.prompt(d["q"], d["k"], d["v"], d["starts"]), dtype, dh, max(lens))
    assert same(a, b)                                                # no order left to chance


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (BF16, 32), (F32, 16)])
def test_prompt_reads_no_other_rows(evs, dtype, dh):
    """Rows of no sequence hold NaN; a sequence's result is the same whatever stands before and behind it."""
    lens = [37, 129, 250]
    d = make_prompt(5, dtype, lens, 4, 2, dh)
    alone = run_prompt(evs, d)
    wide = {k: torch.full((sum(lens) + 70,) + d[k].shape[1:], NAN, device="cuda", dtype=dtype) for k in "qkv"}
    for k in "qkv":
        wide[k][29:29 + sum(lens)] = d[k]
    out = torch.full_like(wide["q"], 3.0)
    starts = i32([29 + s for s in d["starts"]])
    o, lse = evs.prompt_attention(wide["q"], wide["k"], wide["v"], starts, return_lse=True)
    assert torch.equal(o[29:29 + sum(lens)], alone[0]) and torch.equal(lse[29:29 + sum(lens)], alone[1])
    rest = torch.ones(o.shape[0], dtype=torch.bool)
    rest[29:29 + sum(lens)] = False
    assert (o[rest] == 0).all() and torch.isneginf(lse[rest]).all()
    evs.prompt_attention(wide["q"], wide["k"], wide["v"], starts, out=out)
    assert torch.equal(out[29:29 + sum(lens)], alone[0]) and (out[rest] == 3.0).all()
    # packed in another order
    for b, n in enumerate(lens):
        s = d["starts"][b]
        one = {k: d[k][s:s + n].contiguous() for k in "qkv"}
        o1, l1 = evs.prompt_attention(one["q"], one["k"], one["v"], i32([0, n]), return_lse=True)
        assert torch.equal(o1, alone[0][s:s + n]) and torch.equal(l1, alone[1][s:s + n])


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (F32, 64)])
def test_prompt_starts_out_of_order(evs, dtype, dh):
    d = make_prompt(6, dtype, [100, 50], 2, 2, dh)
    flags = i32([0])
    want = run_prompt(evs, d)
    good = [run_prompt(evs, dict(d, starts=s), flags=flags) for s in ([0, 100, 150], [0, 150])]
    assert flags.item() == 0 and same(good[0], want)
    for bad, read in (([0, 100, 500], [0, 100, 150]), ([-7, 100, 150], [0, 100, 150]), ([0, 100, 40], [0, 100, 100]),
                      ([2000, 3, -1], [150, 150, 150])):
        flags.zero_()
        got = run_prompt(evs, dict(d, starts=bad), flags=flags)
        assert flags.item() == 32
        assert same(got, run_prompt(evs, dict(d, starts=read)))


def test_prompt_scores_of_minus_infinity(evs):
    """A query whose scores are all -inf has no output; later keys that are finite do."""
    d = make_prompt(7, BF16, [300], 1, 1, 128)
    q, k, v = (d[x].contiguous().clone() for x in "qkv")
    q.abs_()
    k[:40] = -math.inf
    o, lse = evs.prompt_attention(q, k, v, i32([0, 300]), return_lse=True)
    assert (o[:40] == 0).all() and torch.isneginf(lse[:40]).all()
    want = ref.prompt(q[40:], k[40:], v[40:], [0, 260])
    check((o[40:], lse[40:]), want, BF16, 128, 300)


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 32)])
def test_prompt_large_scores(evs, dtype, dh):
    """Maxima that grow by far more than what is left unscaled, tile after tile."""
    d = make_prompt(8, dtype, [900], 2, 1, dh)
    q, k = d["q"].contiguous(), d["k"].contiguous()
    k *= (1 + torch.arange(900, device="cuda") // 100).to(dtype)[:, None, None] * 2
    got = evs.prompt_attention(q, k, d["v"].contiguous(), i32([0, 900]), return_lse=True)
    check(got, ref.prompt(q, k, d["v"], [0, 900]), dtype, dh, 900)


def test_prompt_scale_and_strides(evs):
    for dtype, dh in ((BF16, 128), (F32, 32)):
        d = make_prompt(9, dtype, [130, 200], 4, 2, dh)
        want = run_prompt(evs, d, scale=0.3)
        check(want, ref.prompt(d["q"], d["k"], d["v"], d["starts"], 0.3), dtype, dh, 200)
        # heads outermost; rows that are off 16 bytes, which no tensor map describes; spaced outputs
        t = {k: d[k].transpose(0, 1).contiguous().transpose(0, 1) for k in "qkv"}
        assert same(run_prompt(evs, dict(d, **t), scale=0.3), want)
        odd = {}
        for k in "qkv":
            n = d[k].shape[1] * dh
            buf = torch.zeros(330, n + 3, device="cuda", dtype=dtype)
            buf[:, 1:1 + n] = d[k].reshape(330, n)
            odd[k] = buf[:, 1:1 + n].unflatten(1, (-1, dh))
        check(run_prompt(evs, dict(d, **odd), scale=0.3), ref.prompt(d["q"], d["k"], d["v"], d["starts"], 0.3), dtype,
              dh, 200)
        for pad in (8, 3):
            wide = torch.full((330, 4 * dh + pad), 7.0, device="cuda", dtype=dtype)
            view = wide[:, :4 * dh].unflatten(1, (4, dh))
            run_prompt(evs, d, scale=0.3, out=view)
            assert torch.equal(view, want[0]) and (wide[:, 4 * dh:] == 7.0).all()


def test_prompt_many_sequences(evs):
    """The most sequences, most of them short: the ring is smaller then."""
    lens = [(i * 7) % 19 for i in range(1023)] + [260]
    d = make_prompt(10, BF16, lens, 2, 1, 128)
    check(run_prompt(evs, d), ref.prompt(d["q"], d["k"], d["v"], d["starts"]), BF16, 128, 260)


def test_prompt_offsets_past_32_bits(evs):
    """Rows further than 2^31 elements into a buffer."""
    N, H, dh = 9000, 2, 128
    big = torch.empty(N, 1 << 18, dtype=BF16, device="cuda")        # 4.7 GB, rows of 512 KB
    d = make_prompt(11, BF16, [300], H, 1, dh)
    q, k, v = big[:, :H * dh].unflatten(1, (H, dh)), big[:, 512:640].unflatten(1, (1, dh)), big[:, 768:896].unflatten(1, (1, dh))
    at = N - 300
    q[at:], k[at:], v[at:] = d["q"], d["k"], d["v"]
    got = evs.prompt_attention(q, k, v, i32([at, N]), return_lse=True)
    check((got[0][at:], got[1][at:]), ref.prompt(d["q"], d["k"], d["v"], d["starts"]), BF16, dh, 300)


RUNS = [
    # few items of uneven length: dealt in runs of tiles, some of which no item begins in, or several do
    ([2048], 8, 8, 128), ([5000], 1, 1, 128), ([5001], 2, 1, 64), ([4096, 700], 2, 2, 128), ([0, 3000, 0, 1, 0, 2999], 3, 1, 128),
    ([8192], 4, 2, 64), ([1, 6000, 1], 2, 2, 64), ([255, 4097, 257], 1, 1, 128), ([300] * 5 + [4000], 1, 1, 64),
]


@pytest.mark.parametrize("case", RUNS, ids=lambda c: "_".join(map(str, c[0][:4])) + f"-{c[1]}-{c[3]}")
def test_prompt_in_runs(evs, case):
    lens, H, G, dh = case
    d = make_prompt(sum(lens) + H, BF16, lens, H, G, dh, before=3, behind=5)
    want = ref.prompt(d["q"], d["k"], d["v"], d["starts"])
    a, b = run_prompt(evs, d), run_prompt(evs, d)
    check(a, want, BF16, dh, max(lens))
    assert same(a, b)
    wide = torch.zeros(d["q"].shape[0], H * dh + 3, device="cuda", dtype=BF16)      # rows off 8 bytes
    view = wide[:, :H * dh].unflatten(1, (H, dh))
    c = run_prompt(evs, d, out=view)
    n = sum(lens)
    assert torch.equal(view[3:3 + n], a[0][3:3 + n]) and torch.equal(c[1], a[1])


@pytest.mark.parametrize("dtype,dh,N,H,starts", [
    (BF16, 128, 2000, 2, [5, 5]), (BF16, 64, 2000, 2, [0, 0, 0]), (BF16, 128, 300, 64, [300, 300]), (F32, 16, 90, 2, [7, 7, 7, 7]),
    (BF16, 128, 2000, 2, [9, 9, 10, 10, 10]), (BF16, 64, 300, 64, [0, 0, 1, 1]), (F32, 64, 70, 1, [69, 69, 70])], ids=str)
def test_prompt_without_rows(evs, dtype, dh, N, H, starts):
    """Sequences of no rows, or of one, which reads itself: its V."""
    g = gen(N + H)
    q, k, v = (randn(g, N, H, dh, dtype=dtype) for _ in range(3))
    flags = i32([0])
    for _ in range(2):
        o, lse = evs.prompt_attention(q, k, v, i32(starts), return_lse=True, flags=flags)
        one = torch.zeros(N, dtype=torch.bool, device="cuda")
        one[starts[0]:starts[-1]] = True
        assert torch.equal(o[one], v[one]) and (o[~one] == 0).all()
        assert torch.isfinite(lse[one]).all() and torch.isneginf(lse[~one]).all() and flags.item() == 0
    out = torch.full_like(q, 2.0)
    evs.prompt_attention(q, k, v, i32(starts), out=out)
    assert torch.equal(out[one], v[one]) and (out[~one] == 2.0).all()


def test_prompt_runs_of_infinities(evs):
    """Partials of a row without any score: the first 2000 keys are -inf for all, the first 2000 rows read nothing else."""
    d = make_prompt(77, BF16, [4000], 1, 1, 128)
    q, k, v = (d[x].contiguous().clone() for x in "qkv")
    q.abs_()
    k[:2000] = -math.inf
    o, lse = evs.prompt_attention(q, k, v, i32([0, 4000]), return_lse=True)
    assert (o[:2000] == 0).all() and torch.isneginf(lse[:2000]).all()
    check((o[2000:], lse[2000:]), ref.prompt(q[2000:], k[2000:], v[2000:], [0, 2000]), BF16, 128, 4000)


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 64), (BF16, 32), (F32, 16)])
@pytest.mark.parametrize("lens,H", [([700, 33], 2), ([3000], 1), ([130], 40), ([257], 1)], ids=str)
def test_prompt_values_that_are_not_finite(evs, dtype, dh, lens, H):
    """Infinities and NaN in V reach the rows that read them, and no other: those are what they are without them."""
    d = make_prompt(78, dtype, lens, H, 1, dh)
    q, k, v = (d[x].contiguous().clone() for x in "qkv")
    n = lens[0]
    bad = {5: (0, math.inf), n - 3: (dh - 1, NAN), n // 2: (dh // 2, -math.inf), min(n - 1, 129): (3, math.inf), n - 20: (3, -math.inf)}
    clean = evs.prompt_attention(q, k, v, i32(d["starts"]), return_lse=True)
    for j, (c, x) in bad.items():
        v[j, 0, c] = x
    o, lse = evs.prompt_attention(q, k, v, i32(d["starts"]), return_lse=True)
    assert torch.equal(lse, clean[1])
    want = clean[0].float()
    hit = torch.zeros_like(want, dtype=torch.bool)
    for j, (c, x) in bad.items():
        want[j:n, :, c] += x                                         # a later one of the other sign: NaN
        hit[j:n, :, c] = True
    assert torch.equal(torch.isnan(o), torch.isnan(want)) and torch.equal(torch.isinf(o), torch.isinf(want))
    assert torch.equal(o[torch.isinf(o)].float(), want[torch.isinf(want)])
    # (a cleared value leaves other values of its row in the sums: the rest is the same to the last bit)
    assert torch.equal(o[~hit], clean[0][~hit])


def test_prompt_refusals(evs):
    d = make_prompt(12, BF16, [20], 4, 2, 64)
    q, k, v, s = d["q"], d["k"], d["v"], i32([0, 20])
    f = evs.prompt_attention
    for bad in (lambda: f(q[0], k, v, s), lambda: f(q.float(), k, v, s), lambda: f(q, k[:10], v, s),
                lambda: f(q[:, :3], k, v, s), lambda: f(q[:, :, :48], k[:, :, :48], v[:, :, :48], s),
                lambda: f(q, k, v.contiguous(), s), lambda: f(q, k, v, s.long()), lambda: f(q, k, v, s[:1]),
                lambda: f(q, k, v, s.cpu()), lambda: f(q, k, v, s[::2]), lambda: f(q, k, v, s, scale=0.0),
                lambda: f(q, k, v, s, scale=math.inf), lambda: f(q, k, v, s, scale=1e-40),
                lambda: f(q, k, v, s, out=torch.empty_like(q, dtype=F32)),
                lambda: f(q, k, v, s, out=torch.empty(20, 64, 4, dtype=BF16, device="cuda").transpose(1, 2)),
                lambda: f(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, s),
                lambda: f(q.half(), k.half(), v.half(), s), lambda: f(q.cpu(), k, v, s),
                lambda: f(q.clone().requires_grad_(), k, v, s), lambda: f(q, k, v, s, flags=i32([0, 0])),
                lambda: f(q[:1].expand(20, 4, 64), k, v, s)):
        with pytest.raises(ValueError):
            bad()
    assert f(q[:0], k[:0], v[:0], i32([0, 0])).shape == (0, 4, 64)


# ---- trees -------------------------------------------------------------------------------------
def shape_of(kind, n, g):
    """Parents of a tree of n nodes."""
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(n)]
    return [int(torch.randint(max(-1, i - 6), i, (1,), generator=g)) if i else -1 for i in range(n)]


def make_tree(seed, dtype, T, H, G, dh, S, cached, kind="random", nodes=True):
    B = len(cached)
    g, host = gen(seed), torch.Generator().manual_seed(seed)
    d = dict(q=randn(g, B, T, H, dh, dtype=dtype) * 1.5, kc=randn(g, B, G, S, dh, dtype=dtype),
             vc=randn(g, B, G, S, dh, dtype=dtype), cached=cached, parents=[shape_of(kind, T, host) for _ in range(B)])
    d["kn"] = randn(g, B, G, T, dh, dtype=dtype) if nodes else None
    d["vn"] = randn(g, B, G, T, dh, dtype=dtype) if nodes else None
    return d


def run_tree(evs, d, **kw):
    lens = d.get("lens")
    return evs.tree_attention(d["q"], d["kc"], d["vc"], i32(d["cached"]), i32(d["parents"]), d["kn"], d["vn"],
                              lens=None if lens is None else i32(lens), return_lse=True, **kw)


def want_tree(d, scale=None):
    return ref.tree(d["q"], d["kc"], d["vc"], d["cached"], d["parents"], d["kn"], d["vn"], d.get("lens"), scale)


TREE = [
    # tensor cores, a worker per lane
    (BF16, 1, 1, 1, 128, 4, [0]), (BF16, 1, 4, 1, 128, 300, [0, 300, 128]), (BF16, 7, 4, 4, 128, 257, [1, 127, 128, 129, 257]),
    (BF16, 13, 8, 2, 64, 1000, [0, 999, 1000, 17]), (BF16, 128, 1, 1, 64, 260, [131, 0]), (BF16, 16, 8, 1, 128, 3000, [2999]),
    (BF16, 1, 32, 8, 128, 700, [(i * 37) % 701 for i in range(33)]),
    # lengths of so many sequences that the ring is smaller
    (BF16, 1, 8, 2, 128, 900, [(i * 371) % 901 for i in range(64)]), (BF16, 33, 8, 2, 128, 500, [(i * 137) % 501 for i in range(50)]),
    # a lane per row tile
    (BF16, 33, 8, 2, 128, 777, [777, 0, 131]), (BF16, 60, 8, 2, 64, 500, [500, 3, 16]), (BF16, 128, 2, 1, 128, 400, [400, 255]),
    # several row tiles
    (BF16, 100, 8, 1, 128, 300, [300, 0]), (BF16, 128, 16, 2, 64, 200, [200]),
    # no cache at all
    (BF16, 20, 4, 2, 128, 0, [0, 0]), (BF16, 1, 2, 2, 64, 0, [0]),
    # CUDA cores
    (F32, 1, 1, 1, 16, 4, [0]), (F32, 7, 4, 4, 16, 256, [256, 0, 40]), (F32, 1, 4, 2, 64, 700, [700, 129]),
    (F32, 65, 2, 1, 32, 130, [130, 1]), (F32, 128, 2, 2, 128, 65, [65]), (F32, 9, 2, 2, 64, 0, [0]),
    (BF16, 12, 4, 2, 32, 99, [99, 0]), (BF16, 3, 4, 4, 16, 64, [64, 63]),
]


def tid(c):
    return ("b" if c[0] == BF16 else "f") + "-" + "-".join(map(str, c[1:6])) + "-" + "_".join(map(str, c[6][:4]))


@pytest.mark.parametrize("case", TREE, ids=tid)
def test_tree_matches_definition(evs, case):
    dtype, T, H, G, dh, S, cached = case
    d = make_tree(T * 1000 + S, dtype, T, H, G, dh, S, cached)
    a, b = run_tree(evs, d), run_tree(evs, d)
    check(a, want_tree(d), dtype, dh, S + T)
    assert same(a, b)


@pytest.mark.parametrize("kind", ["chain", "star", "binary"])
@pytest.mark.parametrize("dtype,dh,T,H", [(BF16, 128, 128, 2), (BF16, 64, 40, 2), (F32, 32, 100, 2)])
def test_tree_shapes(evs, kind, dtype, dh, T, H):
    d = make_tree(3, dtype, T, H, 1, dh, 150, [150, 77], kind)
    check(run_tree(evs, d), want_tree(d), dtype, dh, 150 + T)
    one = evs.tree_attention(d["q"], d["kc"], d["vc"], i32(d["cached"]), i32(d["parents"][0]), d["kn"], d["vn"],
                             return_lse=True)                        # one tree for all
    assert same(one, run_tree(evs, dict(d, parents=[d["parents"][0]] * 2)))


@pytest.mark.parametrize("dtype,dh,T", [(BF16, 128, 5), (BF16, 64, 40), (BF16, 128, 70), (F32, 32, 20), (BF16, 16, 5)])
def test_tree_nodes_in_the_cache(evs, dtype, dh, T):
    S, cached = 400, [0, 400 - T, 128, 130]
    d = make_tree(4, dtype, T, 4, 2, dh, S, cached)
    c = dict(d, kc=d["kc"].clone(), vc=d["vc"].clone(), kn=None, vn=None)
    for b, m in enumerate(cached):
        c["kc"][b, :, m:m + T], c["vc"][b, :, m:m + T] = d["kn"][b], d["vn"][b]
    got = run_tree(evs, c)
    check(got, want_tree(c), dtype, dh, S + T)
    flags = i32([0])
    over = dict(c, cached=[0, 400, 398, 401])                        # nodes past the capacity are no keys
    got = run_tree(evs, over, flags=flags)
    assert flags.item() == 1 | 32
    check(got, want_tree(over), dtype, dh, S + T)


@pytest.mark.parametrize("dtype,dh,T", [(BF16, 128, 20), (BF16, 64, 100), (F32, 16, 33)])
def test_tree_lengths(evs, dtype, dh, T):
    """Trees of fewer nodes: the rest is left alone, or zero; nothing behind any length is read."""
    S, cached, lens = 300, [300, 0, 129, 16, 250], [T, 1, 0, T - 1, 17]
    d = make_tree(5, dtype, T, 4, 2, dh, S, cached)
    d["lens"] = lens
    want = want_tree(d)
    for b in range(5):
        d["q"][b, lens[b]:] = NAN
        for c, n in (("c", cached[b]), ("n", lens[b])):
            d["k" + c][b, :, n:] = NAN
            d["v" + c][b, :, n:] = NAN
    flags = i32([0])
    got = run_tree(evs, d, flags=flags)
    assert flags.item() == 0
    check(got, want, dtype, dh, S + T)
    out = torch.full_like(d["q"], 5.0)
    o, lse = run_tree(evs, d, out=out)
    for b in range(5):
        assert (o[b, lens[b]:] == 5.0).all() and torch.equal(o[b, :lens[b]], got[0][b, :lens[b]])
        assert (got[0][b, lens[b]:] == 0).all() and torch.isneginf(lse[b, lens[b]:]).all()
    bad = dict(d, lens=[T + 5, 1, -3, T - 1, 17], cached=[301, -1, 129, 16, 250])
    again = run_tree(evs, bad, flags=flags)
    assert flags.item() == 32 and same(again, got)


@pytest.mark.parametrize("dtype,dh,T,S,own", [(BF16, 128, 20, 300, True), (BF16, 64, 128, 300, True), (BF16, 128, 1, 40, False),
                                              (F32, 16, 7, 100, True), (F32, 64, 40, 2000, False), (BF16, 64, 90, 0, True)])
def test_tree_without_nodes(evs, dtype, dh, T, S, own):
    """Trees that are all empty, and then but the last, of one node."""
    d = make_tree(8, dtype, T, 4, 2, dh, S, [S // 2, 0, S // 3], nodes=own)
    for last in (0, 1):
        d["lens"] = [0, 0, last]
        flags = i32([0])
        got = run_tree(evs, d, flags=flags)
        check(got, want_tree(d), dtype, dh, S + T)
        assert flags.item() == 0 and (got[0][:2] == 0).all() and torch.isneginf(got[1][:2]).all()
        out = torch.full_like(d["q"], 5.0)
        o, _ = run_tree(evs, d, out=out)
        assert (o[:2] == 5.0).all() and (o[2, last:] == 5.0).all() and torch.equal(o[2, :last], got[0][2, :last])


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (F32, 32)])
def test_tree_bad_parents(evs, dtype, dh):
    d = make_tree(6, dtype, 30, 2, 1, dh, 64, [64, 9])
    want = run_tree(evs, d)
    flags = i32([0])
    assert same(run_tree(evs, d, flags=flags), want) and flags.item() == 0
    bad = dict(d, parents=[list(p) for p in d["parents"]])
    read = dict(d, parents=[list(p) for p in d["parents"]])
    for i, p in ((0, 0), (3, 3), (4, 29), (7, 1 << 30), (9, -2), (11, -(1 << 31))):
        bad["parents"][1][i] = p
        read["parents"][1][i] = -1
    got = run_tree(evs, bad, flags=flags)
    assert flags.item() == 128 and same(got, run_tree(evs, read))


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (F32, 64)])
def test_tree_is_what_a_chain_and_a_step_are(evs, dtype, dh):
    """A chain over a cache is a verify block behind an empty prefix; one node a decode step."""
    for T in (1, 13):
        d = make_tree(7, dtype, T, 4, 2, dh, 500, [500, 0, 333], "chain")
        none = torch.empty(2, 0, dh, device="cuda", dtype=dtype)
        o, lse = evs.shared_prefix_attention(d["q"][:, None], none, none, d["kc"], d["vc"], i32(d["cached"]),
                                             d["kn"][:, None], d["vn"][:, None], return_lse=True)
        want = want_tree(d)
        check((o[:, 0], lse[:, 0]), want, dtype, dh, 513)
        check(run_tree(evs, d), want, dtype, dh, 513)


def test_tree_continues_a_prompt(evs):
    """The last rows of a prompt, as a chain over the cache of the rows before, are the prompt's own."""
    d = make_prompt(8, BF16, [400], 8, 2, 128)
    o, lse = run_prompt(evs, d)
    T = 21
    q, k, v = d["q"], d["k"].transpose(0, 1)[None], d["v"].transpose(0, 1)[None]
    got = evs.tree_attention(q[None, 400 - T:].contiguous(), k, v, i32([400 - T]), i32(list(range(-1, T - 1))), return_lse=True)
    want = ref.prompt(d["q"], d["k"], d["v"], d["starts"])
    check((got[0][0], got[1][0]), tuple(t[400 - T:] for t in want[:3]) + (want[3],), BF16, 128, 400)


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 32)])
def test_tree_large_and_infinite_scores(evs, dtype, dh):
    d = make_tree(9, dtype, 9, 4, 2, dh, 600, [600, 300])
    d["kc"] *= (1 + torch.arange(600, device="cuda") // 60).to(dtype)[:, None] * 2
    check(run_tree(evs, d), want_tree(d), dtype, dh, 609)
    d["q"].abs_()
    d["kc"][:, :, :200] = -math.inf
    d["kc"][1] = -math.inf
    got, want = run_tree(evs, d), want_tree(d)
    want = want[:3] + (max(want_tree(dict(d, kc=torch.where(torch.isinf(d["kc"]), 0.0, d["kc"])))[3], 0.0),)
    check(got, want, dtype, dh, 609)
    d["kn"][:] = -math.inf
    got = run_tree(evs, d)
    assert (got[0][1] == 0).all() and torch.isneginf(got[1][1]).all() and torch.isfinite(got[1][0]).all()


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 16)])
def test_tree_strides(evs, dtype, dh):
    B, T, H, G, S = 3, 6, 4, 2, 140
    d = make_tree(10, dtype, T, H, G, dh, S, [140, 3, 77])
    want = run_tree(evs, d, scale=0.2)
    check(want, want_tree(d, 0.2), dtype, dh, S + T)
    # the cache as [row][batch][head], nodes as [row][head][batch], queries and outputs in wider rows
    c = dict(d)
    for k in ("kc", "vc"):
        c[k] = d[k].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    for k in ("kn", "vn"):
        c[k] = d[k].permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    wide = torch.zeros(B, T, H * dh + 8, device="cuda", dtype=dtype)
    c["q"] = wide[..., :H * dh].unflatten(2, (H, dh))
    c["q"].copy_(d["q"])
    out = torch.full((B, T, H * dh + 3), 9.0, device="cuda", dtype=dtype)
    view = out[..., :H * dh].unflatten(2, (H, dh))
    got = run_tree(evs, c, scale=0.2, out=view)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (out[..., H * dh:] == 9.0).all()
    # strides that no tensor map describes, and queries off 16 bytes
    odd = dict(d)
    for k in ("kc", "vc"):
        buf = torch.zeros(B, G, S, dh + 1, device="cuda", dtype=dtype)
        buf[..., 1:] = d[k]
        odd[k] = buf[..., 1:]
    check(run_tree(evs, odd, scale=0.2), want_tree(d, 0.2), dtype, dh, S + T)
    off = torch.zeros(B * T * H * dh + 1, device="cuda", dtype=dtype)[1:].view(B, T, H, dh)
    off.copy_(d["q"])
    got = run_tree(evs, dict(d, q=off), scale=0.2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one cache for all sequences
    one = dict(d, kc=d["kc"][:1].expand(B, G, S, dh), vc=d["vc"][:1].expand(B, G, S, dh))
    check(run_tree(evs, one, scale=0.2), want_tree(one, 0.2), dtype, dh, S + T)


def test_tree_offsets_past_32_bits(evs):
    """A cache of more than 2^31 elements, read near its end."""
    G, S, dh = 2, 1 << 20, 128
    kc, vc = (torch.zeros(5, G, S, dh, dtype=BF16, device="cuda") for _ in range(2))     # 2.7 GB each
    g = gen(11)
    m = S - 500
    kc[4, 1, m:], vc[4, 1, m:] = randn(g, 500, dh, dtype=BF16), randn(g, 500, dh, dtype=BF16)
    kc[4, 1, :m] = -30.0                     # no weight beside the last rows
    q = randn(g, 5, 3, 4, dh, dtype=BF16).abs_()
    kn, vn = randn(g, 5, G, 3, dh, dtype=BF16), randn(g, 5, G, 3, dh, dtype=BF16)
    args = (i32([5, 0, 0, 0, S]), i32([-1, 0, 0]))
    o, lse = evs.tree_attention(q, kc, vc, *args, kn, vn, return_lse=True)
    want = ref.tree(q[4:, :, 2:].clone(), kc[4:, 1:, m:], vc[4:, 1:, m:], [500], [[-1, 0, 0]], kn[4:, 1:], vn[4:, 1:])
    check((o[4:, :, 2:], lse[4:, :, 2:]), want, BF16, dh, S)


@pytest.mark.parametrize("case", TREE, ids=tid)
def test_tree_keeps_to_its_workspace(evs, case):
    """The bytes asked for and no others, from lengths of nothing to all of the capacity."""
    import ctypes
    from lossless_speculative_verify_gb300 import _lib
    dtype, T, H, G, dh, S, cached = case
    d = make_tree(T + S, dtype, T, H, G, dh, S, cached)
    B, lib = len(cached), evs.load()
    o, lse = torch.empty_like(d["q"]), torch.empty(B, T, H, device="cuda")
    parents, p = i32(d["parents"]), lambda t: t.data_ptr()  # noqa: E731
    for lens in (cached, [0] * B, [S] * B):
        n_cached = i32(lens)
        a = _lib.TreeAttnArgs(batch=B, nodes=T, heads=H, kv_heads=G, head_dim=dh, dtype=1 if dtype == BF16 else 0,
                              capacity=S, q=p(d["q"]), q_ld=H * dh, k_cache=p(d["kc"]), v_cache=p(d["vc"]),
                              cache_row=dh, cache_head=S * dh, cache_seq=G * S * dh, cache_len=p(n_cached),
                              parents=p(parents), parents_seq=T, k_nodes=p(d["kn"]), v_nodes=p(d["vn"]), node_row=dh,
                              node_head=T * dh, node_seq=G * T * dh, o=p(o), o_ld=H * dh, lse=p(lse))
        n = lib.evs_tree_attention_workspace(ctypes.byref(a))
        ws = torch.full((n + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
        a.workspace, a.ws_bytes = p(ws), n
        assert lib.evs_tree_attention(ctypes.byref(a), None) == 0
        torch.cuda.synchronize()
        assert (ws[n:] == 0x5a).all()
        check((o, lse), want_tree(dict(d, cached=lens)), dtype, dh, S + T)


@pytest.mark.parametrize("dtype,dh,T,H", [(BF16, 128, 128, 2), (BF16, 64, 100, 4), (BF16, 128, 30, 2), (BF16, 64, 7, 2),
                                          (F32, 32, 40, 2), (F32, 16, 5, 2), (BF16, 16, 20, 2)])
@pytest.mark.parametrize("own", [True, False], ids=["nodes", "cache"])
def test_tree_values_that_are_not_finite(evs, dtype, dh, T, H, own):
    """A node's V that is not finite reaches the nodes below it alone."""
    cached = [300, 0, 77]
    d = make_tree(79, dtype, T, H, 1, dh, 300 + T, cached)
    vn = d["vn"]
    if not own:
        for b, m in enumerate(cached):
            d["kc"][b, :, m:m + T], d["vc"][b, :, m:m + T] = d["kn"][b], d["vn"][b]
        d["kn"] = d["vn"] = None
    clean = run_tree(evs, d)
    bad = {0: (1, NAN), T // 2: (dh - 1, math.inf), T - 1: (2, -math.inf), T // 3: (2, math.inf)}
    want, hit = clean[0].float(), torch.zeros_like(clean[0], dtype=torch.bool)
    for b in (0, 1):
        sees = ref.ancestry(d["parents"][b], T).cuda()
        for j, (c, x) in bad.items():
            (vn[b, :, j] if own else d["vc"][b, :, cached[b] + j])[:, c] = x
            want[b, sees[:, j], :, c] += x
            hit[b, sees[:, j], :, c] = True
    o, lse = run_tree(evs, d)
    assert torch.equal(lse, clean[1])
    assert torch.equal(torch.isnan(o), torch.isnan(want)) and torch.equal(torch.isinf(o), torch.isinf(want))
    assert torch.equal(o[torch.isinf(o)].float(), want[torch.isinf(want)])
    assert torch.equal(o[~hit], clean[0][~hit])


def test_tree_refusals(evs):
    d = make_tree(12, BF16, 5, 4, 2, 64, 30, [30, 2])
    q, kc, vc, kn, vn = (d[k] for k in ("q", "kc", "vc", "kn", "vn"))
    n, par = i32(d["cached"]), i32(d["parents"])
    f = evs.tree_attention
    big = torch.zeros(2, 129, 4, 64, dtype=BF16, device="cuda")
    for bad in (lambda: f(q[0], kc, vc, n, par, kn, vn), lambda: f(q, kc[:1], vc, n, par, kn, vn),
                lambda: f(q, kc, vc, n, par, kn), lambda: f(q, kc, vc, None, par, kn, vn),
                lambda: f(q, kc, vc, n.long(), par, kn, vn), lambda: f(q, kc, vc, n, par.long(), kn, vn),
                lambda: f(q, kc, vc, n, par[:, :4], kn, vn), lambda: f(q, kc, vc, n, par.cpu(), kn, vn),
                lambda: f(q, kc, vc, n, None, kn, vn), lambda: f(q, kc, vc, n, par.t().contiguous().t(), kn, vn),
                lambda: f(big, kc, vc, n, torch.zeros(129, dtype=torch.int32, device="cuda")),
                lambda: f(q.float(), kc, vc, n, par, kn, vn), lambda: f(q[:, :, :3], kc, vc, n, par, kn, vn),
                lambda: f(q, kc[:, :, :0], vc[:, :, :0], n, par), lambda: f(q, kc, vc, n, par, kn, vn, lens=n[:1]),
                lambda: f(q, kc, vc, n, par, kn, vn, scale=-1.0), lambda: f(q, kc, vc, n, par, kn, vn, scale=NAN),
                lambda: f(q, kc, vc, n, par, kn[:, :, :4], vn[:, :, :4]), lambda: f(q, kc, vc.transpose(0, 1).contiguous().transpose(0, 1), n, par, kn, vn),
                lambda: f(q, kc, vc, n, par, kn, vn, out=q.float()), lambda: f(q, kc, vc, n, par, kn, vn, out=q[0]),
                lambda: f(q.transpose(1, 2).contiguous().transpose(1, 2), kc, vc, n, par, kn, vn),
                lambda: f(q, kc[:, :, :1].expand(2, 2, 30, 64), vc[:, :, :1].expand(2, 2, 30, 64), n, par, kn, vn),
                lambda: f(q, kc, vc, n, par, kn[:, :, :1].expand(2, 2, 5, 64), vn[:, :, :1].expand(2, 2, 5, 64)),
                lambda: f(q, kc.clone().requires_grad_(), vc, n, par, kn, vn)):
        with pytest.raises(ValueError):
            bad()
    assert f(q[:0], kc[:0], vc[:0], n[:0], par[:0], kn[:0], vn[:0]).shape == (0, 5, 4, 64)


# ---- log probabilities -------------------------------------------------------------------------
def check_logprobs(logits, tokens, temperature, top, got):
    want = ref.logprobs(logits, tokens.tolist(), temperature, top)
    lp, ent, tlp, tid_ = [x.cpu() for x in got]
    V = logits.shape[1]
    for r in range(logits.shape[0]):
        # a weight: the exponent's three roundings and the exponential's four; sums: a thread's own tokens and the
        # tree above them; the given token's own exponent and the difference
        soft = U * (3 * want[4][r] + 4 + V / 256 + 64)
        for have, exp, y in [(lp[r].tolist(), want[0][r], want[6][r]), (tlp[r].tolist(), want[2][r], want[7][r])]:
            for a, b, m in zip(have, exp, y):
                b = -math.inf if b < -torch.finfo(F32).max else b     # past fp32's range, whose nearest is -inf
                assert a == b or abs(a - b) <= soft + U * (4 * m + abs(b)), (r, a, b)
        assert abs(float(ent[r]) - want[1][r]) <= 2 * soft * (1 + want[4][r]) + U * (8 * want[5][r] + 4), (r, float(ent[r]), want[1][r])
        assert tid_[r].tolist() == want[3][r], r


def make_logits(seed, R, V, dtype, ruled=0.1):
    g = gen(seed)
    l = (randn(g, R, V) * 3).to(dtype)
    l[torch.rand(R, V, device="cuda", generator=g) < ruled] = -math.inf
    return l


@pytest.mark.parametrize("V", [1, 2, 3, 31, 64, 255, 512, 1000, 1025, 4097, 16385, 50021, 131072, 262144])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprob_sizes(evs, V, dtype):
    R = 5 if V < 20000 else 2
    l = make_logits(V, R, V, dtype)
    g = gen(V + 1)
    tok = torch.randint(0, V, (R, 3), device="cuda", generator=g, dtype=torch.int32)
    temp = torch.rand(R, device="cuda", generator=g) + 0.3
    for top in {0, 1, min(7, V), min(32, V), min(33, V), min(64, V)}:
        a = evs.token_logprobs(l, tok, temperature=temp, top=top, return_entropy=True)
        b = evs.token_logprobs(l, tok, temperature=temp, top=top, return_entropy=True)
        assert same(a, b)
        if top:
            check_logprobs(l, tok, temp, top, a)
    assert torch.equal(evs.token_logprobs(l, tok, temperature=temp), a[0])
    one = evs.token_logprobs(l, tok[:, 0].contiguous())
    assert one.shape == (R,)
    check_logprobs(l, tok[:, :1], None, 1, [one[:, None]] + evs.token_logprobs(l, tok, top=1, return_entropy=True)[1:])


@pytest.mark.parametrize("R", [1, 3, 75, 152, 153, 304, 700])
def test_logprob_rows(evs, R):
    l = make_logits(R, R, 9001, F32)
    tok = torch.randint(0, 9001, (R, 2), device="cuda", generator=gen(R), dtype=torch.int32)
    check_logprobs(l, tok, None, 5, evs.token_logprobs(l, tok, top=5, return_entropy=True))


@pytest.mark.parametrize("V", [40, 3000, 70001])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprob_ties(evs, V, dtype):
    """Equal logits go by their ids: all alike, a few values, -0 beside +0, the largest in one thread's share."""
    l = torch.zeros(5, V, device="cuda", dtype=dtype)
    l[1] = torch.randint(0, 3, (V,), device="cuda", generator=gen(1)).to(dtype)
    l[2, ::2] = -0.0
    l[3, V // 2:] = 5.0
    l[4] = -4.0
    e = 16 // l.element_size()
    for i in range(40):
        l[4, (256 * e * (i // e) + i % e) % V] = 7.0                  # vectors of the same thread
    tok = i32([[0, V - 1]] * 5)
    for top in (1, 20, min(40, V), min(64, V)):
        check_logprobs(l, tok, None, top, evs.token_logprobs(l, tok, top=top, return_entropy=True))


def test_logprob_sorted_rows(evs):
    """Every token larger than all before it, and the other way."""
    up = torch.arange(20000, device="cuda", dtype=F32) * 0.001
    l = torch.stack([up, up.flip(0)])
    tok = i32([[0, 19999]] * 2)
    check_logprobs(l, tok, None, 64, evs.token_logprobs(l, tok, top=64, return_entropy=True))


@pytest.mark.parametrize("V", [60, 3000, 70001])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprob_infinities_and_temperatures(evs, V, dtype):
    l = make_logits(V, 12, V, dtype)
    l[:, 7] = 1.0
    l[0] = -math.inf                                                  # nothing left
    l[1] = NAN
    l[2, 5] = NAN
    l[3, 11] = l[3, 50] = math.inf
    l[4] = -math.inf
    l[4, 9] = -2.0                                                    # one token left
    l[5] = torch.finfo(dtype).min                                     # the type's lowest value is a value
    l[6, ::3] = torch.finfo(dtype).min
    temp = torch.tensor([1, 1, 1, 1, 1, 1, 1, 0.0, -1.0, NAN, 1e-38, math.inf], device="cuda")
    tok = torch.cat([i32([[7, 11, 5, 9, -1, V, 1 << 30]] * 12)], 1)
    flags = i32([0])
    got = evs.token_logprobs(l, tok, temperature=temp, top=20, return_entropy=True, flags=flags)
    assert flags.item() == 8 | 64
    check_logprobs(l, tok, temp, 20, got)
    flags.zero_()
    evs.token_logprobs(l[2:], tok[2:, :4].contiguous(), flags=flags)
    assert flags.item() == 0


def test_logprob_greedy_without_alternatives(evs):
    l = make_logits(3, 4, 50000, F32)
    tok = torch.stack([l.argmax(-1), l.argmin(-1)], 1).int()
    got = evs.token_logprobs(l, tok, temperature=torch.zeros(4, device="cuda"))
    assert (got[:, 0] == 0).all() and torch.isneginf(got[:, 1]).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprob_strides(evs, dtype):
    """Rows off 16 bytes, rows behind each other with gaps, the same row twice."""
    for V, off, ld in ((1000, 1, 1003), (1001, 3, 1007), (5, 2, 9), (30000, 5, 30011)):
        buf = torch.full((4 * ld + off,), 50.0, device="cuda", dtype=dtype)
        l = buf[off:].as_strided((4, V), (ld, 1))
        l.copy_(make_logits(V, 4, V, dtype))
        tok = i32([[0, V - 1]] * 4)
        top = min(V, 9)
        got = evs.token_logprobs(l, tok, top=top, return_entropy=True)
        check_logprobs(l, tok, None, top, got)
        assert torch.equal(got[3], evs.token_logprobs(l.contiguous(), tok, top=top, return_entropy=True)[3])


def test_logprob_agrees_with_the_draw(evs):
    """What `sample` reports of a token that it drew from the whole distribution."""
    l = make_logits(4, 64, 5000, F32)
    temp = torch.rand(64, device="cuda", generator=gen(5)) + 0.5
    token, lp = evs.sample(l, torch.rand(64, device="cuda", generator=gen(6)), temperature=temp, return_logprob=True)
    got = evs.token_logprobs(l, token, temperature=temp)
    assert float((got - lp).abs().max()) <= 64 * U * 20


def test_logprob_refusals(evs):
    l, tok = make_logits(1, 3, 40, F32), i32([[1, 2]] * 3)
    f = evs.token_logprobs
    for bad in (lambda: f(l[0], tok), lambda: f(l.half(), tok), lambda: f(l.t().contiguous().t(), tok), lambda: f(l, tok[:2]),
                lambda: f(l, tok.long()), lambda: f(l, tok, top=41), lambda: f(l, tok, top=2.0), lambda: f(l, tok, top=-1), lambda: f(l.cpu(), tok),
                lambda: f(torch.zeros(3, 100, device="cuda"), tok, top=65), lambda: f(l, tok.cpu()),
                lambda: f(l, tok, temperature=torch.ones(3, device="cuda").double()), lambda: f(l, tok[:, ::2]),
                lambda: f(l, tok, temperature=torch.ones(2, device="cuda")), lambda: f(l, None),
                lambda: f(l[:1].expand(3, 40), tok), lambda: f(l, tok, flags=i32([[0]])),
                lambda: f(l.clone().requires_grad_(), tok)):
        with pytest.raises(ValueError):
            bad()
    assert f(l[:0], tok[:0]).shape == (0, 2) and f(l, tok[:, :0].contiguous()).shape == (3, 0)


# ---- together ----------------------------------------------------------------------------------
def calls(evs):
    """A call of each operator on fixed inputs, as functions of nothing."""
    p = make_prompt(20, BF16, [300, 41], 4, 2, 128)
    f = make_prompt(21, F32, [100], 2, 2, 16)
    t = make_tree(22, BF16, 40, 8, 2, 128, 500, [500, 77])
    s = make_tree(23, BF16, 1, 8, 2, 64, 900, [900, 0, 5])
    l = make_logits(24, 6, 40000, F32)
    tok = i32([[1, 2, 3]] * 6)
    ps, fs = i32(p["starts"]), i32(f["starts"])
    tc, tp, sc, sp = i32(t["cached"]), i32(t["parents"]), i32(s["cached"]), i32(s["parents"])
    return [lambda: evs.prompt_attention(p["q"], p["k"], p["v"], ps, return_lse=True),
            lambda: evs.prompt_attention(f["q"], f["k"], f["v"], fs, return_lse=True),
            lambda: evs.tree_attention(t["q"], t["kc"], t["vc"], tc, tp, t["kn"], t["vn"], return_lse=True),
            lambda: evs.tree_attention(s["q"], s["kc"], s["vc"], sc, sp, s["kn"], s["vn"], return_lse=True),
            lambda: evs.token_logprobs(l, tok, top=9, return_entropy=True)]


def test_captured_and_on_other_streams(evs):
    todo = calls(evs)
    want = [f() for f in todo]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = [f() for f in todo]
    stream.synchronize()
    assert all(same(a, b) for a, b in zip(want, got))
    # two graphs, each with its own workspaces, replayed beside each other
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([f() for f in todo])
        graphs.append(graph)
    other = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            for ts in o:
                for t in ts:
                    t.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(same(a, b) for a, b in zip(want, o))


def test_calls_of_several_threads(evs):
    """Host threads with streams of their own, the first call of each among them."""
    todo = calls(evs)
    want = [f() for f in todo]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for k in range(8):
                    j = (i + k) % len(todo)
                    if not same(todo[j](), want[j]):
                        wrong.append((i, j))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_inputs_written_just_before(evs):
    """The kernels may start before the ones before them end: they have to wait for their inputs."""
    t = make_tree(30, BF16, 12, 4, 2, 128, 300, [300, 20])
    p = make_prompt(31, BF16, [260], 4, 2, 128)
    l = make_logits(32, 4, 30000, F32)
    cached, parents, starts = i32(t["cached"]), i32(t["parents"]), i32(p["starts"])
    zero_t = {k: torch.zeros_like(t[k]) for k in ("q", "kc", "vc", "kn", "vn")}
    zero_p = {k: torch.zeros(p[k].shape, dtype=BF16, device="cuda") for k in "qkv"}
    c0, s0, l0, par0 = torch.zeros_like(cached), torch.zeros_like(starts), torch.zeros_like(l), torch.full_like(parents, -1)
    tok = i32([[3]] * 4)
    want = [run_tree(evs, t), run_prompt(evs, p), evs.token_logprobs(l, tok, top=4, return_entropy=True)]
    for _ in range(5):
        for k in zero_t:
            zero_t[k].copy_(t[k])
        for k in zero_p:
            zero_p[k].copy_(p[k])
        l0.copy_(l)
        par0.copy_(parents)
        s0.copy_(starts)
        c0.copy_(cached)
        got = [evs.tree_attention(zero_t["q"], zero_t["kc"], zero_t["vc"], c0, par0, zero_t["kn"], zero_t["vn"], return_lse=True),
               evs.prompt_attention(zero_p["q"], zero_p["k"], zero_p["v"], s0, return_lse=True),
               evs.token_logprobs(l0, tok, top=4, return_entropy=True)]
        for z in (*zero_t.values(), *zero_p.values(), l0, s0, c0):
            z.zero_()
        par0.fill_(-1)
        assert all(same(a, b) for a, b in zip(got, want))


def test_gradients_are_refused_and_let_in(evs):
    t = make_tree(33, BF16, 2, 2, 1, 64, 10, [10])
    q = t["q"].clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        run_tree(evs, dict(t, q=q))
    with torch.no_grad():
        assert same(run_tree(evs, dict(t, q=q)), run_tree(evs, t))


def test_a_verify_of_a_tree(evs):
    """Prompts fill the cache, a tree of drafts is attended to, its logits give the drafts' log probabilities and the
    next alternatives: a node's logits are those of the prompt that ends with its path."""
    g = gen(40)
    dm, H, G, dh, V = 256, 4, 2, 64, 997
    w = {k: randn(g, *s) * s[0] ** -0.5 for k, s in dict(embed=(V, dm), qkv=(dm, (H + 2 * G) * dh), o=(H * dh, dm), head=(dm, V)).items()}
    w["embed"] *= V ** 0.5
    lens, T, S = [130, 61], 9, 160
    tokens = torch.randint(0, V, (sum(lens),), device="cuda", generator=g)

    def project(ids):
        x = w["embed"][ids]
        return x, (x @ w["qkv"]).to(BF16).unflatten(-1, (H + 2 * G, dh))

    def logits(x, o):
        return (x + o.float().flatten(-2) @ w["o"]) @ w["head"]

    x, qkv = project(tokens)
    starts = i32([0, 130, 191])
    o = evs.prompt_attention(qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:], starts)
    l = logits(x, o)
    scores, entropy = evs.token_logprobs(l[:-1], tokens[1:].int(), return_entropy=True)
    assert float(scores.max()) <= 0 and float(entropy.min()) >= 0 and float(entropy.max()) <= math.log(V) + 1e-3
    cache = torch.zeros(2, 2, G, S, dh, dtype=BF16, device="cuda")    # K and V of each sequence
    for b, n in enumerate(lens):
        s = int(starts[b])
        cache[0, b, :, :n] = qkv[s:s + n, H:H + G].transpose(0, 1)
        cache[1, b, :, :n] = qkv[s:s + n, H + G:].transpose(0, 1)
    # trees grown from the alternatives: three tokens below the prompt's last, two below each of them
    roots = evs.token_logprobs(l[[129, 190]], tokens[:2].int(), top=3)[-1]
    drafts = torch.cat([roots, torch.randint(0, V, (2, 6), device="cuda", generator=g).int()], 1)
    parents = [-1, -1, -1, 0, 0, 1, 1, 2, 2]
    tx, tqkv = project(drafts.long())
    kn, vn = (t.transpose(1, 2).contiguous() for t in (tqkv[:, :, H:H + G], tqkv[:, :, H + G:]))
    cached = i32(lens)
    to = evs.tree_attention(tqkv[:, :, :H].contiguous(), cache[0], cache[1], cached, i32(parents), kn, vn)
    tl = logits(tx, to)
    children = i32([[3, 4], [5, 6], [7, 8]])
    got = evs.token_logprobs(tl[:, :3].reshape(6, V), drafts[:, children.long().flatten()].reshape(6, 2).contiguous(), top=5)
    for b, n in enumerate(lens):
        for i in range(3):
            path = torch.cat([tokens[int(starts[b]):int(starts[b]) + n], drafts[b, i:i + 1].long()])
            px, pqkv = project(path)
            po = evs.prompt_attention(pqkv[:, :H], pqkv[:, H:H + G], pqkv[:, H + G:], i32([0, n + 1]))
            pl = logits(px, po)[-1]
            want = torch.log_softmax(pl.double(), 0)
            # two bf16 roundings of o, through weights whose rows are of unit size: 2^-8 |o| a logit, a few of it
            assert float((tl[b, i] - pl).abs().max()) <= 0.05
            for j, c in enumerate((3 + 2 * i, 4 + 2 * i)):
                assert abs(float(got[0][b * 3 + i, j]) - float(want[drafts[b, c].long()])) <= 0.1


def test_drawn_cases(evs):
    """Calls over the ranges that serving makes, against plain forms."""
    import importlib.util
    import os
    import random
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    rng = random.Random(7)
    for seed in range(12):
        case = mod.draw(rng)
        st = mod.prepare(case, seed)
        mod.own = False
        want = mod.run(st)
        mod.own = True
        got = mod.run(st)
        for a, b in zip(got, want):
            assert a.shape == b.shape and a.dtype == b.dtype, case
            if a.dtype == torch.int32:
                assert torch.equal(a, b), case
            else:
                # both sides' roundings, of the type and of sums of the values' size
                step = 4 * BF if a.dtype == BF16 else 4096 * U
                assert float((a.double() - b.double()).abs().max()) <= step * (1 + float(b.double().abs().max())), case
        del st, want, got
