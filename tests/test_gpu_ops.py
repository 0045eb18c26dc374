"""The stand-alone operators against their 64-bit definitions (tests/ops_reference.py): sizes at
tile and page edges, ragged and empty lengths, ties, masks, infinities and NaN where nothing may
read them, strides, streams, captured graphs, and a run of all four as a decode step uses them.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of fp32 u = 2^-24."""
import contextlib
import math

import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8


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


# ---- attention ---------------------------------------------------------------------------------
def make_attn(seed, dtype, B, C, T, H, G, dh, P, S, own, block=True):
    g = gen(seed)
    d = dict(q=randn(g, B, C, T, H, dh, dtype=dtype) * 1.5, kp=randn(g, G, P, dh, dtype=dtype),
             vp=randn(g, G, P, dh, dtype=dtype), ko=randn(g, B, G, S, dh, dtype=dtype),
             vo=randn(g, B, G, S, dh, dtype=dtype), own=torch.tensor(own, dtype=torch.int32, device="cuda"))
    d["kb"] = randn(g, B, C, G, T, dh, dtype=dtype) if block else None
    d["vb"] = randn(g, B, C, G, T, dh, dtype=dtype) if block else None
    return d


def run_attn(evs, d, **kw):
    return evs.shared_prefix_attention(d["q"], d["kp"], d["vp"], d["ko"], d["vo"], d["own"], d["kb"], d["vb"],
                                       return_lse=True, **kw)


def check_attn(d, got, dtype, scale=None):
    o, lse = got
    ro, rl, mag, qk = ref.attention(d["q"], d["kp"], d["vp"], d["ko"], d["vo"], d["own"].tolist(), d["kb"], d["vb"],
                                    scale)
    dh = d["q"].shape[-1]
    keys = d["kp"].shape[1] + d["ko"].shape[2] + d["q"].shape[2]
    # scores: a dot product of dh terms in fp32; the exponential's argument and value; sums of all keys
    # (in tiles, so the count is far above what is reached)
    soft = U * ((dh + 4) * qk + keys + 128)
    tol = 2 * soft * mag
    if dtype == torch.bfloat16:      # weights and the output rounded to bf16
        tol = tol + BF * mag + BF * ro.abs()
    err = (o.double() - ro).abs()
    assert torch.isfinite(o.float()).all()
    worst = float((err / (tol + 1e-30)).max())
    assert worst <= 1.0, f"o: {worst:.2f} of the tolerance"
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert float((lse.double() - rl)[~empty].abs().max() if (~empty).any() else 0.0) <= 2 * soft + 4 * U * 16


BF16, F32 = torch.bfloat16, torch.float32
ATTN = [
    # tensor cores, a lane per key tile: one row, odd tails of every kind, empty own rows
    (BF16, 1, 1, 1, 1, 1, 128, 1, 4, [0]),
    (BF16, 2, 1, 1, 4, 4, 128, 127, 130, [0, 130]),
    (BF16, 3, 1, 2, 4, 2, 128, 128, 129, [128, 129, 1]),
    (BF16, 3, 1, 5, 8, 2, 128, 129, 300, [15, 16, 17]),
    (BF16, 8, 1, 1, 8, 8, 128, 4097, 511, [0, 1, 511, 127, 128, 129, 255, 300]),
    (BF16, 8, 1, 16, 2, 2, 64, 1000, 200, [0, 200, 64, 63, 65, 3, 100, 199]),
    (BF16, 5, 1, 1, 8, 1, 64, 2049, 77, [77, 0, 5, 76, 1]),
    # a lane per row tile: 129 to 256 query rows, own rows still few
    (BF16, 3, 2, 11, 6, 3, 128, 777, 260, [0, 260, 131]),
    (BF16, 4, 4, 13, 2, 2, 128, 3001, 400, [0, 399, 400, 129]),
    (BF16, 4, 4, 13, 2, 2, 64, 3001, 400, [0, 399, 400, 129]),
    # several row tiles, own rows above 128 too
    (BF16, 4, 4, 17, 8, 2, 128, 640, 300, [300, 17, 0, 150]),
    (BF16, 2, 4, 40, 4, 1, 64, 130, 513, [513, 1]),
    (BF16, 64, 1, 1, 8, 2, 128, 1025, 150, [(37 * i) % 151 for i in range(64)]),
    # one of the parts missing
    (BF16, 3, 1, 4, 4, 4, 128, 0, 200, [0, 200, 77]),
    (BF16, 3, 2, 4, 4, 4, 128, 500, 0, [0, 0, 0]),
    # CUDA cores: fp32 and narrow heads
    (F32, 1, 1, 1, 1, 1, 16, 1, 1, [0]),
    (F32, 4, 1, 7, 4, 4, 16, 256, 40, [0, 40, 13, 1]),
    (F32, 2, 3, 5, 4, 2, 32, 65, 64, [64, 3]),
    (F32, 3, 1, 2, 8, 4, 64, 700, 129, [129, 0, 64]),
    (F32, 2, 1, 3, 2, 1, 128, 129, 33, [33, 2]),
    (BF16, 3, 1, 3, 4, 2, 16, 130, 65, [0, 65, 64]),
    (BF16, 2, 2, 9, 4, 4, 32, 100, 10, [10, 4]),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c[1:9]) + ("b" if c[0] == BF16 else "f"))
def test_attention_matches_definition(evs, case):
    dtype, B, C, T, H, G, dh, P, S, own = case
    d = make_attn(B * 1000 + P, dtype, B, C, T, H, G, dh, P, S, own)
    a, b = run_attn(evs, d), run_attn(evs, d)
    check_attn(d, a, dtype)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])       # no order left to chance


def attn_args(L, d, **kw):
    """The C entry point's arguments for contiguous tensors; the caller keeps o, lse and the workspace."""
    B, C, T, H, dh = d["q"].shape
    (G, P, _), S = d["kp"].shape, d["ko"].shape[2]
    dt = {BF16: 1, F32: 0}
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    base = dict(batch=B, n_cand=C, block=T, heads=H, kv_heads=G, head_dim=dh, dtype=dt[d["kp"].dtype],
                q_dtype=dt[d["q"].dtype], prefix=P, own_max=S, q=p(d["q"]), q_ld=H * dh, k_prefix=p(d["kp"]),
                v_prefix=p(d["vp"]), prefix_row=dh, prefix_head=P * dh, k_own=p(d["ko"]), v_own=p(d["vo"]), own_row=dh,
                own_head=S * dh, own_seq=G * S * dh, own_len=p(d["own"]), k_block=p(d["kb"]), v_block=p(d["vb"]),
                block_row=dh, block_head=T * dh, block_cand=G * T * dh, o_ld=H * dh)
    base.update(kw)
    return L.SharedAttnArgs(**base)


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c[1:9]) + ("b" if c[0] == BF16 else "f"))
def test_attention_keeps_to_its_workspace(evs, case):
    """The bytes asked for and no others, from lengths of nothing to all of the capacity."""
    import ctypes
    from lossless_speculative_verify_gb300 import _lib
    dtype, B, C, T, H, G, dh, P, S, own = case
    d = make_attn(B * 1000 + P, dtype, B, C, T, H, G, dh, P, S, own)
    o, lse = torch.empty_like(d["q"]), torch.empty(B, C, T, H, device="cuda")
    n = evs.load().evs_shared_attention_workspace(ctypes.byref(attn_args(_lib, d)))
    ws = torch.empty(n + 65536, dtype=torch.uint8, device="cuda")
    args = attn_args(_lib, d, o=o.data_ptr(), lse=lse.data_ptr(), workspace=ws.data_ptr(), ws_bytes=n)
    for lens in (own, [0] * B, [S] * B, [S if b % 3 else 1 for b in range(B)]):
        d["own"].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(0xff)                                               # NaN, where a partial was not written
        assert evs.load().evs_shared_attention(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.all(ws[n:] == 0xff)
        want = run_attn(evs, d)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.isfinite(o.float()).all() or S == 0 and P == 0


@pytest.mark.parametrize("dh,dtype", [(128, BF16), (16, F32)])
@pytest.mark.parametrize("block", [True, False], ids=["block", "cache"])
def test_attention_lengths_that_count_other_rows(evs, dh, dtype, block):
    """own_skip of a length are rows elsewhere; differences that pass 32 bits are clamped to their own side."""
    import ctypes
    from lossless_speculative_verify_gb300 import _lib
    own, S = [0, 100, 37], 120
    d = make_attn(19, dtype, 3, 1, 4, 4, 2, dh, 300, S, own, block=block)
    big = 2 ** 31 - 1
    behind = 0 if block else 1                                       # EVS_FLAG_KV_OVERFLOW: no block rows behind the last
    for skip, lens, plain, flag in ((200, [n + 200 for n in own], own, 0), (-3, [n - 3 for n in own], own, 0),
                                    (5, [-big - 1, 4, 50], [0, 0, 45], 32),
                                    (-5, [big, 40, 0], [S, 45, 5], 32 | behind)):
        want = run_attn(evs, dict(d, own=torch.tensor(plain, dtype=torch.int32, device="cuda")))
        e = dict(d, own=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        o, lse, flags = torch.empty_like(d["q"]), torch.empty(3, 1, 4, 4, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        extra = {} if block else dict(block_row=0, block_head=0, block_cand=0)
        args = attn_args(_lib, dict(e, kb=d["kb"], vb=d["vb"]), own_skip=skip, o=o.data_ptr(), lse=lse.data_ptr(),
                         flags=flags.data_ptr(), **extra)
        n = evs.load().evs_shared_attention_workspace(ctypes.byref(args))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        args.workspace, args.ws_bytes = ws.data_ptr(), n
        assert evs.load().evs_shared_attention(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), (skip, lens)
        assert int(flags) == flag


@pytest.mark.parametrize("dh,dtype", [(128, BF16), (64, BF16), (32, BF16), (16, F32)])
def test_attention_block_rows_in_the_cache(evs, dh, dtype):
    """Without block tensors the block is own rows own_len + j; past the capacity they are left out."""
    d = make_attn(5, dtype, 4, 1, 6, 4, 2, dh, 200, 150, [0, 144, 30, 100], block=False)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attn(d, run_attn(evs, d, flags=flags), dtype)
    assert int(flags) == 0
    d["own"] = torch.tensor([0, 147, 150, 100], dtype=torch.int32, device="cuda")
    check_attn(d, run_attn(evs, d, flags=flags), dtype)
    assert int(flags) == 1                                           # EVS_FLAG_KV_OVERFLOW


def test_attention_scores_of_minus_infinity(evs):
    """Keys whose every score is -inf have no weight; a query that has only such keys gives 0 and lse -inf."""
    for dtype, dh in ((BF16, 128), (BF16, 64), (F32, 16)):
        d = make_attn(6, dtype, 2, 1, 2, 2, 2, dh, 150, 140, [140, 9])
        d["q"] = d["q"].abs() + 0.5
        d["kp"][:, :130] = -math.inf              # the whole first tile and some of the second
        d["ko"][0] = -math.inf
        d["kb"][:, :, :, 0] = -math.inf
        got = run_attn(evs, d)
        # the definition's magnitudes with the weightless keys out of the way
        e = dict(d, kp=d["kp"].clone(), vp=d["vp"], own=d["own"])
        o, lse, mag, _ = ref.attention(d["q"], d["kp"], d["vp"], d["ko"], d["vo"], [140, 9], d["kb"], d["vb"])
        _, _, _, qk = ref.attention(d["q"], e["kp"].nan_to_num(neginf=0.0), d["vp"], d["ko"].nan_to_num(neginf=0.0),
                                    d["vo"], [140, 9], d["kb"].nan_to_num(neginf=0.0), d["vb"])
        soft = U * ((dh + 4) * qk + 292 + 128)
        tol = 2 * soft * mag + (BF * (mag + o.abs()) if dtype == BF16 else 0.0)
        assert torch.all((got[0].double() - o).abs() <= tol)
        assert torch.all((got[1].double() - lse).abs() <= 2 * soft + 64 * U)
        for k in ("kp", "ko", "kb"):
            d[k][:] = -math.inf
        o, lse = run_attn(evs, d)
        assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("dh,dtype", [(128, BF16), (64, BF16), (32, F32)])
def test_attention_reads_nothing_behind_the_lengths(evs, dh, dtype):
    """Rows that no query reads hold NaN and infinities, a prefix tile's neighbours among them."""
    d = make_attn(7, dtype, 4, 1, 3, 4, 2, dh, 131, 300, [0, 1, 137, 300])
    clean = run_attn(evs, d)
    for b, n in enumerate(d["own"].tolist()):
        d["ko"][b, :, n:] = float("nan")
        d["vo"][b, :, n:] = float("nan")
        d["vo"][b, :, n + 1::2] = float("inf")
    big_k = torch.full((2, 400, dh), float("nan"), dtype=dtype, device="cuda")
    big_v = big_k.clone()
    big_k[:, :131], big_v[:, :131] = d["kp"], d["vp"]
    d["kp"], d["vp"] = big_k[:, :131], big_v[:, :131]
    dirty = run_attn(evs, d)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("dh", [64, 128])
def test_attention_partials_without_a_value(evs, dh):
    """A partial (m, l) = (-inf, NaN), which a row of NaN scores leaves and a kernel that gave up a wait writes,
    makes its row NaN among any number of sound partials, first, last or between them; the other rows stay sound."""
    P, S = 40000, 300                                                # partials of many runs
    d = make_attn(18, BF16, 3, 2, 2, 4, 2, dh, P, S, [300, 0, 129])
    clean = run_attn(evs, d)
    for at in (0, 20000, P - 1):
        e = dict(d, kp=d["kp"].clone())
        e["kp"][0, at] = float("nan")                                # one K/V head of two
        o, lse = run_attn(evs, e)
        assert torch.isnan(o[:, :, :, :2].float()).all() and torch.isnan(lse[:, :, :, :2]).all()
        assert torch.equal(o[:, :, :, 2:], clean[0][:, :, :, 2:]) and torch.equal(lse[:, :, :, 2:], clean[1][:, :, :, 2:])
    e = dict(d, ko=d["ko"].clone())
    e["ko"][2, 1, 128] = float("nan")                                # the last own row of one sequence
    o, lse = run_attn(evs, e)
    assert torch.isnan(o[2, :, :, 2:].float()).all() and torch.isnan(lse[2, :, :, 2:]).all()
    assert torch.equal(o[:2], clean[0][:2]) and torch.equal(o[2, :, :, :2], clean[0][2, :, :, :2])


def test_attention_values_that_propagate(evs):
    """A NaN or infinity in a readable row does reach the queries that read it, and no others."""
    for dtype, dh in ((BF16, 128), (F32, 32)):
        d = make_attn(8, dtype, 3, 1, 2, 2, 1, dh, 200, 140, [140, 20, 0])
        d["ko"][0, 0, 139] = float("nan")
        d["vo"][1, 0, 3, 5] = float("inf")
        o, lse = run_attn(evs, d)
        assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
        assert torch.isinf(o[1, ..., 5].float()).all() and torch.isfinite(o[1, ..., :5].float()).all()
        assert torch.isfinite(o[2].float()).all()


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_attention_strides(evs, dtype, dh):
    """Token-major K/V, padded rows, a q inside a wider projection, out of the caller's."""
    B, C, T, H, G, P, S = 3, 2, 4, 4, 2, 150, 140
    d = make_attn(9, dtype, B, C, T, H, G, dh, P, S, [0, 140, 70])
    want = run_attn(evs, d)
    e = dict(d)
    for k in ("kp", "vp"):
        e[k] = d[k].transpose(0, 1).contiguous().transpose(0, 1)
    for k in ("ko", "vo"):
        wide = torch.zeros(B, S, G, dh + 8, dtype=dtype, device="cuda")
        wide[..., :dh] = d[k].transpose(1, 2)
        e[k] = wide[..., :dh].transpose(1, 2)
    proj = torch.zeros(B, C, T, 3 * H * dh, dtype=dtype, device="cuda")
    proj[..., :H * dh] = d["q"].flatten(3)
    e["q"] = proj[..., :H * dh].unflatten(3, (H, dh))
    out = torch.full((B, C, T, H, dh), 7.0, dtype=dtype, device="cuda")
    o, lse = run_attn(evs, e, out=out)
    assert o.data_ptr() == out.data_ptr()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # rows that do not start on 16 bytes take the other kernel, to the same tolerance
    odd = torch.zeros(G * P * dh + 1, dtype=dtype, device="cuda")
    odd[1:] = d["kp"].flatten()
    e["kp"] = odd[1:].view(G, P, dh)
    e["vp"] = d["vp"].contiguous()
    check_attn(d, run_attn(evs, e), dtype)
    odd_q = torch.zeros(d["q"].numel() + 1, dtype=dtype, device="cuda")
    odd_q[1:] = d["q"].flatten()
    f = dict(d, q=odd_q[1:].view(d["q"].shape))
    got = run_attn(evs, f)
    assert torch.equal(got[0], want[0])


def test_attention_fp32_queries(evs):
    d = make_attn(10, BF16, 3, 1, 4, 8, 2, 128, 300, 100, [0, 100, 50])
    want = run_attn(evs, d)
    got = run_attn(evs, dict(d, q=d["q"].float()))
    # the same bf16 queries; the block rows' scores are fp32 sums of the same products
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_attn(d, run_attn(evs, d, scale=0.25), BF16, scale=0.25)


@pytest.mark.parametrize("dh", [16, 32, 64, 128])
def test_attention_fp32_queries_are_rounded_to_the_cache(evs, dh):
    """fp32 queries that are no bf16 values give what the rounded ones give, bit for bit: of prefix, own and block
    rows, block rows in the cache, rows on 16 bytes and off them."""
    for block in (True, False):
        d = make_attn(16, BF16, 3, 1, 4, 8, 2, dh, 300, 100, [0, 90, 50], block=block)
        q = randn(gen(17), 3, 1, 4, 8, dh) * 1.5
        odd = dict(d)
        for k in ("kp", "vp"):
            wide = torch.zeros(d[k].numel() + 1, dtype=BF16, device="cuda")
            wide[1:] = d[k].flatten()
            odd[k] = wide[1:].view(d[k].shape)
        for e in (d, odd):
            got, want = run_attn(evs, dict(e, q=q)), run_attn(evs, dict(e, q=q.to(BF16)))
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            check_attn(dict(e, q=q.to(BF16)), got, BF16)


def test_attention_lengths_out_of_range(evs):
    for dtype, dh in ((BF16, 128), (F32, 16)):
        d = make_attn(11, dtype, 3, 1, 2, 2, 2, dh, 140, 60, [0, 60, 7])
        want = run_attn(evs, d)
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_attn(evs, dict(d, own=torch.tensor([-5, 61, 7], dtype=torch.int32, device="cuda")), flags=flags)
        assert int(flags) == 32                                      # EVS_FLAG_BAD_LEN
        assert torch.equal(got[0], want[0])


def test_attention_offsets_past_32_bits(evs):
    """The last sequence's own rows start more than 2^31 elements into the cache."""
    B, G, S, dh = 3, 2, 4_300_000, 128
    assert (B - 1) * G * S * dh > 2 ** 31
    ko = torch.empty(B, G, S, dh, dtype=BF16, device="cuda")
    vo = torch.empty_like(ko)
    own = [100, 0, 290]
    g = gen(12)
    d = make_attn(12, BF16, B, 1, 1, 4, G, dh, 300, 1, [0, 0, 0])
    for b, n in enumerate(own):
        ko[b, :, :n] = randn(g, G, n, dh, dtype=BF16)
        vo[b, :, :n] = randn(g, G, n, dh, dtype=BF16)
    d.update(ko=ko, vo=vo, own=torch.tensor(own, dtype=torch.int32, device="cuda"))
    got = run_attn(evs, d)
    d.update(ko=ko[:, :, :300].contiguous(), vo=vo[:, :, :300].contiguous())
    check_attn(d, got, BF16)
    del ko, vo


def test_attention_captured_and_on_another_stream(evs):
    """Two captured graphs of different sizes replayed in turn, lengths changed between replays."""
    big = make_attn(13, BF16, 4, 4, 13, 2, 2, 128, 1000, 300, [0, 300, 20, 129])
    small = make_attn(14, BF16, 2, 1, 1, 4, 2, 64, 513, 100, [7, 100])
    want = [run_attn(evs, big), run_attn(evs, small)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run_attn(evs, big)
    side.synchronize()
    assert torch.equal(other[0], want[0][0])
    graphs, outs = [], []
    for d in (big, small):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run_attn(evs, d))
        graphs.append(gr)
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    big["own"].copy_(torch.tensor([17, 0, 300, 5], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_attn(big, outs[0], BF16)


def test_attention_many_rows_of_a_head(evs):
    """64 candidates x 128 positions x 32 heads of one K/V head: 65536 groups of four rows to combine."""
    g = gen(77)
    C, T, H, dh = 64, 128, 32, 128
    q = randn(g, 1, C, T, H, dh, dtype=BF16)
    kp, vp = (randn(g, 1, 200, dh, dtype=BF16) for _ in range(2))
    ko, vo = (randn(g, 1, 1, 8, dh, dtype=BF16) for _ in range(2))
    kb, vb = (randn(g, 1, C, 1, T, dh, dtype=BF16) for _ in range(2))
    own = torch.tensor([5], dtype=torch.int32, device="cuda")
    out, lse = evs.shared_prefix_attention(q, kp, vp, ko, vo, own, kb, vb, return_lse=True)
    for c, t, h in ((0, 0, 0), (0, 127, 31), (31, 64, 7), (63, 0, 31), (63, 127, 31)):
        k = torch.cat([kp[0], ko[0, 0, :5], kb[0, c, 0, :t + 1]]).double()
        v = torch.cat([vp[0], vo[0, 0, :5], vb[0, c, 0, :t + 1]]).double()
        s = (k @ q[0, c, t, h].double()) / math.sqrt(dh)
        p = torch.softmax(s, 0)
        # as in check_attn
        qk = float((k.abs() @ q[0, c, t, h].double().abs()).max()) / math.sqrt(dh)
        soft = U * ((dh + 4) * qk + len(k) + 128)
        tol = (2 * soft + BF) * (p @ v.abs()) + BF * (p @ v).abs()
        assert torch.all((out[0, c, t, h].double() - p @ v).abs() <= tol)
        assert abs(float(lse[0, c, t, h]) - float(torch.logsumexp(s, 0))) <= 2 * soft + 4 * U * 16


def test_attention_refusals(evs):
    d = make_attn(15, BF16, 2, 1, 2, 4, 2, 64, 20, 10, [1, 2])
    for bad in (dict(q=d["q"].half()), dict(q=d["q"][..., :32]), dict(kp=d["kp"].float()), dict(vp=d["vp"][:, :10]),
                dict(ko=d["ko"][:1]), dict(own=d["own"].long()), dict(own=d["own"].cpu()), dict(kb=None),
                dict(q=d["q"].transpose(1, 2)), dict(vo=d["vo"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(own=None)):
        with pytest.raises(ValueError):
            run_attn(evs, {**d, **bad})
    with pytest.raises(ValueError):
        run_attn(evs, d, scale=0.0)
    with pytest.raises(ValueError):
        run_attn(evs, d, out=torch.empty_like(d["q"]).float())


# ---- the draw ------------------------------------------------------------------------------------
def check_draw(evs, logits, u, probs=True, **kw):
    """Tokens equal the definition's; logprob and probabilities to fp32 (their sums are exact to 2e-10)."""
    R, V = logits.shape
    out = evs.sample(logits, u, return_logprob=True, return_probs=probs, **kw)
    host = logits.float().cpu().numpy()
    par = {k: v.cpu().numpy() for k, v in kw.items() if v is not None and k != "flags"}
    tok, lp = out[0].cpu().numpy(), out[1].cpu().numpy()
    pr = out[2].cpu().numpy() if probs else None
    for r in range(R):
        p = {k: (int(v[r]) if k == "top_k" else float(v[r])) for k, v in par.items()}
        wt, wl, wp = ref.draw_row(host[r], float(u[r]), **p)
        assert tok[r] == wt, (r, tok[r], wt, p)
        if math.isinf(wl):
            assert lp[r] == wl
        else:
            # logit difference and quotient 2, the log's argument 1.5 and value 2, the sum 1 (both terms are
            # negative); weights below 2^-45 of the largest are left out of the total
            assert abs(lp[r] - wl) <= 5 * U * abs(wl) + 1e-9
        if probs:
            # four roundings (the sum of a table entry and its tail, the total, 1 over it, the product) and one of a term
            # of at most 0.011; weights below 2^-45 of the largest are none
            assert np.all(np.abs(pr[r] - wp) <= 4.05 * U * wp + 2.0 ** -44), r
    return out


def col(R, v, dtype=torch.float32):
    return torch.tensor([v] * R if not isinstance(v, (list, tuple)) else list(v), dtype=dtype, device="cuda")


def make_logits(seed, R, V, dtype=torch.float32, masked=0.0, spread=2.0):
    g = gen(seed)
    l = randn(g, R, V) * spread
    if masked:
        l = l.masked_fill(torch.rand(R, V, device="cuda", generator=g) < masked, -math.inf)
        l[:, V // 2] = 0.5
    return l.to(dtype), torch.rand(R, device="cuda", generator=g)


@pytest.mark.parametrize("V", [1, 2, 31, 512, 1000, 1024, 1025, 2048, 2049, 4097, 16385, 40001, 131072, 262144])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_sample_sizes_and_filters(evs, V, dtype):
    R = 8 if V <= 5000 else 5
    l, u = make_logits(V, R, V, dtype, masked=0.1 if V > 2 else 0.0)
    t = col(R, [0.7, 1.0, 0.0, 1.5, 0.05, 3.0, 1.0, 0.9][:R])
    check_draw(evs, l, u)
    check_draw(evs, l, u, temperature=t)
    for k in (1, 7, 50, 1500):
        check_draw(evs, l, u, probs=False, temperature=t, top_k=col(R, k, torch.int32))
    check_draw(evs, l, u, probs=False, temperature=t, top_p=col(R, 0.9))
    check_draw(evs, l, u, temperature=t, top_k=col(R, 40, torch.int32), top_p=col(R, 0.8), min_p=col(R, 0.02))
    check_draw(evs, l, u, probs=False, temperature=t, top_k=col(R, 3000, torch.int32), top_p=col(R, 0.97))
    check_draw(evs, l, u, probs=False, min_p=col(R, 0.1))


@pytest.mark.parametrize("R", [1, 3, 152, 700])
def test_sample_rows(evs, R):
    """Cluster sizes follow the rows and the vocabulary."""
    for V in (300, 9000, 33000):
        l, u = make_logits(R + V, R, V)
        check_draw(evs, l, u, probs=False, top_p=col(R, 0.95), top_k=col(R, 100, torch.int32))


def test_sample_cut_among_close_logits(evs):
    """Every row of many: the mass above a bin and the tokens in it have to belong to the same bins."""
    for V, R, spread in ((60000, 96, 2.0), (200000, 24, 1.0), (5000, 200, 0.3)):
        l, u = make_logits(V + 5, R, V, spread=spread)
        t = col(R, [0.5 + 0.01 * i for i in range(R)])
        check_draw(evs, l, u, temperature=t, top_p=col(R, [0.05 + 0.9 * i / R for i in range(R)]))
        check_draw(evs, l, u, probs=False, temperature=t, top_k=col(R, 2000, torch.int32), top_p=col(R, 0.6))


def test_sample_equal_but_for_a_last_bit(evs):
    """The largest vocabulary off the 16-byte grid, all weights of a bin one step below the largest."""
    V = 1 << 18
    wide = torch.full((2, V + 3), 1.0 - 2.0 ** -24, device="cuda")
    l = wide[:, 1:V + 1]
    l[:, 1000] = 1.0
    u = torch.tensor([0.3, 0.999], device="cuda")
    for t in (600.0, 300.0, 40.0):
        check_draw(evs, l, u, probs=False, temperature=col(2, t), top_p=col(2, [0.3, 0.7]))


def test_sample_border_at_the_end_of_a_crowded_bin(evs):
    """top-p's border on the last units of 2^-45 of a step of 1/32 in the exponent that holds 3360 tokens whose
    logits spread over 1120 binary orders and quarters: what each of these rounds off must not lose the border.

    Row: one token of weight 1; the crowd A; B of as much mass as both, two of its tokens tuned
    row by row; top_p = 1/2. The tuned mass at which the kernel first keeps one of B is found by refinement; below
    it, in steps of 40 units over the 1120 that could be lost, every row keeps exactly the first token and A."""
    T, p, unit = 64.0, 0.5, 2.0 ** -45
    step = math.log(2.0) / 32.0 * T
    top = np.float32(33 * step)                                      # A, around 0, is in step 33 below the largest
    mags = np.array([2.0 ** -e * (1.0 + q / 4.0 + 0.03 * j) for e in range(2, 142) for q in range(4) for j in range(3)],
                    np.float32)
    a = np.sort(np.concatenate([mags, -mags]))[::-1]
    assert np.all(np.abs(a) < 0.45 * step) and a.size == 3360
    weight = lambda l: np.exp((np.asarray(l, np.float64) - float(top)) / T)  # noqa: E731
    want = 1.0 + weight(a).sum()
    b, left = [], want - 2.0 ** -18 * 1.5
    for depth in range(40, 19 * 32, 8):                              # 2^-1.25 .. 2^-19 of the largest
        l = np.float32(float(top) - depth * step)
        n = min(int(left / weight(l)), 4000)
        b += [l] * n
        left -= n * float(weight(l))
    assert 0 <= left < 2.0 ** -18
    fixed = np.concatenate([[top], a, np.array(b, np.float32)])

    def kept(extra):
        """Kept tokens where B has `extra` (an array) more than `left` + 2^-18, as two tokens each."""
        mass = extra + left + 2.0 ** -18 * 1.5
        coarse = (float(top) + T * np.log(mass * (1.0 - 2.0 ** -12))).astype(np.float32)
        fine = (float(top) + T * np.log(mass - weight(coarse))).astype(np.float32)
        rows = np.tile(fixed, (len(extra), 1))
        l = torch.from_numpy(np.concatenate([rows, coarse[:, None], fine[:, None]], 1)).cuda()
        n = len(extra)
        _, probs = evs.sample(l, torch.full((n,), 0.5, device="cuda"), temperature=col(n, T), top_p=col(n, p),
                              return_probs=True)
        return (probs > 0).sum(1).cpu().numpy()

    first = 1 + a.size
    lo, hi = -2.0 ** -19, 2.0 ** -19
    while hi - lo > 16 * unit:                                       # kept(lo) <= first < kept(hi)
        grid = np.linspace(lo, hi, 66)
        over = np.flatnonzero(kept(grid) > first)
        assert over.size and over[0] > 0
        lo, hi = grid[over[0] - 1], grid[over[0]]
    below = kept(lo - 2.0 * unit * np.arange(0, 1200, 40))
    assert np.all(below == first), below


@pytest.mark.parametrize("V,R", [(301, 512), (3000, 512), (20000, 64)])
def test_sample_tokens_on_the_border_of_a_bin(evs, V, R):
    """300 neighbouring floats around a border between two steps of 1/32 in the exponent, top-p's cut among the
    later ones: whichever step a token is counted in has to be the one that it is ranked in."""
    rng = np.random.default_rng(V)
    n, cut = 300, 225
    rows = np.full((R, V), -np.inf, np.float32)
    t = (0.6 + 0.8 * rng.random(R)).astype(np.float32)
    p = np.empty(R, np.float32)
    for r in range(R):
        top = np.float32(3.0 + 5.0 * rng.random())
        per = math.log(2.0) / 32.0 * float(t[r])                     # logits of a step
        mid = np.float32(float(top) - (rng.integers(20, 200) + 0.5) * per)
        l = (mid.view(np.int32) + np.arange(n, dtype=np.int32) - n // 2).view(np.float32)
        assert np.all(np.abs(l - mid) < per / 4) and len(set(l.tolist())) == n
        l = np.sort(l)[::-1]
        w = np.exp((l.astype(np.float64) - float(top)) / float(t[r]))
        # in the middle of token `cut`: half a token's mass, 1 / 800 of all at least, is 10^4 roundings of p
        p[r] = (1.0 + w[:cut].sum() + 0.5 * w[cut]) / (1.0 + w.sum())
        at = rng.permutation(V)[:n + 1]
        rows[r, at[0]], rows[r, at[1:]] = top, l
    _, probs = evs.sample(torch.from_numpy(rows).cuda(), torch.full((R,), 0.5, device="cuda"),
                          temperature=torch.from_numpy(t).cuda(), top_p=torch.from_numpy(p).cuda(), return_probs=True)
    kept = (probs > 0).sum(1).cpu().numpy()
    assert np.all(kept == 1 + cut + 1), np.bincount(kept)[cut:]


def test_sample_ties(evs):
    """Equal logits go by their ids: cuts inside one value shared by many more tokens than are ranked at once."""
    for V, levels in ((3000, 1), (50021, 1), (50021, 3), (131072, 2), (131072, 40)):
        g = gen(V + levels)
        l = torch.randint(0, levels, (4, V), device="cuda", generator=g).float() * 0.5
        u = torch.rand(4, device="cuda", generator=g)
        for dtype in (F32, BF16):
            x = l.to(dtype)
            check_draw(evs, x, u, probs=False, top_k=col(4, [1, 1023, 1025, 2500], torch.int32))
            check_draw(evs, x, u, probs=False, top_p=col(4, [0.001, 0.3, 0.7, 0.999]))
            check_draw(evs, x, u, probs=False, top_k=col(4, 2000, torch.int32), top_p=col(4, [0.001, 0.3, 0.7, 0.999]))
            check_draw(evs, x, torch.zeros(4, device="cuda"), probs=False, temperature=col(4, 0.0))
    zeros = torch.zeros(2, 5000, device="cuda")
    zeros[:, ::2] = -0.0                                              # one value, not two
    check_draw(evs, zeros, torch.tensor([0.2, 0.9], device="cuda"), top_k=col(2, 7, torch.int32))


def test_sample_parameters_at_their_edges(evs):
    l, u = make_logits(3, 10, 3000)
    nan = float("nan")
    # off: outside [1, vocab), at or above 1 or NaN, at or below 0
    base = evs.sample(l, u)
    for kw in (dict(top_k=col(10, [0, -1, 3000, 3001, 2 ** 31 - 1, -2 ** 31, 0, 0, 0, 0], torch.int32)),
               dict(top_p=col(10, [1.0, 2.0, nan, float("inf"), 1.0, 1.0, 1.0, 1.0, 1.0, 1.0])),
               dict(min_p=col(10, [0.0, -1.0, nan, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]))):
        assert torch.equal(evs.sample(l, u, **kw), base)
    top = l.argmax(-1).int()
    for kw in (dict(top_p=col(10, 0.0)), dict(top_p=col(10, -1.0)), dict(top_k=col(10, 1, torch.int32)),
               dict(min_p=col(10, 1.0)), dict(min_p=col(10, 7.0)), dict(temperature=col(10, 0.0)),
               dict(temperature=col(10, -1.0)), dict(temperature=col(10, nan)), dict(temperature=col(10, 1e-42)),
               dict(temperature=col(10, 1e-8))):
        assert torch.equal(evs.sample(l, u, **kw), top), kw
    # a temperature without bound makes the draw uniform
    flat = evs.sample(l, u, temperature=col(10, float("inf")))
    assert torch.equal(flat, (u.double() * 3000).floor().int())
    # uniforms at and outside the ends: the first and the last token with any mass
    m = l.clone()
    m[:, :5] = -math.inf
    m[:, -7:] = -math.inf
    ends = torch.tensor([0.0, -3.0, nan, 1.0, 5.0, float("inf"), 1.0 - 2.0 ** -24, 2.0 ** -30, 0.0, 1.0], device="cuda")
    got = evs.sample(m, ends, temperature=col(10, 1000.0)).tolist()
    assert got[0] == got[1] == got[2] == 5 and got[3] == got[4] == got[5] == 3000 - 8
    assert got[6] == 3000 - 8 and got[7] == 5


@pytest.mark.parametrize("V", [600, 3000, 70001])
def test_sample_infinities_and_nan(evs, V):
    l, u = make_logits(V, 8, V)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    l[0, ::3] = float("nan")                      # ruled out
    l[1, ::2] = -math.inf
    l[2] = torch.finfo(F32).min                   # a mask of the type's lowest value, everywhere
    l[3, : V - 1] = torch.finfo(F32).min          # and everywhere but for one
    l[4, 5] = l[4, V - 2] = math.inf              # the infinite ones share the mass
    l[5] = -math.inf
    l[5, 17] = -3.0                               # a single token left
    l[6] = torch.finfo(F32).max
    for kw in (dict(), dict(top_k=col(8, 20, torch.int32), top_p=col(8, 0.9)), dict(top_p=col(8, 0.5)),
               dict(min_p=col(8, 0.3), temperature=col(8, 0.6))):
        check_draw(evs, l, u, flags=flags, **kw)
    assert int(flags) == 0
    l[7] = -math.inf                              # nothing left: no draw
    l[0] = float("nan")
    for kw in (dict(), dict(top_p=col(8, 0.5)), dict(temperature=col(8, 0.0))):
        out = check_draw(evs, l, u, flags=flags, **kw)
        assert out[0][7] == -1 and out[0][0] == -1 and int(flags) == 64


def test_sample_draws_the_distribution(evs):
    """Over a fine grid of uniforms every kept token is drawn as often as its share says."""
    l, _ = make_logits(21, 1, 700)
    n = 20000
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    big = l.expand(n, 700)
    with pytest.raises(ValueError):
        evs.sample(big, u)                        # rows that lie on one another
    tok, probs = evs.sample(big.contiguous(), u, top_p=col(n, 0.9), return_probs=True)
    share = torch.bincount(tok.long(), minlength=700).double() / n
    assert float((share - probs[0].double()).abs().max()) <= 2.0 / n       # the two ends of an interval
    assert torch.all(share[probs[0] > 1.01 / n] > 0) and torch.all(probs[0][share > 0] > 0)


def test_sample_strides_and_streams(evs):
    l, u = make_logits(22, 6, 1001)
    want = evs.sample(l, u, top_p=col(6, 0.9))
    for dtype in (F32, BF16):
        w = evs.sample(l.to(dtype), u, top_p=col(6, 0.9))
        for off in (0, 1, 3):
            wide = torch.full((6, 1500), 100.0, device="cuda", dtype=dtype)     # neighbours that would win
            wide[:, off:off + 1001] = l
            assert torch.equal(evs.sample(wide[:, off:off + 1001], u, top_p=col(6, 0.9)), w)
    gr = torch.cuda.CUDAGraph()
    p = col(6, 0.9)
    with torch.cuda.graph(gr):
        tok = evs.sample(l, u, top_p=p)
    l2, u2 = make_logits(23, 6, 1001)
    want2 = evs.sample(l2, u2, top_p=p)
    l.copy_(l2)
    u.copy_(u2)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, want2) and not torch.equal(want, want2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = evs.sample(l, u, top_p=p)
    side.synchronize()
    assert torch.equal(got, want2)
    assert evs.sample(l[:0], u[:0]).shape == (0,)


FIRST_CALL = """
import torch, lossless_speculative_verify_gb300 as evs
g = torch.Generator(device="cuda").manual_seed(1)
for dtype in (torch.float32, torch.bfloat16):
    for rows, vocab in ((200, 7000), (30, 14000)):
        l = torch.randn(rows, vocab, device="cuda", generator=g).to(dtype)
        u = torch.rand(rows, device="cuda", generator=g)
        got = evs.sample(l, u, top_p=torch.full((rows,), 0.9, device="cuda"))
        wide = torch.full((rows, 40000), -float("inf"), device="cuda", dtype=dtype)
        wide[:, :vocab] = l
        assert torch.equal(evs.sample(wide, u, top_p=torch.full((rows,), 0.9, device="cuda")), got), (dtype, vocab)
print("done")
"""


def test_sample_first_call_of_a_process(evs):
    """Slices of 7000 logits need 48 KB of shared memory with the kernel's own: the first call of each instance in a
    process, before a larger one has raised its limit (then alike rows in a wider vocabulary)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-1500:]


def test_sample_refusals(evs):
    l, u = make_logits(24, 4, 100)
    for a, kw in (((l.half(), u), {}), ((l.t(), u), {}), ((l, u[:3]), {}), ((l, u.double()), {}), ((l, None), {}),
                  ((l, u.cpu()), {}), ((l, u), dict(top_k=col(4, 5))), ((l, u), dict(top_p=col(3, 0.5))),
                  ((l, u), dict(temperature=1.0)), ((l, u), dict(out=torch.empty(4, device="cuda"))),
                  ((torch.zeros(1, (1 << 18) + 1, device="cuda"), u[:1]), {}), ((l[0], u), {})):
        with pytest.raises(ValueError):
            evs.sample(*a, **kw)


def test_inputs_written_just_before(evs):
    """Each operator right behind the kernels that write its inputs, over and over, eagerly and in a graph."""
    n = 12
    ds = [make_attn(900 + i, BF16, 4, 2, 5, 4, 2, 128, 300, 40, [0, 40, 17, 3]) for i in range(n)]
    ls = [make_logits(950 + i, 6, 9000) for i in range(n)]
    ss = [make_scan(970 + i, 2, 24, 96, 16, BF16) for i in range(n)]
    w = randn(gen(1), 96, 4)
    p = col(6, 0.9)

    def run(d, l, s):
        y = evs.causal_conv(s["x"], w)
        z = evs.selective_scan(y, s["dt"], s["A"], s["B"], s["C"])
        return [*run_attn(evs, d), evs.sample(*l, top_p=p), y, z]

    want = []
    for d, l, s in zip(ds, ls, ss):
        want.append(run(d, l, s))
        torch.cuda.synchronize()
    d, l, s = ({k: v.clone() for k, v in ds[0].items()}, [v.clone() for v in ls[0]], {k: v.clone() for k, v in ss[0].items()})

    def chain():
        out = []
        for dn, ln, sn in zip(ds, ls, ss):
            for k, v in dn.items():
                d[k].copy_(v)
            for a, b in zip(l, ln):
                a.copy_(b)
            for k, v in sn.items():
                s[k].copy_(v)
            out.append(run(d, l, s))
        return out

    eager = chain()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        captured = chain()
    gr.replay()
    gr.replay()
    torch.cuda.synchronize()
    for got in (eager, captured):
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_first_call_of_a_thread(evs):
    """Each operator as the first use of the device that a host thread makes, through its C entry point."""
    import ctypes
    import threading
    from lossless_speculative_verify_gb300 import _lib
    lib, p = evs.load(), lambda t: t.data_ptr()  # noqa: E731
    d, s = make_attn(65, BF16, 2, 1, 2, 2, 2, 128, 300, 40, [40, 3]), make_scan(66, 1, 3, 64, 16, F32)
    l, u = make_logits(67, 2, 9000)
    o, y, z, w = torch.empty_like(d["q"]), torch.empty_like(s["x"]), torch.empty_like(s["x"]), randn(gen(68), 64, 4)
    tok = torch.empty(2, dtype=torch.int32, device="cuda")
    n = lib.evs_shared_attention_workspace(ctypes.byref(attn_args(_lib, d)))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    calls = [("evs_shared_attention", attn_args(_lib, d, o=p(o), workspace=p(ws), ws_bytes=n)),
             ("evs_sample", _lib.SampleArgs(rows=2, vocab=9000, dtype=0, ld=9000, logits=p(l), uniforms=p(u), token=p(tok))),
             ("evs_causal_conv", _lib.ConvArgs(batch=1, tokens=3, width=64, taps=4, dtype=0, silu=1, x=p(s["x"]), x_ld=64,
                                               x_seq=192, y=p(y), y_ld=64, y_seq=192, weight=p(w))),
             ("evs_selective_scan", _lib.ScanArgs(
                 batch=1, tokens=3, width=64, states=16, dtype=0, softplus=1, x=p(s["x"]), x_ld=64, x_seq=192, dt=p(s["dt"]),
                 dt_ld=64, dt_seq=192, B=p(s["B"]), b_ld=16, b_seq=48, C=p(s["C"]), c_ld=16, c_seq=48, y=p(z), y_ld=64,
                 y_seq=192, A=p(s["A"])))]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, args in calls:
        status = []
        t = threading.Thread(target=lambda: status.append(getattr(lib, name)(ctypes.byref(args), stream.cuda_stream)))
        t.start()
        t.join()
        assert status == [0], name
    torch.cuda.synchronize()
    assert torch.equal(o, run_attn(evs, d)[0]) and torch.equal(tok, evs.sample(l, u))
    assert torch.equal(y, evs.causal_conv(s["x"], w))
    assert torch.equal(z, evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"]))


def test_calls_of_several_threads(evs):
    """Threads with a stream each call one kernel instance with little and with much shared memory at once: no call
    takes from another what it asked for. And a captured large call replays after small ones."""
    import ctypes
    import threading
    from lossless_speculative_verify_gb300 import _lib
    lib, jobs, keep = evs.load(), [], []
    for rows, vocab in ((30, 14000), (1, 131072), (2, 262144)):
        l, u = make_logits(vocab, rows, vocab)
        p, tok = col(rows, 0.9), torch.empty(rows, dtype=torch.int32, device="cuda")
        want = evs.sample(l, u, top_p=p)
        jobs.append((lib.evs_sample, _lib.SampleArgs(
            rows=rows, vocab=vocab, dtype=0, ld=vocab, logits=l.data_ptr(), uniforms=u.data_ptr(), top_p=p.data_ptr(),
            token=tok.data_ptr()), tok, want))
        keep.append((l, u, p))
    for B in (1, 40, 300):
        d = make_attn(64, BF16, B, 1, 1, 2, 2, 128, 300, 40, [i % 41 for i in range(B)])
        o = torch.empty_like(d["q"])
        n = lib.evs_shared_attention_workspace(ctypes.byref(attn_args(_lib, d)))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        jobs.append((lib.evs_shared_attention, attn_args(_lib, d, o=o.data_ptr(), workspace=ws.data_ptr(), ws_bytes=n), o,
                     run_attn(evs, d)[0]))
        keep.append((d, ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    failed = [0] * len(jobs)

    def work(k):
        fn, args, _, _ = jobs[k]
        for i in range(6000):
            failed[k] += fn(ctypes.byref(args), streams[k].cuda_stream) != 0
            if i % 100 == 0:
                streams[k].synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(jobs)
    assert all(torch.equal(got, want) for _, _, got, want in jobs)
    (l1, u1, p1), (l2, u2, p2) = keep[0], keep[2]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = evs.sample(l2, u2, top_p=p2)
    evs.sample(l1, u1, top_p=p1)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, jobs[2][3])


def test_no_gradients(evs):
    l, u = make_logits(25, 2, 100)
    x, w = torch.zeros(1, 4, 8, device="cuda", requires_grad=True), torch.zeros(8, 4, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        evs.sample(l.requires_grad_(), u)
    with pytest.raises(ValueError, match="gradient"):
        evs.causal_conv(x, w)
    with torch.no_grad():
        assert evs.sample(l, u).shape == (2,) and evs.causal_conv(x, w).shape == (1, 4, 8)


def test_no_gradients_of_any_argument(evs):
    """Weights, states and caches that ask for a gradient are refused like the first argument, not detached."""
    l, u = make_logits(26, 2, 100)
    s, d = make_scan(27, 2, 5, 64, 16, F32), make_attn(28, F32, 2, 1, 3, 4, 2, 16, 20, 10, [3, 10])
    x, w, bias, tail = s["x"], torch.ones(64, 4, device="cuda"), torch.zeros(64, device="cuda"), torch.zeros(2, 3, 64, device="cuda")
    t, p, m = col(2, 0.9), col(2, 0.8), col(2, 0.1)
    out, so, to = torch.empty_like(x), torch.empty_like(s["state"]), torch.empty_like(tail)
    o = torch.empty_like(d["q"])
    draw = lambda: evs.sample(l, u, temperature=t, top_p=p, min_p=m)  # noqa: E731
    conv = lambda: evs.causal_conv(x, w, bias, tail=tail, tail_out=to, out=out)  # noqa: E731
    scan = lambda: evs.selective_scan(x, s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],  # noqa: E731
                                      state=s["state"], state_out=so, out=out)
    attn = lambda: run_attn(evs, d, out=o)  # noqa: E731
    for call, tensors in ((draw, (l, u, t, p, m)), (conv, (x, w, bias, tail, to, out)),
                          (scan, (*s.values(), so, out)), (attn, (*(v for k, v in d.items() if k != "own"), o))):
        call()
        for leaf in tensors:
            leaf.requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call()
            with torch.no_grad():
                call()
            leaf.requires_grad_(False)


def test_decode_filtered(evs):
    """The decode step's own path: its logits, drawn with filters; the state as after a plain step."""
    from gpu_harness import Pair
    from synth import LayerSpec, get_workload
    for wl in (get_workload("tiny_d64_fp32").replace(batch=3),
               get_workload("d1024_l8_p8k_bf16").replace(d=256, head_dim=128, batch=2, vocab=2048, layers=(
                   LayerSpec("fir", 3), LayerSpec("iir", 16), LayerSpec("attn", 2)))):
        B, V = wl.batch, wl.vocab
        pair = Pair(wl, t_max=200)
        pair.ver.prefill(torch.randint(65, 85, (B, 30), dtype=torch.int32, device="cuda"))
        start = pair.ver.export_state()
        tok = col(B, 67, torch.int32)
        pair.ver.decode(tok, None if wl.mode == "greedy" else col(B, 0.5))
        plain = pair.ver.export_state()
        pair.ver.import_state(start)
        u = torch.rand(B, device="cuda", generator=gen(3))
        lp, pr = torch.empty(B, device="cuda"), torch.empty(B, V, device="cuda")
        kw = dict(temperature=col(B, 0.8), top_k=col(B, 30, torch.int32), top_p=col(B, 0.9), min_p=col(B, 0.01))
        nxt = pair.ver.decode_filtered(tok, u, logprob=lp, probs=pr, **kw)
        logits = pair.ver.buffer(0, -1, torch.float32, (B, V)).clone()
        want = check_draw(evs, logits, u, **kw)
        assert torch.equal(nxt, want[0]) and torch.equal(lp, want[1]) and torch.equal(pr, want[2])
        after = pair.ver.export_state()
        assert np.array_equal(after["kv_len"], plain["kv_len"])
        for x, y in zip(after["layers"], plain["layers"]):
            for key in ("k", "v", "tail", "s"):
                if key in x:
                    assert np.array_equal(x[key], y[key])
        assert pair.ver.flags() == 0
        with pytest.raises(ValueError):
            pair.ver.decode_filtered(tok, u, top_k=col(B, 3.0))
        from lossless_speculative_verify_gb300 import EvsError
        with pytest.raises(EvsError):
            pair.ver.decode_filtered(tok, None)


# ---- convolution and scan --------------------------------------------------------------------------
CONV = [(1, 1, 1, 2), (2, 1, 64, 4), (3, 2, 72, 3), (2, 5, 8, 16), (3, 33, 136, 7), (2, 64, 520, 4), (1, 100, 1030, 5),
        (2, 70, 33, 4), (64, 1, 256, 4), (2, 32, 128, 8), (1, 40, 24, 9)]


def conv_tolerance(mag, y, dtype, taps):
    # taps + 1 products and sums, then v / (1 + exp(-v)): the exponential to 4 roundings and 2 |v| of its argument,
    # the sum 1, the division 4; the slope of silu is at most 1.1
    t = 1.1 * U * (taps + 2) * mag + U * (12 + 2 * mag) * y.abs() + 1e-12
    return t + BF * y.abs() * (1 + 1e-3) if dtype == BF16 else t


@pytest.mark.parametrize("shape", CONV, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_conv_matches_definition(evs, shape, dtype):
    B, T, D, K = shape
    g = gen(T * 100 + D)
    x, w, bias, tail = randn(g, B, T, D, dtype=dtype), randn(g, D, K), randn(g, D), randn(g, B, K - 1, D)
    lens = [max(0, T - 3 * i) for i in range(B)]
    for use in (None, lens):
        for silu, bs, tl in ((True, bias, tail), (False, None, None)):
            n = [T] * B if use is None else use
            lt = None if use is None else torch.tensor(use, dtype=torch.int32, device="cuda")
            out = torch.full((B, T, D), 9.0, device="cuda", dtype=dtype)
            tout = torch.full((B, K - 1, D), 5.0, device="cuda")
            y = evs.causal_conv(x, w, bs, tail=tl, tail_out=tout, lens=lt, silu=silu, out=out)
            ry, rt, mag = ref.conv(x, w, bs, tl, n, silu)
            assert torch.equal(tout.double(), rt)
            for b in range(B):
                assert torch.all(y[b, n[b]:] == 9.0)                 # left as they were
                err = (y[b, :n[b]].double() - ry[b, :n[b]]).abs()
                assert torch.all(err <= conv_tolerance(mag, ry, dtype, K)[b, :n[b]])
            alone = tail.clone() if tl is not None else torch.zeros(B, K - 1, D, device="cuda")
            if tl is not None:                                       # in place, output not wanted
                assert evs.causal_conv(x, w, bs, tail=alone, tail_out=alone, lens=lt, output=False) is None
                assert torch.equal(alone.double(), rt)


def test_conv_in_pieces_is_the_same(evs):
    """A prompt in pieces, then single tokens, the tail carried in place: the bits of one call. Slicing at k."""
    g = gen(31)
    x, w, bias = randn(g, 2, 77, 128, dtype=BF16), randn(g, 128, 4), randn(g, 128)
    whole_tail = torch.empty(2, 3, 128, device="cuda")
    whole = evs.causal_conv(x, w, bias, tail_out=whole_tail)
    tail = torch.zeros(2, 3, 128, device="cuda")
    at = 0
    for n in (40, 2, 1, 1, 33):
        y = evs.causal_conv(x[:, at:at + n], w, bias, tail=tail, tail_out=tail)
        assert torch.equal(y, whole[:, at:at + n])
        at += n
    assert torch.equal(tail, whole_tail)
    pre = torch.empty(2, 3, 128, device="cuda")
    evs.causal_conv(x[:, :50], w, bias, tail_out=pre)
    k = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    evs.causal_conv(x[:, 50:57], w, bias, tail=pre, tail_out=pre, lens=k + 1, output=False)
    assert torch.equal(pre[0], x[0, 48:51].float()) and torch.equal(pre[1], x[1, 53:56].float())


@pytest.mark.parametrize("T", [17, 29, 31, 33, 47, 200])
def test_conv_tail_in_place_with_long_taps(evs, T):
    """A run of positions may reach no further back than the one before it: the old tail is overwritten meanwhile."""
    g = gen(T)
    x, w, tail = randn(g, 2, T, 4096, dtype=BF16), randn(g, 4096, 16), randn(g, 2, 15, 4096)
    apart = torch.empty_like(tail)
    want = evs.causal_conv(x, w, tail=tail, tail_out=apart)
    for _ in range(5):
        carried = tail.clone()
        assert torch.equal(evs.causal_conv(x, w, tail=carried, tail_out=carried), want) and torch.equal(carried, apart)


def test_conv_strides_and_lengths(evs):
    g = gen(32)
    B, T, D = 3, 50, 96
    for dtype in (F32, BF16):
        x, w = randn(g, B, T, D, dtype=dtype), randn(g, D, 4)
        want = evs.causal_conv(x, w)
        proj = torch.zeros(B, T, 3 * D + 5, device="cuda", dtype=dtype)
        proj[..., 1:1 + D] = x                                       # rows off the 16-byte grid
        got = evs.causal_conv(proj[..., 1:1 + D], w)
        assert float((got.float() - want.float()).abs().max()) <= 1e-5 + (0.0 if dtype == F32 else 2 * BF * float(want.abs().max()))
        tm = x.transpose(0, 1).contiguous().transpose(0, 1)          # token-major
        out = torch.empty(T, B, D, device="cuda", dtype=dtype).transpose(0, 1)
        assert torch.equal(evs.causal_conv(tm, w, out=out), want)
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        evs.causal_conv(x, w, lens=torch.tensor([50, 51, -1], dtype=torch.int32, device="cuda"), flags=flags)
        assert int(flags) == 32
    for bad in (dict(x=x.half()), dict(w=w.double()), dict(w=w[:, :1]), dict(w=w[:5]), dict(out=x),
                dict(x=x.transpose(1, 2)), dict(lens=torch.zeros(B, device="cuda")), dict(output=False),
                dict(tail=torch.zeros(B, 4, D, device="cuda"))):
        kw = {k: v for k, v in bad.items() if k not in ("x", "w")}
        with pytest.raises(ValueError):
            evs.causal_conv(bad.get("x", x), bad.get("w", w), **kw)
    assert evs.causal_conv(x[:, :0], w).shape == (B, 0, D)
    t0 = randn(g, B, 3, D)
    t1 = torch.empty_like(t0)
    evs.causal_conv(x[:, :0], w, tail=t0, tail_out=t1)
    assert torch.equal(t0, t1)


@contextlib.contextmanager
def invalid_capture():
    """A stream in a capture that has become invalid: the host's runtime refuses every launch on it."""
    import ctypes
    # torch's runtime, as loaded into this process
    rt = ctypes.CDLL(next(p for p in open("/proc/self/maps").read().split() if "libcudart.so" in p))
    rt.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    rt.cudaStreamSynchronize.argtypes = rt.cudaStreamDestroy.argtypes = [ctypes.c_void_p]
    rt.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    assert rt.cudaStreamBeginCapture(stream, 2) == 0                 # relaxed: other streams of the thread as ever
    assert rt.cudaStreamSynchronize(stream) != 0                     # not permitted: the capture is invalid now
    yield stream
    assert rt.cudaStreamEndCapture(stream, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()
    assert rt.cudaStreamDestroy(stream) == 0


def test_an_earlier_call_that_failed_is_not_reported_again(evs):
    """A draw on a stream whose capture has become invalid fails, on the host; the calls after it on a sound stream
    succeed. (The runtime that the library links keeps the last error of a thread until somebody asks for it.)"""
    import ctypes
    g = gen(33)
    x, w, tail = randn(g, 2, 9, 64), randn(g, 64, 4), randn(g, 2, 3, 64)
    want = evs.causal_conv(x, w, tail=tail)
    l, u = make_logits(34, 2, 100)
    tok = torch.empty(2, dtype=torch.int32, device="cuda")
    lib = evs.load()
    from lossless_speculative_verify_gb300 import _lib
    a = _lib.SampleArgs(rows=2, vocab=100, dtype=0, ld=100, logits=l.data_ptr(), uniforms=u.data_ptr(),
                        token=tok.data_ptr())
    torch.cuda.synchronize()
    with invalid_capture() as stream:
        assert lib.evs_sample(ctypes.byref(a), stream) == 4          # EVS_ERR_CUDA
    assert torch.equal(evs.causal_conv(x, w, tail=tail), want)
    assert torch.equal(evs.sample(l, u), evs.sample(l, u))


def test_a_failed_operator_leaves_no_error_to_a_handle(evs):
    """Each operator fails on a stream whose capture has become invalid; a Verifier's next decode step is sound."""
    import ctypes
    from gpu_harness import Pair
    from synth import get_workload
    from lossless_speculative_verify_gb300 import _lib
    pair = Pair(get_workload("tiny_d64_fp32"), t_max=100)
    pair.ver.prefill(torch.randint(65, 85, (1, 9), dtype=torch.int32, device="cuda"))
    tok = col(1, 67, torch.int32)
    u = col(1, 0.5)
    d, s = make_attn(35, BF16, 1, 1, 1, 2, 2, 64, 20, 10, [3]), make_scan(36, 1, 3, 64, 16, F32)
    y, w = torch.empty_like(s["x"]), torch.ones(64, 4, device="cuda")
    o, ws = torch.empty_like(d["q"]), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    l = torch.zeros(1, 100, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    calls = [("evs_sample", _lib.SampleArgs(rows=1, vocab=100, dtype=0, ld=100, logits=p(l), uniforms=p(u), token=p(tok))),
             ("evs_causal_conv", _lib.ConvArgs(batch=1, tokens=3, width=64, taps=4, dtype=0, x=p(s["x"]), x_ld=64,
                                               x_seq=192, y=p(y), y_ld=64, y_seq=192, weight=p(w))),
             ("evs_selective_scan", _lib.ScanArgs(
                 batch=1, tokens=3, width=64, states=16, dtype=0, x=p(s["x"]), x_ld=64, x_seq=192, dt=p(s["dt"]), dt_ld=64,
                 dt_seq=192, B=p(s["B"]), b_ld=16, b_seq=48, C=p(s["C"]), c_ld=16, c_seq=48, y=p(y), y_ld=64, y_seq=192,
                 A=p(s["A"]))),
             ("evs_shared_attention", _lib.SharedAttnArgs(
                 batch=1, n_cand=1, block=1, heads=2, kv_heads=2, head_dim=64, dtype=1, q_dtype=1, prefix=20, own_max=10,
                 q=p(d["q"]), q_ld=128, k_prefix=p(d["kp"]), v_prefix=p(d["vp"]), prefix_row=64, prefix_head=1280,
                 k_own=p(d["ko"]), v_own=p(d["vo"]), own_row=64, own_head=640, own_seq=1280, own_len=p(d["own"]),
                 k_block=p(d["kb"]), v_block=p(d["vb"]), block_row=64, block_head=64, block_cand=128, o=p(o), o_ld=128,
                 workspace=p(ws), ws_bytes=1 << 22))]
    torch.cuda.synchronize()
    with invalid_capture() as stream:
        status = [getattr(evs.load(), name)(ctypes.byref(a), stream) for name, a in calls]
    assert status == [4] * 4                                         # EVS_ERR_CUDA
    pair.ver.decode_filtered(tok, u)
    assert pair.ver.flags() == 0
    assert [getattr(evs.load(), name)(ctypes.byref(a), None) for name, a in calls] == [0] * 4
    torch.cuda.synchronize()


def test_outputs_whose_sequences_overlap(evs):
    """An output whose rows lie on one another is refused; sequence-major, token-major and padded ones are not."""
    B, T, D = 3, 5, 32
    s = make_scan(48, B, T, D, 8, F32)
    w = randn(gen(49), D, 4)
    conv = lambda o: evs.causal_conv(s["x"], w, out=o)  # noqa: E731
    scan = lambda o: evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], out=o)  # noqa: E731
    buf = torch.zeros(4096, device="cuda")
    for run in (conv, scan):
        want = run(None)
        for seq, row in ((0, D), (D, D), (2 * D, D), (T * D - 1, D), (D - 1, 3 * D), (D, 3 * D - 1), (D, 2 * D), (4 * D + 3, D)):
            with pytest.raises(ValueError, match="overlap"):
                run(buf.as_strided((B, T, D), (seq, row, 1)))
        for seq, row in ((T * D, D), (D, B * D), (T * D + 7, D), (D + 4, 3 * D + 8), (4 * D + D, D)):
            buf.fill_(7.0)
            got = run(buf.as_strided((B, T, D), (seq, row, 1)))
            assert torch.allclose(got, want, rtol=1e-5, atol=1e-5)     # unaligned rows take another instance
            assert int((buf != 7.0).sum()) <= B * T * D


def make_scan(seed, B, T, D, N, dtype):
    g = gen(seed)
    step = torch.exp(torch.rand(D, device="cuda", generator=g) * math.log(100.0) + math.log(1e-3))
    return dict(x=randn(g, B, T, D, dtype=dtype), dt=randn(g, B, T, D, dtype=dtype),
                A=-(torch.arange(1, N + 1, device="cuda") * (0.5 + torch.rand(D, N, device="cuda", generator=g))),
                B=randn(g, B, T, N, dtype=dtype), C=randn(g, B, T, N, dtype=dtype), D=randn(g, D),
                z=randn(g, B, T, D, dtype=dtype), dt_bias=torch.log(torch.expm1(step)), state=randn(g, B, D, N))


SCAN = [(1, 1, 1, 4), (2, 1, 64, 16), (3, 3, 33, 8), (2, 16, 40, 32), (2, 17, 64, 16), (3, 32, 65, 16), (2, 33, 100, 4),
        (1, 100, 130, 32), (2, 300, 64, 8), (64, 1, 256, 16), (1, 600, 32, 16),
        # enough channels for a lane each, in one piece and in segments; rows on 16, 4 and 2 bytes
        (40, 40, 512, 16), (40, 33, 514, 16), (40, 33, 513, 16), (2, 700, 2048, 16), (40, 40, 488, 8), (24, 40, 420, 32)]


@pytest.mark.parametrize("shape", SCAN, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scan_matches_definition(evs, shape, dtype):
    B, T, D, N = shape
    s = make_scan(T * 10 + D, B, T, D, N, dtype)
    lens = [max(0, T - 5 * i) for i in range(B)]
    for use, part in ((None, s), (lens, s), (lens, {**s, "D": None, "z": None, "dt_bias": None, "state": None})):
        n = [T] * B if use is None else use
        lt = None if use is None else torch.tensor(use, dtype=torch.int32, device="cuda")
        out = torch.full((B, T, D), 9.0, device="cuda", dtype=dtype)
        so = torch.empty(B, D, N, device="cuda")
        kw = {k: part[k] for k in ("D", "z", "dt_bias", "state")}
        y = evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], **kw, state_out=so, lens=lt, out=out)
        ry, ye, rs, se = ref.scan(s["x"], s["dt"], s["A"], s["B"], s["C"], kw["D"], kw["z"], kw["dt_bias"],
                                  kw["state"], n)
        assert torch.all((so.double() - rs).abs() <= se + 1e-30)
        for b in range(B):
            assert torch.all(y[b, n[b]:] == 9.0)
            tol = ye[b] + (BF * (1 + 1e-3) * ry[b].abs() if dtype == BF16 else 0.0) + 1e-30
            assert torch.all((y[b].double() - ry[b]).abs()[:n[b]] <= tol[:n[b]])
    raw = evs.selective_scan(s["x"], s["dt"].abs(), s["A"], s["B"], s["C"], softplus=False)
    ry, ye, _, _ = ref.scan(s["x"], s["dt"].abs(), s["A"], s["B"], s["C"], None, None, None, None, [T] * B, False)
    assert torch.all((raw.double() - ry).abs() <= ye + (BF * (1 + 1e-3) * ry.abs() if dtype == BF16 else 0.0) + 1e-30)


@pytest.mark.parametrize("B,T,N", [(8, 64, 8), (8, 64, 16), (8, 64, 32), (4, 250, 16), (32, 16, 16)])
def test_scan_decays_do_not_lean(evs, B, T, N):
    """A decay may be off by half an ulp or so either way, but not all of them the same way, which would add up.

    With a lean c of every decay the state's error is c L, L_t = a_t (L_{t-1} + s_{t-1}); c is read from the error by
    least squares. Arguments of -2^-14 to -1, where a state remembers anything, lean by 0.1 to -0.25 u, u = 2^-24.
    What scatters, about 1 u a step, is a thousandth of that in a mean over 10^5 states."""
    s = make_scan(60 + N, B, T, 512, N, F32)
    st = torch.empty_like(s["state"])
    evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], dt_bias=s["dt_bias"], state=s["state"], state_out=st)
    d = {k: v.double() for k, v in s.items()}
    dl = torch.nn.functional.softplus(d["dt"] + d["dt_bias"], threshold=50)
    h, lean = d["state"], torch.zeros_like(d["state"])
    for t in range(T):
        a = torch.exp(dl[:, t, :, None] * d["A"])
        lean = a * (lean + h)
        h = a * h + (dl[:, t] * d["x"][:, t])[..., None] * d["B"][:, t, None, :]
    c = float(((st.double() - h) * lean).sum() / (lean * lean).sum()) / U
    assert abs(c) <= 0.25, c


def test_scan_in_pieces_and_sliced(evs):
    """A prompt in pieces with the state carried in place, a verify block that leaves it alone, the slice at k."""
    s = make_scan(41, 2, 90, 96, 16, BF16)
    run = lambda a, b, **kw: evs.selective_scan(s["x"][:, a:b], s["dt"][:, a:b], s["A"], s["B"][:, a:b],  # noqa: E731
                                                s["C"][:, a:b], D=s["D"], z=s["z"][:, a:b], dt_bias=s["dt_bias"], **kw)
    whole = run(0, 90, state=s["state"])
    ry, ye, _, _ = ref.scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["state"], [90, 90])
    st = s["state"].clone()
    for a, b in ((0, 40), (40, 41), (41, 75), (75, 83)):
        y = run(a, b, state=st, state_out=st)
        assert torch.all((y.double() - ry[:, a:b]).abs() <= ye[:, a:b] + BF * 1.001 * ry[:, a:b].abs())
    before = st.clone()
    run(83, 90, state=st)                                            # a verify block: no state out
    assert torch.equal(st, before)
    k = torch.tensor([2, 6], dtype=torch.int32, device="cuda")
    run(83, 90, state=st, state_out=st, lens=k + 1, output=False)
    for b, n in ((0, 86), (1, 90)):
        _, _, rs, se = ref.scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["state"], [n, n])
        assert torch.all((st[b].double() - rs[b]).abs() <= se[b] + 1e-30)
    assert torch.equal(whole, run(0, 90, state=s["state"]))


def poison(*sizes):
    """Freed memory of these sizes, which the next allocations of them get, holds NaN."""
    torch.cuda.synchronize()
    for n in sizes:
        if n:
            t = torch.full((n // 4,), float("nan"), device="cuda")
            del t


# (width, states, tokens, lengths) of prompts that run in segments of 96 to 224 positions
SEGMENTED = [(4096, 16, 4096, [4096, 100]), (1024, 16, 700, [0, 1, 127, 128, 129, 159, 160, 161, 319, 320, 321, 700]),
             (96, 4, 513, [513, 0, 128, 129, 31]), (256, 8, 600, [600, 128, 1]), (64, 32, 900, [1, 900, 127, 257]),
             (33, 16, 400, [400, 128, 2, 399])]


@pytest.mark.parametrize("case", SEGMENTED, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scan_segments_and_short_sequences(evs, case, dtype):
    """Prompts cut into segments beside sequences that end in the first segment, at its end or have no token:
    the carried state apart and in place, with and without outputs, in memory that held NaN."""
    W, N, T, lens = case
    Bn = len(lens)
    s = make_scan(W + T, Bn, T, W, N, dtype)
    n_ws = evs.load().evs_selective_scan_workspace(Bn, T, W, N)
    assert n_ws > 0                                                  # it does run in segments
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    kw = {k: s[k] for k in ("D", "z", "dt_bias")}
    long = lens.index(max(lens))
    ry, ye, rs, se = ref.scan(*args, kw["D"], kw["z"], kw["dt_bias"], s["state"],
                              [0 if T > 2000 and b == long else n for b, n in enumerate(lens)])
    for place in (False, True):
        for output in (True, False):
            st = s["state"].clone()
            so = st if place else torch.full_like(st, 5.0)
            out = torch.full((Bn, T, W), 9.0, device="cuda", dtype=dtype) if output else None
            poison(n_ws)
            y = evs.selective_scan(*args, **kw, state=st, state_out=so, lens=lt, out=out, output=output)
            for b, n in enumerate(lens):
                if T > 2000 and b == long:                           # its definition takes long and has a test
                    assert torch.isfinite(so[b]).all()
                    continue
                assert torch.all((so[b].double() - rs[b]).abs() <= se[b] + 1e-30), (b, n)
                if output:
                    tol = ye[b] + (BF * (1 + 1e-3) * ry[b].abs() if dtype == BF16 else 0.0) + 1e-30
                    assert torch.all((y[b].double() - ry[b]).abs()[:n] <= tol[:n]), (b, n)
                    assert torch.all(y[b, n:] == 9.0)
            if not place:
                assert torch.equal(st, s["state"])
    # a length below zero is one of zero: the state stays
    so = torch.empty_like(s["state"])
    poison(n_ws)
    evs.selective_scan(*args, **kw, state=s["state"], state_out=so, lens=torch.full_like(lt, -3))
    assert torch.equal(so, s["state"])


def test_scan_extremes(evs):
    """Step sizes from none to huge: a decay of exactly one, and of zero."""
    for T in (4, 40):
        s = make_scan(42, 2, T, 64, 16, F32)
        s["dt"][0] = -200.0                                          # softplus 0: the state stays
        s["dt"][1] = 500.0                                           # softplus is the value itself: all forgotten
        so = torch.empty(2, 64, 16, device="cuda")
        evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], state=s["state"], state_out=so)
        assert torch.equal(so[0], s["state"][0])
        last = 500.0 * s["x"][1, -1][:, None] * s["B"][1, -1]
        assert torch.all((so[1] - last).abs() <= 2 * U * last.abs())


def test_scan_strides_lengths_refusals(evs):
    B, T, D, N = 2, 40, 64, 16
    s = make_scan(43, B, T, D, N, BF16)
    want = evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], z=s["z"])
    proj = torch.cat([s["z"], s["x"], s["B"], s["dt"], s["C"]], -1)   # slices of one projection
    x, z, dt = proj[..., D:2 * D], proj[..., :D], proj[..., 2 * D + N:3 * D + N]
    b, c = proj[..., 2 * D:2 * D + N], proj[..., 3 * D + N:]
    out = torch.zeros(T, B, D, device="cuda", dtype=BF16).transpose(0, 1)
    assert torch.equal(evs.selective_scan(x, dt, s["A"], b, c, z=z, out=out), want)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (T, 4):
        flags.zero_()
        evs.selective_scan(x[:, :n], dt[:, :n], s["A"], b[:, :n], c[:, :n], flags=flags,
                           lens=torch.tensor([n + 1, -1], dtype=torch.int32, device="cuda"))
        assert int(flags) == 32
    st = torch.empty(B, D, N, device="cuda")
    evs.selective_scan(x[:, :0], dt[:, :0], s["A"], b[:, :0], c[:, :0], state=s["state"], state_out=st)
    assert torch.equal(st, s["state"])
    args = dict(x=s["x"], dt=s["dt"], A=s["A"], B=s["B"], C=s["C"])
    for bad in (dict(x=s["x"].half()), dict(dt=s["dt"].float()), dict(A=s["A"][:, :12]), dict(B=s["B"][:, :5]),
                dict(C=s["C"].float()), dict(D=s["D"][:5]), dict(z=s["z"].float()), dict(state=s["state"].double()),
                dict(out=s["x"]), dict(output=False), dict(A=s["A"].double()),
                dict(state=torch.empty(B * D * N + 1, device="cuda")[1:].view(B, D, N))):
        with pytest.raises(ValueError):
            evs.selective_scan(**{**args, **bad})


@pytest.mark.parametrize("T", [1, 7, 40, 600])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_past_the_lengths_of_an_own_output(evs, T, dtype):
    """Without an output tensor the rows behind a sequence's length are zero, in memory that held NaN."""
    lens = [T, 0, T // 2]
    s = make_scan(46, 3, T, 64, 16, dtype)
    w = randn(gen(47), 64, 4)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for run in (lambda o: evs.causal_conv(s["x"], w, lens=lt, out=o),
                lambda o: evs.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], lens=lt, out=o)):
        want = run(torch.zeros_like(s["x"]))
        poison(s["x"].numel() * s["x"].element_size())
        got = run(None)
        assert torch.equal(got, want)
        assert all(torch.all(got[b, n:] == 0.0) for b, n in enumerate(lens))


def test_recurrent_captured(evs):
    s = make_scan(44, 2, 50, 64, 16, BF16)
    w = randn(gen(45), 64, 4)
    gr = torch.cuda.CUDAGraph()
    st, tail = s["state"].clone(), torch.zeros(2, 3, 64, device="cuda")
    lens = torch.tensor([50, 13], dtype=torch.int32, device="cuda")

    def step(state, tl):
        xc = evs.causal_conv(s["x"], w, tail=tl, tail_out=tl, lens=lens, out=torch.zeros_like(s["x"]))
        return evs.selective_scan(xc, s["dt"], s["A"], s["B"], s["C"], state=state, state_out=state, lens=lens,
                                  out=torch.zeros_like(s["x"]))

    st2, tail2 = st.clone(), tail.clone()
    want = [step(st2, tail2), step(st2, tail2)]
    with torch.cuda.graph(gr):
        y = step(st, tail)
    for w_ in want:
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w_)
    assert torch.equal(st, st2) and torch.equal(tail, tail2)


# ---- all of them, as a decode step of several continuations of one prompt -----------------------------
def test_a_step_of_continuations(evs):
    """n continuations of one prompt on a small hybrid block: convolution, selective scan, attention over the
    shared prompt and each continuation's own rows, logits, filtered draw; several steps, the caches and states
    carried on the device, against the same steps in fp64."""
    g = gen(51)
    n, d, H, G, dh, N, taps, V, P, steps = 6, 256, 4, 2, 64, 16, 4, 2000, 333, 5
    S = 16
    W = {k: randn(g, *s) / s[0] ** 0.5 for k, s in dict(
        emb=(V, d), x=(d, d), z=(d, d), dt=(d, d), b=(d, N), c=(d, N), q=(d, H * dh), k=(d, G * dh), v=(d, G * dh),
        o=(H * dh, d), head=(d, V)).items()}
    W["emb"] = W["emb"] * V ** 0.5
    cw, cb = randn(g, d, taps) / taps ** 0.5, randn(g, d) * 0.1
    A = -(torch.arange(1, N + 1, device="cuda") * (0.5 + torch.rand(d, N, device="cuda", generator=g)))
    kp, vp = randn(g, G, P, dh, dtype=BF16), randn(g, G, P, dh, dtype=BF16)
    ko = torch.full((n, G, S, dh), float("nan"), dtype=BF16, device="cuda")
    vo = ko.clone()
    own = torch.zeros(n, dtype=torch.int32, device="cuda")
    st, tail = torch.zeros(n, d, N, device="cuda"), torch.zeros(n, taps - 1, d, device="cuda")
    rst, rtail = st.clone(), tail.clone()
    tok = torch.arange(n, device="cuda", dtype=torch.int32)
    kw = dict(temperature=col(n, 0.9), top_k=col(n, 50, torch.int32), top_p=col(n, 0.95))
    for i in range(steps):
        u = torch.rand(n, device="cuda", generator=g)
        h = W["emb"][tok.long()][:, None]
        xin, z, dt = ((h @ W[k]) for k in ("x", "z", "dt"))
        xc = evs.causal_conv(xin, cw, cb, tail=tail, tail_out=tail)
        y = evs.selective_scan(xc, dt, A, xc @ W["b"], xc @ W["c"], z=z, state=st, state_out=st)
        rx, rt, _ = ref.conv(xin, cw, cb, rtail, [1] * n)
        assert torch.equal(rt, tail.double())
        ry, ye, rs, se = ref.scan(xc, dt, A, xc @ W["b"], xc @ W["c"], None, z, None, rst, [1] * n)
        assert torch.all((y.double() - ry).abs() <= ye + 1e-30) and torch.all((st.double() - rs).abs() <= se + 1e-30)
        rst, rtail = st.clone(), tail.clone()
        q = (y @ W["q"]).to(BF16).view(n, 1, 1, H, dh)
        for cache, w in ((ko, "k"), (vo, "v")):
            cache[:, :, i] = (y @ W[w]).to(BF16).view(n, G, dh)
        d_attn = dict(q=q, kp=kp, vp=vp, ko=ko, vo=vo, own=own, kb=None, vb=None)
        got = run_attn(evs, d_attn)
        check_attn({**d_attn, "ko": ko.nan_to_num(), "vo": vo.nan_to_num()}, got, BF16)
        logits = (h[:, 0] + got[0].float().view(n, H * dh) @ W["o"]) @ W["head"]
        tok = check_draw(evs, logits, u, **kw)[0]
        own += 1
