"""Stand-alone operators of the library on torch tensors: attention over a shared prefix, over whole
prompts and of trees of drafts, the filtered draw, log probabilities, the short causal convolution and
the selective scan.

Each function checks its arguments, fills the argument struct of one entry point (include/evs.h
states the mathematics) and enqueues it on the current stream of the tensors' device, like any
torch operator: outputs and workspaces come from torch's allocator, calls may be captured into
CUDA graphs, nothing synchronises. Inputs that are not what an operator takes raise ValueError
before anything is enqueued. Outputs share no memory with inputs, but for the state or tail that
is carried in place. There are no gradients: while they are enabled, a tensor that asks for one is
refused, whichever argument it is (``torch.no_grad()`` or ``detach()`` lets it in).
``flags`` is an int32 tensor of one element that collects EVS_FLAG_* bits.
"""
from __future__ import annotations

import torch

from . import _lib as L

_DT = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _p(t):
    return 0 if t is None else t.data_ptr()


def _no_grad(name, t):
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: this operator has no gradient")


def _vec(name, t, dtype, shape, dev):
    """Address of a contiguous tensor of the given type and shape on dev, or 0."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and
            t.device == dev):
        raise ValueError(f"{name}: want contiguous {dtype} {tuple(shape)} on {dev}")
    _no_grad(name, t)
    return t.data_ptr()


def _rows3(name, t, dtype, shape, dev, written=False):
    """Strides (row, sequence) of a [batch, tokens, n] tensor whose last dimension is contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} on {dev}")
    _no_grad(name, t)
    b, n, w = shape
    sq, ld, one = t.stride()
    ld = ld if n > 1 else w
    sq = sq if b > 1 else 0
    if not (one == 1 or w == 1):
        raise ValueError(f"{name}: the last dimension has to be contiguous")
    if ld < w:
        raise ValueError(f"{name}: rows overlap")
    # one sequence behind the other, or all of them within the distance of two rows
    if written and b > 1 and n > 0 and sq < (n - 1) * ld + w and not (sq >= w and ld >= (b - 1) * sq + w):
        raise ValueError(f"{name}: sequences overlap")
    return ld, sq


def _fresh(b, n, w, x, lens):
    """An output like x; with lengths the operator leaves rows unwritten, which are zero then."""
    make = torch.empty if lens is None else torch.zeros
    return make(b, n, w, dtype=x.dtype, device=x.device)


def _enqueue(fn, where, args, dev):
    # (the stream object that torch.cuda.current_stream builds costs 2 us a call)
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch.cuda.current_device() == dev.index:
        st = fn(args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(args, stream)
    if st:
        L.check(st, where)


def _device(name, t):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name}: want a CUDA tensor")
    _no_grad(name, t)
    return t.device


def sample(logits, uniforms, temperature=None, top_k=None, top_p=None, min_p=None, *, return_logprob=False,
           return_probs=False, out=None, flags=None):
    """Draw one token per row of ``logits`` [rows, vocab] (fp32 or bf16, any row stride).

    uniforms [rows] fp32 in [0, 1); temperature, top_p, min_p [rows] fp32 and top_k [rows] int32, each on the
    device or None (off). Temperatures that are not above zero take the largest logit. Returns the tokens
    [rows] int32, or a list [tokens, logprob fp32 [rows] if asked, probabilities fp32 [rows, vocab] if asked];
    the probabilities are the distribution that was drawn from (what a verify needs as the draft's q). A row
    with every token ruled out gives -1."""
    dev = _device("logits", logits)
    _need(logits.dim() == 2 and logits.dtype in _DT, "logits: want fp32 or bf16 [rows, vocab]")
    R, V = logits.shape
    _need(1 <= V <= 1 << 18 and R <= 1 << 24, "logits: vocabulary of 1 to 262144, at most 2**24 rows")
    _need(logits.stride(1) == 1 or V == 1, "logits: the vocabulary has to be contiguous")
    ld = logits.stride(0) if R > 1 else V
    _need(ld >= V, "logits: rows overlap")
    _need(uniforms is not None, "uniforms: missing")
    token = torch.empty(R, dtype=torch.int32, device=dev) if out is None else out
    logprob = torch.empty(R, dtype=torch.float32, device=dev) if return_logprob else None
    probs = torch.empty(R, V, dtype=torch.float32, device=dev) if return_probs else None
    f32 = torch.float32
    a = L.pack_sample(R, V, _DT[logits.dtype], ld, logits.data_ptr(), _vec("temperature", temperature, f32, (R,), dev),
                     _vec("top_k", top_k, torch.int32, (R,), dev), _vec("top_p", top_p, f32, (R,), dev),
                     _vec("min_p", min_p, f32, (R,), dev), _vec("uniforms", uniforms, f32, (R,), dev),
                     _vec("out", token, torch.int32, (R,), dev), _p(logprob), _p(probs), V,
                     _vec("flags", flags, torch.int32, (1,), dev))
    _enqueue(L.load().evs_sample, "evs_sample", a, dev)
    if logprob is None and probs is None:
        return token
    return [t for t in (token, logprob, probs) if t is not None]


def causal_conv(x, weight, bias=None, *, tail=None, tail_out=None, lens=None, silu=True, out=None, output=True,
                flags=None):
    """Short causal convolution of every channel of x [batch, tokens, width] (fp32 or bf16).

    weight [width, taps] fp32 (2 to 16 taps; weight[c, j] multiplies x[t - j]), bias [width] fp32 or None; tail
    and tail_out [batch, taps - 1, width] fp32, oldest first: the inputs before the first token, and the last
    ones after lens[b] tokens (they may be one tensor). lens [batch] int32 or None. Rows past a sequence's
    length are left as they were in ``out``, and zero where none is given. Returns out, or None with output=False (only the tail moves on:
    slicing at position k is lens = k + 1)."""
    dev = _device("x", x)
    _need(x.dim() == 3 and x.dtype in _DT and x.shape[2] > 0, "x: want fp32 or bf16 [batch, tokens, width]")
    B, T, D = x.shape
    _need(B <= 65535 and T <= 1 << 30 and D <= 1 << 24, "x: at most 65535 x 2**30 x 2**24")
    _need(isinstance(weight, torch.Tensor) and weight.dim() == 2 and 2 <= weight.shape[1] <= 16,
          "weight: want [width, 2..16]")
    taps = weight.shape[1]
    x_ld, x_sq = _rows3("x", x, x.dtype, (B, T, D), dev)
    y_ld = y_sq = 0
    y = None
    if output:
        y = _fresh(B, T, D, x, lens) if out is None else out
        y_ld, y_sq = _rows3("out", y, x.dtype, (B, T, D), dev, written=True)
        _need(y.data_ptr() != x.data_ptr() or y.numel() == 0, "out: may not be x")
    else:
        _need(out is None and tail_out is not None, "output=False wants tail_out and no out")
    f32 = torch.float32
    a = L.pack_conv(B, T, D, taps, _DT[x.dtype], 1 if silu else 0, x.data_ptr(), x_ld, x_sq, _p(y), y_ld, y_sq,
                   _vec("weight", weight, f32, (D, taps), dev), _vec("bias", bias, f32, (D,), dev),
                   _vec("tail", tail, f32, (B, taps - 1, D), dev),
                   _vec("tail_out", tail_out, f32, (B, taps - 1, D), dev),
                   _vec("lens", lens, torch.int32, (B,), dev), _vec("flags", flags, torch.int32, (1,), dev))
    if (T == 0 or B == 0) and tail_out is None:
        return y
    _enqueue(L.load().evs_causal_conv, "evs_causal_conv", a, dev)
    return y


def selective_scan(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, state=None, state_out=None, lens=None,
                   softplus=True, out=None, output=True, flags=None):
    """Selective scan over x [batch, tokens, width] with step sizes dt (same shape), input and output weights B, C
    [batch, tokens, states] and gate z (like x, or None), all fp32 or all bf16; A [width, states] fp32, states
    4, 8, 16 or 32; D, dt_bias [width] fp32 or None; state, state_out [batch, width, states] fp32 or None (they
    may be one tensor); lens [batch] int32 or None. Rows past a sequence's length are left as they were in
    ``out``, and zero where none is given. Returns out, or None with output=False (only the state moves on)."""
    dev = _device("x", x)
    _need(x.dim() == 3 and x.dtype in _DT and x.shape[2] > 0, "x: want fp32 or bf16 [batch, tokens, width]")
    Bn, T, W = x.shape
    _need(Bn <= 65535 and T <= 1 << 30 and W <= 1 << 24, "x: at most 65535 x 2**30 x 2**24")
    _need(isinstance(A, torch.Tensor) and A.dim() == 2 and A.shape[1] in (4, 8, 16, 32), "A: want [width, 4|8|16|32]")
    N = A.shape[1]
    x_ld, x_sq = _rows3("x", x, x.dtype, (Bn, T, W), dev)
    dt_ld, dt_sq = _rows3("dt", dt, x.dtype, (Bn, T, W), dev)
    z_ld, z_sq = (0, 0) if z is None else _rows3("z", z, x.dtype, (Bn, T, W), dev)
    b_ld, b_sq = _rows3("B", B, x.dtype, (Bn, T, N), dev)
    c_ld, c_sq = _rows3("C", C, x.dtype, (Bn, T, N), dev)
    y_ld = y_sq = 0
    y = None
    if output:
        y = _fresh(Bn, T, W, x, lens) if out is None else out
        y_ld, y_sq = _rows3("out", y, x.dtype, (Bn, T, W), dev, written=True)
        if y.data_ptr() in (x.data_ptr(), dt.data_ptr(), _p(z)) and y.numel() > 0:
            raise ValueError("out: may not be x, dt or z")
    else:
        _need(out is None and state_out is not None, "output=False wants state_out and no out")
    f32 = torch.float32
    if (A.data_ptr() | _p(state) | _p(state_out)) % 16:
        raise ValueError("A, state and state_out have to start on 16 bytes")
    lib = L.load()
    n = lib.evs_selective_scan_workspace(Bn, T, W, N)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    a = L.pack_scan(Bn, T, W, N, _DT[x.dtype], 1 if softplus else 0, x.data_ptr(), x_ld, x_sq, dt.data_ptr(), dt_ld,
                    dt_sq, _p(z), z_ld, z_sq, B.data_ptr(), b_ld, b_sq, C.data_ptr(), c_ld, c_sq, _p(y), y_ld, y_sq,
                    _vec("A", A, f32, (W, N), dev), _vec("D", D, f32, (W,), dev),
                    _vec("dt_bias", dt_bias, f32, (W,), dev), _vec("state", state, f32, (Bn, W, N), dev),
                    _vec("state_out", state_out, f32, (Bn, W, N), dev), _vec("lens", lens, torch.int32, (Bn,), dev),
                    _vec("flags", flags, torch.int32, (1,), dev), _p(ws), n)
    if (T == 0 or Bn == 0) and state_out is None:
        return y
    _enqueue(lib.evs_selective_scan, "evs_selective_scan", a, dev)
    return y


def _kv(name, k, v, dtype, shape, dev):
    """Strides of K and V of one kind, which are alike."""
    of = "_" + name if name else ""
    for which, t in (("k", k), ("v", v)):
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
            raise ValueError(f"{which}{of}: want {dtype} {tuple(shape)} on {dev}")
        _no_grad(which + of, t)
    st = k.stride()
    if st[-1] != 1:
        raise ValueError(f"k{of}: the head dimension has to be contiguous")
    if v.stride() != st:
        raise ValueError(f"k{of} and v{of}: want equal strides")
    return st


def _flat(name, t, dtype, shape, dev):
    """Row stride of a [batch, candidates, block, heads, dh] tensor whose rows are evenly spaced."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} on {dev}")
    _no_grad(name, t)
    B, Cn, T, H, dh = shape
    s0, s1, s2, s3, s4 = t.stride()
    if not (s4 == 1 and (H == 1 or s3 == dh)):
        raise ValueError(f"{name}: heads have to be contiguous")
    ld = s2 if T > 1 else s1 if Cn > 1 else s0 if B > 1 else H * dh
    if not (ld >= H * dh and (Cn == 1 or s1 == T * ld) and (B == 1 or s0 == Cn * T * ld)):
        raise ValueError(f"{name}: rows have to be evenly spaced")
    return ld


def shared_prefix_attention(q, k_prefix, v_prefix, k_own, v_own, own_len, k_block=None, v_block=None, *, scale=None,
                            out=None, return_lse=False, flags=None):
    """Attention of q [batch, candidates, block, heads, dh] over rows that the batch shares, k_prefix / v_prefix
    [kv_heads, P, dh], each sequence's own rows k_own / v_own [batch, kv_heads, capacity, dh] up to own_len [batch]
    (int32), and the block rows k_block / v_block [batch, candidates, kv_heads, block, dh] up to the query's own
    position. Without k_block (one candidate) the block rows are own rows own_len[b] + j.

    K and V are fp32 or bf16 with any strides but the last (K and V of a pair alike); q is of their type, or
    fp32 and rounded to it. heads is a multiple of kv_heads; dh 16, 32, 64 or 128. Returns out (the type of K), or [out, lse fp32
    [batch, candidates, block, heads]]."""
    dev = _device("q", q)
    _need(q.dim() == 5 and q.dtype in _DT, "q: want fp32 or bf16 [batch, candidates, block, heads, dh]")
    B, Cn, T, H, dh = q.shape
    _need(isinstance(k_prefix, torch.Tensor) and k_prefix.dim() == 3 and k_prefix.dtype in _DT,
          "k_prefix: want fp32 or bf16 [kv_heads, P, dh]")
    G, P, _ = k_prefix.shape
    dt = k_prefix.dtype
    _need(q.dtype == dt or q.dtype == torch.float32, "q: of the type of K, or fp32")
    _need(dh in (16, 32, 64, 128) and G > 0 and H > 0 and H % G == 0,
          "head dimension 16, 32, 64 or 128, heads a multiple of kv_heads")
    _need(1 <= Cn <= 64 and 1 <= T <= 128 and B <= 1024, "at most 1024 sequences, 64 candidates, 128 block positions")
    _need(isinstance(k_own, torch.Tensor) and k_own.dim() == 4, "k_own: want [batch, kv_heads, capacity, dh]")
    S = k_own.shape[2]
    _need(H <= 1024 and P <= 1 << 30 and S <= 1 << 30, "at most 1024 heads and 2**30 rows")
    ps = _kv("prefix", k_prefix, v_prefix, dt, (G, P, dh), dev)
    os_ = _kv("own", k_own, v_own, dt, (B, G, S, dh), dev)
    _need((k_block is None) == (v_block is None), "k_block and v_block go together")
    if k_block is not None:
        bs = _kv("block", k_block, v_block, dt, (B, Cn, G, T, dh), dev)
        _need(Cn == 1 or B == 1 or bs[0] == Cn * bs[1], "k_block: sequences and candidates have to be evenly spaced")
        b_row, b_head, b_cand = (bs[3] if T > 1 else dh), bs[2], bs[1] if Cn > 1 else bs[0]
    else:
        _need(Cn == 1 and S > 0, "block rows in k_own want one candidate")
        b_row = b_head = b_cand = 0

    q_ld = _flat("q", q, q.dtype, (B, Cn, T, H, dh), dev)
    if out is not None:
        o, o_ld = out, _flat("out", out, dt, (B, Cn, T, H, dh), dev)
    else:
        o, o_ld = torch.empty(B, Cn, T, H, dh, dtype=dt, device=dev), H * dh
    _need(scale is None or scale > 0.0, "scale: above zero")
    _need(own_len is not None, "own_len: missing")
    lengths = _vec("own_len", own_len, torch.int32, (B,), dev)
    flag = _vec("flags", flags, torch.int32, (1,), dev)
    lse = torch.empty(B, Cn, T, H, dtype=torch.float32, device=dev) if return_lse else None
    if B > 0:
        lib = L.load()
        shapes = L.pack_attn_shapes(B, Cn, T, H, G, dh, _DT[dt], _DT[q.dtype], P, S, 0, 0.0 if scale is None else scale)
        n = lib.evs_shared_attention_workspace(shapes + L.NO_REST)
        _need(n > 0, "sizes that the operator does not take")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        a = shapes + L.pack_attn_rest(
            q.data_ptr(), q_ld, k_prefix.data_ptr(), v_prefix.data_ptr(), ps[1] if P > 1 else dh, ps[0],
            k_own.data_ptr(), v_own.data_ptr(), os_[2] if S > 1 else dh, os_[1], os_[0], lengths, _p(k_block),
            _p(v_block), b_row, b_head, b_cand, o.data_ptr(), o_ld, _p(lse), ws.data_ptr(), n, flag)
        _enqueue(lib.evs_shared_attention, "evs_shared_attention", a, dev)
    return o if lse is None else [o, lse]


def _rows4(name, t, dtype, shape, dev):
    """Row stride of a [batch, nodes, heads, dh] tensor whose rows are evenly spaced."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} on {dev}")
    _no_grad(name, t)
    B, T, H, dh = shape
    s0, s1, s2, s3 = t.stride()
    ld = s1 if T > 1 else s0 if B > 1 else H * dh
    if not (s3 == 1 and (H == 1 or s2 == dh)):
        raise ValueError(f"{name}: heads have to be contiguous")
    if not (ld >= H * dh and (B == 1 or s0 == T * ld)):
        raise ValueError(f"{name}: rows have to be evenly spaced")
    return ld


def prompt_attention(q, k, v, starts, *, scale=None, out=None, return_lse=False, flags=None):
    """Causal attention over whole prompts packed behind each other: q [tokens, heads, dh], k and v [tokens, kv_heads,
    dh], all fp32 or all bf16. Sequence b is rows starts[b] up to starts[b + 1] of starts [batch + 1] (int32, on the
    device, ascending); its row i reads its rows j <= i.

    Any strides but the last (k and v alike), so that q, k and v may be parts of one projection's output; bf16 with
    heads of 64 or 128 whose rows start on 16 bytes is what runs on the tensor cores. heads is a multiple of kv_heads; dh 16, 32, 64 or 128; scale None (1 / sqrt(dh)) or 1e-30 to 1e30. Rows of no sequence may hold
    anything; they are left as they were in ``out``, and zero where none is given. Returns out [tokens, heads, dh], or
    [out, lse fp32 [tokens, heads]], whose rows of no sequence are -inf."""
    dev = _device("q", q)
    _need(q.dim() == 3 and q.dtype in _DT, "q: want fp32 or bf16 [tokens, heads, dh]")
    N, H, dh = q.shape
    _need(isinstance(k, torch.Tensor) and k.dim() == 3, "k: want [tokens, kv_heads, dh]")
    G = k.shape[1]
    _need(dh in (16, 32, 64, 128) and G > 0 and 0 < H <= 1024 and H % G == 0,
          "head dimension 16, 32, 64 or 128, at most 1024 heads, a multiple of kv_heads")
    _need(N <= 1 << 24, "at most 2**24 tokens")
    qs = q.stride()
    _need(qs[2] == 1, "q: the head dimension has to be contiguous")
    q_row, q_head = (qs[0] if N > 1 else H * dh), (qs[1] if H > 1 else dh)
    _need(q_row >= dh and q_head >= dh, "q: rows overlap")
    ks = _kv("", k, v, q.dtype, (N, G, dh), dev)
    kv_row, kv_head = (ks[0] if N > 1 else G * dh), (ks[1] if G > 1 else dh)
    _need(kv_row >= dh and kv_head >= dh, "k: rows overlap")
    _need(isinstance(starts, torch.Tensor) and starts.dim() == 1 and 2 <= starts.shape[0] <= 1025,
          "starts: want [batch + 1], at most 1024 sequences")
    at = _vec("starts", starts, torch.int32, starts.shape, dev)
    if out is not None:
        o = out
        _need(isinstance(o, torch.Tensor) and o.dtype is q.dtype and o.shape == q.shape and o.device == dev,
              f"out: want {q.dtype} {tuple(q.shape)} on {dev}")
        _no_grad("out", o)
        s0, s1, s2 = o.stride()
        _need(s2 == 1 and (H == 1 or s1 == dh), "out: heads have to be contiguous")
        o_row = s0 if N > 1 else H * dh
        _need(o_row >= H * dh, "out: rows overlap")
        _need(N == 0 or o.data_ptr() not in (k.data_ptr(), v.data_ptr()), "out: may not be k or v")
    else:
        o, o_row = torch.empty(N, H, dh, dtype=q.dtype, device=dev), H * dh
    _need(scale is None or 1e-30 <= scale <= 1e30, "scale: 1e-30 to 1e30")
    flag = _vec("flags", flags, torch.int32, (1,), dev)
    lse = torch.empty(N, H, dtype=torch.float32, device=dev) if return_lse else None
    if N > 0:
        lib = L.load()
        shapes = L.pack_prompt_shapes(N, starts.shape[0] - 1, H, G, dh, _DT[q.dtype], out is None,
                                      0.0 if scale is None else scale)
        n = lib.evs_prompt_attention_workspace(shapes + L.PROMPT_NO_REST)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        a = shapes + L.pack_prompt_rest(q.data_ptr(), q_row, q_head, k.data_ptr(), v.data_ptr(), kv_row, kv_head, at,
                                        o.data_ptr(), o_row, _p(lse), _p(ws), n, flag)
        _enqueue(lib.evs_prompt_attention, "evs_prompt_attention", a, dev)
    return o if lse is None else [o, lse]


def tree_attention(q, k_cache, v_cache, cache_len, parents, k_nodes=None, v_nodes=None, *, lens=None, scale=None,
                   out=None, return_lse=False, flags=None):
    """Attention of a tree of drafted tokens over each sequence's cache: q [batch, nodes, heads, dh] (at most 128
    nodes), k_cache and v_cache [batch, kv_heads, capacity, dh] of which cache_len [batch] (int32) rows are readable.
    Node i reads those and the nodes on its path to the root, itself included: parents [batch, nodes] or [nodes]
    (int32, on the device) holds the node above it, which comes before it, or -1 below the last cached token. A tree
    of one node is a decode step. lens [batch] (int32) or None: nodes of each tree; the rest is left as it was in
    ``out``, and zero where none is given.

    The nodes' K/V are k_nodes and v_nodes [batch, kv_heads, nodes, dh], or without them the cache's rows
    cache_len[b] + i. All fp32 or all bf16. K and V have any strides but the last (those of a pair alike); q's and out's
    heads are contiguous and their rows evenly spaced over nodes and batch. bf16 with heads of 64 or 128 whose K/V rows
    start on 16 bytes is what runs on the tensor cores; a cache that is expanded over the batch or the heads (a stride
    of 0) does not, and is many times slower than one with rows of its own. heads is a multiple of kv_heads; dh 16,
    32, 64 or 128; scale None (1 / sqrt(dh)) or 1e-30 to 1e30. Returns out [batch, nodes, heads, dh], or [out, lse fp32
    [batch, nodes, heads]]."""
    dev = _device("q", q)
    _need(q.dim() == 4 and q.dtype in _DT, "q: want fp32 or bf16 [batch, nodes, heads, dh]")
    B, T, H, dh = q.shape
    _need(isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4, "k_cache: want [batch, kv_heads, capacity, dh]")
    G, S = k_cache.shape[1:3]
    dt = q.dtype
    _need(dh in (16, 32, 64, 128) and G > 0 and 0 < H <= 1024 and H % G == 0,
          "head dimension 16, 32, 64 or 128, at most 1024 heads, a multiple of kv_heads")
    _need(1 <= T <= 128 and B <= 1024 and S <= 1 << 30, "at most 1024 sequences, 1 to 128 nodes, 2**30 rows")
    cs = _kv("cache", k_cache, v_cache, dt, (B, G, S, dh), dev)
    _need(S <= 1 or cs[2] >= dh, "k_cache: rows overlap")
    _need((k_nodes is None) == (v_nodes is None), "k_nodes and v_nodes go together")
    n_row = n_head = n_seq = 0
    if k_nodes is not None:
        ns = _kv("nodes", k_nodes, v_nodes, dt, (B, G, T, dh), dev)
        n_row, n_head, n_seq = (ns[2] if T > 1 else dh), ns[1], ns[0]
        _need(n_row >= dh, "k_nodes: rows overlap")
    else:
        _need(S > 0, "nodes in the cache want a capacity")
    _need(isinstance(parents, torch.Tensor) and parents.shape in ((B, T), (T,)), "parents: want [batch, nodes] or [nodes]")
    par = _vec("parents", parents, torch.int32, parents.shape, dev)
    _need(cache_len is not None, "cache_len: missing")
    cached = _vec("cache_len", cache_len, torch.int32, (B,), dev)
    sizes = _vec("lens", lens, torch.int32, (B,), dev)
    q_ld = _rows4("q", q, dt, (B, T, H, dh), dev)
    if out is not None:
        o, o_ld = out, _rows4("out", out, dt, (B, T, H, dh), dev)
        _need(B == 0 or o.data_ptr() not in (k_cache.data_ptr(), v_cache.data_ptr(), _p(k_nodes), _p(v_nodes)),
              "out: may not be k or v")
    else:
        o, o_ld = torch.empty(B, T, H, dh, dtype=dt, device=dev), H * dh
    _need(scale is None or 1e-30 <= scale <= 1e30, "scale: 1e-30 to 1e30")
    flag = _vec("flags", flags, torch.int32, (1,), dev)
    lse = torch.empty(B, T, H, dtype=torch.float32, device=dev) if return_lse else None
    if B > 0:
        lib = L.load()
        shapes = L.pack_tree_shapes(B, T, H, G, dh, _DT[dt], S, out is None, 0.0 if scale is None else scale)
        n = lib.evs_tree_attention_workspace(shapes + L.TREE_NO_REST)
        _need(n > 0, "sizes that the operator does not take")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        a = shapes + L.pack_tree_rest(
            q.data_ptr(), q_ld, k_cache.data_ptr(), v_cache.data_ptr(), cs[2] if S > 1 else dh, cs[1], cs[0], cached,
            par, T if parents.dim() == 2 else 0, _p(k_nodes), _p(v_nodes), n_row, n_head, n_seq, sizes, o.data_ptr(),
            o_ld, _p(lse), ws.data_ptr(), n, flag)
        _enqueue(lib.evs_tree_attention, "evs_tree_attention", a, dev)
    return o if lse is None else [o, lse]


def token_logprobs(logits, tokens, *, temperature=None, top=0, return_entropy=False, flags=None):
    """Log probabilities of ``tokens`` [rows, n] or [rows] (int32) under softmax(logits / temperature), logits [rows,
    vocab] (fp32 or bf16, any row stride), temperature [rows] fp32 or None; natural logarithms, fp32.

    Returns them, in the shape of tokens, or a list [logprob, entropy [rows] if asked, top_logprob [rows, top] and
    top_token int32 [rows, top] if top]: the ``top`` (at most 64) largest logits, equal ones by their ids. Logits
    that are NaN or -inf are ruled out. A temperature that is not above zero puts all mass on the first largest
    token. An id outside the vocabulary has -inf; behind the last token that is not ruled out, top_token is -1."""
    dev = _device("logits", logits)
    _need(logits.dim() == 2 and logits.dtype in _DT, "logits: want fp32 or bf16 [rows, vocab]")
    R, V = logits.shape
    _need(1 <= V <= 1 << 24 and R <= 1 << 24, "logits: vocabulary of 1 to 2**24, at most 2**24 rows")
    _need(logits.stride(1) == 1 or V == 1, "logits: the vocabulary has to be contiguous")
    ld = logits.stride(0) if R > 1 else V
    _need(ld >= V, "logits: rows overlap")
    _need(isinstance(tokens, torch.Tensor) and tokens.dim() in (1, 2) and tokens.shape[0] == R,
          "tokens: want int32 [rows] or [rows, n]")
    n = tokens.shape[1] if tokens.dim() == 2 else 1
    _need(n <= 1 << 20, "tokens: at most 2**20 a row")
    _need(isinstance(top, int) and 0 <= top <= min(64, V), "top: 0 to 64, at most the vocabulary")
    f32 = torch.float32
    tok = _vec("tokens", tokens, torch.int32, tokens.shape, dev)
    logprob = torch.empty(tokens.shape, dtype=f32, device=dev)
    entropy = torch.empty(R, dtype=f32, device=dev) if return_entropy else None
    top_lp = torch.empty(R, top, dtype=f32, device=dev) if top else None
    top_id = torch.empty(R, top, dtype=torch.int32, device=dev) if top else None
    if R > 0 and (n > 0 or top or return_entropy):
        a = L.pack_logprob(R, V, n, top, _DT[logits.dtype], ld, logits.data_ptr(),
                           _vec("temperature", temperature, f32, (R,), dev), tok, logprob.data_ptr(), _p(entropy),
                           _p(top_lp), _p(top_id), _vec("flags", flags, torch.int32, (1,), dev))
        _enqueue(L.load().evs_token_logprobs, "evs_token_logprobs", a, dev)
    if entropy is None and not top:
        return logprob
    return [t for t in (logprob, entropy, top_lp, top_id) if t is not None]
