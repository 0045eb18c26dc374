"""Stand-alone operators of the library on torch tensors: attention over a shared prefix, the
filtered draw, the short causal convolution and the selective scan.

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
    for which, t in (("k_", k), ("v_", v)):
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev):
            raise ValueError(f"{which}{name}: want {dtype} {tuple(shape)} on {dev}")
        _no_grad(which + name, t)
    st = k.stride()
    if st[-1] != 1:
        raise ValueError(f"k_{name}: the head dimension has to be contiguous")
    if v.stride() != st:
        raise ValueError(f"k_{name} and v_{name}: want equal strides")
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
