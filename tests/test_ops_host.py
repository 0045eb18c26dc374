"""Refusals of the stand-alone operators, which need no GPU: every bad argument is found on the
host before anything is enqueued, at the C entry points and in the Python functions."""
import ctypes as C
import re

import pytest
import torch

INV, CAP, OK = 1, 2, 0
P = 1 << 20      # a 256-byte aligned address that no refused or empty call reads


@pytest.fixture(scope="module")
def L():
    from lossless_speculative_verify_gb300.build import build
    build()
    from lossless_speculative_verify_gb300 import _lib
    _lib.load()
    return _lib


def test_struct_layouts_follow_the_header(L):
    """Field names and their order in the ctypes mirrors are those of include/evs.h."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "evs.h")).read(), flags=re.S)
    for name, cls in (("evs_sample_args", L.SampleArgs), ("evs_conv_args", L.ConvArgs),
                      ("evs_scan_args", L.ScanArgs), ("evs_shared_attn_args", L.SharedAttnArgs)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, src).group(1)
        fields = [re.sub(r".*[\s*]", "", f.strip()) for decl in body.split(";") if decl.strip()
                  for f in decl.split(",")]
        assert fields == [f for f, _ in cls._fields_], name


def _sample(L, **kw):
    base = dict(rows=2, vocab=100, dtype=0, ld=100, logits=P, uniforms=P, token=P)
    base.update(kw)
    return L.load().evs_sample(C.byref(L.SampleArgs(**base)), None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 18) + 1), dict(ld=99), dict(dtype=2),
                                 dict(logits=None), dict(uniforms=None), dict(token=None), dict(logits=P + 2),
                                 dict(probs=P, probs_ld=99), dict(rows=1 << 25)])
def test_sample_refuses(L, bad):
    assert _sample(L, **bad) == INV


def test_sample_empty_and_null(L):
    assert L.load().evs_sample(None, None) == INV
    assert _sample(L, rows=0, logits=None, uniforms=None, token=None) == OK


def _conv(L, **kw):
    base = dict(batch=2, tokens=3, width=64, taps=4, dtype=1, silu=1, x=P, x_ld=64, x_seq=192, y=P, y_ld=64,
                y_seq=192, weight=P)
    base.update(kw)
    return L.load().evs_causal_conv(C.byref(L.ConvArgs(**base)), None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(width=0), dict(taps=1), dict(taps=17),
                                 dict(dtype=3), dict(weight=None), dict(x=None), dict(y=None), dict(x_ld=63),
                                 dict(y_ld=63), dict(batch=65536), dict(tokens=(1 << 30) + 1),
                                 dict(width=1 << 25, x_ld=1 << 25, y_ld=1 << 25)])
def test_conv_refuses(L, bad):
    assert _conv(L, **bad) == INV


def _scan(L, **kw):
    base = dict(batch=2, tokens=3, width=64, states=16, dtype=1, softplus=1, x=P, x_ld=64, x_seq=192, dt=P, dt_ld=64,
                dt_seq=192, B=P, b_ld=16, b_seq=48, C=P, c_ld=16, c_seq=48, y=P, y_ld=64, y_seq=192, A=P)
    base.update(kw)
    return L.load().evs_selective_scan(C.byref(L.ScanArgs(**base)), None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(width=0), dict(states=12), dict(states=64),
                                 dict(dtype=5), dict(A=None), dict(x=None), dict(dt=None), dict(B=None), dict(C=None),
                                 dict(y=None), dict(x_ld=63), dict(dt_ld=63), dict(b_ld=15), dict(c_ld=15),
                                 dict(y_ld=63), dict(z=P, z_ld=63), dict(A=P + 4), dict(state_in=P + 4),
                                 dict(state_out=P + 8), dict(batch=65536)])
def test_scan_refuses(L, bad):
    assert _scan(L, **bad) == INV


def test_recurrent_empty(L):
    lib = L.load()
    assert lib.evs_causal_conv(None, None) == INV and lib.evs_selective_scan(None, None) == INV
    assert _conv(L, batch=0) == OK and _scan(L, batch=0) == OK
    assert _conv(L, tokens=0) == OK and _scan(L, tokens=0) == OK      # no tokens and no state wanted


def _attn(L, **kw):
    base = dict(batch=2, n_cand=1, block=3, heads=8, kv_heads=4, head_dim=64, dtype=1, q_dtype=1, prefix=100,
                own_max=50, q=P, q_ld=512, k_prefix=P, v_prefix=P, prefix_row=64, prefix_head=6400, k_own=P, v_own=P,
                own_row=64, own_head=3200, own_seq=12800, own_len=P, k_block=P, v_block=P, block_row=64,
                block_head=192, block_cand=768, o=P, o_ld=512, workspace=P, ws_bytes=1 << 30)
    base.update(kw)
    return L.SharedAttnArgs(**base)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=1025), dict(n_cand=0), dict(n_cand=65), dict(block=0),
                                 dict(block=129), dict(heads=0), dict(heads=6), dict(kv_heads=0), dict(head_dim=48),
                                 dict(head_dim=256), dict(dtype=2), dict(q_dtype=2), dict(prefix=-1),
                                 dict(own_max=-1), dict(q=None), dict(o=None), dict(q_ld=511), dict(o_ld=511),
                                 dict(k_prefix=None), dict(v_prefix=None), dict(prefix_row=63), dict(k_own=None),
                                 dict(own_len=None), dict(own_row=63), dict(v_block=None), dict(block_row=63),
                                 dict(k_block=None, v_block=None, n_cand=2),
                                 dict(k_block=None, v_block=None, own_max=0), dict(scale=-1.0),
                                 dict(scale=float("inf")), dict(scale=float("nan")), dict(workspace=None),
                                 dict(workspace=P + 16)])
def test_attention_refuses(L, bad):
    assert L.load().evs_shared_attention(C.byref(_attn(L, **bad)), None) == INV


def test_attention_workspace(L):
    lib = L.load()
    a = _attn(L)
    n = lib.evs_shared_attention_workspace(C.byref(a))
    assert n > 0
    a.ws_bytes = n - 1
    assert lib.evs_shared_attention(C.byref(a), None) == CAP
    assert lib.evs_shared_attention_workspace(C.byref(_attn(L, head_dim=48))) == 0
    assert lib.evs_shared_attention_workspace(None) == 0
    assert lib.evs_shared_attention(C.byref(_attn(L, batch=0)), None) == OK
    # a longer prefix never needs less
    assert lib.evs_shared_attention_workspace(C.byref(_attn(L, prefix=100000))) >= n


def _bytes(L, **kw):
    return L.load().evs_shared_attention_workspace(C.byref(_attn(L, **kw)))


@pytest.mark.parametrize("shape", [
    dict(batch=64, heads=64, kv_heads=8, head_dim=128, block=16, prefix=8192),
    dict(batch=1024, heads=64, kv_heads=8, head_dim=128, block=1, prefix=0),
    dict(batch=256, heads=32, kv_heads=32, head_dim=64, block=13, n_cand=4, prefix=1000),
    dict(batch=3, heads=8, kv_heads=1, head_dim=128, block=128, n_cand=4, prefix=100)], ids=str)
def test_attention_workspace_is_what_the_kernels_can_fill(L, shape):
    """Partials number at most the workers (two on each of 152 SMs) and the segments, of the prefix and of the own
    rows, each of up to 256 query rows; the CUDA-core kernel's, which share the memory, at most four waves of CTAs
    of 16 rows besides one for each. However long the own rows may get, no more is asked for."""
    c = dict(n_cand=1)
    c.update(shape)
    grp, per = c["heads"] // c["kv_heads"], c["n_cand"] * c["block"]

    def partial_rows(rows, segs):
        tensor = (segs * ((rows + 255) // 256) + 2 * 152) * min(rows + 3, 256)
        simt = (segs * ((rows + 15) // 16) + 4 * 152) * 16
        return max(tensor, simt)

    rows = partial_rows(per * grp, c["batch"] * c["kv_heads"])
    if c["prefix"]:
        rows += partial_rows(c["batch"] * per * grp, c["kv_heads"])
    most = rows * (c["head_dim"] + 2) * 4 + 8192
    for own_max in (4096, 32768, 1 << 20):
        n = _bytes(L, own_max=own_max, **shape)
        assert 0 < n <= most, (n, most)


def test_decode_filtered_refuses(L):
    lib = L.load()
    assert lib.evs_decode_filtered(None, None, None, None) == INV


def test_python_functions_want_cuda_tensors():
    import lossless_speculative_verify_gb300 as evs
    x = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        evs.sample(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        evs.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        evs.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(1, 2, 4), torch.zeros(1, 2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        evs.shared_prefix_attention(torch.zeros(1, 1, 1, 2, 16), torch.zeros(2, 4, 16), torch.zeros(2, 4, 16),
                                    torch.zeros(1, 2, 4, 16), torch.zeros(1, 2, 4, 16), torch.zeros(1).int())
