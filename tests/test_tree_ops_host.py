"""Refusals of prompt attention, tree attention and token log probabilities, which need no GPU: every bad argument is
found on the host before anything is enqueued, at the C entry points and in the Python functions."""
import ctypes as C
import os
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
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "evs.h")).read(), flags=re.S)
    for name, cls in (("evs_logprob_args", L.LogprobArgs), ("evs_prompt_attn_args", L.PromptAttnArgs),
                      ("evs_tree_attn_args", L.TreeAttnArgs)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, src).group(1)
        fields = [re.sub(r".*[\s*]", "", f.strip()) for decl in body.split(";") if decl.strip()
                  for f in decl.split(",")]
        assert fields == [f for f, _ in cls._fields_], name


def test_packed_structs_are_the_structs(L):
    """What the Python functions pack is laid out as the C compiler lays the structs out."""
    for cls, pack in ((L.LogprobArgs, L.pack_logprob),
                      (L.PromptAttnArgs, lambda *a: L.pack_prompt_shapes(*a[:8]) + L.pack_prompt_rest(*a[8:])),
                      (L.TreeAttnArgs, lambda *a: L.pack_tree_shapes(*a[:9]) + L.pack_tree_rest(*a[9:]))):
        values = [float(i + 1) if t is C.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        raw = pack(*values)
        assert len(raw) == C.sizeof(cls)
        back = cls.from_buffer_copy(raw)
        assert [getattr(back, f) for f, _ in cls._fields_] == values
    assert len(L.pack_tree_shapes(*[1] * 8, 0.0) + L.TREE_NO_REST) == C.sizeof(L.TreeAttnArgs)


def _logprob(L, **kw):
    base = dict(rows=2, vocab=100, n_tokens=1, top=3, dtype=0, ld=100, logits=P, tokens=P, logprob=P, top_logprob=P,
                top_token=P)
    base.update(kw)
    return L.load().evs_token_logprobs(C.byref(L.LogprobArgs(**base)), None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1),
                                 dict(n_tokens=-1), dict(n_tokens=(1 << 20) + 1), dict(top=-1), dict(top=65),
                                 dict(vocab=2, top=3), dict(dtype=2), dict(ld=99), dict(logits=None),
                                 dict(logits=P + 2), dict(tokens=None), dict(logprob=None), dict(top_logprob=None),
                                 dict(top_token=None), dict(n_tokens=0, top=0)], ids=str)
def test_logprob_refuses(L, bad):
    assert _logprob(L, **bad) == INV


def test_logprob_empty_and_null(L):
    assert L.load().evs_token_logprobs(None, None) == INV
    assert _logprob(L, rows=0, logits=None, tokens=None) == OK


def _prompt(L, **kw):
    base = dict(tokens=10, batch=2, heads=8, kv_heads=4, head_dim=64, dtype=1, q=P, q_row=1024, q_head=64, k=P, v=P,
                kv_row=1024, kv_head=64, starts=P, o=P, o_row=512)
    base.update(kw)
    return L.load().evs_prompt_attention(C.byref(L.PromptAttnArgs(**base)), None)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(batch=-1), dict(batch=0),
                                 dict(batch=1025), dict(heads=0), dict(heads=6), dict(heads=1028), dict(kv_heads=0),
                                 dict(head_dim=48), dict(head_dim=256), dict(dtype=2), dict(q=None), dict(k=None),
                                 dict(v=None), dict(o=None), dict(starts=None), dict(q_row=63), dict(kv_row=63),
                                 dict(q_head=63), dict(kv_head=63), dict(o_row=511), dict(q=P + 1), dict(o=P + 1),
                                 dict(scale=-1.0), dict(scale=1e-40), dict(scale=float("inf")),
                                 dict(scale=float("nan"))], ids=str)
def test_prompt_refuses(L, bad):
    assert _prompt(L, **bad) == INV


def test_prompt_empty_and_null(L):
    assert L.load().evs_prompt_attention(None, None) == INV
    assert _prompt(L, tokens=0, q=None) == OK and _prompt(L, tokens=0, batch=0) == OK


def test_prompt_workspace(L):
    """Sizes whose items are dealt in runs of tiles need one; it follows neither the addresses nor the lengths."""
    lib = L.load()
    base = dict(tokens=2048, batch=1, heads=8, kv_heads=8, head_dim=128, dtype=1, q_row=1024, q_head=128, kv_row=1024,
                kv_head=128, o_row=1024)
    size = lambda **kw: lib.evs_prompt_attention_workspace(C.byref(L.PromptAttnArgs(**{**base, **kw})))  # noqa: E731
    n = size()
    # partials of two slots for each of 152 workers: 256 rows of outputs, maxima and sums; a job of each worker
    assert n >= 2 * 152 * 256 * (128 + 2) * 4 + 152 * 32 and n == size(q=P + 2, k=P + 2, q_row=1 << 20)
    assert _prompt(L, **base, workspace=None, ws_bytes=n) == INV
    assert _prompt(L, **base, workspace=P + 16, ws_bytes=n) == INV
    assert _prompt(L, **base, workspace=P, ws_bytes=n - 1) == CAP and _prompt(L, **base, workspace=P) == CAP
    # none is needed, or the sizes are none
    assert size(tokens=10) == 0 and size(tokens=0) == 0 and size(dtype=0) == 0 and size(head_dim=32) == 0
    assert size(head_dim=48) == 0 and size(heads=6, kv_heads=4) == 0 and size(batch=0) == 0
    assert lib.evs_prompt_attention_workspace(None) == 0


def _tree(L, **kw):
    base = dict(batch=2, nodes=5, heads=8, kv_heads=4, head_dim=64, dtype=1, capacity=50, q=P, q_ld=512, k_cache=P,
                v_cache=P, cache_row=64, cache_head=3200, cache_seq=12800, cache_len=P, parents=P, parents_seq=5,
                k_nodes=P, v_nodes=P, node_row=64, node_head=320, node_seq=1280, o=P, o_ld=512, workspace=P,
                ws_bytes=1 << 30)
    base.update(kw)
    return L.TreeAttnArgs(**base)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=1025), dict(nodes=0), dict(nodes=129, parents_seq=129),
                                 dict(heads=0), dict(heads=6), dict(kv_heads=0), dict(head_dim=48), dict(dtype=2),
                                 dict(capacity=-1), dict(capacity=(1 << 30) + 1), dict(q=None), dict(o=None),
                                 dict(q_ld=511), dict(o_ld=511), dict(k_cache=None), dict(v_cache=None),
                                 dict(cache_row=63), dict(cache_len=None), dict(parents=None), dict(parents_seq=4),
                                 dict(v_nodes=None), dict(k_nodes=None), dict(node_row=63),
                                 dict(k_nodes=None, v_nodes=None, capacity=0), dict(q=P + 1), dict(k_cache=P + 1),
                                 dict(v_nodes=P + 1), dict(scale=-1.0), dict(scale=1e-40), dict(scale=float("inf")),
                                 dict(scale=float("nan")), dict(workspace=None), dict(workspace=P + 16),
                                 dict(batch=1024, nodes=128, heads=1024, kv_heads=1024)], ids=str)
def test_tree_refuses(L, bad):
    a = _tree(L, **bad)
    if "heads" in bad:
        a.q_ld = a.o_ld = 1 << 20
    assert L.load().evs_tree_attention(C.byref(a), None) == INV


@pytest.mark.parametrize("scale", [1.1e30, 3e38, 1e-31, 1e-45])
def test_scales_are_of_a_range(L, scale):
    """In log2 units a scale near the type's largest value is an infinity, which makes a score of 0 NaN."""
    assert _prompt(L, scale=scale) == INV
    assert L.load().evs_tree_attention(C.byref(_tree(L, scale=scale)), None) == INV


def test_tree_workspace(L):
    lib = L.load()
    a = _tree(L)
    n = lib.evs_tree_attention_workspace(C.byref(a))
    assert n > 0
    a.ws_bytes = n - 1
    assert lib.evs_tree_attention(C.byref(a), None) == CAP
    assert lib.evs_tree_attention_workspace(C.byref(_tree(L, head_dim=48))) == 0
    assert lib.evs_tree_attention_workspace(None) == 0
    assert lib.evs_tree_attention(None, None) == INV
    assert lib.evs_tree_attention(C.byref(_tree(L, batch=0)), None) == OK


@pytest.mark.parametrize("shape", [dict(batch=64, heads=64, kv_heads=8, head_dim=128, nodes=64),
                                   dict(batch=1024, heads=64, kv_heads=8, head_dim=128, nodes=1, parents_seq=1),
                                   dict(batch=1, heads=8, kv_heads=8, head_dim=64, nodes=128, parents_seq=128)], ids=str)
def test_tree_workspace_does_not_follow_the_capacity(L, shape):
    """Partials number at most the workers (two on each of 152 SMs) and the segments, of up to 256 query rows each;
    the CUDA-core kernel's, which share the memory, four waves of CTAs besides one for each."""
    lib = L.load()
    sizes = [lib.evs_tree_attention_workspace(C.byref(_tree(L, capacity=c, **shape))) for c in (1 << 15, 1 << 18, 1 << 20)]
    rows = shape["nodes"] * shape["heads"] // shape["kv_heads"]
    segs = shape["batch"] * shape["kv_heads"]
    tensor = (segs * ((rows + 255) // 256) + 2 * 152) * min(rows + 3, 256)
    simt = (segs + 4 * 152) * (rows + 3)
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] <= max(tensor, simt) * (shape["head_dim"] + 2) * 4 + 8192


def test_python_functions_want_cuda_tensors():
    import lossless_speculative_verify_gb300 as evs
    x = torch.zeros(4, 2, 16)
    one = torch.zeros(1).int()
    with pytest.raises(ValueError, match="CUDA"):
        evs.token_logprobs(torch.zeros(2, 8), torch.zeros(2).int())
    with pytest.raises(ValueError, match="CUDA"):
        evs.prompt_attention(x, x, x, torch.tensor([0, 4]).int())
    with pytest.raises(ValueError, match="CUDA"):
        evs.tree_attention(x[None], x[None], x[None], one, one)
