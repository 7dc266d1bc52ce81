"""Refusals of the attention and cache calls (no GPU: every one is refused
before anything is launched), and the list model the GPU tests compare with."""
import ctypes

import pytest
import torch

from ivf_top_key_b200 import _capi as C
from ivf_top_key_b200 import attend_cached, attend_prompt, cache_extend, cache_free
from tests.attention_ref import Pages

P = 1 << 20   # an aligned address that nothing follows


def _cache(**change):
    c = C.AiCache(k=P, v=P, tables=P, lens=P, refs=P, dtype=C.AI_BF16, n_layers=2, n_pages=8, page_size=16,
                  n_kv_heads=2, head_dim=128, n_seqs=3, max_pages=4)
    for k, v in change.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(k=None), "null pages"), (dict(v=None), "null pages"), (dict(tables=None), "null tables"),
    (dict(lens=None), "null tables or lens"), (dict(k=P + 8), "aligned"), (dict(dtype=C.AI_FP32), "bf16 or fp8"),
    (dict(k_scale=P), "k_scale"), (dict(dtype=C.AI_FP8E4M3), "k_scale"),
    (dict(dtype=C.AI_FP8E4M3, k_scale=P), "k_scale"), (dict(n_layers=0), "positive"), (dict(n_pages=0), "positive"),
    (dict(page_size=-1), "positive"), (dict(n_seqs=0), "positive"), (dict(max_pages=0), "positive"),
    (dict(n_pages=(1 << 20) + 1), "pages"), (dict(n_pages=1 << 20, page_size=1 << 11), "slots"),
    (dict(max_pages=1 << 27), "slots"), (dict(head_dim=100), "head_dim"), (dict(n_kv_heads=0), "positive"),
]


@pytest.mark.parametrize("change,match", BAD_CACHES)
def test_bad_caches_are_refused(change, match):
    c = _cache(**change)
    big = 1 << 40
    with pytest.raises(C.AiError, match=match) as e:
        C.ai_attend_cached(c, 0, P, 3, 4, None, 1.0, P, None, P, big, 0)
    assert e.value.code == -1
    with pytest.raises(C.AiError, match=match):
        C.ai_attend_selected(c, 0, P, P, 3, 5, 4, None, 1.0, P, None, P, big, 0)
    with pytest.raises(C.AiError, match=match):
        C.ai_cache_write(c, 0, P, P, P, P, 1, 1, 0)
    with pytest.raises(C.AiError):
        C.ai_cache_fork(c, P, P, 1, P, big, 0)
    with pytest.raises(C.AiError):
        C.ai_cache_compact(c, P, big, 0)


@pytest.mark.parametrize("args,match", [
    (dict(layer=2), "layer"), (dict(layer=-1), "layer"), (dict(q=None), "null"), (dict(out=None), "null"),
    (dict(ws=None), "null"), (dict(ws_bytes=100), "workspace"), (dict(heads=3), "multiple"), (dict(heads=0), "multiple"),
    (dict(rows=2), "seqs"), (dict(scale=float("nan")), "finite"), (dict(scale=float("inf")), "finite"),
    (dict(scale=-0.5), "negative"),
    (dict(q=P + 2), "aligned"), (dict(out=P + 8), "aligned"), (dict(rows=-1, seqs=P), "multiple"),
    (dict(rows=1 << 30, seqs=P), "too many"),
])
def test_bad_attention_arguments_are_refused(args, match):
    a = dict(layer=0, q=P, rows=3, heads=4, seqs=None, scale=1.0, out=P, ws=P, ws_bytes=1 << 40) | args
    with pytest.raises(C.AiError, match=match):
        C.ai_attend_cached(_cache(), a["layer"], a["q"], a["rows"], a["heads"], a["seqs"], a["scale"], a["out"], None,
                           a["ws"], a["ws_bytes"], 0)
    with pytest.raises(C.AiError, match=match):
        C.ai_attend_selected(_cache(), a["layer"], a["q"], P, a["rows"], 7, a["heads"], a["seqs"], a["scale"], a["out"],
                             None, a["ws"], a["ws_bytes"], 0)


def test_selected_needs_ids_and_head_dims_that_the_kernels_have():
    with pytest.raises(C.AiError, match="null"):
        C.ai_attend_selected(_cache(), 0, P, None, 3, 7, 4, None, 1.0, P, None, P, 1 << 40, 0)
    with pytest.raises(C.AiError, match="positive"):
        C.ai_attend_selected(_cache(), 0, P, P, 3, 0, 4, None, 1.0, P, None, P, 1 << 40, 0)
    with pytest.raises(C.AiError, match="head_dim"):
        C.ai_attend_cached(_cache(head_dim=96), 0, P, 3, 4, None, 1.0, P, None, P, 1 << 40, 0)


@pytest.mark.parametrize("args,match", [
    (dict(q=None), "null"), (dict(k=None), "null"), (dict(v=None), "null"), (dict(out=None), "null"),
    (dict(cu_q=None), "null"), (dict(n_seqs=-1), "negative"), (dict(total_q=-1), "negative"), (dict(D=96), "head_dim"),
    (dict(Hq=5), "multiple"), (dict(Hq=258), "128 query heads"), (dict(scale=float("inf")), "finite"), (dict(scale=-0.5), "negative"),
    (dict(q=P + 8), "aligned"), (dict(qs=(257, 128)), "strides"), (dict(ks=(256, 4)), "strides"),
    (dict(vs=(-256, 128)), "strides"), (dict(ks=(0, 128)), "strides"), (dict(qs=(1024, 0)), "strides"),
])
def test_bad_prompt_arguments_are_refused(args, match):
    a = dict(q=P, k=P, v=P, out=P, cu_q=P, n_seqs=1, total_q=4, total_k=4, Hq=4, D=128, scale=1.0, qs=(512, 128),
             ks=(256, 128), vs=(256, 128)) | args
    with pytest.raises(C.AiError, match=match) as e:
        C.ai_attend_prompt(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu_q"], P, a["n_seqs"], a["total_q"],
                           a["total_k"], a["Hq"], 2, a["D"], a["scale"], a["out"], None, None, None, 0, 0)
    assert e.value.code == -1


def test_prompt_workspace_is_needed_only_where_keys_are_divided():
    assert C.ai_attend_prompt_workspace(4, 8192, 8192, 32, 8, 128) == 0    # enough blocks
    assert C.ai_attend_prompt_workspace(1, 3, 900, 4, 2, 128) == 0         # few keys
    need = C.ai_attend_prompt_workspace(1, 3, 100000, 4, 2, 128)
    assert need > 0
    for ws, n in ((None, need), (P, need - 1), (P + 8, need)):
        with pytest.raises(C.AiError, match="workspace"):
            C.ai_attend_prompt(P, (512, 128), P, (256, 128), P, (256, 128), P, P, 1, 3, 100000, 4, 2, 128, 1.0, P, None,
                               None, ws, n, 0)
    for bad in ((-1, 3, 9, 4, 2, 128), (1, 3, 9, 5, 2, 128), (1, 3, 9, 258, 2, 128), (1, 3, 9, 4, 2, 0)):
        with pytest.raises(C.AiError, match="sizes"):
            C.ai_attend_prompt_workspace(*bad)


def test_bad_lists_and_workspaces_are_refused():
    need = C.ai_cache_workspace(_cache(), 5)
    for call in (lambda c, n, b: C.ai_cache_extend(c, P, P, n, P, b, 0), lambda c, n, b: C.ai_cache_fork(c, P, P, n, P, b, 0)):
        with pytest.raises(C.AiError, match="workspace"):
            call(_cache(), 5, need - 1)
        with pytest.raises(C.AiError, match="list"):
            call(_cache(), -1, need)
        with pytest.raises(C.AiError, match="refs"):
            call(_cache(refs=None), 5, need)
    with pytest.raises(C.AiError, match="refs"):
        C.ai_cache_free(_cache(refs=None), P, 1, 0)
    with pytest.raises(C.AiError, match="layer"):
        C.ai_cache_write(_cache(), 2, P, P, P, P, 1, 1, 0)
    with pytest.raises(C.AiError, match="null"):
        C.ai_cache_write(_cache(), 0, P, P, P, None, 1, 1, 0)
    with pytest.raises(C.AiError, match="bad"):
        C.ai_attend_workspace(5, 2, 128)


def test_calls_with_nothing_to_do_launch_nothing():
    before = C.ai_kernel_launches()
    C.ai_cache_extend(_cache(), None, None, 0, P, 1 << 20, 0)
    C.ai_cache_fork(_cache(), None, None, 0, P, 1 << 20, 0)
    C.ai_cache_free(_cache(), None, 0, 0)
    C.ai_cache_write(_cache(), 0, None, None, None, None, 0, 0, 0)
    C.ai_attend_cached(_cache(), 0, P, 0, 4, P, 1.0, P, None, P, 1 << 40, 0)
    C.ai_attend_prompt(None, (512, 128), P, (256, 128), P, (256, 128), P, P, 3, 0, 4, 4, 2, 128, 1.0, None, None, None, None, 0,
                       0)
    assert C.ai_kernel_launches() == before


def test_structure_matches_the_header():
    """Eight pointers and eight int32 in the header's order."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "ai_index.h")).read()
    body = re.search(r"typedef struct ai_cache \{(.*?)\} ai_cache;", src, re.S).group(1)
    names = [n for line in body.split(";") for n in re.findall(r"\b(\w+)\s*(?=,|$)", line.strip().split(" ", 1)[-1])]
    assert [n for n, _ in C.AiCache._fields_] == names
    assert ctypes.sizeof(C.AiCache) == 8 * 8 + 8 * 4


def test_host_tensors_are_refused():
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        attend_prompt(q, q, q, cu)
    t = torch.zeros(1, 2, dtype=torch.int32)
    pool = torch.zeros(3, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        attend_cached(q, pool, pool, t, cu[:1])
    with pytest.raises(ValueError, match="GPU"):
        cache_extend(pool, pool, t, cu[:1], cu[:1], cu, cu)
    with pytest.raises(ValueError, match="GPU"):
        cache_free(t, cu[:1], cu, cu, page_size=4)


def test_list_model_by_hand():
    m = Pages(6, 4, 4, 3)
    m.extend([1, 0], [5, 4])
    assert m.rows == [[2], [0, 1], [], []] and m.refs == [1, 1, 1, 0, 0, 0]
    m.fork([1, 0, 1], [2, 3, 2])          # part page copied, full page shared, dst named twice
    assert m.rows == [[2], [0, 1], [0, 3], [2]] and m.refs == [2, 1, 2, 1, 0, 0]
    m.extend([3, 0, 1], [9, 8, 1])        # too long for the row; the two free pages; a slot that is there
    assert m.lens == [12, 6, 5, 4] and m.rows[0] == [2, 4, 5]
    m.free([1, 3])
    assert m.refs == [1, 0, 1, 1, 1, 1]
    m.compact()                           # the page behind the first five moves into the hole
    assert m.refs == [1, 1, 1, 1, 1, 0] and m.rows[0] == [2, 4, 1]
