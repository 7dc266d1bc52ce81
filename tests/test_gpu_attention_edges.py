"""The attention and cache calls at their edges: what lists ask for, values that are not finite, shared pages, long rows,
tensors that are dropped after the call."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import attention_ref as R

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from ivf_top_key_b200 import (AiError, AttentionIndex, C, PagedCache, attend_cached, attend_check,  # noqa: E402
                              attend_prompt, attend_selected, cache_extend, cache_write)
from tests.test_gpu_attention import DEV, _cache, _gen, _i32, _ids, _prompt, _q  # noqa: E402


@pytest.mark.parametrize("asked", [0, 80, 96, 97, 112, 128, 129, 144, 256])
def test_extend_that_needs_no_page_is_done_whatever_the_list_asks(asked):
    """Eight pages, six of them free: sequences 1 and 3 have room in their own part page."""
    c = PagedCache(n_pages=8, page_size=16, n_kv_heads=1, head_dim=64, n_seqs=4, max_pages=16)
    ref = R.Pages(8, 16, 4, 16)
    for seqs, counts in (([1, 3], [5, 1]), ([0, 1, 2, 3], [asked, 1, 1, 15])):
        ref.extend(seqs, counts)
        c.extend(_i32(seqs), _i32(counts))
        ref.same_as(c)
    assert ref.lens[1] == 6 and ref.lens[3] == 16
    if asked > 80:   # six free pages, one of them for sequence 2
        with pytest.raises(AiError, match="OOM"):
            c.check()
    c.check()


def test_extend_decode_steps_beside_one_request_beyond_the_cache():
    """The same in a list of more than one pass of the planning block."""
    n = 1500
    c = PagedCache(n_pages=2 * n, page_size=2, n_kv_heads=1, head_dim=64, n_seqs=n, max_pages=2 * n + 1)
    ref = R.Pages(2 * n, 2, n, 2 * n + 1)
    for seqs, counts in ((range(1, n), [1 + s % 2 for s in range(1, n)]), (range(n), [4 * n + 1] + [1] * (n - 1))):
        ref.extend(list(seqs), counts)
        c.extend(_i32(list(seqs)), _i32(counts))
        ref.same_as(c)
    assert ref.lens[:5] == [0, 2, 2, 2, 2]


def _spoiled(v, cu_q, cu_k, Hq, places):
    """v with the values of `places` (sequence, key, key head, column, value), and what they make of the outputs
    [total_q, Hq, D]: 0 where no row sees one, else the sum of those that it sees (of a place named twice the last)."""
    v, G = v.clone(), Hq // v.shape[1]
    add = torch.zeros(cu_q[-1], Hq, v.shape[2])
    for (b, j, h, d), x in {tuple(p[:4]): p[4] for p in places}.items():
        v[cu_k[b] + j, h, d] = x
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        first = max(0, j - (lk - lq))   # query i sees the keys up to lk - lq + i
        add[cu_q[b] + first:cu_q[b + 1], h * G:(h + 1) * G, d] += x
    return v, add


@pytest.mark.parametrize("Hq,Hkv,D,ql,kl", [
    (2, 2, 64, [300], [300]),
    (1, 1, 128, [513], [700]),
    (4, 2, 128, [40, 300, 50], [40, 300, 50]),
    (8, 1, 64, [130, 3], [400, 140]),
    (6, 2, 128, [150, 20], [90, 20]),        # the first rows see nothing
    (128, 1, 128, [9], [140]),
    (8, 2, 64, [40, 3], [3000, 5000]),       # keys divided among CTAs
    (2, 1, 128, [5], [9000]),
    (64, 1, 64, [70], [4000]),
])
def test_prompt_values_that_are_not_finite_reach_only_the_rows_that_see_them(Hq, Hkv, D, ql, kl):
    """Bit for bit: every other output is what it is without them, and so it is in every run."""
    q, k, v, cu_q, cu_k = _prompt(ql, kl, Hq, Hkv, D, seed=7 * sum(kl))
    r = random.Random(sum(kl))
    places = []
    for b, (n_q, n_k) in enumerate(zip(ql, kl)):
        near = [n_k - 1, max(0, n_k - n_q), max(0, n_k - n_q // 2), r.randrange(n_k), max(0, n_k - 1 - r.randrange(n_q))]
        for j in near:
            places.append((b, j, r.randrange(Hkv), r.randrange(D), r.choice([torch.nan, torch.inf, -torch.inf])))
        j, h, d = near[2], r.randrange(Hkv), r.randrange(D)
        places += [(b, j, h, d, torch.inf), (b, n_k - 1, h, d, -torch.inf)]
    v2, add = _spoiled(v, cu_q, cu_k, Hq, places)
    dq, dk, cq, ck = q.to(DEV), k.to(DEV), _i32(cu_q), _i32(cu_k)
    lse, lse2 = (torch.empty(len(q), Hq, device=DEV) for _ in range(2))
    status = _i32([0])
    # the two runs differ in these values alone; a finite one has to be a finite one's bits
    out = attend_prompt(dq, dk, v.to(DEV), cq, ck, out_lse=lse, status=status)
    want = out.float() + add.to(DEV)
    for _ in range(5):
        got = attend_prompt(dq, dk, v2.to(DEV), cq, ck, out_lse=lse2, status=status).float()
        assert torch.equal(lse, lse2)
        seen = want.isnan() | want.isinf()
        assert torch.equal(got.where(~seen, 0), want.where(~seen, 0))
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert (got[want.isinf()] == want[want.isinf()]).all()
    assert status.item() == 0


def test_prompt_long_with_bad_values_beside_a_healthy_one():
    """Blocks at the end of a long prompt whose last values are not finite, taken over by CTAs that have others to do."""
    ql = [24000, 300]
    Hq, Hkv, D = 16, 8, 128
    assert C.ai_attend_prompt_workspace(2, sum(ql), sum(ql), Hq, Hkv, D) == 0   # undivided
    q, k, v, cu, _ = _prompt(ql, ql, Hq, Hkv, D, seed=91)
    v2, add = _spoiled(v, cu, cu, Hq, [(0, 23990, 3, 5, torch.nan), (0, 23901, 0, 127, torch.inf),
                                       (0, 12001, 7, 64, torch.nan), (0, 0, 1, 1, -torch.inf)])
    dq, dk, dcu = q.to(DEV), k.to(DEV), _i32(cu)
    status = _i32([0])
    want = attend_prompt(dq, dk, v.to(DEV), dcu, status=status).float() + add.to(DEV)
    got = attend_prompt(dq, dk, v2.to(DEV), dcu, status=status).float()
    assert status.item() == 0
    good = want.isfinite()
    assert torch.equal(got.isfinite(), good) and torch.equal(got[good], want[good])
    assert good[24000:].all()


def test_calls_without_a_status_word_are_checked_by_device():
    args, _, _ = _cache([40, 50], 16, 1, 64, "bf16", seed=5)
    q = _q(2, 2, 64, 8).to(DEV)
    x = _q(30, 2, 64, 9).to(DEV)
    attend_check()
    ok = [lambda: attend_cached(q, **args), lambda: attend_prompt(x, x, x, _i32([0, 10, 30]))]
    bad = [lambda: attend_cached(q, seqs=_i32([7, -1]), **args), lambda: attend_selected(q, _i32([[1], [50]]), **args),
           lambda: attend_prompt(x, x, x, _i32([0, 40, 30])), lambda: attend_prompt(x, x, x, _i32([0, 10, 31]))]
    lens = args["lens"]
    for wrong in (-1, 10 ** 9):
        def call(n=wrong):
            args["lens"] = _i32([n, 50])
            attend_cached(q, **args)
            args["lens"] = lens
        bad.append(call)
    for call in bad:
        ok[0](), call(), ok[1]()
        with pytest.raises(AiError, match="DEVICE_CHECK"):
            attend_check(DEV)
        attend_check()   # once
    status = _i32([0])   # with a word of its own a call says it there
    attend_cached(q, seqs=_i32([7, -1]), status=status, **args)
    attend_check(torch.device("cuda", 0))
    assert status.item() == 2
    c = PagedCache(n_pages=2, page_size=4, n_kv_heads=1, head_dim=64, n_seqs=2, max_pages=3)
    cache_extend(c.k, c.v, c.tables, c.lens, c.refs, _i32([0]), _i32([9]))
    with pytest.raises(AiError, match="OOM"):
        attend_check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    seqs = _i32([7, -1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        attend_cached(q, seqs=seqs, **args)
    attend_check()
    g.replay()
    with pytest.raises(AiError, match="DEVICE_CHECK"):
        attend_check()


def test_the_first_call_of_a_process_may_be_a_captured_one():
    code = """
import torch
from ivf_top_key_b200 import PagedCache, attend_cached, attend_check, attend_prompt
c = PagedCache(n_pages=2, page_size=4, n_kv_heads=1, head_dim=64, n_seqs=1, max_pages=2)
q, cu = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = attend_cached(q, c.k, c.v, c.tables, c.lens)
    b = attend_prompt(q, q[:, :1], q[:, :1], cu)
g.replay()
attend_check()
assert (a == 0).all() and (b == 1).all()
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=200,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_write_leaves_pages_alone_that_another_sequence_holds(dtype):
    c = PagedCache(n_pages=8, page_size=4, n_kv_heads=2, head_dim=64, n_seqs=3, max_pages=4, dtype=dtype)
    x = torch.randn(16, 2, 64, generator=_gen(1)).bfloat16().to(DEV)
    c.extend(_i32([0]), _i32([8]))
    c.write(_i32([0]), _i32([0, 8]), x[:8], x[:8])
    c.fork(_i32([0]), _i32([1]))          # two full pages, held by both
    c.extend(_i32([1, 0]), _i32([2, 6]))
    c.check()
    before = [t.clone() for t in (c.k, c.v)]
    # sequence 1's last five tokens: three of them lie in a page that sequence 0 holds too; sequence 0's own are written
    c.write(_i32([1, 0]), _i32([0, 5, 11]), x[:11], x[:11])
    with pytest.raises(AiError, match="DEVICE_CHECK"):
        c.check()
    own = c.tables[0, 2:4].tolist()
    for t, b in zip((c.k, c.v), before):
        rest = [p for p in range(8) if p not in own]
        assert torch.equal(t[:, rest], b[:, rest]) and not torch.equal(t[:, own], b[:, own])
    c.write(_i32([1]), _i32([0, 2]), x[:2], x[:2])   # what it owns alone
    c.check()
    c.free(_i32([0]))
    c.write(_i32([1]), _i32([0, 10]), x[:10], x[:10])   # now it owns all of it
    c.check()
    if dtype == "bf16":
        pages = c.tables[1, :3].tolist()
        assert torch.equal(c.k[0, pages].reshape(12, 2, 64)[:10], x[:10])


@pytest.mark.parametrize("refs", [False, True])
def test_write_of_more_tokens_than_a_sequence_has_writes_the_last_ones(refs):
    c = PagedCache(n_pages=4, page_size=4, n_kv_heads=1, head_dim=64, n_seqs=2, max_pages=2)
    c.extend(_i32([0, 1]), _i32([3, 2]))
    x = torch.randn(9, 1, 64, generator=_gen(2)).bfloat16().to(DEV)
    status = _i32([0])
    cache_write(c.k, c.v, c.tables, c.lens, _i32([0, 1]), _i32([0, 7, 9]), x, x, refs=c.refs if refs else None,
                status=status)
    assert status.item() == 2
    assert torch.equal(c.k[0, 0, :3], x[4:7]) and torch.equal(c.k[0, 1, :2], x[7:]) and (c.k[0, :2, 3] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 5), (8, 1, 31), (8, 2, 300), (24, 1, 20), (40, 1, 200), (4, 1, 30000),
                                      (16, 1, 30000)])
def test_rows_whose_scores_are_all_minus_infinity_are_zero(Hq, Hkv, n, kv):
    """Whatever the values hold; the heads beside them are as they would be."""
    D = 64
    args, _, _ = _cache([n], 64, Hkv, D, kv, seed=n, layers=1, layer=0)
    page = args["tables"][0].long()
    k, v = args["k"], args["v"]
    if kv == "bf16":
        k[0, :, :, :, 0] = 1
        v[0, :, :, :, 1] = torch.nan
        v[0, :, :, :, 2] = torch.inf
    else:
        k[0, :, :, :, 0] = 0x38            # 1.0
        v[0, :, :, :, 1] = 0x7F            # NaN
    q = torch.zeros(1, Hq, D, dtype=torch.bfloat16, device=DEV)
    q[0, 0, 0] = -torch.inf
    lse = torch.empty(1, Hq, device=DEV)
    ids = _i32([list(range(n))])
    for out in (attend_cached(q, out_lse=lse, **args), attend_selected(q, ids, out_lse=lse, **args)):
        assert (out[0, 0] == 0).all() and lse[0, 0] == -torch.inf
        assert out[0, 1:, 1].isnan().all() and lse[0, 1:].isfinite().all()
    if kv == "bf16":
        at = (page[:, None] * 64 + torch.arange(64, device=DEV)).flatten()[:n]
        kk, vv = (t[0].flatten(0, 1)[at].contiguous() for t in (k, v))
        out = attend_prompt(q, kk, vv, _i32([0, 1]), _i32([0, n]), out_lse=lse)
        assert (out[0, 0] == 0).all() and lse[0, 0] == -torch.inf and out[0, 1:, 1].isnan().all()


@pytest.mark.parametrize("Hq", [2, 16])
def test_a_row_of_almost_2_31_keys(Hq):
    """49981 times the same page of 42966 tokens, 2^31 - 2 in all: the last tile's end is past 2^31.  All weights are 1
    and the values small whole numbers, so sums are exact where a warp adds up (2^31 / (148 * 8) keys, below 2^24)."""
    page, width = 42966, 49981
    n = page * width
    assert n == 2 ** 31 - 2
    k = torch.ones(1, page, 1, 64, dtype=torch.bfloat16, device=DEV)
    v = (torch.arange(64, device=DEV) % 5 - 2).to(torch.bfloat16).expand(1, page, 1, 64).contiguous()
    tables = torch.zeros(1, width, dtype=torch.int32, device=DEV)
    q = torch.zeros(1, Hq, 64, dtype=torch.bfloat16, device=DEV)
    lse, status = torch.empty(1, Hq, device=DEV), _i32([0])
    out = attend_cached(q, k, v, tables, _i32([n]), out_lse=lse, status=status)
    assert status.item() == 0
    assert torch.equal(out, v[:, 0].expand_as(out))
    # the joined parts' sum: at most 300 roundings; then a step of the logarithm, and the product's
    assert (lse.double() - math.log(n)).abs().max() < 300 * 2.0 ** -24 + 4 * 22 * 2.0 ** -24


def test_extend_to_almost_2_31_tokens():
    page, width = 42966, 49981
    tables = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    lens, refs, status = _i32([0, 0]), torch.zeros(width, dtype=torch.int32, device=DEV), _i32([0])
    c = C.AiCache(tables=tables.data_ptr(), lens=lens.data_ptr(), refs=refs.data_ptr(), status=status.data_ptr(),
                  n_pages=width, page_size=page, n_seqs=2, max_pages=width)
    n = C.ai_cache_workspace(c, 1)
    ws, seqs = torch.empty(n, dtype=torch.uint8, device=DEV), _i32([1])
    for more in (2 ** 31 - 2 - page - 5, page, 5):
        C.ai_cache_extend(c, seqs.data_ptr(), _i32([more]).data_ptr(), 1, ws.data_ptr(), n, 0)
    torch.cuda.synchronize()
    assert status.item() == 0 and lens.tolist() == [0, 2 ** 31 - 2] and (refs == 1).all()
    assert torch.equal(tables[1], torch.arange(width, dtype=torch.int32, device=DEV)) and (tables[0] == -1).all()


def test_inputs_of_a_call_on_another_stream_may_be_dropped_after_it():
    args, _, _ = _cache([700, 65], 64, 2, 64, "bf16", seed=71, layers=1, layer=0)
    q = _q(2, 8, 64, 72).to(DEV)
    ids = _i32(_ids(2, 65, 60, 73))
    k, v = (torch.randn(2, 2, 64, generator=_gen(s)).bfloat16().to(DEV) for s in (74, 75))
    cu = _i32([0, 1, 2])
    c = PagedCache(n_pages=4, page_size=4, n_kv_heads=2, head_dim=64, n_seqs=2, max_pages=2)
    s = torch.cuda.Stream()

    def dropped(call, *inputs):
        held = [x.clone() for x in inputs]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(40_000_000)
        out = call(*[held.pop(0) for _ in inputs], stream=s)
        junk = [torch.full_like(x, 3) for x in inputs for _ in range(4)]   # where the inputs were, if that is free
        torch.cuda.synchronize()
        del junk
        return out

    assert torch.equal(dropped(lambda x, stream: attend_cached(x, stream=stream, **args), q), attend_cached(q, **args))
    assert torch.equal(dropped(lambda x, i, stream: attend_selected(x, i, stream=stream, **args), q, ids),
                       attend_selected(q, ids, **args))
    assert torch.equal(dropped(attend_prompt, q, k, v, cu), attend_prompt(q, k, v, cu))
    seqs, ones = _i32([1, 0]), _i32([1, 1])
    dropped(c.extend, seqs, ones)
    assert c.lens.tolist() == [1, 1] and c.tables[:, 0].tolist() == [1, 0]
    dropped(c.write, seqs, cu, k, v)
    assert torch.equal(c.k[0, :2, 0], k) and torch.equal(c.v[0, :2, 0], v)
    dropped(c.fork, _i32([0]), _i32([1]))
    dropped(c.free, _i32([0]))
    assert c.lens.tolist() == [0, 1]


def test_an_output_of_another_stream_may_be_dropped_while_it_is_read():
    args, _, _ = _cache([700, 65], 64, 2, 64, "bf16", seed=76, layers=1, layer=0)
    q = _q(2, 8, 64, 77).to(DEV)
    k, cu = q[:, :2].contiguous(), _i32([0, 1, 2])
    s = torch.cuda.Stream()
    minus = -q
    for call in (lambda x: attend_cached(x, stream=s, **args), lambda x: attend_prompt(x, k, k, cu, stream=s)):
        s.wait_stream(torch.cuda.current_stream())
        want = call(q)
        torch.cuda.synchronize()
        want + 0   # (the kernel's first launch may wait for the device)
        out = call(q)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(40_000_000)
        got = out + 0
        del out
        others = [call(minus) for _ in range(4)]   # on s, which does not wait for the copy
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del others


def test_attend_of_an_index_with_its_own_stream():
    """The queries may be dropped after the call, the output while the current stream still reads it."""
    d, H, D, n, T, k = 128, 32, 64, 512, 64, 40
    ik, iq = (torch.randn(m, *t, d, generator=_gen(80 + m)).bfloat16().to(DEV) for m, t in ((n, ()), (T, (H,))))
    w, q = torch.randn(T, H, generator=_gen(81)).to(DEV), _q(T, 4, D, 82).to(DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        idx = AttentionIndex(d=d, H=H, window=128, clusters_per_window=4, refit_period=0, max_query_chunk=T, max_budget=256,
                             max_k=k, max_keys=n)
    c = PagedCache(n_pages=40, page_size=16, n_kv_heads=2, head_dim=D, n_seqs=1, max_pages=32)
    c.extend(_i32([0]), _i32([n]))
    kv = torch.randn(n, 2, D, generator=_gen(83)).bfloat16().to(DEV)
    c.write(_i32([0]), _i32([0, n]), kv, kv)
    torch.cuda.synchronize()
    idx.append_keys(ik)
    idx.seal()
    want = idx.attend(iq, w, n - T, k, 256, q, c)
    minus = -q
    idx.sync()
    torch.cuda.synchronize()
    assert want.isfinite().all() and want.abs().max() > 0
    want + 0   # (the kernel's first launch may wait for the device)
    # inputs
    held = [iq.clone(), w.clone(), q.clone()]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    out = idx.attend(held.pop(0), held.pop(0), n - T, k, 256, held.pop(0), c)
    junk = [torch.full_like(x, 3) for x in (iq, w, q) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del junk, out
    # the output
    out = idx.attend(iq, w, n - T, k, 256, q, c)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(40_000_000)
    got = out + 0
    del out
    others = [idx.attend(iq, w, n - T, k, 256, minus, c) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del others
    c.check()
    idx.close()


def test_no_rows_and_empty_lists_of_ids():
    c = PagedCache(n_pages=2, page_size=4, n_kv_heads=1, head_dim=64, n_seqs=1, max_pages=2)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert c.attend_selected(q, torch.empty(0, 5, dtype=torch.int32, device=DEV)).shape == (0, 2, 64)
    assert c.attend(q, _i32([])).shape == (0, 2, 64)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_compact_moves_all_layers_and_scales(dtype):
    page, n = 8, [13, 30, 8, 21]
    c = PagedCache(n_pages=16, page_size=page, n_kv_heads=2, head_dim=64, n_seqs=5, max_pages=4, dtype=dtype, n_layers=3)
    c.extend(_i32(list(range(4))), _i32(n))
    cu = _i32([0, 13, 43, 51, 72])
    for layer in range(3):
        x = torch.randn(72, 2, 64, generator=_gen(layer)).bfloat16().to(DEV)
        c.write(_i32(list(range(4))), cu, x, x * 2, layer=layer)
    c.fork(_i32([1]), _i32([4]))
    c.free(_i32([0, 2]))
    c.check()
    parts = [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]

    def tokens(s, length):
        at = c.tables[s, :-(-length // page)].long()
        return [t[:, at].flatten(1, 2)[:, :length].clone() for t in parts]

    before = {s: tokens(s, m) for s, m in ((1, 30), (3, 21), (4, 30))}
    c.compact()
    c.check()
    assert c.refs.tolist() == [1, 1, 2, 2, 2, 1, 1, 1] + [0] * 8
    for s, want in before.items():
        for a, b in zip(tokens(s, 21 if s == 3 else 30), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 2), (24, 1), (64, 1)])
@pytest.mark.parametrize("what", ["zero", "every fourth zero", "outlier"])
def test_fp8_values_beside_far_larger_scales_keep_their_weights(Hq, Hkv, what):
    """Values 2^-30 of ordinary ones beside some that are zero (scale 1, as quantize_fp8 makes it), and ordinary values
    beside some of 2^30 that weigh nothing (a score 100 below the others): what the others give is as exact as ever."""
    D, n = 64, 3000
    args, kd, vd = _cache([n], 64, Hkv, D, "fp8", seed=90, layers=1, layer=0)
    page = args["tables"][0].tolist()
    q = _q(1, Hq, D, 91)
    q[:, :, 0] = 8
    if what != "outlier":
        args["v_scale"] *= 2.0 ** -30
        vd[0] *= 2.0 ** -30
    for j in range(0, n, 4) if what == "every fourth zero" else (0, 700, 701, 1500, n - 1):
        at = 0, page[j // 64], j % 64
        if what != "outlier":
            args["v"][at] = 0
            args["v_scale"][at] = 1
            vd[0][j] = 0
        else:
            args["k"][at] = 0
            args["k"][at][:, 0] = 0xFE    # -448
            args["k_scale"][at] = 0.25
            kd[0][j] = 0
            kd[0][j, :, 0] = -112
            args["v_scale"][at] *= 2.0 ** 30
            vd[0][j] *= 2.0 ** 30
    lse, status = torch.empty(1, Hq, device=DEV), _i32([0])
    want = [R.attend(q[0].double(), kd[0], vd[0], D ** -0.5)]
    for out in (attend_cached(q.to(DEV), out_lse=lse, status=status, **args),
                attend_selected(q.to(DEV), _i32([list(range(n))]), out_lse=lse, status=status, **args)):
        R.check(out, lse, want)
    assert status.item() == 0


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (24, 1), (64, 1)])
def test_fp8_value_scales_of_every_size_end_and_reach_only_their_rows(Hq, Hkv):
    """Scales over all of fp32's exponents, zero and infinity among them: rows of infinite ones are not finite, the other
    sequence's rows are as exact as ever."""
    D, n = 64, 700
    args, kd, vd = _cache([n, n], 64, Hkv, D, "fp8", seed=95, layers=1, layer=0)
    r = random.Random(96)
    for s in range(2):
        page = args["tables"][s].tolist()
        for j in range(n):
            at = 0, page[j // 64], j % 64
            x = r.choice([0.0, 2.0 ** r.randint(-140, 90), 2.0 ** r.randint(-140, -100), 1.0, torch.inf if s == 0 else 3.0])
            args["v_scale"][at] = x
            vd[s][j] = args["v"][at].view(torch.float8_e4m3fn).double().cpu() * x
    q = _q(2, Hq, D, 97)
    lse, status = torch.empty(2, Hq, device=DEV), _i32([0])
    want = R.attend(q[1].double(), kd[1], vd[1], D ** -0.5)
    ids = _i32([list(range(n))] * 2)
    for out in (attend_cached(q.to(DEV), out_lse=lse, status=status, **args),
                attend_selected(q.to(DEV), ids, out_lse=lse, status=status, **args)):
        assert not out[0].isfinite().any()
        R.check(out[1:], lse[1:], [want])
    assert status.item() == 0
