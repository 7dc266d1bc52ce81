"""Attention over cached, selected and packed keys against float64, and the
pages of the cache against plain lists."""
import random

import numpy as np
import pytest
import torch

from tests import attention_ref as R

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from ivf_top_key_b200 import (AiError, AttentionIndex, PagedCache, attend_cached, attend_prompt,  # noqa: E402
                              attend_selected, cache_compact, cache_extend, cache_fork, cache_free, cache_write)

DEV = "cuda"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cache(lens, page, Hkv, D, kv, seed, spare=3, layers=2, layer=1):
    """Pages in no order, NaN (or NaN codes and scales) wherever no token lies.  Returns the tensors of the call
    and each sequence's float64 keys and values."""
    g = _gen(seed)
    need = [-(-n // page) for n in lens]
    width = max(max(need), 1) + 1
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g)[:sum(need)].tolist()
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    shape = (layers, n_pages, page, Hkv, D)
    pools, scales, vals = [], [], []
    for _ in range(2):
        if kv == "bf16":
            pool, sc = torch.full(shape, torch.nan, dtype=torch.bfloat16), None
        else:
            pool, sc = torch.full(shape, 0x7F, dtype=torch.uint8), torch.full(shape[:-1], torch.nan)
        at, seqs = 0, []
        for i, n in enumerate(lens):
            pages = order[at:at + need[i]]
            at += need[i]
            tables[i, :need[i]] = torch.tensor(pages, dtype=torch.int32)
            x = torch.randn(n, Hkv, D, generator=g) * (1 + torch.rand(n, Hkv, 1, generator=g) * 2)
            if kv == "bf16":
                x = x.bfloat16()
                val = x.double()
            else:
                s = x.abs().amax(-1) / 448
                x = (x / s[..., None]).to(torch.float8_e4m3fn)
                val = x.double() * s[..., None].double()
            for j in range(n):
                p, o = pages[j // page], j % page
                if kv == "bf16":
                    pool[layer, p, o] = x[j]
                else:
                    pool[layer, p, o] = x[j].view(torch.uint8)
                    sc[layer, p, o] = s[j]
            seqs.append(val)
        pools.append(pool.to(DEV))
        scales.append(None if sc is None else sc.to(DEV))
        vals.append(seqs)
    args = dict(k=pools[0], v=pools[1], tables=tables.to(DEV), lens=_i32(lens), k_scale=scales[0], v_scale=scales[1],
                layer=layer)
    return args, vals[0], vals[1]


def _q(rows, Hq, D, seed):
    return (torch.randn(rows, Hq, D, generator=_gen(seed)) * 2).bfloat16()


# ------------------------------------------------------------------ cached
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,page,lens", [
    (1, 1, 1, [1]),
    (8, 2, 16, [0, 1, 15, 16, 17, 63, 64, 65, 0]),
    (6, 2, 48, [700, 5, 129]),
    (34, 2, 32, [300, 64, 1]),
    (64, 1, 256, [1000, 255]),
    (80, 1, 16, [130, 0, 77]),
    (128, 2, 64, [190]),
])
def test_cached_matches_float64(Hq, Hkv, page, lens, D, kv):
    args, kd, vd = _cache(lens, page, Hkv, D, kv, seed=Hq + page)
    q = _q(len(lens), Hq, D, 5)
    lse = torch.empty(len(lens), Hq, device=DEV)
    status = _i32([0])
    out = attend_cached(q.to(DEV), out_lse=lse, status=status, **args)
    want = [R.attend(q[i].double(), kd[i], vd[i], D ** -0.5) for i in range(len(lens))]
    R.check(out, lse, want)
    assert status.item() == 0


def test_cached_long_uneven_batch_divides_rows_among_ctas():
    lens = [9000, 1, 0, 4097, 333, 20000]
    args, kd, vd = _cache(lens, 64, 2, 128, "bf16", seed=3, layers=1, layer=0)
    q = _q(len(lens), 16, 128, 6)
    lse = torch.empty(len(lens), 16, device=DEV)
    out = attend_cached(q.to(DEV), out_lse=lse, **args)
    R.check(out, lse, [R.attend(q[i].double(), kd[i], vd[i], 128 ** -0.5) for i in range(len(lens))])
    again = attend_cached(q.to(DEV), **args)
    assert torch.equal(out, again)   # no order of arrival in it


@pytest.mark.parametrize("n,Hq,Hkv", [(33, 4, 2), (300, 2, 1), (700, 20, 1)])
def test_cached_many_sequences_with_empty_ones(n, Hq, Hkv):
    """A padded batch: more sequences than a warp, and than a block, looks up at once; some are empty."""
    r = random.Random(n)
    lens = [r.choice([0, 1, 31, 33, 64, 100]) for _ in range(n)]
    lens[n // 2] = 900
    args, kd, vd = _cache(lens, 32, Hkv, 64, "bf16", seed=n, layers=1, layer=0)
    q = _q(n, Hq, 64, 15)
    lse = torch.empty(n, Hq, device=DEV)
    status = _i32([0])
    out = attend_cached(q.to(DEV), out_lse=lse, status=status, **args)
    R.check(out, lse, [R.attend(q[i].double(), kd[i], vd[i], 0.125) for i in range(n)])
    assert status.item() == 0


def test_cached_rows_of_chosen_sequences_and_other_scales():
    lens = [40, 200, 3]
    args, kd, vd = _cache(lens, 16, 2, 64, "bf16", seed=4)
    seqs = [2, 0, 2, 1, 1]
    q = _q(len(seqs), 4, 64, 7)
    for scale in (0.0, 0.3):
        lse = torch.empty(len(seqs), 4, device=DEV)
        out = attend_cached(q.to(DEV), seqs=_i32(seqs), scale=scale, out_lse=lse, **args)
        R.check(out, lse, [R.attend(q[i].double(), kd[s], vd[s], scale) for i, s in enumerate(seqs)])


def test_cached_flags_bad_sequences_pages_and_lengths():
    args, kd, vd = _cache([40, 50], 16, 1, 64, "bf16", seed=5)
    q = _q(2, 2, 64, 8)
    status = _i32([0])
    out = attend_cached(q.to(DEV), seqs=_i32([7, -1]), status=status, **args)
    assert status.item() == 2 and (out == 0).all()
    status.zero_()
    args["tables"][1, 1] = 1 << 19   # a page that the cache does not have: its tokens are left out
    lse = torch.empty(2, 2, device=DEV)
    out = attend_cached(q.to(DEV), status=status, out_lse=lse, **args)
    assert status.item() == 2
    keep = [i for i in range(50) if not 16 <= i < 32]
    R.check(out, lse, [R.attend(q[0].double(), kd[0], vd[0], 0.125),
                       R.attend(q[1].double(), kd[1][keep], vd[1][keep], 0.125)])
    status.zero_()
    args["lens"][0] = 10 ** 9
    attend_cached(q.to(DEV), status=status, **args)
    assert status.item() == 2


def test_cached_infinite_and_nan_keys_that_are_seen():
    """+inf and NaN scores make a row NaN as the formula does; a key whose score is -inf has no weight."""
    args, kd, vd = _cache([100], 16, 1, 64, "bf16", seed=6)
    q = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    page = int(args["tables"][0, 2])
    args["k"][1, page, 3, 0, 0] = -torch.inf
    out = attend_cached(q, **args)
    keep = [i for i in range(100) if i != 35]
    lse = torch.empty(1, 2, device=DEV)
    out = attend_cached(q, out_lse=lse, **args)
    R.check(out, lse, [R.attend(q[0].cpu().double(), kd[0][keep], vd[0][keep], 0.125)])
    args["k"][1, page, 3, 0, 0] = torch.nan
    assert attend_cached(q, **args).isnan().all()


# ---------------------------------------------------------------- selected
def _ids(T, n, k, seed, empty=()):
    r = random.Random(seed)
    rows = []
    for t in range(T):
        row = [r.randrange(n) if r.random() < 0.5 else j % n for j in range(k)]
        for _ in range(r.randrange(k + 1)):
            row[r.randrange(k)] = -1
        rows.append([-1] * k if t in empty else row)
    return rows


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,D,T,k,n", [
    (1, 1, 64, 1, 1, 1),
    (8, 2, 128, 5, 63, 100),
    (24, 8, 64, 33, 65, 700),
    (32, 1, 128, 4, 200, 150),
    (64, 1, 128, 3, 700, 900),
    (72, 1, 64, 7, 64, 90),
])
def test_selected_matches_float64(Hq, Hkv, D, T, k, n, kv):
    args, kd, vd = _cache([n], 32, Hkv, D, kv, seed=k)
    ids = _ids(T, n, k, seed=T, empty=(2,))
    q = _q(T, Hq, D, 9)
    lse = torch.empty(T, Hq, device=DEV)
    status = _i32([0])
    out = attend_selected(q.to(DEV), _i32(ids), out_lse=lse, status=status, **args)
    want = []
    for t in range(T):
        at = [j for j in ids[t] if j >= 0]
        want.append(R.attend(q[t].double(), kd[0][at], vd[0][at], D ** -0.5))
    R.check(out, lse, want)
    assert status.item() == 0


def test_selected_many_rows_whole_and_divided():
    """More rows than CTAs: whole rows dealt out, the rest divided and joined."""
    n, T, k = 600, 700, 130
    args, kd, vd = _cache([n], 16, 2, 64, "bf16", seed=11, layers=1, layer=0)
    ids = _ids(T, n, k, seed=12, empty=(0, 699))
    q = _q(T, 4, 64, 10)
    lse = torch.empty(T, 4, device=DEV)
    out = attend_selected(q.to(DEV), _i32(ids), out_lse=lse, **args)
    want = []
    for t in range(T):
        at = [j for j in ids[t] if j >= 0]
        want.append(R.attend(q[t].double(), kd[0][at], vd[0][at], 0.125))
    R.check(out, lse, want)


def test_selected_rows_of_several_sequences_and_bad_ids():
    lens = [50, 90, 7]
    args, kd, vd = _cache(lens, 16, 1, 64, "bf16", seed=13)
    ids = [[0, 5, 49, -1], [89, 3, 90, 1 << 30], [6, 6, 6, 0]]
    q = _q(3, 2, 64, 11)
    lse = torch.empty(3, 2, device=DEV)
    status = _i32([0])
    out = attend_selected(q.to(DEV), _i32(ids), out_lse=lse, status=status, **args)
    good = [[0, 5, 49], [89, 3], [6, 6, 6, 0]]
    R.check(out, lse, [R.attend(q[i].double(), kd[i][a], vd[i][a], 0.125) for i, a in enumerate(good)])
    assert status.item() == 2
    seqs = [1, 1, 0]
    out = attend_selected(q.to(DEV), _i32([[1, 2, 3, 4]] * 3), seqs=_i32(seqs), out_lse=lse, **args)
    R.check(out, lse, [R.attend(q[i].double(), kd[s][1:5], vd[s][1:5], 0.125) for i, s in enumerate(seqs)])


# ------------------------------------------------------------------ prompt
def _prompt(ql, kl, Hq, Hkv, D, seed, pad=0):
    g = _gen(seed)
    nq, nk = sum(ql) + 2 * pad, sum(kl) + 2 * pad
    q = (torch.randn(nq, Hq, D, generator=g) * 2).bfloat16()
    k, v = (torch.randn(nk, Hkv, D, generator=g).bfloat16() for _ in range(2))
    return q, k, v, np.cumsum([pad] + list(ql)).tolist(), np.cumsum([pad] + list(kl)).tolist()


def _prompt_want(q, k, v, cu_q, cu_k, scale):
    want = []
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(lq):
            n = max(0, lk - lq + i + 1)
            want.append(R.attend(q[cu_q[b] + i].double(), k[cu_k[b]:cu_k[b] + n].double(),
                                 v[cu_k[b]:cu_k[b] + n].double(), scale))
    return want


@pytest.mark.parametrize("Hq,Hkv,D,ql,kl", [
    (1, 1, 64, [1], [1]),
    (4, 4, 128, [1, 17, 0, 130, 3], None),
    (8, 2, 64, [200, 1, 64], [260, 500, 64]),
    (8, 2, 128, [129, 40, 5], [129, 10, 0]),
    (6, 2, 128, [150, 33], [170, 33]),
    (14, 2, 64, [75, 300], [400, 300]),
    (16, 1, 128, [90], [350]),
    (48, 1, 64, [20, 7], [150, 7]),
    (128, 1, 128, [9], [140]),
    (100, 1, 64, [5, 1], [5, 64]),
])
def test_prompt_matches_float64(Hq, Hkv, D, ql, kl):
    kl = ql if kl is None else kl
    q, k, v, cu_q, cu_k = _prompt(ql, kl, Hq, Hkv, D, seed=sum(ql))
    lse = torch.empty(len(q), Hq, device=DEV)
    status = _i32([0])
    out = attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), None if cu_k == cu_q else _i32(cu_k), out_lse=lse,
                        status=status)
    R.check(out, lse, _prompt_want(q, k, v, cu_q, cu_k, D ** -0.5))
    assert status.item() == 0


@pytest.mark.parametrize("Hq,Hkv,D,ql,kl", [
    (2, 1, 128, [1], [3000]),
    (8, 2, 64, [40, 0, 3], [3000, 2000, 5000]),
    (6, 2, 128, [5, 30], [100, 9000]),
    (128, 1, 64, [4], [4000]),
])
def test_prompt_few_queries_divide_the_keys(Hq, Hkv, D, ql, kl):
    q, k, v, cu_q, cu_k = _prompt(ql, kl, Hq, Hkv, D, seed=sum(kl), pad=2)
    n = len(q)
    for bad in (None, torch.nan):
        if bad is not None:   # a value that the last sequence's last query alone sees
            v[cu_k[-1] - 1, 0, 5] = bad
        out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((n, Hq), 7.0, device=DEV)
        attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k), out=out, out_lse=lse)
        want = _prompt_want(q, k, v, cu_q, cu_k, D ** -0.5)
        rows = len(want) if bad is None else len(want) - 1
        if rows:
            R.check(out[2:2 + rows], lse[2:2 + rows], want[:rows])
        assert (out[:2] == 7).all() and (out[-2:] == 7).all() and (lse[-2:] == 7).all()
        if bad is not None:
            assert out[n - 3, :Hq // Hkv, 5].isnan().all()


def test_prompt_long_sampled_rows():
    L, Hq, Hkv, D = 5000, 4, 1, 128
    q, k, v, cu_q, _ = _prompt([L], [L], Hq, Hkv, D, seed=21)
    lse = torch.empty(L, Hq, device=DEV)
    out = attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), out_lse=lse)
    rows = [0, 1, 127, 128, 2047, 2048, 4095, 4863, 4864, 4999] + random.Random(1).sample(range(L), 40)
    want = [R.attend(q[i].double(), k[:i + 1].double(), v[:i + 1].double(), D ** -0.5) for i in rows]
    R.check(out[rows], lse[rows], want)


def test_prompt_strided_views_and_rows_of_no_sequence():
    """q, k, v as slices of one projection; rows before the first and behind the last sequence stay as they were."""
    ql = [70, 1, 33]
    Hq, Hkv, D, pad = 6, 2, 64, 5
    n = sum(ql) + 2 * pad
    x = torch.randn(n, (Hq + 2 * Hkv) * D, generator=_gen(22)).bfloat16()
    dx = x.to(DEV)
    parts = [t.split([Hq * D, Hkv * D, Hkv * D], 1) for t in (x, dx)]
    (q, k, v), (dq, dk, dv) = ([t.view(n, -1, D) for t in p] for p in parts)
    cu = np.cumsum([pad] + ql).tolist()
    out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, Hq), 7.0, device=DEV)
    attend_prompt(dq, dk, dv, _i32(cu), out=out, out_lse=lse, scale=0.2)
    R.check(out[pad:-pad], lse[pad:-pad], _prompt_want(q, k, v, cu, cu, 0.2))
    for t in (out, lse):
        assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()
    # heads outermost in memory
    h = torch.randn(Hkv, n, D, generator=_gen(23)).bfloat16()
    lse2 = torch.empty(n, Hq, device=DEV)
    out2 = attend_prompt(dq, h.to(DEV).transpose(0, 1), dv, _i32(cu), out_lse=lse2)
    R.check(out2[pad:-pad], lse2[pad:-pad], _prompt_want(q, h.transpose(0, 1), v, cu, cu, 0.125))


@pytest.mark.parametrize("bad", [torch.nan, torch.inf, -torch.inf])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_unseen_keys_and_values_have_no_influence(bad, D):
    """A bad key and value at a position: earlier rows as without them, later rows and their heads NaN (values)."""
    L, Hq, Hkv, at = 300, 4, 2, 171
    q, k, v, cu, _ = _prompt([40, L, 50], [40, L, 50], Hq, Hkv, D, seed=24)
    want = _prompt_want(q, k, v, cu, cu, D ** -0.5)
    k2, v2 = k.clone(), v.clone()
    v2[40 + at, 1, 3] = bad
    k2[40 + at, 1] = bad
    lse = torch.empty(len(q), Hq, device=DEV)
    out = attend_prompt(q.to(DEV), k.to(DEV), v2.to(DEV), _i32(cu), out_lse=lse)
    sick = out[40 + at:40 + L, 2:, 3]
    assert (sick.isnan() if bad != bad else sick == bad).all() or (sick.isnan() | (sick == bad)).all()
    good = [i for i in range(len(q)) if not 40 + at <= i < 40 + L]
    R.check(out[good], lse[good], [want[i] for i in good])
    rest = list(range(40 + at, 40 + L))
    R.check(out[rest][:, :2], lse[rest][:, :2], [tuple(t[:2] for t in want[i]) for i in rest])
    out = attend_prompt(q.to(DEV), k2.to(DEV), v.to(DEV), _i32(cu), out_lse=lse)
    R.check(out[good], lse[good], [want[i] for i in good])


def test_prompt_flags_bad_offsets():
    q, k, v, cu, _ = _prompt([10, 20], [10, 20], 2, 1, 64, seed=25)
    for bad in ([0, 10, 31], [0, 40, 30], [-1, 10, 30], [5, 4, 30]):
        out = torch.full_like(q, 7.0, device=DEV)
        status = _i32([0])
        attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), _i32(bad), out=out, status=status)
        assert status.item() == 2
    ok = torch.empty(30, 2, device=DEV)
    out = attend_prompt(q.to(DEV), k.to(DEV), v.to(DEV), _i32([0, 10, 30]), out_lse=ok)
    R.check(out, ok, _prompt_want(q, k, v, cu, cu, 0.125))


# ------------------------------------------------------------------- pages
def _tokens(cache, ref, Hkv, D):
    """Contents of every live sequence's pages, all layers, as token values."""
    k, v = cache.k.float().cpu(), cache.v.float().cpu()
    for s in range(len(ref.rows)):
        for pos, x in enumerate(ref.read(s)):
            p, o = ref.rows[s][pos // ref.page], pos % ref.page
            for layer in range(k.shape[0]):
                assert (k[layer, p, o] == x + layer).all() and (v[layer, p, o] == -x - layer).all(), (s, pos)


@pytest.mark.parametrize("page", [1, 5, 16])
def test_pages_random_program_matches_lists(page):
    """extend, write, fork, free and compact in a random order, with lists that hold bad entries."""
    n_seqs, width, n_pages, Hkv, D, layers = 9, 12, 40, 1, 64, 2
    c = PagedCache(n_pages=n_pages, page_size=page, n_kv_heads=Hkv, head_dim=D, n_seqs=n_seqs, max_pages=width,
                   n_layers=layers)
    ref = R.Pages(n_pages, page, n_seqs, width)
    r = random.Random(page)
    for step in range(60):
        op = r.choice(["extend", "extend", "fork", "free", "compact"])
        if op == "extend":
            seqs = [r.randrange(-1, n_seqs + 1) for _ in range(r.randint(1, 4))]
            counts = [r.choice([0, 1, page, r.randrange(3 * page + 2)]) for _ in seqs]
            before = list(ref.lens)
            ref.extend(seqs, counts)
            c.extend(_i32(seqs), _i32(counts))
            grown = [s for s in range(n_seqs) if ref.lens[s] > before[s]]
            new = [[float(r.randrange(100)) for _ in range(ref.lens[s] - before[s])] for s in grown]
            for s, x in zip(grown, new):
                ref.write(s, x)
            flat = torch.tensor([y for x in new for y in x], device=DEV)
            cu = np.cumsum([0] + [len(x) for x in new]).tolist()
            for layer in range(layers):
                x = (flat + layer).to(torch.bfloat16)[:, None, None].expand(-1, Hkv, D).contiguous()
                c.write(_i32(grown), _i32(cu), x, -x, layer=layer)
        elif op == "fork":
            n = r.randint(1, 4)
            src, dst = ([r.randrange(-1, n_seqs + 1) for _ in range(n)] for _ in range(2))
            ref.fork(src, dst)
            c.fork(_i32(src), _i32(dst))
        elif op == "free":
            seqs = [r.randrange(-1, n_seqs + 1) for _ in range(r.randint(1, 3))]
            ref.free(seqs)
            c.free(_i32(seqs))
        else:
            ref.compact()
            c.compact()
        ref.same_as(c)
    _tokens(c, ref, Hkv, D)


def test_pages_many_sequences_and_pages():
    """Lists and pools beyond one pass of the planning block."""
    n, page = 1500, 2
    c = PagedCache(n_pages=9000, page_size=page, n_kv_heads=1, head_dim=64, n_seqs=3100, max_pages=7)
    ref = R.Pages(9000, page, 3100, 7)
    r = random.Random(2)
    for _ in range(2):
        seqs = r.sample(range(n), n)
        counts = [r.randrange(6) for _ in range(n)]
        ref.extend(seqs, counts)
        c.extend(_i32(seqs), _i32(counts))
        ref.same_as(c)
    gone = r.sample(range(n), 900) + [3]
    ref.free(gone)
    c.free(_i32(gone))
    src, dst = list(range(n)), [1500 + i for i in range(n)]
    ref.fork(src, dst)
    c.fork(_i32(src), _i32(dst))
    ref.same_as(c)
    ref.compact()
    c.compact()
    ref.same_as(c)
    # exhaust the pages: what fits in list order is lengthened, the rest is flagged and as it was
    c.check()
    ref.extend(list(range(n)), [8] * n)
    c.extend(_i32(list(range(n))), _i32([8] * n))
    ref.same_as(c)
    with pytest.raises(AiError, match="OOM"):
        c.check()
    c.check()


def test_pages_behind_four_gib():
    """Written, forked, attended and moved where byte offsets pass 32 bits (4.7 GB of keys and of values)."""
    n_pages, page, Hkv, D, n = 36000, 64, 8, 128, 300
    c = PagedCache(n_pages=n_pages, page_size=page, n_kv_heads=Hkv, head_dim=D, n_seqs=3, max_pages=n_pages)
    c.extend(_i32([0, 1]), _i32([(n_pages - 8) * page, n]))
    k, v = (torch.randn(n, Hkv, D, generator=_gen(s)).bfloat16() for s in (60, 61))
    c.write(_i32([1]), _i32([0, n]), k.to(DEV), v.to(DEV))
    c.fork(_i32([1]), _i32([2]))
    assert c.tables[1, :5].tolist() == list(range(n_pages - 8, n_pages - 3))
    q = _q(2, 16, D, 62)
    ids = [list(range(0, n, 3)), list(range(n - 1, n - 101, -1))]
    all_keys = [R.attend(q[i].double(), k.double(), v.double(), D ** -0.5) for i in range(2)]
    some = [R.attend(q[i].double(), k[ids[i]].double(), v[ids[i]].double(), D ** -0.5) for i in range(2)]
    for moved in (False, True):
        if moved:
            c.free(_i32([0]))
            c.compact()
            assert sorted(c.tables[1, :5].tolist() + c.tables[2, 4:5].tolist()) == list(range(6))
        lse = torch.empty(2, 16, device=DEV)
        out = c.attend(q.to(DEV), _i32([2, 1]), out_lse=lse)
        R.check(out, lse, all_keys)
        out = c.attend_selected(q.to(DEV), _i32(ids), _i32([1, 2]), out_lse=lse)
        R.check(out, lse, some)
    c.check()


def test_prompt_few_queries_behind_a_long_prefix():
    L, T, Hq, Hkv, D = 400_000, 3, 2, 1, 64
    g = torch.Generator(device=DEV).manual_seed(63)
    k, v = (torch.randn(L, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(T, Hq, D, generator=g, device=DEV).bfloat16()
    lse = torch.empty(T, Hq, device=DEV)
    out = attend_prompt(q, k, v, _i32([0, T]), _i32([0, L]), out_lse=lse)
    want = [R.attend(q[i].cpu().double(), k[:L - T + i + 1].cpu().double(), v[:L - T + i + 1].cpu().double(), D ** -0.5)
            for i in range(T)]
    R.check(out, lse, want)


def test_write_quantises_like_the_key_store():
    from ivf_top_key_b200 import quantize_fp8
    c = PagedCache(n_pages=8, page_size=4, n_kv_heads=3, head_dim=64, n_seqs=2, max_pages=4, dtype="fp8", n_layers=2)
    c.extend(_i32([1, 0]), _i32([5, 9]))
    k, v = (torch.randn(14, 3, 64, generator=_gen(s)).bfloat16().to(DEV) for s in (1, 2))
    k[3] = 0
    c.write(_i32([1, 0]), _i32([0, 5, 14]), k, v, layer=1)
    c.check()
    tables = c.tables.cpu()
    for x, pool, sc in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        codes, scales = quantize_fp8(x.view(-1, 64))
        codes, scales = codes.view(14, 3, 64), scales.view(14, 3)
        for s, t0, n in ((1, 0, 5), (0, 5, 9)):
            for i in range(n):
                p = int(tables[s, i // 4])
                assert torch.equal(pool[1, p, i % 4], codes[t0 + i])
                assert torch.equal(sc[1, p, i % 4], scales[t0 + i])
    assert (c.k[0] == 0).all()


def test_write_refuses_repeated_and_unknown_sequences():
    c = PagedCache(n_pages=8, page_size=4, n_kv_heads=1, head_dim=64, n_seqs=2, max_pages=4)
    c.extend(_i32([0, 1]), _i32([3, 3]))
    x = torch.arange(1, 13, device=DEV).to(torch.bfloat16)[:, None, None].expand(-1, 1, 64).contiguous()
    c.write(_i32([0, 0, 5, 1]), _i32([0, 3, 6, 9, 12]), x, x)
    assert c.k[0, 0, :3, 0, 0].tolist() == [1, 2, 3] and c.k[0, 1, :3, 0, 0].tolist() == [10, 11, 12]
    with pytest.raises(AiError, match="DEVICE_CHECK"):
        c.check()
    c.write(_i32([0]), _i32([0, 12]), x, x)   # more tokens than the sequence has
    assert c.k[0, 0, :3, 0, 0].tolist() == [10, 11, 12]
    with pytest.raises(AiError, match="DEVICE_CHECK"):
        c.check()


def test_fork_copies_filled_slots_only_and_all_layers_fp8():
    c = PagedCache(n_pages=6, page_size=8, n_kv_heads=2, head_dim=64, n_seqs=3, max_pages=3, dtype="fp8", n_layers=3)
    c.extend(_i32([0]), _i32([13]))
    for layer in range(3):
        x = torch.randn(13, 2, 64, generator=_gen(layer)).bfloat16().to(DEV)
        c.write(_i32([0]), _i32([0, 13]), x, x + 1, layer=layer)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    c.fork(_i32([0, 0]), _i32([2, 1]))
    c.check()
    assert c.tables.tolist() == [[0, 1, -1], [0, 3, -1], [0, 2, -1]] and c.refs.tolist() == [3, 1, 1, 1, 0, 0]
    for t, b in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        for p in (2, 3):
            assert torch.equal(t[:, p, :5], b[:, 1, :5]) and torch.equal(t[:, p, 5:], b[:, p, 5:])
        assert torch.equal(t[:, :2], b[:, :2]) and torch.equal(t[:, 4:], b[:, 4:])


# --------------------------------------------------- streams, graphs, refusals
def test_calls_on_another_stream_and_in_graphs():
    """Two captured steps (take a page slot, write, attend) replayed in turn, and an eager call on a third stream."""
    D, Hq, Hkv = 64, 4, 2
    caches, graphs, outs, news, qs, held = [], [], [], [], [], []
    for i in range(2):
        c = PagedCache(n_pages=20, page_size=4, n_kv_heads=Hkv, head_dim=D, n_seqs=2, max_pages=10)
        one, seqs, cu = _i32([1, 1]), _i32([1, 0]), _i32([0, 1, 2])
        x = torch.zeros(2, Hkv, D, dtype=torch.bfloat16, device=DEV)
        q = _q(2, Hq, D, 30 + i).to(DEV)
        lse = torch.empty(2, Hq, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.extend(seqs, one)
                c.write(seqs, cu, x, 2 * x)
                out = c.attend(q, seqs, out_lse=lse)
        caches.append(c), graphs.append(g), outs.append((out, lse)), news.append(x), qs.append(q)
        held.append((one, seqs, cu))   # the graphs read them at every replay
    torch.cuda.synchronize()
    hist = [[], []]
    for step in range(11):
        for i in range(2):
            x = torch.randn(2, Hkv, D, generator=_gen(100 * i + step)).bfloat16()
            hist[i].append(x)
            news[i].copy_(x)
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            k = torch.stack(hist[i]).double()
            want = [R.attend(qs[i][b].cpu().double(), k[:, b], 2 * k[:, b], 0.125) for b in range(2)]
            R.check(outs[i][0], outs[i][1], want)
            caches[i].check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lse = torch.empty(2, Hq, device=DEV)
    out = caches[1].attend(qs[1], _i32([1, 0]), out_lse=lse, stream=s)
    s.synchronize()
    R.check(out, lse, want)


def test_two_streams_at_once():
    """Cached rows, divided among CTAs and joined, and prompts, on two streams that overlap: as one after the other."""
    args, _, _ = _cache([5000, 17, 3000], 64, 2, 128, "bf16", seed=41, layers=1, layer=0)
    qc = [_q(3, 16, 128, 42 + i).to(DEV) for i in range(2)]
    q, k, v, cu, _ = _prompt([700, 900], [700, 900], 8, 2, 128, seed=43)
    dq, dk, dv, dcu = q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu)
    alone = [attend_cached(x, **args) for x in qc], attend_prompt(dq, dk, dv, dcu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for i, s in enumerate(streams):
            got.append((i, attend_cached(qc[i], stream=s, **args), attend_prompt(dq, dk, dv, dcu, stream=s)))
    torch.cuda.synchronize()
    for i, c, p in got:
        assert torch.equal(c, alone[0][i]) and torch.equal(p, alone[1])


def test_prompt_in_a_graph():
    ql = [50, 140]
    q, k, v, cu, _ = _prompt(ql, ql, 4, 2, 64, seed=40)
    dq, dk, dv, dcu = q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu)
    lse = torch.empty(len(q), 4, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = attend_prompt(dq, dk, dv, dcu, out_lse=lse)
    cu = [0, 90, 190]   # other lengths, same memory
    dcu.copy_(_i32(cu))
    g.replay()
    torch.cuda.synchronize()
    R.check(out, lse, _prompt_want(q, k, v, cu, cu, 0.125))


def test_divided_prompts_in_graphs_and_between_them():
    # each call has its own workspace: two graphs, and eager calls of other sizes between their replays
    shapes = [([3], [4000]), ([17, 2], [2500, 3100])]
    graphs, s = [], torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for ql, kl in shapes:
        q, k, v, cu_q, cu_k = _prompt(ql, kl, 8, 2, 64, seed=kl[0])
        d = [x.to(DEV) for x in (q, k, v)] + [_i32(cu_q), _i32(cu_k)]
        lse = torch.empty(len(q), 8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = attend_prompt(*d, out_lse=lse)
        graphs.append((g, d, out, lse, (q, k, v, cu_q, cu_k)))
    for turn in range(3):
        for g, d, out, lse, host in graphs:
            out.fill_(7), lse.fill_(7)
            g.replay()
        eager = [attend_prompt(*d) for _, d, _, _, _ in graphs]
        torch.cuda.synchronize()
        for (g, d, out, lse, host), e in zip(graphs, eager):
            assert torch.equal(out, e)
            if turn == 0:
                R.check(out, lse, _prompt_want(*host, 0.125))


def test_empty_calls():
    c = PagedCache(n_pages=2, page_size=4, n_kv_heads=1, head_dim=64, n_seqs=1, max_pages=2)
    none = _i32([])
    c.extend(none, none), c.fork(none, none), c.free(none), c.compact()
    c.write(none, _i32([0]), *(torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV),) * 2)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert c.attend(e, none).shape == (0, 2, 64)
    assert attend_prompt(e, e[:, :1], e[:, :1], _i32([0])).shape == (0, 2, 64)
    assert attend_prompt(e, e[:, :1], e[:, :1], _i32([0, 0, 0])).shape == (0, 2, 64)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert (attend_prompt(q, e[:, :1], e[:, :1], _i32([0, 3]), _i32([0, 0])) == 0).all()
    c.check()


# ------------------------------------------------------------ together
def test_index_selects_and_cache_attends():
    """A request as it is served: chunked prefill (index and cache side by side), then decode steps, a fork and its
    continuation; the attention over the selected keys against float64 on the ids the index returned."""
    d, H, Hq, Hkv, D, T, k, C = 128, 32, 8, 2, 128, 256, 96, 384
    g = _gen(50)
    n, steps = 3 * T, 5
    ik = torch.randn(n + steps, d, generator=g).bfloat16().to(DEV)
    iq = torch.randn(n + steps, H, d, generator=g).bfloat16().to(DEV)
    w = torch.randn(n + steps, H, generator=g).to(DEV)
    q = torch.randn(n + steps, Hq, D, generator=g).bfloat16()
    kk, vv = (torch.randn(n + steps, Hkv, D, generator=g).bfloat16() for _ in range(2))
    dq, dk, dv = q.to(DEV), kk.to(DEV), vv.to(DEV)
    idx = AttentionIndex(d=d, H=H, window=128, clusters_per_window=4, refit_period=0, max_query_chunk=T, max_budget=C,
                         max_k=k, max_keys=n + steps)
    c = PagedCache(n_pages=80, page_size=32, n_kv_heads=Hkv, head_dim=D, n_seqs=3, max_pages=30)

    def check(rows, ids, out, lse):
        want = []
        for j, t in enumerate(rows):
            at = [i for i in ids[j].tolist() if i >= 0]
            assert max(at) <= t
            want.append(R.attend(q[t].double(), kk[at].double(), vv[at].double(), D ** -0.5))
        R.check(out, lse, want)

    spans = [(p, p + T) for p in range(0, n, T)] + [(n + i, n + i + 1) for i in range(steps)]
    for p0, p1 in spans:
        m = p1 - p0
        idx.append_keys(ik[p0:p1])
        idx.seal()
        c.extend(_i32([0]), _i32([m]))
        c.write(_i32([0]), _i32([0, m]), dk[p0:p1], dv[p0:p1])
        lse = torch.empty(m, Hq, device=DEV)
        ids = torch.empty(m, k, dtype=torch.int32, device=DEV)
        out = idx.attend(iq[p0:p1], w[p0:p1], p0, k, C, dq[p0:p1], c, seq=0, out_ids=ids, out_lse=lse)
        rows = list(range(0, m, 37)) + [m - 1]
        check([p0 + i for i in rows], ids[rows].cpu(), out[rows], lse[rows])
    idx.sync()
    # branch, take one more token in each, attend over everything
    c.fork(_i32([0]), _i32([2]))
    c.extend(_i32([2, 0]), _i32([1, 1]))
    new = torch.randn(2, Hkv, D, generator=g).bfloat16()
    c.write(_i32([2, 0]), _i32([0, 1, 2]), new.to(DEV), -new.to(DEV))
    c.free(_i32([1]))
    c.compact()
    lse = torch.empty(2, Hq, device=DEV)
    out = c.attend(dq[:2], _i32([2, 0]), out_lse=lse)
    want = []
    for b in range(2):
        ke, ve = torch.cat([kk, new[b:b + 1]]).double(), torch.cat([vv, -new[b:b + 1]]).double()
        want.append(R.attend(q[b].double(), ke, ve, D ** -0.5))
    R.check(out, lse, want)
    c.check()
    idx.close()
