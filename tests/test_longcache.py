"""CPU tests of the operators that read less of a long cache: refusals of bad
arguments, and the shared plan.  No kernel is launched."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def mla():
    import __graft_entry__
    __graft_entry__._builder().build()
    import mla_decode_stage1_gb300 as m
    m.mla_shared_run         # loads longcache.py, which declares the argument types
    return m


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    mem.keep = buf
    return (ctypes.addressof(buf) + 255) & ~255


def plan(mla, groups, prefix, kvp, last=None, ps=8, q_len=1, qd="bf16", kd="bf16", sms=152, form="once"):
    return mla.mla_shared_plan(np.asarray(groups, np.int32), np.asarray(prefix, np.int32),
                               np.asarray(kvp, np.int32), last, page_size=ps, q_len=q_len,
                               q_dtype=qd, kv_dtype=kd, num_sms=sms, form=form)


@pytest.mark.parametrize("groups,prefix,kvp,last,kw,status", [
    ([1, 2], [0, 4], [0, 1, 2], None, {}, 1),            # groups do not begin at 0
    ([0, 2, 1], [0, 4, 8], [0, 1], None, {}, 1),         # decreasing
    ([0, 0], [0, 4], [0], None, {}, 1),                  # no request
    ([0, 2], [-1, 4], [0, 1, 2], None, {}, 1),
    ([0, 2], [4, 0], [0, 1, 2], None, {}, 1),
    ([0, 2], [0, 4], [0, 2, 1], None, {}, 1),
    ([0, 2], [0, 4], [-1, 1, 2], None, {}, 1),
    ([0, 2], [0, 4], [0, 1, 2], [0, 1], {}, 1),
    ([0, 2], [0, 4], [0, 1, 2], [1, 9], {}, 1),
    ([0, 2], [0, 4], [0, 1, 2], None, dict(ps=0), 1),
    ([0, 2], [0, 4], [0, 1, 2], None, dict(q_len=0), 1),
    ([0, 2], [0, 4], [0, 1, 2], None, dict(q_len=65), 1),
    ([0, 2], [0, 4], [0, 1, 2], None, dict(sms=-1), 1),
    ([0, 2], [0, 4], [0, 1, 2], [3, 2], dict(q_len=4), 1),    # a token would not see all of the prefix
    ([0, 2], [0, 2 ** 29], [0, 1, 2], None, {}, 1),
    ([0, 2], [0, 4], [0, 1, 2], None, dict(qd="fp8", kd="mxfp4"), 2),
    ([0, 2], [0, 4], [0, 1, 2], None, dict(qd="mxfp4"), 2)])
def test_shared_plan_refuses(mla, groups, prefix, kvp, last, kw, status):
    with pytest.raises(mla.MlaError) as e:
        plan(mla, groups, prefix, kvp, last, **kw)
    assert e.value.status == status


def test_shared_plan_refuses_mismatched_batches(mla):
    with pytest.raises(ValueError):
        plan(mla, [0, 2], [0, 4, 5], [0, 1, 2])
    with pytest.raises(ValueError):
        plan(mla, [0, 2], [0, 4], [0, 1])
    with pytest.raises(ValueError):
        plan(mla, [0, 2], [0, 4], [0, 1, 2], [1])
    with pytest.raises(ValueError):
        plan(mla, [0], [0], [0])
    f = mla._lib.mla_shared_plan
    assert f(None, None, 1, None, None, 1, 8, 0, 0, 8, 0, None) == 1
    h = ctypes.c_void_p()
    assert f(None, None, 1, None, None, 1, 8, 0, 0, 8, 0, ctypes.byref(h)) == 1 and not h
    at = (ctypes.c_int32 * 2)(0, 1)
    for form, status in ((-1, 1), (0, 0), (1, 0), (2, 0), (3, 1)):
        assert f(at, at, 1, at, None, 1, 8, 0, 0, 8, form, ctypes.byref(h)) == status
        mla._lib.mla_shared_destroy(h)
    with pytest.raises(ValueError):
        plan(mla, [0, 2], [0, 4], [0, 1, 2], form="never")


def test_shared_plan_allows_short_ends(mla):
    # query tokens need q_len - 1 own tokens, and none where there is no prefix
    plan(mla, [0, 2], [0, 4], [0, 1, 2], [3, 3], q_len=4)
    plan(mla, [0, 2], [0, 4], [0, 0, 1])
    plan(mla, [0, 1, 2], [0, 0, 4], [0, 0, 1], q_len=4)
    with pytest.raises(mla.MlaError):
        plan(mla, [0, 1, 2], [0, 4, 4], [0, 0, 1], q_len=4)


def test_shared_plan_sizes(mla):
    # groups of 9 and 20 requests (two and three blocks of 8 tokens), one without a prefix
    p = plan(mla, [0, 9, 10, 30], [0, 50, 50, 113], list(range(31)), sms=152)
    info = p.info()
    assert (info.batch_size, info.num_groups, info.q_len) == (30, 3, 1)
    assert info.prefix_tokens == 113 * 8 and info.own_tokens == 30 * 8
    # 4 and 4 tiles of 128 keys: 2 x 4 + 3 x 4 of them at most
    assert 3 <= info.num_items <= 20 and info.num_clusters <= 76
    assert info.block_rows in (128, 256) and p.query_tokens == 30
    assert p.workspace_bytes >= 8 * 128 * 1152 + info.num_items * info.block_rows * 2052
    # a bf16 pool in pages of a multiple of 64 is not gathered, others are
    size = [plan(mla, [0, 2], [0, 1000], [0, 1, 2], ps=ps, kd=kd).workspace_bytes
            for ps, kd in ((64, "bf16"), (64, "fp8"), (32, "bf16"))]
    assert size[0] < 64000 * 1152 < size[1] and size[2] > 32000 * 1152
    # prefixes of groups without requests are not gathered
    assert plan(mla, [0, 0, 2], [0, 50, 60], [0, 1, 2]).info().prefix_tokens == 80
    assert plan(mla, [0, 2], [0, 0], [0, 1, 2]).info().num_items == 0


@pytest.mark.parametrize("sms", [1, 2, 3, 4, 7, 64, 152])
def test_shared_plan_uses_the_clusters(mla, sms):
    p = plan(mla, [0, 40], [0, 1000], list(range(41)), sms=sms).info()
    clusters = max(1, sms // (2 if p.block_rows == 128 else 4))
    # 640 rows, 63 tiles
    blocks = -(-640 // p.block_rows)
    assert p.num_clusters <= clusters and p.num_clusters >= min(clusters, blocks) * 3 // 4
    assert blocks <= p.num_items <= blocks + clusters


def test_shared_plan_takes_blocks_of_256_rows_where_they_fill(mla):
    assert plan(mla, [0, 256], [0, 1000], list(range(257))).info().block_rows == 256
    assert plan(mla, [0, 8], [0, 1000], list(range(9))).info().block_rows == 128
    assert plan(mla, [0, 256], [0, 1000], list(range(257)), sms=3).info().block_rows == 128


def test_shared_plan_for_each_request(mla):
    kw = dict(groups=[0, 9, 10, 30], prefix=[0, 50, 50, 113], kvp=list(range(31)))
    p = plan(mla, form="each", **kw).info()
    assert (p.num_items, p.num_clusters, p.prefix_tokens, p.own_tokens) == (0, 0, 113 * 8, 240)
    assert plan(mla, form="auto", **kw).info().num_items == 0
    assert plan(mla, [0, 64], [0, 4096], [0] * 65, form="auto").info().num_items > 0
    # no rows are kept, whatever the pool
    assert plan(mla, [0, 2], [0, 1000], [0, 1, 2], form="each").workspace_bytes < 152 * 2 * 33000 + 65536


def test_shared_plan_leaves_sms_for_the_own_ends(mla):
    # 64 requests with 500 own tokens behind 16,384: the decode kernel's CTAs and the
    # clusters' fit the SMs together; without own tokens the clusters have them all
    p = plan(mla, [0, 64], [0, 2048], [63 * i for i in range(65)]).info()
    alone = plan(mla, [0, 64], [0, 2048], [0] * 65).info()
    assert p.num_clusters < alone.num_clusters == 38
    assert plan(mla, [0, 64], [0, 2048], [63 * i for i in range(65)], sms=3).info().num_clusters == 1
    # any number of CTAs is planned for in no time
    assert plan(mla, [0, 64], [0, 2048], [63 * i for i in range(65)], sms=1 << 20).info().num_items > 0


def run_args(p, a, **kw):
    d = dict(plan=p.handle, q=a, qs=None, kv=a, ks=None, e8=None, e8s=0, rows=1 << 20, pidx=a, idx=a,
             ws=a, wsb=p.workspace_bytes, out=a, lse=None)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), 1), (dict(q=None), 1), (dict(kv=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(rows=0), 1), (dict(rows=1 << 31), 1), (dict(rows=(1 << 20) + 1), 1),
    (dict(wsb=1000), 3)])
def test_shared_run_refuses(mla, mem, kw, status):
    p = plan(mla, [0, 2], [0, 4], [0, 1, 2])
    assert mla._lib.mla_shared_run(*run_args(p, mem, **kw)) == status


@pytest.mark.parametrize("name,by", [("q", 8), ("kv", 8), ("out", 8), ("ws", 128), ("lse", 2),
                                     ("pidx", 2), ("idx", 2)])
def test_shared_run_refuses_misaligned(mla, mem, name, by):
    p = plan(mla, [0, 2], [0, 4], [0, 1, 2])
    assert mla._lib.mla_shared_run(*run_args(p, mem, **{name: mem + by})) == 1


def test_shared_run_refuses_missing_scales_and_short_pools(mla, mem):
    f = mla._lib.mla_shared_run
    p = plan(mla, [0, 2], [0, 4], [0, 1, 2], qd="fp8", kd="fp8")
    assert f(*run_args(p, mem, ks=mem)) == 1
    assert f(*run_args(p, mem, qs=mem)) == 1
    p = plan(mla, [0, 2], [0, 4], [0, 1, 2], kd="mxfp4")
    assert f(*run_args(p, mem)) == 1
    assert f(*run_args(p, mem, e8=mem, e8s=17)) == 1
    assert f(*run_args(p, mem, e8=mem, e8s=19)) == 2
    # identity tables must lie in the pool
    p = plan(mla, [0, 2], [2, 6], [0, 1, 2])
    assert f(*run_args(p, mem, pidx=None, rows=47)) == 1
    p = plan(mla, [0, 2], [0, 1], [5, 6, 7])
    assert f(*run_args(p, mem, idx=None, rows=48)) == 1


def test_shared_info_and_check_refuse(mla, mem):
    assert mla._lib.mla_shared_get_info(None, None) == 1
    assert mla._lib.mla_shared_check(None, mem, None) == 1
    p = plan(mla, [0, 2], [0, 4], [0, 1, 2])
    assert mla._lib.mla_shared_check(p.handle, None, None) == 1


def bounds_args(a, **kw):
    d = dict(kv=a, dtype=0, e8=None, e8s=0, rows=64, page=8, old=a, new=a, bs=2, table=a, stride=4,
             cols=4, bounds=a, pages=8, err=a)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw", [
    dict(kv=None), dict(dtype=3), dict(dtype=-1), dict(dtype=2), dict(dtype=2, e8=1, e8s=17),
    dict(rows=0), dict(rows=1 << 31), dict(page=0), dict(old=None), dict(bs=0), dict(table=None),
    dict(stride=3), dict(cols=-1), dict(bounds=None), dict(pages=0),
    dict(bs=1 << 20, cols=2048, stride=2048)])
def test_page_bounds_refuses(mla, mem, kw):
    assert mla._lib.mla_page_bounds(*bounds_args(mem, **kw)) == 1


@pytest.mark.parametrize("name,by", [("kv", 8), ("old", 2), ("new", 1), ("table", 2), ("bounds", 16),
                                     ("err", 2)])
def test_page_bounds_refuses_misaligned(mla, mem, name, by):
    assert mla._lib.mla_page_bounds(*bounds_args(mem, **{name: mem + by})) == 1


def scores_args(a, **kw):
    d = dict(q=a, dtype=0, qs=None, ks=None, bounds=a, pages=8, lens=a, bs=2, q_len=1, page=8, table=a,
             stride=4, cols=4, scores=a, sstride=4, err=a)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(dtype=1), 1), (dict(dtype=2), 2), (dict(dtype=7), 2),
    (dict(bounds=None), 1), (dict(pages=0), 1), (dict(lens=None), 1), (dict(bs=0), 1),
    (dict(q_len=0), 1), (dict(q_len=65), 1), (dict(page=0), 1), (dict(table=None), 1),
    (dict(stride=3), 1), (dict(cols=-1), 1), (dict(scores=None), 1), (dict(sstride=3), 1),
    (dict(bs=1 << 30, cols=4096, stride=4096, sstride=4096), 1),
    (dict(cols=0), 0)])
def test_page_scores_refuses(mla, mem, kw, status):
    assert mla._lib.mla_page_scores(*scores_args(mem, **kw)) == status


@pytest.mark.parametrize("name,by", [("q", 8), ("bounds", 16), ("lens", 2), ("table", 1), ("scores", 2),
                                     ("ks", 2), ("err", 1)])
def test_page_scores_refuses_misaligned(mla, mem, name, by):
    assert mla._lib.mla_page_scores(*scores_args(mem, **{name: mem + by})) == 1


def select_args(a, **kw):
    d = dict(scores=a, sstride=4, lens=a, bs=2, q_len=1, page=8, table=a, stride=4, cols=4, top=3,
             first=1, last=1, kvp=a, lastp=a, idx=a, nidx=6, columns=a, err=a)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw", [
    dict(scores=None), dict(sstride=3), dict(lens=None), dict(bs=0), dict(q_len=0), dict(q_len=65),
    dict(page=0), dict(table=None), dict(stride=3), dict(cols=-1), dict(top=0), dict(first=-1),
    dict(last=0), dict(first=2, last=2), dict(first=2 ** 31 - 1, last=1), dict(kvp=None),
    dict(lastp=None), dict(idx=None), dict(nidx=-1),
    dict(bs=1 << 30, cols=4096, stride=4096, sstride=4096, top=2048)])
def test_page_select_refuses(mla, mem, kw):
    assert mla._lib.mla_page_select(*select_args(mem, **kw)) == 1


@pytest.mark.parametrize("name", ["scores", "lens", "table", "kvp", "lastp", "idx", "columns", "err"])
def test_page_select_refuses_misaligned(mla, mem, name):
    assert mla._lib.mla_page_select(*select_args(mem, **{name: mem + 2})) == 1


def test_the_binding_refuses_tensors_that_do_not_fit(mla):
    import torch
    p = plan(mla, [0, 2], [0, 4], [0, 1, 2])
    q = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):           # not on a GPU
        mla.mla_shared_run(p, q, q, q, workspace=q)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_page_bounds(q, q, i32, i32, page_size=8, kv_dtype="bf16")
    with pytest.raises(ValueError):
        mla.mla_page_scores(q, q, i32, i32, q, page_size=8)
    with pytest.raises(ValueError):
        mla.mla_page_select(q, i32, i32, page_size=8, top_pages=2, kv_indptr=i32, kv_last_page_len=i32,
                            kv_indices=i32)
