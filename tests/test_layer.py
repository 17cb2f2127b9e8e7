"""CPU tests of the operators around the decode call: refusals of bad
arguments, and the prefill plan.  No kernel is launched."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def mla():
    import __graft_entry__
    __graft_entry__._builder().build()
    import mla_decode_stage1_gb300 as m
    m.mla_error_check        # loads layer.py, which declares the argument types
    return m


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    mem.keep = buf
    return (ctypes.addressof(buf) + 255) & ~255


def step_args(a, **kw):
    d = dict(old=a, new=a, bs=2, page=8, table=a, stride=4, cols=4, free=a, nfree=3, kvp=a, last=a,
             idx=a, nidx=8, qo=a, slots=a, pos=a, ntok=4, used=a, err=a)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw", [
    dict(old=None), dict(bs=0), dict(page=0), dict(table=None), dict(stride=3), dict(cols=-1),
    dict(free=None), dict(nfree=-1), dict(kvp=None), dict(last=None), dict(idx=None),
    dict(nidx=-1), dict(qo=None), dict(slots=None), dict(pos=None), dict(ntok=-1)])
def test_cache_step_refuses(mla, mem, kw):
    assert mla._lib.mla_cache_step(*step_args(mem, **kw)) == 1


@pytest.mark.parametrize("name,by", [("old", 2), ("new", 1), ("table", 2), ("slots", 4), ("err", 1)])
def test_cache_step_refuses_misaligned(mla, mem, name, by):
    assert mla._lib.mla_cache_step(*step_args(mem, **{name: mem + by})) == 1


def write_args(a, **kw):
    d = dict(latent=a, ls=512, rope=a, rs=64, weight=a, eps=1e-6, cs=a, npos=8, pos=a, style=0,
             slots=a, tokens=4, dtype=0, kv=a, scale=None, e8=None, e8s=0, rows=16, out=None,
             err=None)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw", [
    dict(latent=None), dict(ls=511), dict(ls=516), dict(rope=None), dict(rs=63), dict(eps=-1.0),
    dict(eps=float("nan")), dict(cs=None), dict(pos=None), dict(npos=0), dict(style=2),
    dict(slots=None), dict(tokens=-1), dict(dtype=3), dict(dtype=-1), dict(kv=None),
    dict(dtype=1), dict(dtype=2), dict(rows=0), dict(rows=1 << 31)])
def test_cache_write_refuses(mla, mem, kw):
    assert mla._lib.mla_cache_write(*write_args(mem, **kw)) == 1


@pytest.mark.parametrize("kw", [dict(latent=8), dict(kv=8), dict(weight=8), dict(slots=4),
                                dict(out=8), dict(rope=1)])
def test_cache_write_refuses_misaligned(mla, mem, kw):
    assert mla._lib.mla_cache_write(*write_args(mem, **{k: mem + v for k, v in kw.items()})) == 1


def test_cache_write_refuses_narrow_scale_rows(mla, mem):
    assert mla._lib.mla_cache_write(*write_args(mem, dtype=2, e8=mem, e8s=17)) == 1


def q_args(a, **kw):
    d = dict(q=a, ts=16 * 192, hs=192, w=a, tokens=2, heads=16, scale=0.07, cs=a, npos=8, pos=a,
             style=0, dtype=0, qs=None, out=a, err=None)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(ts=191), 1), (dict(ts=196), 1),
    (dict(hs=190), 1), (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(heads=1025), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(cs=None), 1), (dict(pos=None), 1), (dict(npos=0), 1), (dict(style=-1), 1),
    (dict(dtype=1), 1), (dict(dtype=2), 2), (dict(dtype=9), 2)])
def test_absorb_q_refuses(mla, mem, kw, status):
    assert mla._lib.mla_absorb_q(*q_args(mem, **kw)) == status


@pytest.mark.parametrize("name", ["q", "w", "out"])
def test_absorb_q_refuses_misaligned(mla, mem, name):
    assert mla._lib.mla_absorb_q(*q_args(mem, **{name: mem + 8})) == 1


def test_absorb_out_refuses(mla, mem):
    f = mla._lib.mla_absorb_out
    assert f(None, mem, 1, 16, mem, None) == 1
    assert f(mem, None, 1, 16, mem, None) == 1
    assert f(mem, mem, 1, 16, None, None) == 1
    assert f(mem, mem, -1, 16, mem, None) == 1
    assert f(mem, mem, 1, 0, mem, None) == 1
    assert f(mem + 8, mem, 1, 16, mem, None) == 1
    assert f(mem, mem, 0, 16, mem, None) == 0


def test_error_check_refuses(mla, mem):
    assert mla._lib.mla_error_check(None, None) == 1
    assert mla._lib.mla_error_check(mem + 2, None) == 1


def plan(mla, qo, kvp, last=None, ps=1, heads=2, kd="bf16", sms=8):
    return mla.mla_prefill_plan(np.asarray(qo, np.int32), np.asarray(kvp, np.int32), last,
                                page_size=ps, kv_dtype=kd, heads=heads, num_sms=sms)


@pytest.mark.parametrize("qo,kvp,last,ps,heads", [
    ([1, 3], [0, 3], None, 1, 2), ([0, 3, 2], [0, 3, 5], None, 1, 2), ([0, 3], [-1, 3], None, 1, 2),
    ([0, 3], [4, 3], None, 1, 2), ([0, 3], [0, 2], [0], 4, 2), ([0, 3], [0, 2], [5], 4, 2),
    ([0, 3], [0, 3], None, 0, 2), ([0, 3], [0, 3], None, 1, 0), ([0, 3], [0, 3], None, 1, 1025),
    ([0, 3], [0, 2 ** 30], None, 8, 2)])
def test_prefill_plan_refuses(mla, qo, kvp, last, ps, heads):
    with pytest.raises(mla.MlaError) as e:
        plan(mla, qo, kvp, last, ps, heads)
    assert e.value.status == 1


def test_prefill_plan_refuses_mismatched_batches(mla):
    with pytest.raises(ValueError):
        plan(mla, [0, 3], [0, 3, 4])
    with pytest.raises(ValueError):
        plan(mla, [0, 3], [0, 3], [1, 1])
    assert mla._lib.mla_prefill_plan(None, None, None, 1, 1, 1, 0, 1, None) == 1


def test_prefill_plan_sizes(mla):
    p = plan(mla, [0, 300, 300, 301], [0, 300, 400, 400], heads=3, sms=8)
    info = p.info()
    assert (info.batch_size, info.heads, info.query_tokens, info.key_tokens) == (3, 3, 301, 400)
    # request 0: two row blocks x three heads, split or not; request 2 has no keys
    assert info.num_items >= 9 and info.num_ctas <= 8
    # 3 key tiles of 128 are expanded (request 1 has no queries)
    assert p.workspace_bytes >= 3 * 128 * (3 * 256 + 64) * 2


def test_prefill_plan_splits_long_keys_over_the_ctas(mla):
    p = plan(mla, [0, 4], [0, 1 << 16], heads=2, sms=152)
    # (items of at most 128 rows hold two partial results)
    assert 100 <= p.info().num_items <= 2 * 152
    assert p.info().num_partials == 2 * p.info().num_items
    # a batch with enough whole items is not split
    assert plan(mla, [0, 8192], [0, 8192], heads=16, sms=152).info().num_partials == 0


def test_prefill_plan_of_nothing(mla):
    info = plan(mla, [0, 0], [0, 5]).info()
    assert (info.num_items, info.num_ctas, info.num_partials) == (0, 0, 0)


def run_args(p, a, **kw):
    d = dict(plan=p.handle, q=a, ts=2 * 192, hs=192, kv=a, scale=a, e8=None, e8s=0, rows=64,
             idx=None, w=a, sm=0.07, cs=None, npos=0, pos=None, style=0, ws=a, wsb=1 << 40, out=a,
             lse=None)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), 1), (dict(q=None), 1), (dict(kv=None), 1), (dict(w=None), 1),
    (dict(ws=None), 1), (dict(out=None), 1), (dict(ts=100), 1), (dict(ts=2 * 192 + 4), 1),
    (dict(ts=1 << 39), 1), (dict(hs=180), 1), (dict(scale=None), 1), (dict(rows=0), 1),
    (dict(rows=1 << 31), 1), (dict(rows=63), 1), (dict(sm=0.0), 1), (dict(sm=float("inf")), 1),
    (dict(style=7), 1), (dict(npos=5, cs=1), 1), (dict(wsb=256), 3)])
def test_prefill_run_refuses(mla, mem, kw, status):
    p = plan(mla, [0, 16], [0, 16], ps=4, kd="fp8")       # identity rows 0..63
    assert mla._lib.mla_prefill_run(*run_args(p, mem, **kw)) == status


@pytest.mark.parametrize("name", ["q", "kv", "w", "out", "ws"])
def test_prefill_run_refuses_misaligned(mla, mem, name):
    p = plan(mla, [0, 16], [0, 16], ps=4, kd="fp8")
    assert mla._lib.mla_prefill_run(*run_args(p, mem, **{name: mem + 8})) == 1


def test_prefill_run_refuses_out_and_tables_off_their_alignment(mla, mem):
    p = plan(mla, [0, 16], [0, 16], ps=4, kd="fp8")
    assert mla._lib.mla_prefill_run(*run_args(p, mem, out=mem + 16)) == 1
    assert mla._lib.mla_prefill_run(*run_args(p, mem, cs=mem + 8, npos=4, pos=mem)) == 1


def test_prefill_run_refuses_pools(mla, mem):
    p = plan(mla, [0, 16], [0, 16], ps=4, kd="fp8")
    assert mla._lib.mla_prefill_run(*run_args(p, mem, idx=mem, rows=66)) == 1     # not whole pages
    p = plan(mla, [0, 16], [0, 16], ps=4, kd="mxfp4")
    assert mla._lib.mla_prefill_run(*run_args(p, mem)) == 1                       # no scale rows
    assert mla._lib.mla_prefill_run(*run_args(p, mem, e8=mem, e8s=17)) == 1
    assert mla._lib.mla_prefill_run(*run_args(p, mem, e8=mem, e8s=19)) == 2
    assert mla._lib.mla_prefill_run(*run_args(p, mem, e8=mem + 1, e8s=18)) == 2


def test_bindings_refuse_host_tensors_and_types(mla):
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_error_check(i[:1])
    with pytest.raises(ValueError):
        mla.mla_cache_step(i, i, i.view(1, 2), i, page_size=1, kv_indptr=i, kv_last_page_len=i,
                           kv_indices=i, qo_indptr=i, slots=i, positions=i)
    b = torch.zeros(1, 16, 192, dtype=torch.bfloat16)
    w = torch.zeros(16, 256, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_absorb_q(b, w, b, sm_scale=1.0)
    with pytest.raises(ValueError):
        mla.mla_absorb_out(b, w, b)


def test_no_tokens_with_a_rotation(mla, mem):
    # an empty tensor of positions has no address
    none = dict(tokens=0, cs=mem, npos=8, pos=None)
    assert mla._lib.mla_cache_write(*write_args(mem, slots=None, latent=None, rope=None, **none)) == 0
    assert mla._lib.mla_absorb_q(*q_args(mem, q=None, out=None, **none)) == 0
    assert mla._lib.mla_absorb_q(*q_args(mem, **dict(none, style=2))) == 1
    assert mla._lib.mla_absorb_q(*q_args(mem, **dict(none, tokens=1))) == 1


def test_absorb_out_ex_refuses(mla, mem):
    f = mla._lib.mla_absorb_out_ex
    assert f(mem, mem, 1, 16, None, mem, None) == 1
    assert f(mem, mem, 0, 16, mem, mem + 2, None) == 1
    assert f(mem, mem, 0, 16, mem, mem, None) == 0
    g = mla._lib.mla_selftest_absorb_wait
    assert g(mem, mem, 0, 16, None, mem, 0, 0, mem, None) == 1
    assert g(mem, mem, 0, 16, None, mem, 1, 20001, mem, None) == 1
    assert g(mem, mem, 1, 16, None, None, 1, 100, mem, None) == 1
    import torch
    b = torch.zeros(1, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_absorb_out(b, torch.zeros(16, 256, 512, dtype=torch.bfloat16), b, err=b)


class OnDevice:
    """A host tensor that says that it is on CUDA device `dev`."""

    is_cuda = True

    def __init__(self, t, dev):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def calls_of_the_layer(mla):
    """name -> (call, its tensors), all of them with right shapes."""
    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)          # noqa: E731
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64)          # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)        # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)           # noqa: E731
    f32 = lambda *s: torch.zeros(*s)                             # noqa: E731
    rope = dict(positions=i32(2), cos_sin=f32(4, 64))
    p = plan(mla, [0, 2], [0, 2], heads=2, kd="fp8")
    return dict(
        mla_cache_step=(lambda **a: mla.mla_cache_step(
            a.pop("old"), a.pop("new"), a.pop("table"), a.pop("free"), page_size=1, **a), dict(
            old=i32(2), new=i32(2), table=i32(2, 3), free=i32(4), kv_indptr=i32(3),
            kv_last_page_len=i32(2), kv_indices=i32(4), qo_indptr=i32(3), slots=i64(4),
            positions=i32(4), pages_used=i32(1), err=i32(1))),
        mla_cache_write=(lambda **a: mla.mla_cache_write(
            a.pop("latent"), a.pop("k_rope"), a.pop("kv"), a.pop("slots"), kv_dtype="fp8", **a),
            dict(latent=bf(2, 512), k_rope=bf(2, 64), kv=u8(4, 576), slots=i64(2), err=i32(1),
                 norm_weight=bf(512), kv_scale=f32(1), rows=bf(2, 576), **rope)),
        mla_cache_write_mxfp4=(lambda **a: mla.mla_cache_write(
            a.pop("latent"), a.pop("k_rope"), a.pop("kv"), a.pop("slots"), kv_dtype="mxfp4", **a),
            dict(latent=bf(2, 512), k_rope=bf(2, 64), kv=u8(4, 288), slots=i64(2),
                 kv_e8m0=u8(4, 18))),
        mla_absorb_q=(lambda **a: mla.mla_absorb_q(
            a.pop("q"), a.pop("w"), a.pop("q_out"), sm_scale=1.0, **a),
            dict(q=bf(2, 2, 192), w=bf(2, 256, 512), q_out=u8(2, 2, 576), q_scale=f32(1),
                 err=i32(1), **rope)),
        mla_absorb_out=(lambda **a: mla.mla_absorb_out(a.pop("o"), a.pop("w"), a.pop("out"), **a),
                        dict(o=bf(2, 2, 512), w=bf(2, 256, 512), out=bf(2, 2, 128), err=i32(1))),
        mla_prefill_run=(lambda **a: mla.mla_prefill_run(
            p, a.pop("q"), a.pop("kv"), a.pop("w"), a.pop("out"), sm_scale=1.0, **a),
            dict(q=bf(2, 2, 192), kv=u8(2, 576), w=bf(2, 256, 512), out=bf(2, 2, 128),
                 workspace=u8(256), kv_scale=f32(1), kv_indices=i32(2), lse=f32(2, 2), **rope)),
        mla_prefill_check=(lambda workspace: mla.mla_prefill_check(p, workspace),
                           dict(workspace=u8(256))),
        mla_error_check=(mla.mla_error_check, dict(err=i32(1))))


@pytest.mark.parametrize("name", ["mla_cache_step", "mla_cache_write", "mla_cache_write_mxfp4",
                                  "mla_absorb_q", "mla_absorb_out", "mla_prefill_run",
                                  "mla_prefill_check", "mla_error_check"])
def test_tensors_of_another_device_are_refused(mla, monkeypatch, name):
    # the library launches on the current device: every tensor has to be there
    from mla_decode_stage1_gb300 import layer
    call, tensors = calls_of_the_layer(mla)[name]
    launched = []

    def library(*args):
        launched.append(args)
        return 0

    for f in ("_cache_step", "_cache_write", "_absorb_q", "_absorb_out", "_prefill_run"):
        monkeypatch.setattr(layer, f, library)
    monkeypatch.setattr(layer, "_lib", type("Library", (), dict(
        mla_prefill_check=staticmethod(library), mla_error_check=staticmethod(library),
        mla_prefill_destroy=staticmethod(library))))
    monkeypatch.setattr(layer, "_raw_stream", lambda dev: 0)
    current = [0]
    monkeypatch.setattr(layer, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(layer, "_several_devices", True, raising=False)
    def on(dev, other=None):
        return {k: OnDevice(t, 1 if k == other else dev) for k, t in tensors.items()}

    call(**on(0))
    assert len(launched) == 1
    for other in tensors:
        with pytest.raises(ValueError):
            call(**on(0, other))
    with pytest.raises(ValueError):
        call(**on(1))
    with pytest.raises(ValueError):
        call(**tensors)                        # on the host
    if "check" not in name:
        with pytest.raises(ValueError):
            call(**on(0), stream=type("Stream", (), dict(
                device=type("Device", (), dict(index=1)), cuda_stream=0)))
    assert len(launched) == 1
    current[0] = 1
    call(**on(1))
    assert len(launched) == 2


@pytest.mark.parametrize("qo,heads", [([0, 2 ** 31 - 1], 1024), ([0, 2 ** 30, 2 ** 31 - 1], 8),
                                      ([0, 8 * 2 ** 20, 16 * 2 ** 20], 1024)])
def test_prefill_plan_refuses_more_blocks_than_it_can_list(mla, qo, heads):
    import resource
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    with pytest.raises(mla.MlaError) as e:
        plan(mla, qo, [0] * len(qo), heads=heads)
    assert e.value.status == 1
    # the first 2^25 items at most (1 GB a list) have been built
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 5 * 2 ** 20
