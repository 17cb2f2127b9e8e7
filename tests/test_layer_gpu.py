"""GPU tests of the operators around the decode call against plain
implementations in 64 bits.

Tolerances count roundings: u = 2^-8 bounds one rounding to bf16 (half of
torch.finfo's eps), 2^-4 one to e4m3, F = 2^-24 one to fp32.  Each test states
the roundings of its path; sums of n fp32 products get n F of the sum of their
magnitudes.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -24
SCALE = 1 / math.sqrt(192)


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_decode_stage1_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def rotation_table(n):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, table, pos, rope):
    """x [t, ..., 64] in x's precision."""
    cs = table[pos.long()].to(x.dtype).reshape(len(pos), *([1] * (x.dim() - 2)), 64)
    c, s = cs[..., :32], cs[..., 32:]
    if rope == "half":
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


# ------------------------------------------------------------------ cache step
def plain_step(old, new, page, table, free):
    """Lists in, (table, outputs) out; pages missing from `free` are -1."""
    table = [list(r) for r in table]
    used, kvp, qo, idx, last, slots, pos = 0, [0], [0], [], [], [], []
    for b, (o, n) in enumerate(zip(old, new)):
        have, pages = -(-o // page), -(-(o + n) // page)
        for j in range(have, pages):
            table[b][j] = free[used] if used < len(free) else -1
            used += 1
        idx += table[b][:pages]
        kvp.append(kvp[-1] + pages)
        qo.append(qo[-1] + n)
        last.append(o + n - (pages - 1) * page if pages else 0)
        for p in range(o, o + n):
            pg = table[b][p // page]
            slots.append(pg * page + p % page if pg >= 0 else -1)
            pos.append(p)
    return table, dict(kvp=kvp, qo=qo, idx=idx, last=last, slots=slots, pos=pos,
                       used=min(used, len(free)))


def run_step(mla, old, new, page, table, free, pad_idx=0, pad_tok=0, stride=None, err=None):
    bs, cols = len(old), len(table[0])
    nnew = new if new is not None else [1] * bs
    store = torch.full((bs, stride or cols), -7, dtype=torch.int32, device="cuda")
    t = store[:, :cols]
    t.copy_(i32(table))
    npages = sum(-(-(a + b) // page) for a, b in zip(old, nnew))
    o = dict(kvp=torch.full((bs + 1,), -9, dtype=torch.int32, device="cuda"),
             qo=torch.full((bs + 1,), -9, dtype=torch.int32, device="cuda"),
             last=torch.full((bs,), -9, dtype=torch.int32, device="cuda"),
             idx=torch.full((npages + pad_idx,), -9, dtype=torch.int32, device="cuda"),
             slots=torch.full((sum(nnew) + pad_tok,), -9, dtype=torch.int64, device="cuda"),
             pos=torch.full((sum(nnew) + pad_tok,), -9, dtype=torch.int32, device="cuda"),
             used=torch.full((1,), -9, dtype=torch.int32, device="cuda"))
    args = (i32(old), None if new is None else i32(new), t, i32(free))
    kw = dict(page_size=page, kv_indptr=o["kvp"], kv_last_page_len=o["last"], kv_indices=o["idx"],
              qo_indptr=o["qo"], slots=o["slots"], positions=o["pos"], pages_used=o["used"],
              err=err)
    mla.mla_cache_step(*args, **kw)
    mla.mla_cache_step(*args, **kw)          # a repeated call changes nothing
    if stride and stride > cols:
        assert (store[:, cols:] == -7).all()
    return t.tolist(), {k: v.tolist() for k, v in o.items()}


def step_case(bs, page, old_hi, new_hi, seed):
    g = gen(seed)
    old = torch.randint(0, old_hi + 1, (bs,), generator=g).tolist()
    new = torch.randint(0, new_hi + 1, (bs,), generator=g).tolist()
    have = [-(-a // page) for a in old]
    pages = [-(-(a + b) // page) for a, b in zip(old, new)]
    ids = torch.randperm(sum(pages) + 5, generator=g).tolist()
    cols, at, table = max(max(pages), 1) + 2, 0, []
    for h in have:
        table.append(ids[at: at + h] + [0] * (cols - h))
        at += h
    return old, new, table, ids[at:]


@pytest.mark.parametrize("bs,page,old_hi,new_hi", [
    (1, 1, 0, 1), (1, 8, 5000, 3000), (2, 64, 63, 64), (5, 1, 40, 3), (300, 8, 100, 20),
    (1300, 16, 50, 5), (2500, 3, 7, 2)])
def test_cache_step(mla, bs, page, old_hi, new_hi):
    old, new, table, free = step_case(bs, page, old_hi, new_hi, bs + page)
    err = word()
    t, o = run_step(mla, old, new, page, table, free, stride=len(table[0]) + 3, err=err)
    rt, ro = plain_step(old, new, page, table, free)
    assert t == rt
    for k, v in ro.items():
        assert o[k] == (v if isinstance(v, list) else [v]), k
    mla.mla_error_check(err)


def test_cache_step_one_token_each_and_padding(mla):
    old, _, table, free = step_case(9, 4, 30, 1, 3)
    table = [r + [0] for r in table]
    free = free + list(range(1000, 1010))
    t, o = run_step(mla, old, None, 4, table, free, pad_idx=3, pad_tok=5)
    rt, ro = plain_step(old, [1] * 9, 4, table, free)
    assert t == rt and o["kvp"] == ro["kvp"] and o["last"] == ro["last"]
    assert o["idx"] == ro["idx"] + [-9] * 3
    assert o["slots"] == ro["slots"] + [-1] * 5 and o["pos"] == ro["pos"] + [0] * 5


def test_cache_step_reports_missing_pages(mla):
    err = word()
    t, o = run_step(mla, [3, 0, 8], [6, 10, 1], 4, [[5, 0, 0], [0, 0, 0], [6, 7, 0]], [9, 8, 1],
                    err=err)
    rt, ro = plain_step([3, 0, 8], [6, 10, 1], 4, [[5, 0, 0], [0, 0, 0], [6, 7, 0]], [9, 8, 1])
    assert t == rt and o["slots"] == ro["slots"] and o["idx"] == ro["idx"] and o["used"] == [3]
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 6
    mla.mla_error_check(err)                 # read and cleared


def test_cache_step_reports_short_tables_and_outputs(mla):
    err = word()
    # 2 columns of 4 tokens: the second request's tokens 8, 9 have no column
    old, new, table = i32([1, 6]), i32([1, 4]), i32([[3, 0], [4, 5]])
    o = dict(kv_indptr=i32([0, 0, 0]), kv_last_page_len=i32([0, 0]), kv_indices=i32([-9, -9]),
             qo_indptr=i32([0, 0, 0]), slots=torch.full((4,), -9, device="cuda"),
             positions=i32([0] * 4))
    mla.mla_cache_step(old, new, table, i32([8]), page_size=4, err=err, **o)
    assert o["kv_indptr"].tolist() == [0, 1, 3] and o["kv_last_page_len"].tolist() == [2, 4]
    assert o["kv_indices"].tolist() == [3, 4] and o["slots"].tolist() == [13, 22, 23, -1]
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 6


def test_cache_step_reports_bad_lengths_and_pages(mla):
    err = word()
    o = dict(kv_indptr=i32([0, 0, 0]), kv_last_page_len=i32([0, 0]), kv_indices=i32([-9] * 4),
             qo_indptr=i32([0, 0, 0]), slots=torch.full((4,), -9, device="cuda"),
             positions=i32([0] * 4))
    mla.mla_cache_step(i32([-5, 2]), i32([1, 1]), i32([[0], [-3]]), i32([8]), page_size=4, err=err,
                       **o)
    assert o["kv_indptr"].tolist() == [0, 1, 2] and o["slots"].tolist() == [32, -1, -1, -1]
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 1


# ----------------------------------------------------------------- cache write
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def plain_row(latent, k_rope, weight, eps, table, pos, rope):
    """The row in plain 32-bit arithmetic (the mean of squares in 64 bits)."""
    x = latent.float()
    if weight is not None:
        ms = (x.double() ** 2).mean(-1, keepdim=True).float()
        x = x * (1.0 / torch.sqrt(ms + torch.tensor(eps, dtype=torch.float32))) * weight.float()
    r = k_rope.float()
    return torch.cat([x, rotate(r, table, pos, rope) if table is not None else r], 1)


def new_pool(kv, rows):
    if kv == "bf16":
        return torch.full((rows, 576), 7.0, dtype=torch.bfloat16, device="cuda"), None
    if kv == "fp8":
        return torch.full((rows, 576), 0x55, dtype=torch.uint8, device="cuda"), None
    return (torch.full((rows, 288), 0x55, dtype=torch.uint8, device="cuda"),
            torch.full((rows, 20), 3, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("tokens,rope,norm,fused", [
    (1, "interleaved", True, True), (7, "half", True, False), (33, "interleaved", False, True),
    (300, "half", True, True), (129, None, True, False)])
def test_cache_write(mla, kv, tokens, rope, norm, fused):
    import workloads as synth
    g = gen(tokens)
    if fused:                                 # slices of one projection's output
        proj = torch.randn(tokens, 584, generator=g).bfloat16()
        latent, k_rope = proj[:, :512], proj[:, 512:576]
    else:
        latent = torch.randn(tokens, 512, generator=g).bfloat16() * 3
        k_rope = torch.randn(tokens, 65, generator=g).bfloat16()[:, :64]
    weight = (1 + 0.2 * torch.randn(512, generator=g)).bfloat16() if norm else None
    table = rotation_table(500) if rope else None
    pos = torch.randint(0, 500, (tokens,), generator=g).int() if rope else None
    rows = tokens + 9
    slots = torch.randperm(rows, generator=g)[:tokens]
    slots[tokens // 2] = -1                   # one token is not stored
    pool, e8 = new_pool(kv, rows)
    before, e8_before = pool.clone(), None if e8 is None else e8.clone()
    scale = torch.tensor([0.013])
    out = torch.full((tokens, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    dev = lambda x: None if x is None else x.cuda()      # noqa: E731
    if fused:
        pd = proj.cuda()
        dl, dr = pd[:, :512], pd[:, 512:576]
    else:
        dl = latent.cuda()
        dr = torch.zeros(tokens, 65, dtype=torch.bfloat16, device="cuda")[:, :64]
        dr.copy_(k_rope)
    err = word()
    mla.mla_cache_write(dl, dr, pool, slots.cuda(), kv_dtype=kv, norm_weight=dev(weight), eps=1e-5,
                        positions=dev(pos), cos_sin=dev(table), rope=rope or "half",
                        kv_scale=scale.cuda() if kv == "fp8" else None, kv_e8m0=e8, rows=out,
                        err=err)
    mla.mla_error_check(err)
    y = plain_row(latent, k_rope, weight, 1e-5, table, pos, rope)
    keep = slots >= 0
    where = slots[keep].cuda()
    touched = torch.zeros(rows, dtype=torch.bool)
    touched[slots[keep]] = True
    assert torch.equal(pool.cpu()[~touched], before.cpu()[~touched])
    if kv == "bf16":
        assert torch.equal(pool[where].cpu(), y.bfloat16()[keep])
        assert torch.equal(out.cpu(), y.bfloat16())
    elif kv == "fp8":
        q = (y / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(pool[where].cpu(), q.view(torch.uint8)[keep])
        assert torch.equal(out.cpu(), (q.float() * scale).bfloat16())
    else:
        packed, e = synth.quant_mxfp4_rows(y)
        assert torch.equal(pool[where].cpu(), packed[keep])
        assert torch.equal(e8[where, :18].cpu(), e[keep])
        assert torch.equal(e8[:, 18:], e8_before[:, 18:])
        assert torch.equal(e8.cpu()[~touched], e8_before.cpu()[~touched])
        codes = torch.stack([packed & 15, packed >> 4], -1).reshape(tokens, 18, 32)
        vals = E2M1[codes.long()] * torch.exp2(e.float() - 127)[..., None]
        assert torch.equal(out.cpu(), vals.reshape(tokens, 576).bfloat16())
    # and against 64 bits: an e4m3 / e2m1 rounding aside, the value itself
    x = latent.double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * weight.double()
    r = rotate(k_rope.double(), table, pos, rope) if rope else k_rope.double()
    ref = torch.cat([x, r], 1)
    # norm: sqrt, reciprocal, two products, eps: 5 F; rotation: 3 F of both terms
    slack = 6 * F * ref.abs() + 4 * F * k_rope.double().abs().amax()
    assert ((y.double() - ref).abs() <= slack).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
def test_cache_write_values_that_are_not_finite(mla, kv):
    import workloads as synth
    latent = torch.randn(6, 512, generator=gen(1)).bfloat16()
    k_rope = torch.randn(6, 64, generator=gen(2)).bfloat16()
    latent[1, 40] = float("nan")
    latent[2, 300] = float("inf")
    k_rope[3, 5] = float("-inf")
    latent[4] = 0
    latent[5] = 1e30
    pool, e8 = new_pool(kv, 6)
    out = torch.empty(6, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_write(latent.cuda(), k_rope.cuda(), pool, torch.arange(6, device="cuda"),
                        kv_dtype=kv, kv_scale=torch.ones(1, device="cuda") if kv == "fp8" else None,
                        kv_e8m0=e8, rows=out)
    y = torch.cat([latent, k_rope], 1).float()
    if kv == "bf16":
        assert torch.equal(torch.isnan(pool.cpu()), torch.isnan(y))
        ok = ~torch.isnan(y)
        assert torch.equal(pool.cpu()[ok], y.bfloat16()[ok])
    elif kv == "fp8":
        ref = y.clamp(-448, 448).to(torch.float8_e4m3fn).float()
        got = pool.view(torch.float8_e4m3fn).float().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(y))
        assert torch.equal(got.nan_to_num(0), ref.nan_to_num(0))
    else:
        bad = ~torch.isfinite(y).reshape(6, 18, 32).all(-1)
        assert (e8[:, :18].cpu()[bad] == 255).all()
        packed, e = synth.quant_mxfp4_rows(torch.where(bad[..., None], 0.0, y.reshape(6, 18, 32))
                                           .reshape(6, 576))
        assert torch.equal(pool.cpu(), packed) and torch.equal(e8[:, :18].cpu()[~bad], e[~bad])
        assert torch.equal(torch.isnan(out).reshape(6, 18, 32).any(-1).cpu(), bad)


def test_cache_write_reports_bad_slots_and_positions(mla):
    latent = torch.randn(3, 512, generator=gen(1)).bfloat16()
    k_rope = torch.randn(3, 64, generator=gen(2)).bfloat16()
    for slots, pos in (([0, 4, 1], [0, 1, 2]), ([0, -2, 1], [0, 1, 2]), ([0, 2, 1], [0, 9, 2]),
                       ([0, 2, 1], [0, -1, 2])):
        pool, _ = new_pool("bf16", 4)
        err = word()
        mla.mla_cache_write(latent.cuda(), k_rope.cuda(), pool, torch.tensor(slots).cuda(),
                            kv_dtype="bf16", positions=i32(pos), cos_sin=rotation_table(9).cuda(),
                            err=err)
        with pytest.raises(mla.MlaError) as e:
            mla.mla_error_check(err)
        assert e.value.status == 1
        # the others are written
        y = plain_row(latent, k_rope, None, 0, rotation_table(9), torch.tensor([0, 0, 2]),
                      "interleaved").bfloat16()
        assert torch.equal(pool[[0, 1]].cpu(), y[[0, 2]])
        assert (pool[3] == 7).all()


def test_cache_write_of_nothing(mla):
    pool, _ = new_pool("bf16", 4)
    e = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_write(e.view(0, 512), e.view(0, 64), pool,
                        torch.empty(0, dtype=torch.int64, device="cuda"), kv_dtype="bf16")
    assert (pool == 7).all()


# --------------------------------------------------------------- absorbed form
def make_w(heads, g):
    return (torch.randn(heads, 256, 512, generator=g) / math.sqrt(512)).bfloat16()


@pytest.mark.parametrize("tokens,heads,rope,layout", [
    (1, 16, "interleaved", "dense"), (2, 1, "half", "dense"), (17, 16, "half", "heads"),
    (64, 3, "interleaved", "wide"), (128, 16, "half", "dense"), (129, 5, "interleaved", "heads"),
    (300, 16, None, "wide"), (1000, 2, "interleaved", "dense")])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_absorb_q(mla, tokens, heads, rope, layout, dtype):
    g = gen(tokens)
    q = torch.randn(tokens, heads, 192, generator=g).bfloat16()
    w = make_w(heads, g)
    table = rotation_table(300) if rope else None
    pos = torch.randint(0, 300, (tokens,), generator=g).int() if rope else None
    if layout == "heads":                     # [heads, tokens, 192] seen as [tokens, heads, 192]
        dq = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    elif layout == "wide":                    # a slice of wider rows
        dq = torch.full((tokens, heads, 208), float("nan"), dtype=torch.bfloat16, device="cuda")
        dq = dq[..., 8:200]
        dq.copy_(q)
    else:
        dq = q.cuda()
    fp8 = dtype == "fp8"
    # guard rows around the output must stay as they are
    store = torch.full((tokens + 2, heads, 576), 0x55 if fp8 else 7.0,
                       dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    out = store[1:-1]
    scale = torch.tensor([0.02])
    mla.mla_absorb_q(dq, w.cuda(), out, sm_scale=SCALE, rope=rope or "half",
                     positions=None if pos is None else pos.cuda(),
                     cos_sin=None if table is None else table.cuda(),
                     q_scale=scale.cuda() if fp8 else None)
    f = 24 * SCALE
    qd, wd = q.double(), w.double()
    ref = torch.einsum("thd,hdc->thc", qd[..., :128], wd[:, :128]) * f
    mag = torch.einsum("thd,hdc->thc", qd[..., :128].abs(), wd[:, :128].abs()) * f
    rot = rotate(qd[..., 128:], table, pos, rope) if rope else qd[..., 128:]
    ref = torch.cat([ref, rot * f], -1)
    mag = torch.cat([mag, 3 * f * qd[..., 128:].abs().amax().expand(tokens, heads, 64)], -1)
    got = out.view(torch.float8_e4m3fn).cpu().double() * scale.double() if fp8 else out.cpu().double()
    # fp32 sums of 128 products, the factor and (fp8) the division; one
    # rounding to the output type (e4m3 subnormals: half of 2^-9 steps)
    acc = 132 * F * mag
    tol = acc + (2 ** -4 * (ref.abs() + acc) + 2 ** -10 * scale.double() if fp8 else U * (ref.abs() + acc))
    assert ((got - ref).abs() <= tol).all()
    edge = store[[0, -1]]
    assert (edge == (0x55 if fp8 else 7.0)).all()


def test_absorb_q_saturates_and_reports(mla):
    g = gen(5)
    q = (torch.randn(3, 2, 192, generator=g) * 1000).bfloat16()
    w = make_w(2, g)
    out = torch.empty(3, 2, 576, dtype=torch.uint8, device="cuda")
    err = word()
    mla.mla_absorb_q(q.cuda(), w.cuda(), out, sm_scale=SCALE, q_scale=torch.full((1,), 0.5).cuda(),
                     positions=i32([0, 3, 1]), cos_sin=rotation_table(3).cuda(), err=err)
    v = out.view(torch.float8_e4m3fn).float()
    assert torch.isfinite(v).all() and (v.abs() == 448).any()
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 1


@pytest.mark.parametrize("tokens", [1, 3, 40, 130])
def test_absorb_rows_do_not_mix(mla, tokens):
    # a token whose query is not finite leaves the others alone
    g = gen(6)
    q = torch.randn(tokens + 1, 16, 192, generator=g).bfloat16()
    q[tokens] = float("nan")
    w = make_w(16, g).cuda()
    a = torch.empty(tokens + 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_q(q.cuda(), w, a, sm_scale=SCALE)
    assert torch.isfinite(a[:tokens]).all() and torch.isnan(a[tokens]).all()
    b = torch.empty(tokens + 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_out(a[..., :512].contiguous(), w, b)
    assert torch.isfinite(b[:tokens]).all() and torch.isnan(b[tokens]).all()


@pytest.mark.parametrize("tokens,heads", [(1, 16), (2, 1), (17, 16), (64, 3), (128, 16), (129, 5),
                                          (300, 16), (1000, 2)])
def test_absorb_out(mla, tokens, heads):
    g = gen(tokens)
    o = torch.randn(tokens, heads, 512, generator=g).bfloat16()
    w = make_w(heads, g)
    store = torch.full((tokens + 2, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_out(o.cuda(), w.cuda(), store[1:-1])
    ref = torch.einsum("thc,hvc->thv", o.double(), w[:, 128:].double())
    mag = torch.einsum("thc,hvc->thv", o.double().abs(), w[:, 128:].double().abs())
    acc = 512 * F * mag
    assert ((store[1:-1].cpu().double() - ref).abs() <= acc + U * (ref.abs() + acc)).all()
    assert (store[[0, -1]] == 7).all()


# --------------------------------------------------------------- expanded form
def prefill_case(q_lens, kv_lens, heads, kv, page, rope, seed, layout="dense", table=True,
                 kv_std=1.0):
    """Inputs on the host: q, w, pool in `kv` encoding, and the stored rows in 64 bits."""
    import workloads as synth
    g = gen(seed)
    bs = len(q_lens)
    w = synth.make_workload(bs=bs, lengths=kv_lens, page_size=page, kv_dtype=kv,
                            permute_pages=table, seed=seed, extra_pool_pages=2 if table else 0)
    if kv_std != 1.0:
        w.kv = (w.kv.float() * kv_std).bfloat16()
    if kv == "bf16":
        rows = w.kv.double()
    elif kv == "fp8":
        rows = w.kv.view(torch.float8_e4m3fn).double() * w.kv_scale.double()
    else:
        codes = torch.stack([w.kv & 15, w.kv >> 4], -1).reshape(-1, 18, 32)
        rows = (E2M1[codes.long()].double() * torch.exp2(w.kv_e8m0[:, :18].double() - 127)[..., None]
                ).reshape(-1, 576)
    qo = [0]
    pos = []
    for m, n in zip(q_lens, kv_lens):
        qo.append(qo[-1] + m)
        pos += [max(0, n - m + t) for t in range(m)]
    q = torch.randn(qo[-1], heads, 192, generator=g).bfloat16()
    return dict(w=w, qo=qo, q=q, weights=make_w(heads, g), rows=rows, heads=heads, page=page,
                kv_lens=kv_lens, q_lens=q_lens, rope=rope, table=rotation_table(max(pos + [0]) + 1),
                pos=torch.tensor(pos, dtype=torch.int32), layout=layout)


def request_rows(c, b):
    w, page = c["w"], c["page"]
    pages = torch.arange(int(w.kv_indptr[b]), int(w.kv_indptr[b + 1]))
    if w.kv_indices is not None:
        pages = w.kv_indices[pages].long()
    return (pages[:, None] * page + torch.arange(page)).reshape(-1)[: c["kv_lens"][b]]


def plain_prefill(c):
    """out, lse in 64 bits and the bound of each output's error."""
    q, w = c["q"].double(), c["weights"].double()
    if c["rope"]:
        q = torch.cat([q[..., :128], rotate(q[..., 128:], c["table"], c["pos"], c["rope"])], -1)
    outs, lses, bounds, lse_bounds = [], [], [], []
    for b, (m, n) in enumerate(zip(c["q_lens"], c["kv_lens"])):
        x = c["rows"][request_rows(c, b)]
        qb = q[c["qo"][b]: c["qo"][b + 1]]
        kv = torch.einsum("nc,hdc->hnd", x[:, :512], w)
        k = torch.cat([kv[..., :128], x[:, 512:].expand(c["heads"], -1, -1)], -1)
        s = torch.einsum("mhd,hnd->hmn", qb, k) * SCALE
        mag = torch.einsum("mhd,hnd->hmn", qb.abs(), k.abs()) * SCALE
        see = torch.arange(n)[None] < (n - m + 1 + torch.arange(m))[:, None]
        s = s.masked_fill(~see, -math.inf)
        lse = torch.logsumexp(s, -1) if n else torch.full((c["heads"], m), -math.inf).double()
        p = torch.exp(s - lse[..., None]).masked_fill(~see, 0.0).nan_to_num(0.0)
        # key, query (rotated dims) rounded to bf16: scores off by e; p to bf16
        # and v to bf16: 2 u; out to bf16; exp2, sums in fp32: n F and a few F
        e = (mag.masked_fill(~see, 0.0).amax(-1) if n else torch.zeros(c["heads"], m).double()) * (
            2 * U + 400 * F)
        o = torch.einsum("hmn,hnd->mhd", p, kv[..., 128:])
        pv = torch.einsum("hmn,hnd->mhd", p, kv[..., 128:].abs())
        inner = pv * (torch.expm1(2 * e).T[..., None] + 2 * U + U * U + (n + 64) * F)
        outs.append(o)
        lses.append(lse.T)
        bounds.append(inner + U * (o.abs() + inner))
        lse_bounds.append((e + U * 0 + (n + 64) * F + 8 * F * lse.abs().nan_to_num(0, 0, 0)).T)
    return torch.cat(outs), torch.cat(lses), torch.cat(bounds), torch.cat(lse_bounds)


def run_prefill(mla, c, num_sms=0, want_lse=True, check=True):
    w = c["w"].to("cuda")
    t, h = c["qo"][-1], c["heads"]
    dq = c["q"].cuda()
    if c["layout"] == "heads":
        dq = dq.transpose(0, 1).contiguous().transpose(0, 1)
    elif c["layout"] == "wide":
        wide = torch.full((t, h, 208), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[..., 8:200] = dq
        dq = wide[..., 8:200]
    plan = mla.mla_prefill_plan(c["qo"], w.kv_indptr.cpu(), w.kv_last_page_len.cpu() if
                                w.kv_last_page_len is not None else None, page_size=c["page"],
                                heads=h, kv_dtype=w.kv_dtype, num_sms=num_sms)
    # workspaces come as they are: fill it with NaN patterns
    ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    store = torch.full((t + 2, h, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((t, h), 7.0, device="cuda") if want_lse else None
    rope = {} if not c["rope"] else dict(positions=c["pos"].cuda(), cos_sin=c["table"].cuda(),
                                         rope=c["rope"])
    mla.mla_prefill_run(plan, dq, w.kv, c["weights"].cuda(), store[1:-1], workspace=ws,
                        sm_scale=SCALE, kv_scale=w.kv_scale, kv_e8m0=w.kv_e8m0,
                        kv_indices=w.kv_indices, lse=lse, **rope)
    if check:
        mla.mla_prefill_check(plan, ws)
    assert (store[[0, -1]] == 7).all()
    return store[1:-1].cpu().double(), None if lse is None else lse.cpu().double(), plan


def check_prefill(mla, c, num_sms=0):
    o, lse, plan = run_prefill(mla, c, num_sms)
    ref, ref_lse, bound, lse_bound = plain_prefill(c)
    empty = torch.isneginf(ref_lse)
    assert (o[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    assert torch.isfinite(o).all()
    assert ((o - ref).abs() <= bound).all()
    assert ((lse - ref_lse)[~empty].abs() <= lse_bound[~empty]).all()
    # the same roundings as independent errors: 4 of u / sqrt 3 and the scores'
    # sqrt(2) u / sqrt 3 stay near 0.4 %; a structural error does not
    # (over the whole output: a row whose values cancel has a small norm)
    assert (o - ref).norm() <= 1e-2 * ref.norm()
    return plan


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("q_lens,kv_lens,heads,page,rope,layout", [
    ([1], [1], 1, 1, "interleaved", "dense"),
    ([5], [5], 2, 8, "half", "heads"),
    ([1, 1, 1], [300, 128, 129], 3, 16, "interleaved", "dense"),
    ([128], [128], 2, 8, "interleaved", "wide"),
    ([129, 0, 40], [129, 77, 200], 2, 1, "half", "dense"),
    ([257, 256], [700, 256], 2, 64, "interleaved", "heads"),
    ([3, 200, 1, 0], [1, 130, 0, 5], 2, 8, "interleaved", "dense"),   # queries without keys
    ([600], [640], 1, 3, None, "dense"),
])
def test_prefill(mla, kv, q_lens, kv_lens, heads, page, rope, layout):
    check_prefill(mla, prefill_case(q_lens, kv_lens, heads, kv, page, rope, 31, layout))


@pytest.mark.parametrize("q_lens,kv_lens,heads,rope", [
    ([512], [512], 1, "interleaved"), ([385], [385], 2, "half"), ([400, 1100], [5000, 1111], 1, None),
    ([897, 3, 450], [1000, 300, 449], 2, "interleaved")])
def test_prefill_blocks_of_512_rows(mla, q_lens, kv_lens, heads, rope):
    # more than 384 rows: an item of two CTAs; the third case has a query without keys
    check_prefill(mla, prefill_case(q_lens, kv_lens, heads, "bf16", 8, rope, 41))


def test_prefill_blocks_of_512_rows_on_few_ctas(mla):
    c = prefill_case([1500, 600], [1500, 2500], 2, "fp8", 16, "interleaved", 42)
    for num_sms in (2, 5, 152):
        check_prefill(mla, c, num_sms=num_sms)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
def test_prefill_without_a_page_table(mla, kv):
    check_prefill(mla, prefill_case([70, 300], [200, 333], 2, kv, 1, "interleaved", 5, table=False))


@pytest.mark.parametrize("num_sms", [1, 2, 5, 40])
def test_prefill_on_few_and_many_ctas(mla, num_sms):
    # few: several items a CTA; many: keys cut into ranges and joined
    c = prefill_case([130, 9, 300], [900, 6000, 400], 2, "bf16", 8, "interleaved", 6)
    plan = check_prefill(mla, c, num_sms=num_sms)
    if num_sms == 40:
        assert plan.info().num_partials > 0


@pytest.mark.parametrize("q_lens,kv_lens,num_sms", [
    ([1], [5000], 152), ([128], [4000], 152), ([127, 3], [3000, 700], 8), ([9], [1300], 3),
    ([100, 40, 1], [1000, 2001, 1153], 5)])
def test_prefill_few_rows_against_many_keys(mla, q_lens, kv_lens, num_sms):
    # at most 128 rows: both query tiles hold them, each against half of a key range
    plan = check_prefill(mla, prefill_case(q_lens, kv_lens, 2, "bf16", 8, "interleaved", 15),
                         num_sms=num_sms)
    assert plan.info().num_partials > 0


def test_prefill_split_keys_with_rows_that_see_few(mla):
    # more query rows than keys in the first ranges: some rows see no key of a range
    c = prefill_case([250], [1400], 1, "fp8", 8, "half", 7)
    assert check_prefill(mla, c).info().num_partials > 0
    c = prefill_case([255, 700], [260, 700], 1, "bf16", 8, "half", 8)
    check_prefill(mla, c)


def test_prefill_scores_that_grow_and_large_ones(mla):
    # a running maximum that keeps moving, and scores of tens
    c = prefill_case([200], [900], 2, "bf16", 8, "interleaved", 9)
    ramp = torch.linspace(0.1, 6.0, 900)
    at = request_rows(c, 0)
    c["w"].kv[at] = (c["w"].kv[at].float() * ramp[:, None]).bfloat16()
    c["rows"] = c["w"].kv.double()
    o, lse, _ = run_prefill(mla, c)
    ref, ref_lse, bound, lse_bound = plain_prefill(c)
    assert torch.isfinite(o).all()
    assert ((o - ref).abs() <= bound).all() and ((lse - ref_lse).abs() <= lse_bound).all()


@pytest.mark.parametrize("q_lens,kv_lens", [([300], [640]), ([700], [1100]), ([40], [2000])])
def test_prefill_values_of_any_size(mla, q_lens, kv_lens):
    # values far above and below one (their type is chosen by groups of 32 keys):
    # by head through the weights, and by key through short rows
    c = prefill_case(q_lens, kv_lens, 6, "bf16", 8, "interleaved", 17)
    for h, f in enumerate((1.0, 1e6, 1e-6, 3e4, 1e-12, 0.0)):
        c["weights"][h, 128:] = (c["weights"][h, 128:].float() * f).bfloat16()
    at = request_rows(c, 0)
    short = torch.arange(len(at)) // 40 % 3 == 1
    c["w"].kv[at[short], :512] = (c["w"].kv[at[short], :512].float() * 1e-3).bfloat16()
    c["rows"] = c["w"].kv.double()
    o, lse, _ = run_prefill(mla, c)
    ref, ref_lse, bound, lse_bound = plain_prefill(c)
    # (fp16 values: half a step of 2^-25 of 32 keys' largest magnitude; far below)
    assert ((o - ref).abs() <= bound).all() and ((lse - ref_lse).abs() <= lse_bound).all()
    for h in range(5):
        assert (o[:, h] - ref[:, h]).norm() <= 1e-2 * ref[:, h].norm()


@pytest.mark.parametrize("q_lens,kv_lens", [([40], [1500]), ([300], [1500]), ([600], [1500])])
@pytest.mark.parametrize("at", [0, 700])
def test_prefill_small_weights_count(mla, q_lens, kv_lens, at):
    # one key takes nearly all of the weight and has no value: the output is what
    # the others' weights of 2^-23.3 leave.  Scores are exact: 16 x 14 or zero.
    c = prefill_case(q_lens, kv_lens, 2, "bf16", 8, None, 21)
    rows = request_rows(c, 0)
    c["w"].kv[rows, 512:] = 0
    c["w"].kv[rows[at], :512] = 0
    c["w"].kv[rows[at], 512] = 16
    c["rows"] = c["w"].kv.double()
    c["q"][:] = 0
    c["q"][..., 128] = 14
    o, lse, _ = run_prefill(mla, c)
    ref, ref_lse, _, lse_bound = plain_prefill(c)
    # the weights: half a step of 2^-24 on 2^-17 or more; values 2^-11, output 2^-8
    assert (o - ref).norm() <= (2**-8 + 2**-11 + 2**-8) * ref.norm()
    assert ((lse - ref_lse).abs() <= lse_bound).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefill_values_that_are_not_finite(mla, kv):
    # request 0: token 150 is poisoned, seen by query rows 50.. only; request
    # 1: untouched; pool rows that no request uses are poisoned too
    c = prefill_case([100, 60], [200, 90], 2, kv, 8, "interleaved", 10)
    ref, _, bound, _ = plain_prefill(c)
    bad = float("nan")
    pool = c["w"].kv
    used = torch.cat([request_rows(c, 0), request_rows(c, 1)])
    unused = torch.ones(len(pool), dtype=torch.bool)
    unused[used] = False
    assert unused.any()
    token = request_rows(c, 0)[150]
    if kv == "bf16":
        pool[unused] = bad
        pool[token, 17] = float("inf")
    else:
        pool[unused] = 0x7F
        pool[token, 17] = 0x7F
    o, _, _ = run_prefill(mla, c)
    clean = torch.ones(160, dtype=torch.bool)
    clean[50:100] = False
    assert torch.isnan(o[50:100]).all()
    assert ((o - ref).abs()[clean] <= bound[clean]).all()
    # poisoned rotated dims: the scores alone
    c = prefill_case([100, 60], [200, 90], 2, kv, 8, "interleaved", 10)
    c["w"].kv[token, 512 + 9] = bad if kv == "bf16" else 0x7F
    o, _, _ = run_prefill(mla, c)
    assert torch.isnan(o[50:100]).all()
    assert ((o - ref).abs()[clean] <= bound[clean]).all()


def test_prefill_query_that_is_not_finite(mla):
    c = prefill_case([300], [300], 2, "bf16", 8, "interleaved", 11)
    ref, _, bound, _ = plain_prefill(c)
    c["q"][140, 1, 3] = float("nan")
    o, _, _ = run_prefill(mla, c)
    assert torch.isnan(o[140, 1]).all()
    ok = torch.ones(300, 2, dtype=torch.bool)
    ok[140, 1] = False
    assert ((o - ref).abs()[ok] <= bound[ok]).all()


def test_prefill_reports_bad_pages_positions_and_workspaces(mla):
    c = prefill_case([20, 30], [40, 50], 2, "fp8", 8, "interleaved", 12)
    ref, _, bound, _ = plain_prefill(c)
    good = c["w"].kv_indices.clone()
    for bad in (-1, 10 ** 6):
        c["w"].kv_indices[1] = bad
        c["w"].kv_indices[len(good) - 1] = good[-1]
        o, _, plan = run_prefill(mla, c, check=False)
        assert ((o - ref).abs()[20:] <= bound[20:]).all()        # the other request
    c["w"].kv_indices = good
    w = c["w"].to("cuda")
    plan = mla.mla_prefill_plan(c["qo"], w.kv_indptr.cpu(), w.kv_last_page_len.cpu(), page_size=8,
                                heads=2, kv_dtype="fp8")
    other = mla.mla_prefill_plan(c["qo"], w.kv_indptr.cpu(), w.kv_last_page_len.cpu(), page_size=8,
                                 heads=2, kv_dtype="fp8")
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.full((50, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(workspace=ws, sm_scale=SCALE, kv_scale=w.kv_scale, kv_indices=w.kv_indices)
    pos = c["pos"].clone()
    pos[3] = len(c["table"])
    args = (c["q"].cuda(), w.kv, c["weights"].cuda(), out)
    mla.mla_prefill_run(plan, *args, positions=pos.cuda(), cos_sin=c["table"].cuda(), **kw)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_prefill_check(plan, ws)
    assert e.value.status == 1
    w.kv_indices[0] = -5
    mla.mla_prefill_run(plan, *args, **kw)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_prefill_check(plan, ws)
    assert e.value.status == 1
    mla.mla_prefill_check(plan, ws)
    # another plan takes the workspace: the first one's next run writes nothing
    mla.mla_prefill_run(other, *args, **kw)
    torch.cuda.synchronize()
    out.fill_(7.0)
    mla.mla_prefill_run(plan, *args, **kw)
    assert (out == 7).all()
    with pytest.raises(mla.MlaError) as e:
        mla.mla_prefill_check(plan, ws)
    assert e.value.status == 3
    mla.mla_prefill_run(plan, *args, **kw)
    assert not (out == 7).all()


def test_captured_into_a_graph_and_on_another_stream(mla):
    c = prefill_case([150], [400], 2, "bf16", 8, "interleaved", 13)
    ref, _, bound, _ = plain_prefill(c)
    w = c["w"].to("cuda")
    plan = mla.mla_prefill_plan(c["qo"], w.kv_indptr.cpu(), w.kv_last_page_len, page_size=8,
                                heads=2, kv_dtype="bf16")
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.zeros(150, 2, 128, dtype=torch.bfloat16, device="cuda")
    q, weights, pos, table = c["q"].cuda(), c["weights"].cuda(), c["pos"].cuda(), c["table"].cuda()
    o = torch.empty(150, 2, 128, dtype=torch.bfloat16, device="cuda")
    qa = torch.empty(150, 2, 576, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        mla.mla_prefill_run(plan, q, w.kv, weights, out, workspace=ws, sm_scale=SCALE,
                            positions=pos, cos_sin=table, kv_indices=w.kv_indices, stream=stream)
        mla.mla_absorb_q(q, weights, qa, sm_scale=SCALE, positions=pos, cos_sin=table,
                         stream=stream)
        mla.mla_absorb_out(qa[..., :512].contiguous() if stream is None else lat, weights, o,
                           stream=stream)

    side = torch.cuda.Stream()
    lat = torch.zeros(150, 2, 512, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    assert ((out.cpu().double() - ref).abs() <= bound).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.zero_()
    qa.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert ((out.cpu().double() - ref).abs() <= bound).all()
    assert qa.abs().sum() > 0


@pytest.mark.parametrize("kv,q_dtype", [("bf16", "bf16"), ("fp8", "bf16"), ("fp8", "fp8"),
                                        ("mxfp4", "bf16")])
def test_both_forms_give_the_same_attention(mla, kv, q_dtype):
    # the last token of each request: expanded form, and absorb - decode - absorb
    kv_lens = [5, 300, 1, 777]
    c = prefill_case([1] * 4, kv_lens, 16, kv, 8, "interleaved", 14)
    o, _, _ = run_prefill(mla, c)
    w = c["w"].to("cuda")
    fp8 = q_dtype == "fp8"
    weights = c["weights"].cuda()
    qa = torch.empty(4, 16, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    qs = torch.full((1,), 0.02, device="cuda") if fp8 else None
    mla.mla_absorb_q(c["q"].cuda(), weights, qa, sm_scale=SCALE, positions=c["pos"].cuda(),
                     cos_sin=c["table"].cuda(), q_scale=qs)
    plan = mla.mla_decode_plan(w.kv_indptr.cpu(), w.kv_last_page_len.cpu(), page_size=8,
                               q_dtype=q_dtype, kv_dtype=kv)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    lat = torch.empty(4, 16, 512, dtype=torch.bfloat16, device="cuda")
    mla.mla_decode_run(plan, qa, w.kv, lat, workspace=ws, q_scale=qs, kv_scale=w.kv_scale,
                       kv_e8m0=w.kv_e8m0, kv_indices=w.kv_indices)
    mla.mla_decode_check(plan, ws)
    out = torch.empty(4, 16, 128, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_out(lat, weights, out)
    # an e4m3 query moves scores of order one by 2^-4 / sqrt 3 of their terms
    assert torch.allclose(out.cpu().double(), o, atol=0.2 if fp8 else 3e-2, rtol=5e-2)


# The cache's encoding sets the error: bf16 u / sqrt 3 a stage, e4m3 2^-4 / sqrt 3
# of every stored value, e2m1 up to a quarter of one.
@pytest.mark.parametrize("kv,limit", [("bf16", 1e-2), ("fp8", 6e-2), ("mxfp4", 2.5e-1)])
def test_the_layer_example(mla, kv, limit):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for e in example.main([70, 3, 400], 3, kv):
        assert e <= limit


def test_rows_past_4_gb_of_a_pool(mla):
    # the same request in the last pages of a pool of 4.6 GB and in a small one
    n, page = 200, 8
    g = torch.Generator(device="cuda").manual_seed(31)
    lat = torch.randn(n, 512, generator=g, device="cuda").bfloat16()
    rope = torch.randn(n, 64, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, 2, 192, generator=g, device="cuda").bfloat16()
    weights = make_w(2, gen(31)).cuda()
    outs = []
    for rows in (n, 4_000_000):
        pool = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
        first = (rows - n) // page
        mla.mla_cache_write(lat, rope, pool, first * page + torch.arange(n, device="cuda"),
                            kv_dtype="bf16")
        assert torch.equal(pool[-n:], torch.cat([lat, rope], 1))
        assert rows == n or not pool[:n].any()
        plan = mla.mla_prefill_plan([0, n], [0, n // page], page_size=page, heads=2,
                                    kv_dtype="bf16")
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        out = torch.empty(n, 2, 128, dtype=torch.bfloat16, device="cuda")
        mla.mla_prefill_run(plan, q, pool, weights, out, workspace=ws, sm_scale=SCALE,
                            kv_indices=first + torch.arange(n // page, device="cuda").int())
        mla.mla_prefill_check(plan, ws)
        outs.append(out.clone())
        del pool
    assert torch.equal(outs[0], outs[1]) and outs[0].abs().sum() > 0


def test_prefill_keys_past_4_gb_of_the_workspace(mla):
    # 600,000 keys of 16 heads expand into 4.9 GB; the last heads stand behind 2^32
    n, m, heads, page = 600_000, 5, 16, 64
    g = torch.Generator(device="cuda").manual_seed(32)
    pages = n // page
    pool = torch.randn(n, 576, generator=g, device="cuda").bfloat16()
    table = torch.randperm(pages, generator=g, device="cuda").int()
    q = torch.randn(m, heads, 192, generator=g, device="cuda").bfloat16()
    weights = make_w(heads, gen(32)).cuda()
    plan = mla.mla_prefill_plan([0, m], [0, pages], page_size=page, heads=heads, kv_dtype="bf16")
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(m, heads, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(m, heads, device="cuda")
    mla.mla_prefill_run(plan, q, pool, weights, out, workspace=ws, sm_scale=SCALE,
                        kv_indices=table, lse=lse)
    mla.mla_prefill_check(plan, ws)
    rows = pool.view(pages, page, 576)[table.long()].view(n, 576)
    see = torch.arange(n, device="cuda")[None] < n - m + 1 + torch.arange(m, device="cuda")[:, None]
    for h in (0, heads - 1):
        x = rows[:, :512].double() @ weights[h].double().T
        k = torch.cat([x[:, :128], rows[:, 512:].double()], 1)
        s = (q[:, h].double() @ k.T * SCALE).masked_fill(~see, -math.inf)
        mag = (q[:, h].double().abs() @ k.abs().T).amax() * SCALE
        o = torch.softmax(s, -1) @ x[:, 128:]
        # independent roundings, as for the other prefill tests; scores off by e
        assert (out[:, h].double() - o).norm() <= 1e-2 * o.norm()
        assert ((lse[:, h].double() - torch.logsumexp(s, -1)).abs() <= mag * (2 * U + 400 * F)
                + (n + 64) * F).all()


def prefill_calls(mla, cases, num_sms=0):
    """Cases of the same lengths on the device: (plan, workspace, calls), a call
    of case i being calls[i](out)."""
    c = cases[0]
    ws = [x["w"].to("cuda") for x in cases]
    plan = mla.mla_prefill_plan(c["qo"], ws[0].kv_indptr, ws[0].kv_last_page_len,
                                page_size=c["page"], heads=c["heads"], kv_dtype=ws[0].kv_dtype,
                                num_sms=num_sms)
    space = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def call(x, w):
        q, weights = x["q"].cuda(), x["weights"].cuda()
        rope = {} if not x["rope"] else dict(positions=x["pos"].cuda(), cos_sin=x["table"].cuda(),
                                             rope=x["rope"])

        def run(out, kv=w.kv, **kw):
            mla.mla_prefill_run(plan, q, kv, weights, out, workspace=space, sm_scale=SCALE,
                                kv_scale=w.kv_scale, kv_e8m0=w.kv_e8m0, kv_indices=w.kv_indices,
                                **rope, **kw)
        return run

    return plan, space, [call(x, w) for x, w in zip(cases, ws)]


def repeats(mla, cases, times, num_sms=0):
    """Calls of the cases in turn, many times without a pause, give each case's
    first output bit by bit: a row or a result of the call before would show."""
    plan, space, calls = prefill_calls(mla, cases, num_sms)
    shape = (cases[0]["qo"][-1], cases[0]["heads"], 128)
    first = []
    for run in calls:
        out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        run(out)
        torch.cuda.synchronize()
        first.append(out)
    differing = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for i in range(times):
        out.fill_(7.0)
        calls[i % len(calls)](out)
        differing += (out.view(torch.int16) != first[i % len(calls)].view(torch.int16)).sum()
    mla.mla_prefill_check(plan, space)
    assert differing.item() == 0
    return [f.cpu().double() for f in first]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
def test_prefill_expansion_takes_every_new_row(mla, kv):
    # few heads against many keys on few CTA pairs: rows are replaced every two
    # units, in both CTAs of a pair, and the products wait for them each time
    cases = [prefill_case([64], [6000], 2, kv, 8, "interleaved", s) for s in (51, 52)]
    for c, o in zip(cases, repeats(mla, cases, 200, num_sms=8)):
        ref, _, bound, _ = plain_prefill(c)
        assert ((o - ref).abs() <= bound).all()


def test_prefill_on_pairs_and_single_ctas_repeats(mla):
    # blocks of 512 rows on CTA pairs and the rest on CTAs of their own, which
    # start beside the pairs' last items: more CTAs in all than planned for
    cases = [prefill_case([1300, 400, 900], [2300, 4400, 900], 2, "bf16", 8, "interleaved", s)
             for s in (53, 54)]
    plan = mla.mla_prefill_plan(cases[0]["qo"], cases[0]["w"].kv_indptr,
                                cases[0]["w"].kv_last_page_len, page_size=8, heads=2,
                                kv_dtype="bf16", num_sms=4)
    assert plan.info().num_ctas > 4
    for c, o in zip(cases, repeats(mla, cases, 200, num_sms=4)):
        ref, _, bound, _ = plain_prefill(c)
        assert ((o - ref).abs() <= bound).all()


@pytest.mark.parametrize("q_lens,kv_lens,num_sms", [
    ([130, 9, 300], [900, 6000, 400], 40), ([1300, 400, 900], [2300, 4400, 900], 4)])
def test_prefill_notices_an_overwritten_work_table(mla, q_lens, kv_lens, num_sms):
    # 256 bytes of the workspace at a time, the header with the plan's stamp left
    # as it was: what the records say is not followed, and the next run is right
    c = prefill_case(q_lens, kv_lens, 2, "bf16", 8, "interleaved", 55)
    plan, space, (run,) = prefill_calls(mla, [c], num_sms)
    out = torch.empty(c["qo"][-1], 2, 128, dtype=torch.bfloat16, device="cuda")
    run(out)
    mla.mla_prefill_check(plan, space)
    clean = out.clone()
    info = plan.info()
    # tiles, CTAs, items (32 bytes each at least) are in there, each from 256 bytes on
    records = sum(-(-n // 128) for n in kv_lens) + info.num_items
    noticed = 0
    for block in range(1, records * 32 // 256 + 8):
        for value in (-1, 5):
            space.view(torch.int32)[64 * block: 64 * block + 64] = value
            out.fill_(7.0)
            run(out)
            try:
                mla.mla_prefill_check(plan, space)
                assert torch.equal(out, clean)        # behind the table: nothing is kept there
            except mla.MlaError as e:
                assert e.status == 3
                noticed += 1
            run(out)
            mla.mla_prefill_check(plan, space)
            assert torch.equal(out, clean)
    assert noticed >= 2 * (records * 32 // 256)


@pytest.mark.parametrize("f", [2.0**-9, 2.0**-16, 2.0**-22, 2.0**-40])
@pytest.mark.parametrize("n", [40, 300, 700])
def test_prefill_a_short_value_among_long_ones(mla, n, f):
    # tokens 0 and 1 are far shorter than the 30 beside them, with which they
    # share a type: query rows 0 and 1 see nothing else
    c = prefill_case([n], [n], 2, "bf16", 8, "interleaved", 22)
    at = request_rows(c, 0)
    c["w"].kv[at[:2], :512] *= f
    c["rows"] = c["w"].kv.double()
    o, lse, _ = run_prefill(mla, c)
    ref, ref_lse, bound, lse_bound = plain_prefill(c)
    assert ((o - ref).abs() <= bound).all() and ((lse - ref_lse).abs() <= lse_bound).all()
    # roundings of values, weights and output as independent errors, as elsewhere
    for t in (0, 1):
        assert (o[t] - ref[t]).norm() <= 1e-2 * ref[t].norm()


def test_a_step_without_new_tokens(mla):
    # every call of a step in which no request gets a token, rotation and all
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rope = dict(positions=none, cos_sin=rotation_table(8).cuda())
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    err, w = word(), make_w(16, gen(1)).cuda()
    o = dict(kv_indptr=i32([-9] * 3), kv_last_page_len=i32([-9] * 2), kv_indices=i32([-9] * 3),
             qo_indptr=i32([-9] * 3), slots=torch.empty(0, dtype=torch.int64, device="cuda"),
             positions=none)
    mla.mla_cache_step(i32([3, 5]), i32([0, 0]), i32([[1, 0], [0, 2]]), i32([3]), page_size=4,
                       err=err, **o)
    assert o["kv_indptr"].tolist() == [0, 1, 3] and o["qo_indptr"].tolist() == [0, 0, 0]
    assert o["kv_indices"].tolist() == [1, 0, 2] and o["kv_last_page_len"].tolist() == [3, 1]
    pool, _ = new_pool("bf16", 16)
    mla.mla_cache_write(torch.empty(0, 512, **bf16), torch.empty(0, 64, **bf16), pool, o["slots"],
                        kv_dtype="bf16", err=err, **rope)
    assert (pool == 7).all()
    q = torch.empty(0, 16, 192, **bf16)
    mla.mla_absorb_q(q, w, torch.empty(0, 16, 576, **bf16), sm_scale=SCALE, err=err, **rope)
    mla.mla_absorb_out(torch.empty(0, 16, 512, **bf16), w, torch.empty(0, 16, 128, **bf16))
    attend = mla.MlaPrefill([0, 0, 0], [0, 1, 3], [3, 1], page_size=4, kv_dtype="bf16")
    attend(q, pool, w, torch.empty(0, 16, 128, **bf16), sm_scale=SCALE,
           kv_indices=o["kv_indices"], **rope)
    mla.mla_prefill_check(attend.plan, attend.workspace)
    mla.mla_error_check(err)


def test_cache_step_refuses_arrays_that_are_not_lists(mla):
    # a [requests, k] tensor of lengths must not pass for its first entries
    def call(**kw):
        a = dict(old=i32([3, 5]), new=i32([1, 1]), table=i32([[1, 0], [0, 2]]), free=i32([3, 4]),
                 idx=i32([0] * 4), slots=torch.zeros(2, dtype=torch.int64, device="cuda"),
                 pos=i32([0] * 2))
        a.update(kw)
        mla.mla_cache_step(a["old"], a["new"], a["table"], a["free"], page_size=4,
                           kv_indptr=i32([0] * 3), kv_last_page_len=i32([0] * 2),
                           kv_indices=a["idx"], qo_indptr=i32([0] * 3), slots=a["slots"],
                           positions=a["pos"])

    call()
    for bad in (dict(old=i32([[3, 5], [7, 9]])), dict(old=i32([[3], [5]])),
                dict(free=i32([[3, 4]])), dict(idx=i32([[0, 0], [0, 0]])),
                dict(slots=torch.zeros(2, 1, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            call(**bad)


@pytest.mark.parametrize("report", [True, False])
@pytest.mark.parametrize("tokens,heads", [(5, 16), (130, 16), (300, 40)])
def test_absorbed_products_whose_wait_gives_up(mla, tokens, heads, report):
    # the waits for operands run out: nothing of the output before them is left,
    # the error word says so, and the next call is right
    g = torch.Generator(device="cuda").manual_seed(tokens)
    w = make_w(heads, gen(tokens)).cuda()
    q = torch.randn(tokens, heads, 192, generator=g, device="cuda").bfloat16()
    o = torch.randn(tokens, heads, 512, generator=g, device="cuda").bfloat16()
    err = word() if report else None
    scale = torch.full((1,), 0.02, device="cuda")
    outs = [torch.full((tokens + 2, heads, n), 7.0, dtype=torch.bfloat16, device="cuda")
            for n in (576, 128)]
    qa, out = (x[1:-1] for x in outs)
    q8 = torch.full((tokens, heads, 576), 0x11, dtype=torch.uint8, device="cuda")
    for x, y, s in ((q, qa, None), (q, q8, scale), (o, out, None)):
        mla.mla_selftest_absorb_wait(x, w, y, q_scale=s, err=err)
        if report:
            with pytest.raises(mla.MlaError) as e:
                mla.mla_error_check(err)
            assert e.value.status == 5
            mla.mla_error_check(err)
    torch.cuda.synchronize()
    assert torch.isnan(qa[..., :512]).all() and torch.isnan(out).all()
    assert torch.isnan(q8.view(torch.float8_e4m3fn).float()[..., :512]).all()
    assert all((x[[0, -1]] == 7).all() for x in outs)
    # the rotated dims wait for nothing
    assert torch.equal(qa[..., 512:], (q[..., 128:].float() * 24).bfloat16())
    mla.mla_absorb_q(q, w, qa, sm_scale=1.0, err=err)
    mla.mla_absorb_q(q, w, q8, sm_scale=1.0, q_scale=scale, err=err)
    mla.mla_absorb_out(o, w, out, err=err)
    if report:
        mla.mla_error_check(err)
    assert torch.isfinite(qa).all() and torch.isfinite(q8.view(torch.float8_e4m3fn).float()).all()
    ref = torch.einsum("thc,hvc->thv", o.double(), w[:, 128:].double())
    mag = torch.einsum("thc,hvc->thv", o.double().abs(), w[:, 128:].double().abs())
    acc = 512 * F * mag
    assert ((out.double() - ref).abs() <= acc + U * (ref.abs() + acc)).all()


@pytest.mark.parametrize("scale", [0.013, 1.0, 2.0**-59, 2.0**-61, 2.0**61, 3e-30, -0.5])
@pytest.mark.parametrize("norm", [True, False])
def test_cache_write_zeros_and_scales_of_any_size(mla, scale, norm):
    # bytes of the plain 32-bit quotient: signed zeros, and scales on both sides
    # of the range in which it is had without a division
    g = gen(61)
    latent = torch.randn(40, 512, generator=g).bfloat16()
    k_rope = torch.randn(40, 64, generator=g).bfloat16()
    for x in (latent, k_rope):
        x[:, 0::7] = 0.0
        x[:, 3::7] = -0.0
        x[5] = -0.0
        x[6, 1::2] *= 2.0**-30
    weight = (1 + 0.2 * torch.randn(512, generator=g)).bfloat16() if norm else None
    sc = torch.tensor([scale])
    pool, _ = new_pool("fp8", 40)
    out = torch.empty(40, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_write(latent.cuda(), k_rope.cuda(), pool, torch.arange(40, device="cuda"),
                        kv_dtype="fp8", eps=1e-5, norm_weight=None if weight is None
                        else weight.cuda(), kv_scale=sc.cuda(), rows=out)
    y = plain_row(latent, k_rope, weight, 1e-5, None, None, None)
    q = (y / sc).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(pool.cpu(), q.view(torch.uint8))
    assert torch.equal(out.cpu().view(torch.int16), (q.float() * sc).bfloat16().view(torch.int16))


# ------------------------------------- rows one by one, more heads, whole chains
def row_errors(c):
    """For every row (token, head): out and lse in 64 bits and the standard
    deviation of their errors if every rounding is an error of its own, uniform
    over its step: u / sqrt 3 for key, query, value, probability and output."""
    q, w = c["q"].double(), c["weights"].double()
    if c["rope"]:
        q = torch.cat([q[..., :128], rotate(q[..., 128:], c["table"], c["pos"], c["rope"])], -1)
    r = U / math.sqrt(3)
    outs, lses, sd_o, sd_l = [], [], [], []
    for b, (m, n) in enumerate(zip(c["q_lens"], c["kv_lens"])):
        x = c["rows"][request_rows(c, b)]
        qb = q[c["qo"][b]: c["qo"][b + 1]]
        kv = torch.einsum("nc,hdc->hnd", x[:, :512], w)
        k = torch.cat([kv[..., :128], x[:, 512:].expand(c["heads"], -1, -1)], -1)
        s = torch.einsum("mhd,hnd->hmn", qb, k) * SCALE
        see = torch.arange(n)[None] < (n - m + 1 + torch.arange(m))[:, None]
        p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
        v = kv[..., 128:]
        o = p @ v
        # score: either factor of each product; (v - o): what a weight moves
        var_s = 2 * r * r * SCALE ** 2 * torch.einsum("mhd,hnd->hmn", qb.square(), k.square())
        far = v.square().sum(-1)[:, None] - 2 * o @ v.transpose(1, 2) + o.square().sum(-1)[..., None]
        sd_o.append((torch.einsum("hmn,hmn->hm", p.square() * var_s, far)
                     + 2 * r * r * torch.einsum("hmn,hn->hm", p.square(), v.square().sum(-1))
                     + r * r * o.square().sum(-1)).sqrt().T)
        sd_l.append((p.square() * var_s).sum(-1).sqrt().T)
        outs.append(o.transpose(0, 1))
        lses.append(torch.logsumexp(s.masked_fill(~see, -math.inf), -1).T)
    return torch.cat(outs), torch.cat(lses), torch.cat(sd_o), torch.cat(sd_l)


def check_rows(mla, c, num_sms=0):
    o, lse, _ = run_prefill(mla, c, num_sms)
    ref, ref_lse, sd_o, sd_l = row_errors(c)
    # six standard deviations; sums, exponents and logarithms in fp32: 64 F each
    off = (o - ref).norm(dim=-1) / (6 * sd_o + 64 * F * ref.norm(dim=-1))
    assert off.max() <= 1, (off.max(), off.argmax())
    off = (lse - ref_lse).abs() / (6 * sd_l + 64 * F * (1 + ref_lse.abs()))
    assert off.max() <= 1, (off.max(), off.argmax())
    return o


@pytest.mark.parametrize("q_lens,kv_lens,num_sms", [
    ([300, 1, 40], [300, 200, 131], 0), ([70], [900], 0), ([70, 9], [900, 1300], 40),
    ([600], [700], 0), ([900, 400], [1000, 400], 4)])
@pytest.mark.parametrize("kv", ["bf16", "mxfp4"])
def test_prefill_row_by_row(mla, kv, q_lens, kv_lens, num_sms):
    # a row of its own, not the whole output: one lost key of 1000 would show
    check_rows(mla, prefill_case(q_lens, kv_lens, 3, kv, 8, "interleaved", 71), num_sms)


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([33, 5], [33, 200], 33), ([520, 3], [520, 64], 20),
                                                  ([17], [150], 128), ([3], [40], 1024)])
def test_prefill_with_more_heads(mla, q_lens, kv_lens, heads):
    check_rows(mla, prefill_case(q_lens, kv_lens, heads, "bf16", 8, "half", 72))


@pytest.mark.parametrize("tokens,heads", [(1, 17), (5, 128), (130, 64), (2, 1024)])
def test_absorbed_products_with_more_heads(mla, tokens, heads):
    g = gen(heads)
    q = torch.randn(tokens, heads, 192, generator=g).bfloat16()
    o = torch.randn(tokens, heads, 512, generator=g).bfloat16()
    w = make_w(heads, g).cuda()
    qa = torch.full((tokens + 2, heads, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((tokens + 2, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_q(q.cuda(), w, qa[1:-1], sm_scale=SCALE)
    mla.mla_absorb_out(o.cuda(), w, out[1:-1])
    f = 24 * SCALE
    for got, x, y in ((qa[1:-1, :, :512], q[..., :128].double().cuda() * f, w[:, :128].double()),
                      (out[1:-1], o.double().cuda(), w[:, 128:].double().transpose(1, 2))):
        ref = torch.einsum("thk,hkn->thn", x, y)
        # sums of at most 512 products and the factor; one rounding
        acc = 516 * F * torch.einsum("thk,hkn->thn", x.abs(), y.abs())
        assert ((got.double() - ref).abs() <= acc + U * (ref.abs() + acc)).all()
    f32 = torch.tensor(24.0) * torch.tensor(SCALE)
    assert torch.equal(qa[1:-1, :, 512:].cpu(), (q[..., 128:].float() * f32).bfloat16())
    assert (qa[[0, -1]] == 7).all() and (out[[0, -1]] == 7).all()


# Roundings of the absorbed chain as independent errors of u / sqrt 3 (query,
# its low part, probabilities, latent output, output, key): sqrt 6 of them stay
# near 0.6 %.  An e4m3 query moves a score by 2^-4 / sqrt 3 of its terms, which
# are 0.87 x 1 / 24 in size and 576: 0.031, and the output by as much of its norm.
@pytest.mark.parametrize("kv,q_dtype,limit", [("bf16", "bf16", 2e-2), ("fp8", "bf16", 2e-2),
                                              ("fp8", "fp8", 1e-1), ("mxfp4", "bf16", 2e-2)])
def test_absorbed_form_request_by_request(mla, kv, q_dtype, limit):
    kv_lens = [5, 300, 1, 777, 130]
    c = prefill_case([1] * 5, kv_lens, 16, kv, 8, "interleaved", 73)
    ref = row_errors(c)[0]
    w = c["w"].to("cuda")
    fp8 = q_dtype == "fp8"
    weights, err = c["weights"].cuda(), word()
    qa = torch.empty(5, 16, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    qs = torch.full((1,), 0.02, device="cuda") if fp8 else None
    mla.mla_absorb_q(c["q"].cuda(), weights, qa, sm_scale=SCALE, positions=c["pos"].cuda(),
                     cos_sin=c["table"].cuda(), q_scale=qs, err=err)
    decode = mla.MlaDecoder(w.kv_indptr, w.kv_last_page_len, page_size=8, q_dtype=q_dtype,
                            kv_dtype=kv)
    lat = torch.empty(5, 16, 512, dtype=torch.bfloat16, device="cuda")
    decode(qa, w.kv, lat, q_scale=qs, kv_scale=w.kv_scale, kv_e8m0=w.kv_e8m0,
           kv_indices=w.kv_indices)
    mla.mla_decode_check(decode.plan, decode.workspace)
    out = torch.empty(5, 16, 128, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_out(lat, weights, out, err=err)
    mla.mla_error_check(err)
    for b in range(5):
        off = out[b].cpu().double() - ref[b]
        assert off.norm() <= limit * ref[b].norm(), (b, off.norm() / ref[b].norm())


def test_replayed_calls_give_the_eager_bits(mla):
    # a whole step in one graph: cache write, both forms, on new inputs each replay
    c = prefill_case([150], [400], 16, "bf16", 8, "interleaved", 74)
    w = c["w"].to("cuda")
    weights, pos, table = c["weights"].cuda(), c["pos"].cuda(), c["table"].cuda()
    attend = mla.MlaPrefill(c["qo"], w.kv_indptr, w.kv_last_page_len, page_size=8,
                            kv_dtype="bf16")
    slots = request_rows(c, 0)[250:].cuda()
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    q, latent, k_rope = (torch.zeros(150, *s, **bf16) for s in ((16, 192), (512,), (64,)))
    lat = torch.zeros(150, 16, 512, **bf16)
    outs = [torch.zeros(150, 16, n, **bf16) for n in (128, 576, 128)]
    err = word()

    def step():
        mla.mla_cache_write(latent, k_rope, w.kv, slots, kv_dtype="bf16", positions=pos,
                            cos_sin=table, err=err)
        attend(q, w.kv, weights, outs[0], sm_scale=SCALE, positions=pos, cos_sin=table,
               kv_indices=w.kv_indices)
        mla.mla_absorb_q(q, weights, outs[1], sm_scale=SCALE, positions=pos, cos_sin=table, err=err)
        mla.mla_absorb_out(lat, weights, outs[2], err=err)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2, 3):
        r = torch.Generator(device="cuda").manual_seed(seed)
        for x in (q, latent, k_rope, lat):
            x.copy_(torch.randn(x.shape, generator=r, device="cuda"))
        step()
        eager = [x.clone() for x in outs]
        for x in outs:
            x.fill_(7.0)
        w.kv[slots] = 7.0
        g.replay()
        torch.cuda.synchronize()
        for x, e in zip(outs, eager):
            assert torch.equal(x, e) and x.float().abs().sum() > 0
    mla.mla_error_check(err)
    mla.mla_prefill_check(attend.plan, attend.workspace)
