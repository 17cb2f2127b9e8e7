"""GPU tests of the operators that read less of a long cache against plain
implementations in 64 bits.

Tolerances count roundings: U = 2^-8 bounds one rounding to bf16 (half of
torch.finfo's eps), F = 2^-24 one to fp32.  A matrix instruction's sums round
towards zero: 2 F of the sum of magnitudes for each term.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -24
INF, NAN = math.inf, math.nan
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FORMATS = [("bf16", "bf16"), ("bf16", "fp8"), ("fp8", "fp8"), ("fp8", "bf16"), ("bf16", "mxfp4")]


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mla_decode_stage1_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def indptr(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def make_pool(kv, x):
    """(pool arguments, stored values in 64 bits without the scale, scale) of rows x [n, 576] fp32."""
    n = len(x)
    if kv == "bf16":
        p = x.bfloat16()
        return dict(kv=p), p.double(), 1.0
    if kv == "fp8":
        scale = torch.full((1,), 0.0131, device="cuda")
        e = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        return dict(kv=e.view(torch.uint8), kv_scale=scale), e.double(), float(scale.double())
    b = x.reshape(n, 18, 32)
    e = (torch.frexp(b.abs().amax(-1))[1].int() + 124).clamp(0, 254)
    e = torch.where(torch.isfinite(b).all(-1), e, 255)
    v = torch.ldexp(b, (127 - e)[..., None].float())
    m = v.abs()
    code = sum((m > t).int() for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0))
    code = (code | (torch.signbit(v).int() << 3)).reshape(n, 576)
    lut = torch.tensor(E2M1 + tuple(-t for t in E2M1), dtype=torch.float64, device="cuda")
    val = lut[code.long()].reshape(n, 18, 32) * torch.exp2(e.double() - 127)[..., None]
    val = torch.where((e == 255)[..., None], NAN, val).reshape(n, 576)
    c = code.to(torch.uint8)
    return (dict(kv=(c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), kv_e8m0=e.to(torch.uint8)), val, 1.0)


def make_query(kind, shape, g, std=1.5):
    x = std * torch.randn(*shape, generator=g, device="cuda")
    if kind == "fp8":
        scale = torch.full((1,), 0.017, device="cuda")
        e = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        return dict(q=e.view(torch.uint8), q_scale=scale), e.double() * scale.double()
    return dict(q=x.bfloat16()), x.bfloat16().double()


# ------------------------------------------------------------- shared prefixes
class Case:
    """Groups of requests: per (requests), prefix (pages), own (tokens)."""

    def __init__(self, per, prefix, own, page, q="bf16", kv="bf16", q_len=1, seed=1, table=True,
                 rows=None, std=1.5, extra=2, form="once"):
        g = gen(seed)
        self.per, self.prefix, self.own, self.page, self.q_len = per, prefix, own, page, q_len
        self.qd, self.kd, self.table, self.form = q, kv, table, form
        self.bs = sum(per)
        own_pages = [-(-n // page) for n in own]
        total = sum(prefix) + sum(own_pages)
        self.prefix_at, self.own_at = indptr(prefix), indptr(own_pages)
        if table:
            ids = torch.randperm(total + extra, generator=g, device="cuda")[:total].int()
        else:                                # the prefixes first, the ends behind them
            ids = torch.arange(total, dtype=torch.int32, device="cuda")
            self.own_at = [a + sum(prefix) for a in self.own_at]
        self.prefix_ids, self.own_ids = ids[: sum(prefix)].clone(), ids[sum(prefix):].clone()
        if rows is None:
            rows = torch.randn((total + extra) * page, 576, generator=g, device="cuda")
        self.pool, self.stored, self.scale = make_pool(kv, rows)
        self.query, self.qv = make_query(q, (self.bs * q_len, 16, 576), g, std)
        self.last = [n - (p - 1) * page if p else 0 for n, p in zip(own, own_pages)]
        self.group = [i for i, n in enumerate(per) for _ in range(n)]

    def rows_of(self, ids, n=None):
        at = (ids.long()[:, None] * self.page + torch.arange(self.page, device="cuda")).reshape(-1)
        return at if n is None else at[:n]

    def keys_of(self, b):
        """Pool rows of a request: its group's prefix, its own."""
        g = self.group[b]
        base = 0 if self.table else sum(self.prefix)
        own = self.own_ids[self.own_at[b] - base: self.own_at[b + 1] - base]
        return (self.rows_of(self.prefix_ids[self.prefix_at[g]: self.prefix_at[g + 1]]),
                self.rows_of(own, self.own[b]))

    def reference(self):
        """out, lse in 64 bits, the bounds of their errors, and the variances of out's
        errors in units of U^2 / 3."""
        outs, lses, ob, lb, var = [], [], [], [], []
        for b in range(self.bs):
            pre, own = self.keys_of(b)
            for t in range(self.q_len):
                q = self.qv[b * self.q_len + t]
                mine = own[: max(0, len(own) - self.q_len + 1 + t)]
                k = self.stored[torch.cat([pre, mine])] * self.scale
                if len(k) == 0:
                    outs.append(torch.zeros(16, 512, dtype=torch.float64, device="cuda"))
                    lses.append(torch.full((16,), -INF, dtype=torch.float64, device="cuda"))
                    ob.append(outs[-1])
                    var.append(outs[-1])
                    lb.append(torch.zeros_like(lses[-1]))
                    continue
                s = q @ k.T / 24
                lse = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                o = p @ k[:, :512]
                # scores: 576 products (twice that where a bf16 query is two e4m3
                # terms, good to 2^-13 of a step), then a few operations on
                # s log2 e and the maximum
                mag = (q.abs() @ k.abs().T / 24).amax(1)
                e = mag * 2400 * F + 16 * F * s.abs().amax(1)
                e = e + q.abs().amax(1) * 2.0 ** -21 * k.abs().sum(1).max() / 24
                # probabilities to bf16 (or two e4m3 terms, at worst 2^-14 of
                # 2^4), sums of n terms, the output to bf16
                n = len(k)
                pv = p @ k[:, :512].abs()
                inner = pv * (torch.expm1(2 * e)[:, None] + U + (3 * n + 64) * F)
                decoded = torch.cat([pre, mine]) if self.form == "each" else mine
                if len(decoded) and self.kd != "bf16":
                    inner = inner + 2.0 ** -17 * (self.stored[decoded][:, :512].abs() * self.scale).sum(0)
                outs.append(o)
                lses.append(lse)
                var.append(p.square() @ k[:, :512].square() + o.square())
                ob.append(inner + U * (o.abs() + inner))
                lb.append(e + (n + 64) * F + 8 * F * lse.abs())
        return [torch.stack(x) for x in (outs, lses, ob, lb, var)]

    def plan(self, mla, num_sms=0):
        return mla.mla_shared_plan(indptr(self.per), self.prefix_at, self.own_at, self.last,
                                   page_size=self.page, q_dtype=self.qd, kv_dtype=self.kd,
                                   q_len=self.q_len, num_sms=num_sms, form=self.form)

    def run(self, mla, num_sms=0, check=True, plan=None, ws=None, want_lse=True):
        plan = self.plan(mla, num_sms) if plan is None else plan
        # workspaces come as they are: fill it with NaN patterns
        if ws is None:
            ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        rows = self.bs * self.q_len
        store = torch.full((rows + 2, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows + 2, 16), 7.0, device="cuda")
        mla.mla_shared_run(plan, self.query["q"], self.pool["kv"], store[1:-1], workspace=ws,
                           q_scale=self.query.get("q_scale"), kv_scale=self.pool.get("kv_scale"),
                           kv_e8m0=self.pool.get("kv_e8m0"),
                           prefix_indices=self.prefix_ids if self.table else None,
                           kv_indices=self.own_ids if self.table else None,
                           lse=lse[1:-1] if want_lse else None)
        if check:
            mla.mla_shared_check(plan, ws)
        assert (store[[0, -1]] == 7).all() and (lse[[0, -1]] == 7).all()
        return store[1:-1], lse[1:-1]


def check_shared(mla, c, num_sms=0):
    o, lse = c.run(mla, num_sms)
    ref, ref_lse, bound, lse_bound, var = c.reference()
    none = torch.isneginf(ref_lse)
    assert (o[none] == 0).all() and torch.isneginf(lse[none]).all()
    o, lse = o.double(), lse.double()
    assert torch.isfinite(o).all()
    assert ((o - ref).abs() <= bound).all()
    assert ((lse - ref_lse)[~none].abs() <= lse_bound[~none]).all()
    # Roundings: p_k (1 + e_k) with |e_k| <= U, the same e_k in all dims of a row, and
    # one of each output.  The mean square over 64 dims of sum_k e_k p_k v_kd is at
    # most U^2 sum_k p_k^2 v_kd^2 (three times the mean with e_k spread evenly) for the
    # squares, and its mixed terms average over 64 dims: a relative standard deviation
    # of sqrt(2 / 64) at most, six of which are 1.06.  With the output's own rounding
    # sqrt(3 x 2.06) < 2.5 times the standard deviation bounds the root mean square.
    # (What fp32 adds is 10^-3 of it.)  A structural error is larger.
    rms = (o - ref).square().unflatten(-1, (8, 64)).mean(-1).sqrt()
    assert (rms <= 2.5 * U / math.sqrt(3) * var.unflatten(-1, (8, 64)).mean(-1).sqrt()).all()


@pytest.mark.parametrize("q,kv", FORMATS)
@pytest.mark.parametrize("per,prefix,own,page,q_len", [
    ([3], [30], [5, 0, 130], 8, 1),
    ([1, 9, 0, 20], [17, 4, 9, 3], [1] + list(range(0, 90, 10)) + [3] * 20, 64, 1),
    ([2, 1, 3, 1], [127, 128, 129, 1], [3, 300, 1, 0, 2, 1, 40], 1, 1),
    ([2, 2], [0, 11], [9, 200, 0, 17], 16, 1),
    ([5], [20], [4, 3, 64, 77, 5], 16, 4),
    ([3, 2], [9, 14], [2, 70, 33, 2, 2], 24, 3),
    ([4], [6], [1, 2, 130, 40], 32, 2)])
@pytest.mark.parametrize("form", ["once", "each"])
def test_shared(mla, q, kv, per, prefix, own, page, q_len, form):
    check_shared(mla, Case(per, prefix, own, page, q, kv, q_len, form=form))


@pytest.mark.parametrize("q,kv", FORMATS)
@pytest.mark.parametrize("form,q_len", [("once", 1), ("each", 1), ("each", 2)])
def test_shared_without_page_tables(mla, q, kv, form, q_len):
    c = Case([2, 3], [13, 2], [40, 1, 1, 200, 9], 16, q, kv, q_len, table=False, form=form)
    check_shared(mla, c)
    # one of the two tables: the other's pages are still those of its offsets
    o, lse = [x.clone() for x in c.run(mla)]
    every = torch.arange(10000, dtype=torch.int32, device="cuda")
    for pre, own in ((every, None), (None, every), (every, every)):
        plan = c.plan(mla)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        mla.mla_shared_run(plan, c.query["q"], c.pool["kv"], o2, workspace=ws, lse=lse2,
                           q_scale=c.query.get("q_scale"), kv_scale=c.pool.get("kv_scale"),
                           kv_e8m0=c.pool.get("kv_e8m0"), prefix_indices=pre, kv_indices=own)
        mla.mla_shared_check(plan, ws)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("per,prefix,form", [([4], [64], "each"), ([40, 1], [700, 3], "once")])
def test_shared_takes_the_faster_form(mla, per, prefix, form):
    own = [5 * i for i in range(sum(per))]
    auto = Case(per, prefix, own, 16, "fp8", "fp8", form="auto")
    named = Case(per, prefix, own, 16, "fp8", "fp8", form=form)
    assert (auto.plan(mla).info().num_items == 0) == (form == "each")
    for x, y in zip(auto.run(mla), named.run(mla)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("num_sms", [1, 2, 5, 8, 40, 152])
def test_shared_on_few_and_many_ctas(mla, num_sms):
    # 3 + 1 + 2 blocks of rows of 7, 20 and 1 tiles, cut anywhere
    own = [(7 * i) % 50 for i in range(44)]
    check_shared(mla, Case([20, 8, 16], [100, 313, 4], own, 8, "fp8", "fp8"), num_sms)
    check_shared(mla, Case([20, 8, 16], [100, 313, 4], own, 8), num_sms)
    check_shared(mla, Case([20, 8, 16], [100, 313, 4], own, 8, "bf16", "fp8", form="each"), num_sms)


def test_shared_many_rows_and_long_prefixes(mla):
    check_shared(mla, Case([41], [150], [(11 * i) % 70 for i in range(41)], 16))
    check_shared(mla, Case([1], [3001], [17], 8, "bf16", "fp8"))
    check_shared(mla, Case([1], [64], [64], 64, q_len=64))


def test_shared_is_the_decode_call_on_whole_tables(mla):
    """The same attention through mla_decode_run, each request with all its pages."""
    c = Case([4, 7], [40, 25], [3 * i + 1 for i in range(11)], 16, "fp8", "fp8", seed=3)
    o, lse = c.run(mla)
    ids, at = [], [0]
    for b in range(c.bs):
        g = c.group[b]
        ids += [c.prefix_ids[c.prefix_at[g]: c.prefix_at[g + 1]], c.own_ids[c.own_at[b]: c.own_at[b + 1]]]
        at.append(at[-1] + c.prefix[g] + c.own_at[b + 1] - c.own_at[b])
    plan = mla.mla_decode_plan(at, c.last, page_size=16, q_dtype="fp8", kv_dtype="fp8")
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    mla.mla_decode_run(plan, c.query["q"], c.pool["kv"], o2, workspace=ws, q_scale=c.query["q_scale"],
                       kv_scale=c.pool["kv_scale"], kv_indices=torch.cat(ids), lse=lse2)
    mla.mla_decode_check(plan, ws)
    # each is within the bound
    ref, ref_lse, bound, lse_bound, var = c.reference()
    assert ((o.double() - o2.double()).abs() <= 2 * bound).all()
    assert ((lse.double() - lse2.double()).abs() <= 2 * lse_bound).all()


@pytest.mark.parametrize("num_sms", [2, 152])
@pytest.mark.parametrize("order", ["up", "down", "peak"])
def test_shared_scores_that_grow(mla, num_sms, order):
    """Rows' maxima that move in many tiles: the output is rescaled each time."""
    n = 2000
    g = gen(9)
    x = torch.randn(n + 128, 576, generator=g, device="cuda")
    w = torch.linspace(0.02, 4, n, device="cuda")
    w = w if order == "up" else w.flip(0) if order == "down" else torch.minimum(w, w.flip(0)) * 2
    x[:n] *= w[:, None]
    c = Case([9], [n // 8], [3] * 9, 8, rows=x, table=False, extra=7, std=6.0)
    check_shared(mla, c, num_sms)


def test_shared_equal_and_extreme_scores(mla):
    # queries of zero: the mean of all values; and scores of some thousands
    c = Case([2], [50], [20, 0], 8)
    c.query["q"].zero_()
    c.qv.zero_()
    check_shared(mla, c)
    c = Case([2], [50], [20, 0], 8, std=1000.0)
    check_shared(mla, c)


@pytest.mark.parametrize("form", ["once", "each"])
@pytest.mark.parametrize("power", [10, 22, 28, 29, 36, 70])
@pytest.mark.parametrize("q,kv", FORMATS)
def test_shared_scores_of_any_size(mla, q, kv, power, form):
    """Values -2 .. 2 times a power of two: products and their sums are exact, and scores
    so far apart that the largest ones of a row have all the weight."""
    g = gen(34)
    for per, prefix, own, page in (([3], [170], [30, 0, 9], 8), ([20], [40], [11] * 20, 64)):
        total = sum(prefix) + sum(-(-n // page) for n in own) + 2
        k = torch.randint(-2, 3, (total * page, 576), generator=g, device="cuda").float()
        c = Case(per, prefix, own, page, q, kv, rows=k * 2.0 ** power if kv != "fp8" else k, form=form)
        x = torch.randint(-2, 3, c.query["q"].shape, generator=g, device="cuda").float()
        if q == "fp8":
            c.query["q"].copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
            c.query["q_scale"].fill_(1.0)
        else:
            c.query["q"].copy_(x.bfloat16())
        if kv == "fp8":
            c.pool["kv"].copy_(k.to(torch.float8_e4m3fn).view(torch.uint8))
            c.pool["kv_scale"].fill_(2.0 ** power)
        o, lse = c.run(mla)
        for b in range(c.bs):
            keys = k[torch.cat(c.keys_of(b))].double()
            s = x[b].double() @ keys.T
            w = (s == s.amax(1, keepdim=True)).double()
            ref = w @ keys[:, :512] / w.sum(1, keepdim=True)
            # probabilities and output to bf16; the products of scale and score, the sums
            assert ((o[b].double() / 2.0 ** power - ref).abs() <= 2 * (2 * U + 64 * F)).all()
            top = s.amax(1) * 2.0 ** power / 24
            assert ((lse[b].double() - top - w.sum(1).log()).abs() <= 16 * F * (top.abs() + 8)).all()


@pytest.mark.parametrize("form", ["once", "each"])
@pytest.mark.parametrize("q,kv,q_scale,kv_scale,std", [
    ("bf16", "fp8", 1.0, 0.0, 1.5), ("fp8", "fp8", 0.0, 0.0131, 1.5), ("fp8", "bf16", 0.0, 1.0, 1.5),
    ("bf16", "fp8", 1.0, -0.0131, 1.5), ("bf16", "fp8", 1.0, -0.0131, 60.0),
    ("fp8", "fp8", -0.8, 0.0131, 1.5), ("fp8", "fp8", -0.8, -0.0131, 1.5), ("fp8", "bf16", -0.8, 1.0, 1.5)])
def test_shared_scales_of_zero_and_below(mla, q, kv, q_scale, kv_scale, std, form):
    """Scales are factors like any other: 0 (that of a pool of zeros) makes all scores
    equal, a negative one turns their order around."""
    for per, prefix, page in (([3], [31], 8), ([20], [64], 16), ([2, 9], [0, 3], 64)):
        c = Case(per, prefix, [(7 * i) % 40 for i in range(sum(per))], page, q, kv, std=std, form=form)
        if q == "fp8":
            c.query["q_scale"].fill_(q_scale)
            c.qv = c.query["q"].view(torch.float8_e4m3fn).double() * c.query["q_scale"].double()
        if kv == "fp8":
            # (the reference's bounds take a positive scale: its sign with the values)
            c.pool["kv_scale"].fill_(kv_scale)
            c.scale = abs(float(c.pool["kv_scale"].double()))
            c.stored = c.stored * math.copysign(1.0, kv_scale)
        check_shared(mla, c)


@pytest.mark.parametrize("form", ["once", "each"])
@pytest.mark.parametrize("scale", [0, 2, 8, 27, 87, 127])
def test_shared_mxfp4_tokens_of_zeros(mla, scale, form):
    """Blocks of zeros have the smallest scale byte: such tokens have scores of 0 and
    their full weight."""
    for std in (0.3, 1.5):
        c = Case([3, 17], [33, 9], [20, 3, 1] + [5] * 17, 8, "bf16", "mxfp4", std=std, form=form)
        zero = torch.rand(len(c.stored), generator=gen(35), device="cuda") < 0.6
        c.pool["kv"][zero] = 0
        c.pool["kv_e8m0"][zero] = scale
        c.stored[zero] = 0
        check_shared(mla, c)
    # nothing but zeros
    c.pool["kv"].zero_()
    c.pool["kv_e8m0"].fill_(scale)
    o, lse = c.run(mla)
    n = torch.tensor([len(torch.cat(c.keys_of(b))) for b in range(c.bs)], device="cuda").double()
    assert (o == 0).all() and ((lse.double() - n.log()[:, None]).abs() <= 64 * F * (1 + n.log()[:, None])).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
def test_shared_values_that_are_not_finite(mla, kv):
    """A bad row reaches exactly the requests that attend to it."""
    per, prefix, own = [9, 3], [40, 33], [20] * 12
    c = Case(per, prefix, own, 8, kv=kv, seed=4)
    rows = torch.randn(len(c.stored), 576, generator=gen(5), device="cuda")
    bad_prefix = int(c.keys_of(10)[0][130])            # of group 1
    bad_own = int(c.keys_of(2)[1][7])                  # of request 2
    rows[bad_prefix, 3] = NAN
    rows[bad_own, 500] = NAN
    d = Case(per, prefix, own, 8, kv=kv, seed=4, rows=rows)
    o, lse = d.run(mla)
    hit = torch.tensor([b >= 9 or b == 2 for b in range(12)], device="cuda")
    assert torch.isnan(lse[hit]).all() and torch.isnan(o[hit]).flatten(1).any(1).all()
    assert torch.isfinite(o[~hit]).all() and torch.isfinite(lse[~hit]).all()


def test_shared_rows_behind_a_request_end_do_not_count(mla):
    """NaN in the page's rows that a request does not reach yet."""
    c = Case([3], [9], [20, 3, 1], 16, seed=6)
    rows = torch.randn(len(c.stored), 576, generator=gen(7), device="cuda")
    d = Case([3], [9], [20, 3, 1], 16, seed=6, rows=rows)
    o, _ = d.run(mla)
    used = torch.zeros(len(rows), dtype=torch.bool, device="cuda")
    for b in range(3):
        for k in d.keys_of(b):
            used[k] = True
    rows[~used] = NAN
    e = Case([3], [9], [20, 3, 1], 16, seed=6, rows=rows)
    o2, _ = e.run(mla)
    assert (o == o2).all()


def test_shared_a_query_that_is_not_finite(mla):
    c = Case([20], [30], [9] * 20, 8)
    clean, _ = c.run(mla)
    c.query["q"][7, 5, 100] = NAN
    o, lse = c.run(mla)
    hit = torch.zeros(20, 16, dtype=torch.bool, device="cuda")
    hit[7, 5] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert (o[~hit] == clean[~hit]).all()


def test_shared_reports_bad_pages_and_workspaces(mla):
    c = Case([3], [30], [5, 0, 130], 8)
    plan = c.plan(mla)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    clean, _ = c.run(mla, plan=plan, ws=ws)
    clean = clean.clone()
    for ids in (c.prefix_ids, c.own_ids):
        for bad in (-1, len(c.stored) // 8, 2 ** 31 - 1):
            keep = int(ids[3])
            ids[3] = bad
            c.run(mla, check=False, plan=plan, ws=ws)
            with pytest.raises(mla.MlaError) as e:
                mla.mla_shared_check(plan, ws)
            assert e.value.status == 1
            ids[3] = keep
    assert (c.run(mla, plan=plan, ws=ws)[0] == clean).all()
    # another plan's table at the same address
    d = Case([2], [9], [5, 7], 8)
    other = d.plan(mla)
    assert other.workspace_bytes <= plan.workspace_bytes
    d.run(mla, plan=other, ws=ws)
    c.run(mla, check=False, plan=plan, ws=ws)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_shared_check(plan, ws)
    assert e.value.status == 3
    assert (c.run(mla, plan=plan, ws=ws)[0] == clean).all()


def test_shared_notices_an_overwritten_work_table(mla):
    c = Case([20, 3], [100, 30], [5] * 23, 8)
    plan = c.plan(mla)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    clean = c.run(mla, plan=plan, ws=ws)[0].clone()
    # behind the header: tiles of 128 gathered rows, clusters' ranges, items, tokens' jobs
    info = plan.info()
    at = 256
    for size, count in ((32, 7 + 2), (16, info.num_clusters), (32, info.num_items), (32, 23)):
        for k in {0, count // 2, count - 1}:
            for word in range(3):
                field = ws[at + k * size + 4 * word: at + k * size + 4 * word + 4]
                keep = field.clone()
                field.copy_(keep ^ 0x11)
                c.run(mla, check=False, plan=plan, ws=ws)
                with pytest.raises(mla.MlaError) as e:
                    mla.mla_shared_check(plan, ws)
                assert e.value.status == 3
                # (the next run uploads the table again)
                assert torch.equal(c.run(mla, plan=plan, ws=ws)[0], clean)
        at += -(-size * count // 256) * 256


def test_shared_repeats_bit_by_bit(mla):
    """Hundreds of calls of several plans in turn."""
    cases = [Case([9, 3], [77, 12], [(5 * i) % 40 for i in range(12)], 16, "bf16", "fp8"),
             Case([1], [130], [0], 8), Case([30], [64], [1] * 30, 64, "fp8", "fp8"),
             Case([4], [31], [64, 3, 5, 9], 8, "bf16", "mxfp4", q_len=2)]
    plans = [c.plan(mla) for c in cases]
    wss = [torch.full((p.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda") for p in plans]
    first = [[x.clone() for x in c.run(mla, plan=p, ws=w)] for c, p, w in zip(cases, plans, wss)]
    for _ in range(100):
        for c, p, w, f in zip(cases, plans, wss, first):
            o, lse = c.run(mla, check=False, plan=p, ws=w)
            assert torch.equal(o, f[0]) and torch.equal(lse, f[1])
    for p, w in zip(plans, wss):
        mla.mla_shared_check(p, w)


@pytest.mark.parametrize("per,q", [(1, "bf16"), (1, "fp8"), (16, "fp8"), (33, "bf16")])
def test_shared_first_calls_of_plans_on_cold_memory(mla, per, q):
    """Loads of very different latencies: new workspaces, tables and caches without any
    of it, the call's kernels all enqueued before the first begins."""
    c = Case([per], [3001], [17] * per, 8, q, "fp8")
    rows = c.bs
    plans = [c.plan(mla) for _ in range(12)]
    wss = [torch.full((p.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda") for p in plans]
    outs = [torch.zeros(rows, 16, 512, dtype=torch.bfloat16, device="cuda") for _ in plans]
    lses = [torch.zeros(rows, 16, device="cuda") for _ in plans]
    other = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for p, w, o, lse in zip(plans, wss, outs, lses):
        other.fill_(1)
        mla.mla_shared_run(p, c.query["q"], c.pool["kv"], o, workspace=w, lse=lse,
                           q_scale=c.query.get("q_scale"), kv_scale=c.pool["kv_scale"],
                           prefix_indices=c.prefix_ids, kv_indices=c.own_ids)
    ref, ref_lse, bound, lse_bound, _ = c.reference()
    for p, w, o, lse in zip(plans, wss, outs, lses):
        mla.mla_shared_check(p, w)
        assert ((o.double() - ref).abs() <= bound).all()
        assert ((lse.double() - ref_lse).abs() <= lse_bound).all()
        assert torch.equal(o, outs[0]) and torch.equal(lse, lses[0])


def test_shared_plans_on_several_streams_at_once(mla):
    cases = [Case([9, 3], [77, 12], [(5 * i) % 40 for i in range(12)], 16, "bf16", "fp8"),
             Case([40], [700], [3 * i for i in range(40)], 16, "fp8", "fp8"),
             Case([2, 30], [90, 64], [100] * 32, 64), Case([4], [31], [64, 3, 5, 9], 8, "bf16", "mxfp4", q_len=2),
             Case([17], [300], [30] * 17, 8, "fp8", "fp8", form="each"), Case([1], [2000], [1], 8)]
    plans = [c.plan(mla) for c in cases]
    wss = [torch.full((p.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda") for p in plans]
    first = [[x.clone() for x in c.run(mla, plan=p, ws=w)] for c, p, w in zip(cases, plans, wss)]
    outs = [torch.empty_like(o) for o, _ in first]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(40):
        for k, (c, p, w, o) in enumerate(zip(cases, plans, wss, outs)):
            mla.mla_shared_run(p, c.query["q"], c.pool["kv"], o, workspace=w, stream=streams[k % 3],
                               q_scale=c.query.get("q_scale"), kv_scale=c.pool.get("kv_scale"),
                               kv_e8m0=c.pool.get("kv_e8m0"), prefix_indices=c.prefix_ids,
                               kv_indices=c.own_ids)
        if i % 8 == 7:
            torch.cuda.synchronize()
            for o, f in zip(outs, first):
                assert torch.equal(o, f[0])
                o.zero_()
            torch.cuda.synchronize()
    for p, w in zip(plans, wss):
        mla.mla_shared_check(p, w)


def test_calls_wait_for_what_is_in_the_stream(mla):
    """Inputs that a kernel, a copy or another stream writes just before the call, eagerly
    and in a graph."""
    g = gen(21)
    lens, pages, page = i32([900, 64, 3000]), 256, 16
    table = torch.randperm(pages * 3, generator=g, device="cuda")[: 3 * 200].int().reshape(3, 200)
    kv = torch.randn(pages * 3 * page, 576, generator=g, device="cuda").bfloat16()
    bounds = torch.zeros(pages * 3, 2, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(3, 16, 576, generator=g, device="cuda").bfloat16()
    scores = torch.randn(3, 200, generator=g, device="cuda")
    ptr, last, idx = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 3, 90))

    def bounds_call():
        mla.mla_page_bounds(kv, bounds, table, torch.zeros_like(lens), lens, page_size=page, kv_dtype="bf16")
        return [bounds]

    def scores_call():
        mla.mla_page_scores(q, bounds, table, lens, scores, page_size=page)
        return [scores]

    def select_call():
        mla.mla_page_select(scores, table, lens, page_size=page, top_pages=30, kv_indptr=ptr,
                            kv_last_page_len=last, kv_indices=idx)
        return [ptr, last, idx]

    shared = []
    for kd, size, form in (("bf16", 64, "once"), ("fp8", 16, "once"), ("bf16", 16, "each")):
        c = Case([9], [40], [5] * 9, size, kv=kd, form=form)
        plan = c.plan(mla)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        out = torch.empty(9, 16, 512, dtype=torch.bfloat16, device="cuda")

        def call(c=c, plan=plan, ws=ws, out=out):
            mla.mla_shared_run(plan, c.query["q"], c.pool["kv"], out, workspace=ws,
                               kv_scale=c.pool.get("kv_scale"), prefix_indices=c.prefix_ids,
                               kv_indices=c.own_ids)
            return [out]
        shared.append((c.query["q"], call))
    side = torch.cuda.Stream()
    for x, call in [(kv, bounds_call), (q, scores_call), (scores, select_call)] + shared:
        keep = x.clone()
        ref = [o.clone() for o in call()]

        def produce(how):
            if how == "copy":
                x.copy_(keep)
            elif how == "kernel":
                torch.add(keep, 0, out=x)
            else:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    torch.add(keep, 0, out=x)
                torch.cuda.current_stream().wait_stream(side)

        for how in ("copy", "kernel", "stream"):
            for _ in range(4):
                x.zero_()
                torch.cuda._sleep(100000)
                produce(how)
                got = [o.clone() for o in call()]
                assert all(torch.equal(a, b) for a, b in zip(got, ref))
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                produce(how)
                outs = call()
            for _ in range(4):
                x.zero_()
                for o in outs:
                    if o is not x:
                        o.zero_()
                graph.replay()
                assert all(torch.equal(a, b) for a, b in zip(outs, ref))


@pytest.mark.parametrize("q,kv,page,q_len,form", [
    ("bf16", "bf16", 16, 1, "each"), ("fp8", "fp8", 8, 1, "each"), ("bf16", "fp8", 12, 1, "each"),
    ("bf16", "fp8", 16, 2, "each"), ("fp8", "fp8", 5, 2, "each"), ("fp8", "bf16", 8, 1, "each"),
    ("bf16", "mxfp4", 16, 1, "each"), ("bf16", "mxfp4", 7, 2, "each"),
    ("bf16", "bf16", 64, 1, "once"), ("fp8", "fp8", 12, 1, "once"), ("bf16", "mxfp4", 16, 1, "once")])
def test_shared_reads_what_was_written_just_before(mla, q, kv, page, q_len, form):
    """Every input in turn, pages and scales among them, is produced by the kernel that the
    call follows, eagerly and in a graph."""
    c = Case([5, 2], [33, 40], [5, 30, 2, 9, 70, 3, 1], page, q, kv, q_len=q_len, form=form, seed=31)
    plan = c.plan(mla)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    inputs = dict(c.query, **c.pool, prefix=c.prefix_ids, own=c.own_ids)
    out = torch.empty(c.bs * q_len, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(c.bs * q_len, 16, device="cuda")

    def call():
        mla.mla_shared_run(plan, inputs["q"], inputs["kv"], out, workspace=ws, lse=lse,
                           q_scale=inputs.get("q_scale"), kv_scale=inputs.get("kv_scale"),
                           kv_e8m0=inputs.get("kv_e8m0"), prefix_indices=inputs["prefix"],
                           kv_indices=inputs["own"])
    call()
    mla.mla_shared_check(plan, ws)
    ref, ref_lse = out.clone(), lse.clone()
    for name, x in inputs.items():
        keep = x.clone()
        # (other pages of the pool, another scale, zeros)
        other = x.flip(0) if name in ("prefix", "own") else 3 * x if name.endswith("_scale") else 0 * x
        x.copy_(other)
        call()
        assert not torch.equal(lse, ref_lse) or not torch.equal(out, ref)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            torch.mul(keep, 1, out=x)
            call()
        for step in range(4):
            x.copy_(other)
            out.zero_()
            if step % 2:
                graph.replay()
            else:
                torch.cuda._sleep(100000)
                torch.mul(keep, 1, out=x)
                call()
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    mla.mla_shared_check(plan, ws)


@pytest.mark.parametrize("form", ["once", "each"])
def test_shared_call_with_nothing_cached(mla, form):
    """The join is then the call's only kernel: it too comes behind what the stream holds,
    which here writes the outputs, and the work table."""
    c = Case([3, 2], [0, 0], [0] * 5, 16, form=form)
    plan = c.plan(mla)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(5, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(5, 16, device="cuda")

    def call():
        mla.mla_shared_run(plan, c.query["q"], c.pool["kv"], out, workspace=ws, lse=lse,
                           prefix_indices=c.prefix_ids, kv_indices=c.own_ids)
    call()
    mla.mla_shared_check(plan, ws)
    for _ in range(5):
        torch.cuda._sleep(100000)
        out.fill_(7)
        lse.fill_(7)
        call()
        assert (out == 0).all() and torch.isneginf(lse).all()
    mla.mla_shared_check(plan, ws)
    table = ws.clone()
    zeros = torch.zeros_like(ws)
    for _ in range(3):
        torch.cuda._sleep(100000)
        torch.mul(zeros, 1, out=ws)
        call()
        with pytest.raises(mla.MlaError) as e:
            mla.mla_shared_check(plan, ws)
        assert e.value.status == 3
        torch.cuda._sleep(100000)
        torch.mul(table, 1, out=ws)
        call()
        mla.mla_shared_check(plan, ws)


def test_shared_captured_and_on_another_stream(mla):
    c = Case([9, 3], [77, 12], [(5 * i) % 40 for i in range(12)], 16, "bf16", "fp8")
    plan = c.plan(mla)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    clean, clean_lse = [x.clone() for x in c.run(mla, plan=plan, ws=ws)]
    side = torch.cuda.Stream()
    out, lse = torch.zeros_like(clean), torch.zeros_like(clean_lse)
    kw = dict(workspace=ws, kv_scale=c.pool["kv_scale"], prefix_indices=c.prefix_ids,
              kv_indices=c.own_ids, lse=lse)
    side.wait_stream(torch.cuda.current_stream())
    mla.mla_shared_run(plan, c.query["q"], c.pool["kv"], out, stream=side, **kw)
    side.synchronize()
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        mla.mla_shared_run(plan, c.query["q"], c.pool["kv"], out, **kw)
    keep = c.query["q"].clone()
    for i in range(5):
        c.query["q"].copy_(keep * (0 if i % 2 else 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, clean) == (i % 2 == 0)
    mla.mla_shared_check(plan, ws)


@pytest.mark.parametrize("form", ["once", "each"])
def test_shared_owner_and_optional_outputs(mla, form):
    c = Case([4], [9], [3, 2, 0, 1], 8, form=form)
    o, _ = c.run(mla)
    owner = mla.MlaShared([0, 4], c.prefix_at, c.own_at, c.last, page_size=8, q_dtype="bf16",
                          kv_dtype="bf16", form=form)
    out = torch.empty(4, 16, 512, dtype=torch.bfloat16, device="cuda")
    assert owner(c.query["q"], c.pool["kv"], out, prefix_indices=c.prefix_ids,
                 kv_indices=c.own_ids) is out
    assert torch.equal(out, o)
    assert torch.equal(c.run(mla, want_lse=False)[0], o)


def test_shared_refuses_tensors_that_do_not_fit(mla):
    c = Case([4], [9], [3, 2, 0, 1], 8)
    plan = c.plan(mla)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(4, 16, 512, dtype=torch.bfloat16, device="cuda")
    good = dict(q=c.query["q"], kv=c.pool["kv"], out=out, workspace=ws, prefix_indices=c.prefix_ids,
                kv_indices=c.own_ids)
    for bad in (dict(q=good["q"][:3]), dict(q=good["q"].float()), dict(q=good["q"].transpose(0, 1)),
                dict(kv=good["kv"][:, :512]), dict(out=out[:3]), dict(out=out.float()),
                dict(prefix_indices=c.prefix_ids[:8]), dict(kv_indices=c.own_ids[:2]),
                dict(kv_indices=c.own_ids.long()), dict(lse=torch.empty(4, 8, device="cuda")),
                dict(workspace=ws.cpu())):
        k = dict(good, **bad)
        with pytest.raises(ValueError):
            mla.mla_shared_run(plan, k.pop("q"), k.pop("kv"), k.pop("out"), **k)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_shared_run(plan, good["q"], good["kv"], out, workspace=ws[:-256],
                           prefix_indices=c.prefix_ids, kv_indices=c.own_ids)
    assert e.value.status == 3


@pytest.mark.parametrize("page,own", [(64, 40), (32, 30)])
@pytest.mark.parametrize("form", ["once", "each"])
def test_shared_pool_rows_and_gathered_rows_past_4_gb(mla, page, own, form):
    """Two requests on 3.8 million tokens, in reverse order of the pool's pages, which
    are read where they stand or gathered."""
    n = 3_800_064
    pages = n // page + 1
    kv = torch.empty(pages * page, 576, dtype=torch.bfloat16, device="cuda")
    g = gen(11)
    for i in range(0, len(kv), 1 << 19):
        kv[i: i + (1 << 19)] = torch.randn(len(kv[i: i + (1 << 19)]), 576, generator=g, device="cuda").bfloat16()
    ids = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")
    q = (2 * torch.randn(2, 16, 576, generator=g, device="cuda")).bfloat16()
    plan = mla.mla_shared_plan([0, 2], [0, pages - 1], [0, 1, 1], [own, 0], page_size=page,
                               q_dtype="bf16", kv_dtype="bf16", form=form)
    assert page == 64 or form == "each" or plan.workspace_bytes > 1 << 32
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 16, device="cuda")
    mla.mla_shared_run(plan, q, kv, out, workspace=ws, prefix_indices=ids[:-1].contiguous(),
                       kv_indices=ids[-1:].contiguous(), lse=lse)
    mla.mla_shared_check(plan, ws)
    m = torch.full((2, 16), -INF, dtype=torch.float64, device="cuda")
    l, o, pv = torch.zeros_like(m), torch.zeros(2, 16, 512, dtype=torch.float64, device="cuda"), 0
    top = torch.zeros_like(m)
    for i in list(range(0, len(kv), 1 << 17)):
        k = kv[i: i + (1 << 17)].double()
        s = q.double() @ k.T / 24
        if i < page:                          # page 0: request 0's own tokens
            s[0, :, own:page] = -INF
            s[1, :, :page] = -INF
        top = torch.maximum(top, s.masked_fill(s == -INF, 0).abs().amax(-1))
        nm = torch.maximum(m, s.amax(-1))
        f, p = torch.exp(m - nm), torch.exp(s - nm[..., None])
        l, m = l * f + p.sum(-1), nm
        o = o * f[..., None] + p @ k[:, :512]
        pv = pv * f[..., None] + p @ k[:, :512].abs()
    o, pv = o / l[..., None], pv / l[..., None]
    # errors of the probabilities are independent: of ~ 10^6 that count, U / sqrt 3
    # each, the sum's is far below U of the mean of magnitudes; the fp32 sums of a
    # range of 50,000 keys round towards zero, 2 F of the running sum each
    e = 2400 * F * 40 + 16 * F * top.max()
    bound = pv * (2 * e + 2.0 ** -14 + 50_000 / 16 * 2 * F) + U * o.abs()
    assert ((out.double() - o).abs() <= bound).all()
    assert ((lse.double() - m - l.log()).abs() <= e + 1e-4).all()


# --------------------------------------------------------------------- bounds
def plain_bounds(stored, bounds, table, old, new, page):
    out = bounds.double().clone()
    for row, a, n in zip(table, old, new):
        for j in range(a // page, -(-(a + n) // page) if n else 0):
            p, first, end = row[j], max(a, j * page) - j * page, min(a + n, (j + 1) * page) - j * page
            x = stored[p * page + first: p * page + end]
            if first:
                x = torch.cat([x, out[p]])
            lo, hi = x.min(0)[0], x.max(0)[0]
            # a dim with a value that is not finite (or beyond bf16)
            bad = ~torch.isfinite(x.float().bfloat16()).all(0)
            out[p] = torch.stack([lo.masked_fill(bad, NAN), hi.masked_fill(bad, NAN)])
    return out


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("old,new,page,stride", [
    ([0, 5, 63, 64, 65, 200], [1, 1, 1, 1, 1, 1], 64, 0),
    ([0, 0, 17, 31, 100], [300, 0, 15, 2, 501], 32, 3),
    ([0], [1], 1, 0), ([7, 0], [9, 4], 1, 0),
    ([0, 3, 50], [129, 400, 7], 13, 1),
    ([10], [5000], 128, 0),
    (list(range(300)), [1 + i % 3 for i in range(300)], 16, 0)])
def test_page_bounds(mla, kv, old, new, page, stride):
    g = gen(3)
    pages = [-(-(a + n) // page) for a, n in zip(old, new)]
    total = sum(pages)
    ids = torch.randperm(total + 3, generator=g, device="cuda")[:total].tolist()
    at = indptr(pages)
    table = [ids[at[i]: at[i + 1]] for i in range(len(old))]
    width = max(pages)
    t = torch.full((len(old), width + stride), -5, dtype=torch.int32)
    for i, row in enumerate(table):
        t[i, : len(row)] = torch.tensor(row, dtype=torch.int32)
    t = t.cuda()[:, :width]
    x = torch.randn((total + 3) * page, 576, generator=g, device="cuda")
    pool, stored, _ = make_pool(kv, x * torch.exp2(torch.randint(-9, 9, (len(x), 1), generator=g, device="cuda").float()))
    b = (3 * torch.randn(total + 3, 2, 576, generator=g, device="cuda")).sort(1)[0].bfloat16()
    got = b.clone()
    err = word()
    e8 = pool.get("kv_e8m0")
    if e8 is not None and stride:
        wide = torch.full((len(e8), 18 + stride), 99, dtype=torch.uint8, device="cuda")
        wide[:, :18] = e8
        e8 = wide
    ref = plain_bounds(stored, b, table, old, new, page)
    for _ in range(2):                        # a repeated call writes the same
        mla.mla_page_bounds(pool["kv"], got, t, i32(old), i32(new), page_size=page, kv_dtype=kv,
                            kv_e8m0=e8, err=err)
        mla.mla_error_check(err)
        assert same(got.double(), ref)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "mxfp4"])
def test_page_bounds_token_by_token(mla, kv):
    """Any cut of the tokens into calls gives the same bounds."""
    g = gen(4)
    n, page = 150, 32
    pool, stored, _ = make_pool(kv, torch.randn(160, 576, generator=g, device="cuda"))
    table = i32([[3, 0, 4, 1, 2]])
    def run(steps):
        b = torch.full((5, 2, 576), NAN, dtype=torch.bfloat16, device="cuda")
        at = 0
        for k in steps:
            mla.mla_page_bounds(pool["kv"], b, table, i32([at]), i32([k]) if k != 1 else None,
                                page_size=page, kv_dtype=kv, kv_e8m0=pool.get("kv_e8m0"))
            at += k
        return b
    whole = run([n])
    assert torch.isfinite(whole.float()).all()
    assert torch.equal(whole, run([1] * n)) and torch.equal(whole, run([31, 2, 32, 1, 0, 84]))


def test_page_bounds_values_that_are_not_finite(mla):
    x = torch.randn(64, 576, generator=gen(5), device="cuda")
    for row, dim, v in ((3, 0, NAN), (20, 7, INF), (40, 575, -INF), (63, 64, NAN), (5, 100, 3.3895e38)):
        x[row, dim] = v
    pool, stored, _ = make_pool("bf16", x)
    b = torch.zeros(4, 2, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_page_bounds(pool["kv"], b, i32([[0, 1, 2, 3]]), i32([0]), i32([64]), page_size=16, kv_dtype="bf16")
    assert same(b.double(), plain_bounds(stored, b, [[0, 1, 2, 3]], [0], [64], 16))
    assert b.isnan().sum() == 2 * 4
    # and stays so, until the page is begun anew
    pool["kv"].zero_()
    mla.mla_page_bounds(pool["kv"], b, i32([[0]]), i32([8]), i32([8]), page_size=16, kv_dtype="bf16")
    assert b[0].isnan().sum() == 2
    mla.mla_page_bounds(pool["kv"], b, i32([[0]]), i32([0]), i32([1]), page_size=16, kv_dtype="bf16")
    assert (b[0] == 0).all()


def test_page_bounds_reports(mla):
    pool, _, _ = make_pool("fp8", torch.randn(64, 576, generator=gen(6), device="cuda"))
    b = torch.full((4, 2, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    err = word()
    def run(table, old, new, bounds=b, page=16):
        mla.mla_page_bounds(pool["kv"], bounds, i32(table), i32(old), i32(new), page_size=page,
                            kv_dtype="fp8", err=err)
        with pytest.raises(mla.MlaError) as e:
            mla.mla_error_check(err)
        return e.value.status
    assert run([[-1]], [0], [3]) == 1
    assert run([[4]], [0], [3]) == 1
    assert run([[2 ** 31 - 1]], [0], [3]) == 1
    assert run([[2]], [0], [3], bounds=b[:2]) == 1           # more pages in the pool than bounds
    assert run([[0]], [0], [17]) == 6 and (b[1:] == 7).all()  # beyond the table
    assert run([[0]], [0], [-1]) == 1
    assert run([[0]], [2 ** 31 - 1], [2 ** 31 - 1]) == 6
    b.fill_(7)
    assert run([[0, 1], [2, 3]], [-4, 0], [5, 0]) == 1        # as 0 old tokens
    assert (b[0] != 7).any() and (b[1:] == 7).all()


def test_page_bounds_pages_past_4_gb(mla):
    page, pages = 64, 120_000                                # 4.4 GB of rows
    kv = torch.zeros(page * pages, 576, dtype=torch.uint8, device="cuda")
    one = torch.randn(page, 576, generator=gen(7), device="cuda").to(torch.float8_e4m3fn)
    kv[-page:] = one.view(torch.uint8)
    b = torch.zeros(pages, 2, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_page_bounds(kv, b, i32([[pages - 1]]), i32([0]), i32([page]), page_size=page, kv_dtype="fp8")
    assert (b[-1, 0].float() == one.float().amin(0)).all() and (b[-1, 1].float() == one.float().amax(0)).all()
    assert (b[:-1] == 0).all()


# --------------------------------------------------------------------- scores
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,page,q_len,pad", [
    ([64], 64, 1, 0), ([1], 64, 1, 0), ([0, 65, 640, 2000], 64, 1, 3), ([5000, 37], 16, 1, 0),
    ([3, 700, 2, 0], 32, 4, 5), ([260] * 40, 2, 2, 1), ([70_000], 16, 3, 0), ([9000] * 37, 16, 1, 0)])
def test_page_scores(mla, kind, lens, page, q_len, pad):
    g = gen(8)
    width = max(1, max(-(-n // page) for n in lens)) + pad
    bs = len(lens)
    b = (torch.randn(50, 1, 576, generator=g, device="cuda")
         + torch.randn(50, 2, 576, generator=g, device="cuda").sort(1)[0]).bfloat16()
    table = torch.randint(0, 50, (bs, width + pad), generator=g, device="cuda").int()[:, :width]
    query, qv = make_query(kind, (bs * q_len, 16, 576), g)
    store = torch.full((bs * q_len, width + 2 * pad), 7.0, device="cuda")
    err = word()
    kvs = torch.full((1,), 0.3, device="cuda") if pad else None
    mla.mla_page_scores(query["q"], b, table, i32(lens), store[:, pad:], page_size=page, q_len=q_len,
                        q_scale=query.get("q_scale"), kv_scale=kvs, err=err)
    mla.mla_error_check(err)
    assert (store[:, :pad] == 7).all() and (store[:, pad + width:] == 7).all()
    got = store[:, pad: pad + width].double()
    for r in range(bs * q_len):
        seen = max(0, lens[r // q_len] - q_len + 1 + r % q_len)
        n = -(-seen // page)
        assert torch.isneginf(got[r, n:]).all()
        lo, hi = b[table[r // q_len, :n].long()].double().unbind(1)
        q = qv[r]
        s = (q.clamp(min=0) @ hi.T + q.clamp(max=0) @ lo.T) / 24
        mag = (q.clamp(min=0) @ hi.abs().T - q.clamp(max=0) @ lo.abs().T) / 24
        k = 0.3 if pad else 1.0
        k = float(kvs.double()) if pad else 1.0
        # 12 x 16 terms in a row, each of which may round towards zero; six sums
        bound = k * (mag * (12 * 16 * 2 + 6) * F).amax(0) + 4 * F * s.abs().amax(0) * k
        assert ((got[r, :n] - s.amax(0) * k).abs() <= bound).all()


def test_page_scores_bound_the_scores_of_every_token(mla):
    g = gen(9)
    n, page = 500, 16
    pool, stored, scale = make_pool("fp8", torch.randn(512, 576, generator=g, device="cuda"))
    table = torch.randperm(32, generator=g, device="cuda").int()[None]
    b = torch.empty(32, 2, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_page_bounds(pool["kv"], b, table, i32([0]), i32([n]), page_size=page, kv_dtype="fp8")
    query, qv = make_query("fp8", (1, 16, 576), g)
    s = torch.empty(1, 32, device="cuda")
    mla.mla_page_scores(query["q"], b, table, i32([n]), s, page_size=page, q_scale=query["q_scale"],
                        kv_scale=pool["kv_scale"])
    rows = (table[0].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
    exact = (qv[0] @ stored[rows].T).amax(0) * scale / 24
    best = torch.full((512,), -INF, dtype=torch.float64, device="cuda")
    best[:n] = exact
    best = best.reshape(32, page).amax(1)
    assert (s[0].double() >= best - 1e-5 * best.abs()).all()
    # a page of one token: the token's own score
    assert -(-n // page) * page - n < page
    one = torch.empty(1, 1, device="cuda")
    mla.mla_page_bounds(pool["kv"], b, table, i32([0]), i32([1]), page_size=page, kv_dtype="fp8")
    mla.mla_page_scores(query["q"], b, table[:, :1], i32([1]), one, page_size=page,
                        q_scale=query["q_scale"], kv_scale=pool["kv_scale"])
    assert abs(float(one) - float(exact[0])) <= 1e-5 * abs(float(exact[0]))


def test_page_scores_values_that_are_not_finite(mla):
    g = gen(10)
    b = torch.randn(9, 2, 576, generator=g, device="cuda").sort(1)[0].bfloat16()
    b[4, :, 77] = NAN
    query, qv = make_query("bf16", (2, 16, 576), g)
    query["q"][0, :, 77] = 0                   # a dim that the query does not use
    table = torch.arange(9, dtype=torch.int32, device="cuda").repeat(2, 1)
    s = torch.empty(2, 9, device="cuda")
    mla.mla_page_scores(query["q"], b, table, i32([9 * 8, 4 * 8]), s, page_size=8)
    assert s[0].isnan().tolist() == [False] * 4 + [True] + [False] * 4
    assert torch.isneginf(s[1, 4:]).all() and torch.isfinite(s[1, :4]).all()
    query["q"][1, 3, 0] = NAN
    mla.mla_page_scores(query["q"], b, table, i32([9 * 8, 4 * 8]), s, page_size=8)
    assert s[1, :4].isnan().all() and torch.isneginf(s[1, 4:]).all() and s[0, 0].isfinite()


def test_page_scores_report(mla):
    b = torch.randn(4, 2, 576, device="cuda").sort(1)[0].bfloat16()
    q = torch.randn(1, 16, 576, device="cuda").bfloat16()
    s, err = torch.empty(1, 2, device="cuda"), word()
    def run(table, lens):
        mla.mla_page_scores(q, b, i32(table), i32(lens), s, page_size=8, err=err)
        with pytest.raises(mla.MlaError) as e:
            mla.mla_error_check(err)
        return e.value.status
    assert run([[0, 4]], [16]) == 1 and run([[-1, 0]], [16]) == 1
    assert run([[0, 1]], [17]) == 6 and torch.isfinite(s).all()
    assert run([[0, 1]], [-1]) == 1 and torch.isneginf(s).all()
    # a bad page that no token reaches is not looked at
    mla.mla_page_scores(q, b, i32([[0, 99]]), i32([8]), s, page_size=8, err=err)
    mla.mla_error_check(err)


@pytest.mark.parametrize("lens,q_len,page,columns", [
    # the first query token's pages fit, the last one's do not
    ([6401], 4, 64, 100), ([16, 17, 3], 2, 8, 2), ([8 * 64 + 3], 64, 8, 64), ([9, 0], 2, 1, 8)])
def test_page_scores_report_pages_that_only_later_query_tokens_lack(mla, lens, q_len, page, columns):
    g = gen(32)
    b = torch.randn(4, 2, 576, generator=g, device="cuda").sort(1)[0].bfloat16()
    q = torch.randn(len(lens) * q_len, 16, 576, generator=g, device="cuda").bfloat16()
    table = torch.randint(0, 4, (len(lens), columns), generator=g, device="cuda").int()
    s, err = torch.empty(len(lens) * q_len, columns, device="cuda"), word()
    mla.mla_page_scores(q, b, table, i32(lens), s, page_size=page, q_len=q_len, err=err)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 6
    for r, x in enumerate(s):
        n = min(columns, -(-max(0, lens[r // q_len] - q_len + 1 + r % q_len) // page))
        assert torch.isfinite(x[:n]).all() and torch.isneginf(x[n:]).all()
    # one token less, and everything fits
    mla.mla_page_scores(q, b, table, i32([min(n, page * columns) for n in lens]), s, page_size=page,
                        q_len=q_len, err=err)
    mla.mla_error_check(err)


def test_page_scores_take_the_type_of_the_query(mla):
    """A bf16 query's scale is ignored, as by the decode call; e4m3 bytes need one."""
    g = gen(33)
    b = torch.randn(4, 2, 576, generator=g, device="cuda").sort(1)[0].bfloat16()
    q = torch.randn(1, 16, 576, generator=g, device="cuda").bfloat16()
    table, n = i32([[2, 1, 3]]), i32([20])
    s, t, scale = (torch.empty(1, 3, device="cuda"), torch.empty(1, 3, device="cuda"),
                   torch.full((1,), 0.25, device="cuda"))
    mla.mla_page_scores(q, b, table, n, s, page_size=8)
    mla.mla_page_scores(q, b, table, n, t, page_size=8, q_scale=scale)
    assert torch.equal(s, t)
    e = q.to(torch.float8_e4m3fn)
    mla.mla_page_scores(e.bfloat16(), b, table, n, s, page_size=8)
    mla.mla_page_scores(e.view(torch.uint8), b, table, n, t, page_size=8, q_scale=scale)
    assert torch.equal(0.25 * s, t)
    with pytest.raises(ValueError):
        mla.mla_page_scores(e.view(torch.uint8), b, table, n, t, page_size=8)


# --------------------------------------------------------------------- select
def plain_select(scores, table, lens, page, q_len, top, first, last):
    ptr, last_len, idx, cols = [0], [], [], []
    for r, row in enumerate(scores):
        seen = max(0, lens[r // q_len] - q_len + 1 + r % q_len)
        n = -(-seen // page)
        if n <= top:
            keep = list(range(n))
        else:
            def rank(j):
                return -INF if row[j] != row[j] else -row[j]
            mid = sorted(range(first, n - last), key=lambda j: (rank(j) if row[j] == row[j] else -INF, j))
            nan = [j for j in range(first, n - last) if row[j] != row[j]]
            mid = nan + [j for j in mid if row[j] == row[j]]
            keep = sorted(list(range(first)) + list(range(n - last, n)) + mid[: top - first - last])
        ptr.append(ptr[-1] + len(keep))
        last_len.append(seen - (n - 1) * page if n else 0)
        idx += [table[r // q_len][j] for j in keep]
        cols.append(keep + [-1] * (top - len(keep)))
    return ptr, last_len, idx, cols


def run_select(mla, scores, table, lens, page, q_len, top, first, last, cap=None, err=None, want=True):
    rows = len(scores)
    need = sum(min(top, -(-max(0, lens[r // q_len] - q_len + 1 + r % q_len) // page)) for r in range(rows))
    cap = need + 3 if cap is None else cap
    ptr, ll = torch.full((rows + 1,), 9, dtype=torch.int32, device="cuda"), torch.full((rows,), 9, dtype=torch.int32, device="cuda")
    idx = torch.full((cap,), -7, dtype=torch.int32, device="cuda")
    cols = torch.full((rows, top), 9, dtype=torch.int32, device="cuda") if want else None
    mla.mla_page_select(scores, table, i32(lens), page_size=page, q_len=q_len, top_pages=top,
                        first_pages=first, last_pages=last, kv_indptr=ptr, kv_last_page_len=ll,
                        kv_indices=idx, columns=cols, err=err)
    return ptr.tolist(), ll.tolist(), idx.tolist(), None if cols is None else cols.tolist(), need


SELECT_CASES = [
    ([0, 1, 64, 65, 1000], 8, 1, 8, 1, 1), ([5000] * 3, 8, 1, 100, 0, 1), ([5000], 8, 1, 100, 3, 7),
    ([4099], 1, 1, 4097, 1, 1), ([300_000], 16, 1, 2000, 1, 1), ([40_000, 7], 1, 1, 5, 4, 1),
    ([700, 3, 0, 64], 16, 4, 9, 2, 3), ([2048 + 13] * 70, 8, 1, 256, 1, 2),
    ([16 * 8 + 1], 8, 1, 16, 1, 1), ([640], 64, 1, 1, 0, 1), ([9 * 64] * 5, 64, 64, 4, 1, 1),
    # around the sizes where another way of selecting begins
    ([256, 255, 33, 32, 0], 1, 1, 31, 0, 1), ([257, 256, 40], 1, 1, 40, 1, 1),
    ([4096, 5], 1, 1, 700, 2, 2), ([4097, 9], 1, 2, 700, 2, 2), ([4100 + i for i in range(160)], 1, 1, 33, 1, 1),
    ([32768], 1, 1, 3000, 5, 5), ([32769, 100], 1, 1, 32768, 0, 1), ([70_001], 1, 1, 40_000, 1, 1),
    ([70_000, 33_000], 1, 1, 300, 1, 1), ([9000, 4, 4104], 1, 1, 4099, 1, 1), ([400_123, 50], 1, 1, 5000, 2, 1)]


@pytest.mark.parametrize("lens,page,q_len,top,first,last", SELECT_CASES)
@pytest.mark.parametrize("kind", ["random", "ties", "special", "equal"])
def test_page_select(mla, lens, page, q_len, top, first, last, kind):
    g = gen(12)
    rows, width = len(lens) * q_len, max(1, max(-(-n // page) for n in lens))
    x = torch.randn(rows, width + 5, generator=g, device="cuda")
    if kind == "ties":
        x = x.round()
    if kind == "equal":
        x = torch.full_like(x, -3.5)
    if kind == "special":
        pick = torch.randint(0, 12, x.shape, generator=g, device="cuda")
        for i, v in enumerate((NAN, INF, -INF, 0.0, -0.0, 1e-42, -1e-42)):
            x = torch.where(pick == i, v, x)
    table = torch.randint(0, 1 << 20, (len(lens), width + 2), generator=g, device="cuda").int()
    got = run_select(mla, x[:, 2:], table[:, :width], lens, page, q_len, top, first, last)
    ref = plain_select(x[:, 2:].tolist(), table.tolist(), lens, page, q_len, top, first, last)
    assert got[0] == ref[0] and got[1] == ref[1] and got[3] == ref[3]
    assert got[2] == ref[2] + [-7] * 3


def test_page_select_reports_and_leaves_what_is_not_its_own(mla):
    x = torch.randn(3, 40, generator=gen(13), device="cuda")
    table = torch.arange(120, dtype=torch.int32, device="cuda").reshape(3, 40)
    lens = [320, 50, 100]
    err = word()
    ref = plain_select(x.tolist(), table.tolist(), lens, 8, 1, 10, 1, 1)
    for cap in (0, 5, 10, 16, 26):            # 10 + 7 + 10 are needed
        ptr, ll, idx, cols, need = run_select(mla, x, table, lens, 8, 1, 10, 1, 1, cap=cap, err=err)
        assert need == 27 and (ptr, ll, cols) == (ref[0], ref[1], ref[3]) and idx == ref[2][:cap]
        with pytest.raises(mla.MlaError) as e:
            mla.mla_error_check(err)
        assert e.value.status == 6
    # columns are optional
    assert run_select(mla, x, table, lens, 8, 1, 10, 1, 1, want=False)[2] == ref[2] + [-7] * 3
    # negative lengths as 0; tokens beyond the table do not count
    ptr = run_select(mla, x, table, [-5, 50, 100], 8, 1, 10, 1, 1, err=err)[0]
    assert ptr == [0, 0, 7, 17]
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 1
    ptr, ll = run_select(mla, x, table, [321, 50, 100], 8, 1, 10, 1, 1, err=err)[:2]
    assert ptr == ref[0] and ll[0] == 8
    with pytest.raises(mla.MlaError) as e:
        mla.mla_error_check(err)
    assert e.value.status == 6


def test_pages_refuse_tensors_that_do_not_fit(mla):
    kv = torch.zeros(64, 576, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(8, 2, 576, dtype=torch.bfloat16, device="cuda")
    t, n = i32([[0, 1], [2, 3]]), i32([8, 16])
    for bad in (dict(kv=kv.float()), dict(kv=kv[:, :288]), dict(bounds=b[:, :1]), dict(bounds=b.float()),
                dict(table=t.long()), dict(table=t[:1]), dict(table=t.T), dict(old=n.long()),
                dict(new=i32([1])), dict(err=i32([0, 0]))):
        k = dict(dict(kv=kv, bounds=b, table=t, old=n, new=n, err=None), **bad)
        with pytest.raises(ValueError):
            mla.mla_page_bounds(k["kv"], k["bounds"], k["table"], k["old"], k["new"], page_size=8,
                                kv_dtype="bf16", err=k["err"])
    q, s = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, device="cuda")
    for bad in (dict(q=q[:1]), dict(q=q.float()), dict(q=q.view(torch.uint8)), dict(s=s[:1]),
                dict(s=s[:, :1]), dict(s=s.T), dict(s=s.double()), dict(bounds=kv), dict(lens=n.long())):
        k = dict(dict(q=q, bounds=b, table=t, lens=n, s=s), **bad)
        with pytest.raises(ValueError):
            mla.mla_page_scores(k["q"], k["bounds"], k["table"], k["lens"], k["s"], page_size=8)
    out = dict(kv_indptr=i32([0] * 3), kv_last_page_len=i32([0] * 2), kv_indices=i32([0] * 4))
    for bad in (dict(kv_indptr=i32([0] * 2)), dict(kv_last_page_len=i32([0] * 3)),
                dict(kv_indices=t), dict(columns=t[:1]), dict(kv_indices=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            mla.mla_page_select(s, t, n, page_size=8, top_pages=2, **dict(out, **bad))


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("kv,q_dtype", FORMATS[:3] + FORMATS[4:])
def test_selected_pages_step_by_step(mla, kv, q_dtype):
    """Prompts, then single tokens: cache step, cache write, bounds, scores,
    selection and the decode call over what was selected, replayed as a graph."""
    import numpy as np
    if (q_dtype, kv) not in FORMATS:
        kv, q_dtype = q_dtype, kv
    g = gen(14)
    bs, page, top, columns = 5, 16, 6, 40
    pages = bs * columns
    pool, _, _ = make_pool(kv, torch.zeros(pages * page, 576, device="cuda"))
    scale, e8 = pool.get("kv_scale"), pool.get("kv_e8m0")
    table = torch.full((bs, columns), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").int()
    bounds = torch.full((pages, 2, 576), NAN, dtype=torch.bfloat16, device="cuda")
    err = word()
    old = torch.zeros(bs, dtype=torch.int32, device="cuda")
    prompt = i32([3, 16, 100, 333, 61])
    dense = torch.zeros(bs, columns * page, 576, dtype=torch.float64, device="cuda")

    def write(old, new, tokens, free):
        n = int(tokens)
        out = dict(kv_indptr=torch.zeros(bs + 1, dtype=torch.int32, device="cuda"),
                   kv_last_page_len=torch.zeros(bs, dtype=torch.int32, device="cuda"),
                   kv_indices=torch.zeros(pages, dtype=torch.int32, device="cuda"),
                   qo_indptr=torch.zeros(bs + 1, dtype=torch.int32, device="cuda"),
                   slots=torch.zeros(n, dtype=torch.int64, device="cuda"),
                   positions=torch.zeros(n, dtype=torch.int32, device="cuda"), pages_used=word())
        mla.mla_cache_step(old, new, table, free, page_size=page, err=err, **out)
        latent = (0.5 * torch.randn(n, 512, generator=g, device="cuda")).bfloat16()
        rope = (0.5 * torch.randn(n, 64, generator=g, device="cuda")).bfloat16()
        rows = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
        mla.mla_cache_write(latent, rope, pool["kv"], out["slots"], kv_dtype=kv, kv_scale=scale,
                            kv_e8m0=e8, rows=rows, err=err)
        mla.mla_page_bounds(pool["kv"], bounds, table, old, new, page_size=page, kv_dtype=kv,
                            kv_e8m0=e8, err=err)
        mla.mla_error_check(err)
        return out, rows

    lens = np.zeros(bs, np.int64)
    new = prompt
    for step in range(4):
        out, rows = write(old, new, int(new.sum()), free)
        free = free[int(out["pages_used"]):].contiguous()
        at = out["qo_indptr"].tolist()
        for b in range(bs):
            dense[b, lens[b]: lens[b] + at[b + 1] - at[b]] = rows[at[b]: at[b + 1]].double()
            lens[b] += at[b + 1] - at[b]
        old = old + new
        new = torch.ones_like(prompt)
        # the plan knows the counts from the lengths alone
        n = -(-lens // page)
        kept = np.minimum(n, top)
        plan = mla.mla_decode_plan(np.concatenate([[0], kept.cumsum()]), lens - (n - 1) * page,
                                   page_size=page, q_dtype=q_dtype, kv_dtype=kv)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        query, qv = make_query(q_dtype, (bs, 16, 576), g)
        scores = torch.empty(bs, columns, device="cuda")
        sel = dict(kv_indptr=torch.zeros(bs + 1, dtype=torch.int32, device="cuda"),
                   kv_last_page_len=torch.zeros(bs, dtype=torch.int32, device="cuda"),
                   kv_indices=torch.zeros(bs * top, dtype=torch.int32, device="cuda"),
                   columns=torch.zeros(bs, top, dtype=torch.int32, device="cuda"))
        o = torch.empty(bs, 16, 512, dtype=torch.bfloat16, device="cuda")

        def attend():
            mla.mla_page_scores(query["q"], bounds, table, old, scores, page_size=page,
                                q_scale=query.get("q_scale"), kv_scale=scale, err=err)
            mla.mla_page_select(scores, table, old, page_size=page, top_pages=top, err=err, **sel)
            mla.mla_decode_run(plan, query["q"], pool["kv"], o, workspace=ws,
                               q_scale=query.get("q_scale"), kv_scale=scale, kv_e8m0=e8,
                               kv_indices=sel["kv_indices"])
        attend()
        eager = o.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attend()
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager)
        mla.mla_error_check(err)
        mla.mla_decode_check(plan, ws)
        assert sel["kv_indptr"].tolist() == [0] + kept.cumsum().tolist()
        assert sel["kv_last_page_len"].tolist() == (lens - (n - 1) * page).tolist()
        for b in range(bs):
            cols = [c for c in sel["columns"][b].tolist() if c >= 0]
            # the first, the last, and the best between them
            s = scores[b, : n[b]].tolist()
            if n[b] > top:
                best = sorted(range(1, n[b] - 1), key=lambda j: (-s[j], j))[: top - 2]
                assert cols == sorted([0, n[b] - 1] + best)
            else:
                assert cols == list(range(n[b]))
            tok = torch.tensor([c * page + i for c in cols for i in range(page) if c * page + i < lens[b]],
                               device="cuda")
            k = dense[b, tok]
            if kv == "fp8":                     # (the rows' bf16 is a rounding of e4m3 times the scale)
                ids = table[b, tok // page].long() * page + tok % page
                k = pool["kv"].view(torch.float8_e4m3fn)[ids].double() * scale.double()
            ref = torch.softmax(qv[b] @ k.T / 24, 1) @ k[:, :512]
            # the decode call's roundings: two of bf16 (p, out), and with a bf16
            # query against fp8 or MXFP4 rows the query's terms (2^-10 of its largest)
            assert (o[b].double() - ref).norm() <= 1e-2 * ref.norm()
