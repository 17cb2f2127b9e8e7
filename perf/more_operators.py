"""Measured cases of the operators that read less of a long latent cache.

Shared prefixes: decode attention for groups of requests whose first pages are
the same, with the prefix's keys read and multiplied once for all of a group.
Selected pages: the smallest and largest value of every dim of a page's rows
(bounds), a score of each page for each query from them, and the pages with the
best scores as the page table of a decode call.

`run` computes a case in plain torch operations, or, with `own` true, through
the library's calls.  `exact` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

HEADS, LATENT, ROW = 16, 512, 576
SCALE = 1.0 / math.sqrt(ROW)
FP8_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # four users of a short system prompt, a few words into their own: latency
        dict(name="shared_4x1024", op="shared", groups=1, per_lo=4, per_hi=4, prefix_lo=1024, prefix_hi=1024,
             own_lo=64, own_hi=64, q_len=1, page=64, q="bf16", kv="bf16", shape=1),
        # 64 users of one long document
        dict(name="shared_64x32768", op="shared", groups=1, per_lo=64, per_hi=64, prefix_lo=32768, prefix_hi=32768,
             own_lo=1, own_hi=512, q_len=1, page=64, q="bf16", kv="bf16", shape=2),
        # the headline batch with its 8192 tokens in common, own ends of any length
        dict(name="shared_fp8_256x8192", op="shared", groups=1, per_lo=256, per_hi=256, prefix_lo=8192, prefix_hi=8192,
             own_lo=0, own_hi=400, q_len=1, page=8, q="fp8", kv="fp8", shape=3),
        # prompts of three applications served together, odd sizes
        dict(name="shared_groups_mxfp4", op="shared", groups=3, per_lo=5, per_hi=19, prefix_lo=1500, prefix_hi=6000,
             own_lo=1, own_hi=700, q_len=1, page=16, q="bf16", kv="mxfp4", shape=4),
        # four query tokens for each of 13 requests (multi-token decode) against a long prefix
        dict(name="shared_q4_13x16384", op="shared", groups=1, per_lo=13, per_hi=13, prefix_lo=16384, prefix_hi=16384,
             own_lo=4, own_hi=300, q_len=4, page=16, q="bf16", kv="fp8", shape=5),
        # one decode step of the headline batch: a row more on each request's last page
        dict(name="bounds_step_256", op="bounds", bs=256, old_lo=4000, old_hi=8191, new_lo=1, new_hi=1, page=64,
             kv="fp8", shape=6),
        # prompts of different lengths after their rows were written
        dict(name="bounds_prompts_9", op="bounds", bs=9, old_lo=0, old_hi=100, new_lo=300, new_hi=8192, page=32,
             kv="bf16", shape=7),
        # the headline batch's pages
        dict(name="scores_256x8192", op="scores", bs=256, len_lo=8192, len_hi=8192, q_len=1, page=64, q="fp8", shape=8),
        # two query tokens of three requests of very different, long lengths
        dict(name="scores_q2_3x131072", op="scores", bs=3, len_lo=9000, len_hi=131072, q_len=2, page=32, q="bf16",
             shape=9),
        # a quarter of the headline batch's pages
        dict(name="select_256x128", op="select", bs=256, len_lo=8192, len_hi=8192, q_len=1, page=64, top=32, first=1,
             last=2, shape=10),
        # one request of a million tokens, an eighth of its pages
        dict(name="select_1x16384", op="select", bs=1, len_lo=1048576, len_hi=1048576, q_len=1, page=64, top=2048, first=4,
             last=16, shape=11),
        # a ragged batch with two query tokens each, some of it shorter than what is kept
        dict(name="select_q2_37", op="select", bs=37, len_lo=3, len_hi=65536, q_len=2, page=32, top=77, first=1,
             last=4, shape=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "bounds", "scores", "select"])
    shape = rng.randint(0, 1 << 20)
    if op == "shared":
        groups, q_len = rng.randint(1, 4), rng.choice([1, 1, 1, 2, 3, 4])
        per = _log_int(rng, 1, 256 // groups // q_len)
        prefix = _log_int(rng, 16, min(32768, (1 << 20) // (groups * per * q_len)))
        own_hi = _log_int(rng, max(1, q_len - 1), 700)
        q, kv = rng.choice([("bf16", "bf16"), ("bf16", "fp8"), ("fp8", "fp8"), ("bf16", "mxfp4"), ("fp8", "bf16")])
        return dict(op=op, groups=groups, per_lo=max(1, per // 2), per_hi=per, prefix_lo=max(1, prefix // 2),
                    prefix_hi=prefix, own_lo=q_len - 1, own_hi=own_hi, q_len=q_len, page=rng.choice([1, 8, 16, 64]),
                    q=q, kv=kv, shape=shape)
    if op == "bounds":
        kv, page = rng.choice(["bf16", "fp8", "mxfp4"]), rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            old_hi = _log_int(rng, 1, 8191)
            return dict(op=op, bs=_log_int(rng, 1, 300), old_lo=rng.randint(0, old_hi), old_hi=old_hi, new_lo=1,
                        new_hi=rng.choice([1, 4]), page=page, kv=kv, shape=shape)
        return dict(op=op, bs=rng.randint(1, 9), old_lo=0, old_hi=_log_int(rng, 1, 700), new_lo=0,
                    new_hi=_log_int(rng, 1, 8192), page=page, kv=kv, shape=shape)
    page = rng.choice([16, 32, 64, 128])
    bs, q_len = _log_int(rng, 1, 256), rng.choice([1, 1, 2, 4])
    len_hi = _log_int(rng, page, 32768 * page // bs if op == "scores" else 16384 * page)
    case = dict(op=op, bs=bs, len_lo=rng.randint(1, len_hi), len_hi=len_hi, q_len=q_len, page=page, shape=shape)
    if op == "scores":
        return dict(case, q=rng.choice(["bf16", "fp8"]))
    top = _log_int(rng, 8, 2048)
    return dict(case, bs=min(bs, max(1, (1 << 17) * page // (len_hi * q_len))), top=top, first=rng.randint(0, 4),
                last=rng.randint(1, 4))


def _pages(n, page):
    return -(-n // page)


def _lengths(case):
    """Lengths of a case, as lists: they belong to the case, not to its inputs."""
    r = random.Random(case["shape"])
    if case["op"] == "shared":
        per = [r.randint(case["per_lo"], case["per_hi"]) for _ in range(case["groups"])]
        prefix = [_pages(r.randint(case["prefix_lo"], case["prefix_hi"]), case["page"]) for _ in per]   # pages
        return per, prefix, [r.randint(case["own_lo"], case["own_hi"]) for _ in range(sum(per))]
    if case["op"] == "bounds":
        return ([r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["bs"])],
                [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["bs"])])
    return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["bs"])]


def _row_lengths(case):
    """Tokens that each query row sees."""
    t = case["q_len"]
    return [max(0, n - t + 1 + i) for n in _lengths(case) for i in range(t)]


def _row_bytes(kv):
    return {"bf16": 2 * ROW, "fp8": ROW, "mxfp4": ROW // 2 + ROW // 32}[kv]


def work(case):
    op, page = case["op"], case["page"]
    if op == "shared":
        per, prefix, ends = _lengths(case)
        t = case["q_len"]
        rows = HEADS * t * len(ends)
        keys = page * sum(prefix) + sum(ends)
        pairs = HEADS * t * page * sum(a * b for a, b in zip(per, prefix))
        pairs += HEADS * sum(max(0, n - t + 1 + i) for n in ends for i in range(t))
        pages = sum(prefix) + sum(_pages(n, page) for n in ends)
        return {"bytes": keys * _row_bytes(case["kv"]) + 4 * pages
                + rows * (ROW * (1 if case["q"] == "fp8" else 2) + 2 * LATENT + 4),
                "flops": 2 * pairs * (ROW + LATENT)}
    if op == "bounds":
        old, new = _lengths(case)
        full = sum(_pages(a + b, page) - a // page for a, b in zip(old, new) if b)
        begun = sum(a % page > 0 for a, b in zip(old, new) if b)
        return {"bytes": sum(new) * _row_bytes(case["kv"]) + (full + begun) * 4 * ROW + 4 * full + 8 * len(old),
                "flops": 2 * ROW * sum(new)}
    seen = [_pages(n, page) for n in _row_lengths(case)]
    whole = [_pages(n, page) for n in _lengths(case)]
    if op == "scores":
        return {"bytes": sum(whole) * (4 * ROW + 4) + 4 * len(whole) + len(seen) * 4 * max(whole)
                + len(seen) * HEADS * ROW * (1 if case["q"] == "fp8" else 2),
                "flops": 2 * HEADS * 2 * ROW * sum(seen)}
    kept = sum(min(n, case["top"]) for n in seen)
    # scores of every page; of the pages kept their table entry in, column and page out
    return {"bytes": 4 * sum(seen) + 12 * kept + 12 * len(seen), "flops": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _e2m1_codes(v):
    m = v.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int()
            + (m > 2.5).int() + (m >= 3.5).int() + (m > 5.0).int())
    return code | (torch.signbit(v).int() << 3)


def _pool(s, kv, rows, g):
    """A pool of random rows."""
    x = torch.randn(rows, ROW, generator=g, device="cuda")
    if kv == "bf16":
        s["pool"] = x.bfloat16()
    elif kv == "fp8":
        s["kv_scale"] = torch.full((1,), 6.0 / FP8_MAX, device="cuda")
        s["pool"] = (x / s["kv_scale"]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        b = x.reshape(rows, ROW // 32, 32)
        e = (torch.frexp(b.abs().amax(-1))[1].int() + 124).clamp(0, 254)
        c = _e2m1_codes(torch.ldexp(b, (127 - e)[..., None].float())).reshape(rows, ROW).to(torch.uint8)
        s["pool"], s["e8m0"] = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), e.to(torch.uint8)


def _queries(s, kind, shape, g):
    x = 1.5 * torch.randn(*shape, generator=g, device="cuda")
    if kind == "fp8":
        s["q_scale"] = torch.full((1,), 8.0 / FP8_MAX, device="cuda")
        s["q"] = (x / s["q_scale"]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["q"] = x.bfloat16()


def _prefix_sum(x):
    out = [0]
    for n in x:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = _gen(seed)
    op, page = case["op"], case["page"]
    s = dict(case=case)
    if op == "shared":
        per, prefix, ends = _lengths(case)
        t, bs = case["q_len"], len(ends)
        ends_pages = [_pages(n, page) for n in ends]
        s.update(group_indptr=_prefix_sum(per), prefix_indptr=_prefix_sum(prefix), kv_indptr=_prefix_sum(ends_pages),
                 last=[n - (p - 1) * page if p else 0 for n, p in zip(ends, ends_pages)])
        total = sum(prefix) + sum(ends_pages)
        ids = torch.randperm(total + 2, generator=g, device="cuda").int()
        s.update(prefix_indices=ids[: sum(prefix)].contiguous(), kv_indices=ids[sum(prefix): total].contiguous(),
                 group_at=_i32(s["group_indptr"]), prefix_at=_i32(s["prefix_indptr"]), kv_at=_i32(s["kv_indptr"]),
                 ends=_i32(ends), shape=(max(per), page * max(prefix), max(ends)))
        _pool(s, case["kv"], (total + 2) * page, g)
        _queries(s, case["q"], (bs * t, HEADS, ROW), g)
        s["out"] = torch.empty(bs * t, HEADS, LATENT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(bs * t, HEADS, dtype=torch.float32, device="cuda")
        if own:
            import mla_decode_stage1_gb300 as mla
            s["plan"] = mla.mla_shared_plan(s["group_indptr"], s["prefix_indptr"], s["kv_indptr"], s["last"],
                                            page_size=page, q_len=t, q_dtype=case["q"], kv_dtype=case["kv"])
            s["workspace"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
        return s
    if op == "bounds":
        old, new = _lengths(case)
        pages = [_pages(a + b, page) for a, b in zip(old, new)]
        width = max(max(pages), 1)
        total = sum(pages)
        ids = torch.randperm(total + 2, generator=g, device="cuda").int()
        table = torch.zeros(case["bs"], width, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda")[None] < _i32(pages)[:, None]] = ids[:total]
        _pool(s, case["kv"], (total + 2) * page, g)
        # bounds of what was cached before: those of any earlier rows
        b = torch.randn(total + 2, 2, ROW, generator=g, device="cuda").abs() * 2
        b[:, 0] *= -1
        s.update(table=table, old=_i32(old), new=_i32(new), bounds=b.bfloat16(), most=max(max(new), 1),
                 err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return s
    lens, t = _lengths(case), case["q_len"]
    pages = [_pages(n, page) for n in lens]
    width = max(pages)
    s.update(lens=_i32(lens), err=torch.zeros(1, dtype=torch.int32, device="cuda"),
             table=torch.randint(0, sum(pages) + 2, (case["bs"], width), generator=g, device="cuda").int())
    if op == "scores":
        # a page's values lie around its own mean
        mean = 0.5 * torch.randn(sum(pages) + 2, 1, ROW, generator=g, device="cuda")
        half = 2.5 * torch.rand(sum(pages) + 2, 2, ROW, generator=g, device="cuda")
        half[:, 0] *= -1
        s["bounds"] = (mean + half).bfloat16()
        _queries(s, case["q"], (case["bs"] * t, HEADS, ROW), g)
        s["kv_scale"] = torch.full((1,), 0.75, device="cuda")
        s["scores"] = torch.empty(case["bs"] * t, width, dtype=torch.float32, device="cuda")
        return s
    x = 4 + torch.randn(case["bs"] * t, width, generator=g, device="cuda")
    # pages with equal bounds have equal scores
    s["scores"] = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.1, x.bfloat16().float(), x)
    kept = [min(_pages(n, page), case["top"]) for n in _row_lengths(case)]
    s.update(kv_indptr=_i32([0] * (len(kept) + 1)), last=_i32([0] * len(kept)),
             kv_indices=_i32([0] * sum(kept)), columns=_i32([0] * (len(kept) * case["top"])).view(len(kept), -1))
    return s


# --------------------------------------------------------------------- run
def _own(s):
    import mla_decode_stage1_gb300 as mla
    case = s["case"]
    op = case["op"]
    if op == "shared":
        mla.mla_shared_run(s["plan"], s["q"], s["pool"], s["out"], workspace=s["workspace"],
                           prefix_indices=s["prefix_indices"], kv_indices=s["kv_indices"], q_scale=s.get("q_scale"),
                           kv_scale=s.get("kv_scale"), kv_e8m0=s.get("e8m0"), lse=s["lse"])
        return s["out"], s["lse"]
    if op == "bounds":
        mla.mla_page_bounds(s["pool"], s["bounds"], s["table"], s["old"], s["new"], page_size=case["page"],
                            kv_dtype=case["kv"], kv_e8m0=s.get("e8m0"), err=s["err"])
        return s["bounds"]
    if op == "scores":
        mla.mla_page_scores(s["q"], s["bounds"], s["table"], s["lens"], s["scores"], page_size=case["page"],
                            q_len=case["q_len"], q_scale=s.get("q_scale"), kv_scale=s["kv_scale"], err=s["err"])
        return s["scores"]
    mla.mla_page_select(s["scores"], s["table"], s["lens"], page_size=case["page"], q_len=case["q_len"],
                        top_pages=case["top"], first_pages=case["first"], last_pages=case["last"],
                        kv_indptr=s["kv_indptr"], kv_last_page_len=s["last"], kv_indices=s["kv_indices"],
                        columns=s["columns"], err=s["err"])
    return s["kv_indptr"], s["last"], s["kv_indices"], s["columns"]


def _stored_rows(s, at, dtype):
    """Values of pool rows `at`, without the pool's scale."""
    kv = s["case"]["kv"]
    if kv == "bf16":
        return s["pool"][at].to(dtype)
    if kv == "fp8":
        return s["pool"].view(torch.float8_e4m3fn)[at].to(dtype)
    c, e = s["pool"][at], s["e8m0"][at]
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device="cuda")
    v = lut[torch.stack([c & 15, c >> 4], -1).long()].reshape(*c.shape[:-1], ROW // 32, 32)
    return torch.ldexp(v, (e.int() - 127)[..., None].to(dtype)).reshape(*c.shape[:-1], ROW)


def _query_values(s, dtype):
    if "q_scale" in s:
        return s["q"].view(torch.float8_e4m3fn).to(dtype) * s["q_scale"].to(dtype)
    return s["q"].to(dtype)


def _padded_rows(s, indices, at, lens, width, dtype):
    """Rows of the requests (or groups) of a page list, [n, width, 576], and which of them count."""
    page = s["case"]["page"]
    tok = torch.arange(width, device="cuda")
    there = tok < lens[:, None]
    # (a token that does not count reads the list's first page)
    entry = torch.where(there, at[:-1, None].long() + tok // page, 0)
    if indices.numel() == 0:
        return torch.zeros(len(lens), width, ROW, dtype=dtype, device="cuda"), there
    rows = _stored_rows(s, indices.long()[entry] * page + tok % page, dtype)
    scale = s["kv_scale"].to(dtype) if "kv_scale" in s else 1.0
    return torch.where(there[..., None], rows * scale, 0.0), there


def _plain_shared(s):
    case = s["case"]
    t, page = case["q_len"], case["page"]
    per, plen, elen = s["shape"]
    q = _query_values(s, torch.float32).reshape(-1, t * HEADS, ROW) * SCALE
    bs = len(q)
    counts = s["group_at"].diff()
    group = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), counts.long(), output_size=bs)
    place = torch.arange(bs, device="cuda") - s["group_at"][group]
    # every group's queries against its prefix
    qg = torch.zeros(len(counts), per, t * HEADS, ROW, device="cuda")
    qg[group, place] = q
    k, there = _padded_rows(s, s["prefix_indices"], s["prefix_at"], s["prefix_at"].diff() * page, plen, torch.float32)
    sc = (qg.flatten(1, 2) @ k.transpose(1, 2)).masked_fill_(~there[:, None], -math.inf)
    # every request's queries against its own end
    ke, there = _padded_rows(s, s["kv_indices"], s["kv_at"], s["ends"], elen, torch.float32)
    tok = torch.arange(elen, device="cuda")
    seen = s["ends"][:, None] - t + 1 + torch.arange(t, device="cuda")
    see = (tok < seen[..., None]).repeat_interleave(HEADS, 1)
    se = (q @ ke.transpose(1, 2)).masked_fill_(~see, -math.inf)
    # one softmax over both
    mg = sc.amax(-1).unflatten(1, (per, t * HEADS))[group, place]
    m = torch.maximum(mg, torch.cat([se, mg[..., None]], -1).amax(-1))
    mp = torch.zeros(len(counts), per, t * HEADS, device="cuda")
    mp[group, place] = m
    p = sc.sub_(mp.flatten(1, 2)[..., None]).exp_()
    pe = se.sub_(m[..., None]).exp_()
    o = (p @ k[..., :LATENT]).unflatten(1, (per, t * HEADS))[group, place] + pe @ ke[..., :LATENT]
    l = p.sum(-1).unflatten(1, (per, t * HEADS))[group, place] + pe.sum(-1)
    return ((o / l[..., None]).bfloat16().reshape(bs * t, HEADS, LATENT),
            (m + l.log()).reshape(bs * t, HEADS))


def _plain_bounds(s):
    page = s["case"]["page"]
    old, new = s["old"].long(), s["new"].long()
    n = int(s["most"])
    tok = torch.arange(n, device="cuda")
    there = tok < new[:, None]
    pos = old[:, None] + tok
    ids = torch.gather(s["table"].long(), 1, torch.where(there, pos // page, 0))
    rows = _stored_rows(s, (ids * page + pos % page)[there], torch.float32)
    # pages whose first row is new begin anew, others go on from their bounds
    b = s["bounds"].float()
    fresh = ids[there & (pos % page == 0)]
    b[fresh, 0], b[fresh, 1] = math.inf, -math.inf
    at = ids[there][:, None].expand(-1, ROW)
    lo = b[:, 0].scatter_reduce(0, at, rows, "amin")
    hi = b[:, 1].scatter_reduce(0, at, rows, "amax")
    s["bounds"].copy_(torch.stack([lo, hi], 1))
    return s["bounds"]


def _seen_tokens(s):
    t = s["case"]["q_len"]
    return (s["lens"][:, None] - t + 1 + torch.arange(t, device="cuda")).clamp(min=0).flatten()


def _plain_scores(s):
    case = s["case"]
    q = _query_values(s, torch.float32).unflatten(0, (-1, case["q_len"]))
    b = s["bounds"][s["table"].long()].float() * s["kv_scale"]
    x = (torch.einsum("bthd,bpd->btph", q.clamp(min=0), b[:, :, 1])
         + torch.einsum("bthd,bpd->btph", q.clamp(max=0), b[:, :, 0]))
    x = x.amax(-1).flatten(0, 1) * SCALE
    pages = (_seen_tokens(s) + case["page"] - 1) // case["page"]
    return x.masked_fill_(torch.arange(x.shape[1], device="cuda") >= pages[:, None], -math.inf)


def _plain_select(s):
    case = s["case"]
    page, top = case["page"], case["top"]
    x = s["scores"]
    seen = _seen_tokens(s).long()
    n = ((seen + page - 1) // page)[:, None]
    col = torch.arange(x.shape[1], device="cuda")
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits)
    key = torch.where(x.isnan(), 1 << 40, key)
    key = torch.where((col < case["first"]) | (col >= n - case["last"]), 1 << 41, key)
    key = torch.where(col < n, key, -(1 << 41))
    order = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :top]
    kept = torch.zeros(x.shape, dtype=torch.bool, device="cuda").scatter_(1, order, True) & (col < n)
    count = n[:, 0].clamp(max=top)
    rank = kept.long().cumsum(1) - 1
    columns = torch.full((len(x), top + 1), -1, device="cuda")
    columns.scatter_(1, torch.where(kept, rank, top), torch.where(kept, col, -1))
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    table = s["table"].repeat_interleave(case["q_len"], 0)
    return (torch.cat([zero, count.cumsum(0)]).int(), (seen - (n[:, 0] - 1).clamp(min=0) * page).int(), table[kept],
            columns[:, :top].int())


def run(state):
    if own:
        return _own(state)
    return {"shared": _plain_shared, "bounds": _plain_bounds, "scores": _plain_scores,
            "select": _plain_select}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact
def exact(case, seed):
    op, page = case["op"], case["page"]
    if op == "select":
        return None                                   # whole numbers: compared as they are
    s = prepare(case, seed)
    if op == "bounds":
        out = s["bounds"].double()
        old, new = _lengths(case)
        table = s["table"].tolist()
        for row, a, n in zip(table, old, new):
            for j in range(a // page, _pages(a + n, page) if n else 0):
                first, end = max(a, j * page), min(a + n, (j + 1) * page)
                x = _stored_rows(s, row[j] * page + torch.arange(first - j * page, end - j * page, device="cuda"),
                                 torch.float64)
                if first > j * page:
                    x = torch.cat([x, out[row[j]]])
                out[row[j]] = torch.stack([x.min(0)[0], x.max(0)[0]])
        return out
    q = _query_values(s, torch.float64)
    if op == "scores":
        out = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for r, n in enumerate(_row_lengths(case)):
            p = _pages(n, page)
            lo, hi = s["bounds"][s["table"][r // case["q_len"], :p].long()].double().unbind(1)
            for i in range(0, p, 512):
                best = torch.maximum(q[r][:, None] * lo[i: i + 512], q[r][:, None] * hi[i: i + 512]).sum(-1)
                out[r, i: i + len(best[0])] = best.max(0)[0] * s["kv_scale"].double() * SCALE
        return out
    per, prefix, ends = _lengths(case)
    t = case["q_len"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    scale = s["kv_scale"].double() if "kv_scale" in s else 1.0
    tok = torch.arange(page, device="cuda")

    def rows(ids):
        return _stored_rows(s, (ids.long()[:, None] * page + tok).reshape(-1), torch.float64) * scale

    for g in range(len(per)):
        kp = rows(s["prefix_indices"][s["prefix_indptr"][g]: s["prefix_indptr"][g + 1]])
        for b in range(s["group_indptr"][g], s["group_indptr"][g + 1]):
            ke = rows(s["kv_indices"][s["kv_indptr"][b]: s["kv_indptr"][b + 1]])[: ends[b]]
            for i in range(t):
                k = torch.cat([kp, ke[: max(0, ends[b] - t + 1 + i)]])
                z = q[b * t + i] @ k.T * SCALE
                lse[b * t + i] = torch.logsumexp(z, 1)
                out[b * t + i] = torch.softmax(z, 1) @ k[:, :LATENT]
    return out, lse
