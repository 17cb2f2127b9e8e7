"""Measured cases of the operators around the MLA decode kernel.

The operators make an MLA attention layer of the decode call: the cache step
(pages handed out, page table and slots built from request lengths), the cache
write (norm, rotation, storage encoding, scatter), the absorbed form's two
products, and the expanded form (ragged causal attention with keys and values
expanded from the cached latent rows).

`run` computes a case in plain torch operations, or, with `own` true, through
the library's calls.  `exact` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
ROW = LATENT + ROPE
SM_SCALE = 1.0 / math.sqrt(NOPE + ROPE)
DECODE_SCALE = 1.0 / math.sqrt(ROW)          # the decode call's own softmax scale
EPS = 1e-6
FP8_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the headline batch: 256 requests near 8192 tokens, one new token each
        dict(name="step_decode_256", op="step", bs=256, page=8, old_lo=4000, old_hi=8191, new_lo=1,
             new_hi=1, shape=1),
        # admission of a batch of prompts of very different lengths
        dict(name="step_prompts_32", op="step", bs=32, page=64, old_lo=0, old_hi=700, new_lo=1,
             new_hi=8192, shape=2),
        # one token's row for each of 32 requests, every decode step of every layer
        dict(name="write_bf16_32", op="write", tokens=32, kv="bf16", page=8, rope="interleaved"),
        # the rows of a large prompt batch into an fp8 cache
        dict(name="write_fp8_16384", op="write", tokens=16384, kv="fp8", page=8, rope="interleaved"),
        # an odd-sized chunk into an MXFP4 cache, rotation in halves
        dict(name="write_mxfp4_5003", op="write", tokens=5003, kv="mxfp4", page=16, rope="half"),
        # the smallest batch's query, before the bf16 decode
        dict(name="absorb_q_4_bf16", op="absorb_q", tokens=4, heads=16, q="bf16", rope="interleaved"),
        # the headline batch's query, to fp8
        dict(name="absorb_q_256_fp8", op="absorb_q", tokens=256, heads=16, q="fp8", rope="interleaved"),
        # decode output of a middle batch, odd
        dict(name="absorb_out_61", op="absorb_out", tokens=61, heads=16),
        # four query tokens for each of 256 requests (multi-token decode)
        dict(name="absorb_out_1024", op="absorb_out", tokens=1024, heads=16),
        # one whole prompt
        dict(name="prefill_prompt_8192", op="prefill", bs=1, q_lo=8192, q_hi=8192, past_lo=0, past_hi=0,
             heads=16, kv="bf16", page=8, rope="interleaved", shape=3),
        # a ragged batch of prompts, some continuing a cached prefix
        dict(name="prefill_ragged_fp8", op="prefill", bs=9, q_lo=33, q_hi=1500, past_lo=0, past_hi=4000,
             heads=16, kv="fp8", page=16, rope="interleaved", shape=4),
        # a short turn after a long conversation: few rows, many keys
        dict(name="prefill_turn_mxfp4", op="prefill", bs=1, q_lo=77, q_hi=77, past_lo=32768,
             past_hi=32768, heads=16, kv="mxfp4", page=1, rope="half", shape=5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["step", "write", "absorb_q", "absorb_out", "prefill", "prefill"])
    rope = rng.choice(["interleaved", "half"])
    if op == "step":
        bs = _log_int(rng, 1, 300)
        if rng.random() < 0.5:
            old_hi = _log_int(rng, 1, 8191)
            return dict(op="step", bs=bs, page=rng.choice([1, 8, 16, 64]), old_lo=rng.randint(0, old_hi),
                        old_hi=old_hi, new_lo=1, new_hi=rng.choice([1, 4]), shape=rng.randint(0, 1 << 20))
        return dict(op="step", bs=min(bs, 32), page=rng.choice([1, 8, 16, 64]), old_lo=0,
                    old_hi=_log_int(rng, 1, 700), new_lo=0, new_hi=_log_int(rng, 1, 8192),
                    shape=rng.randint(0, 1 << 20))
    if op == "write":
        return dict(op="write", tokens=_log_int(rng, 1, 16384), kv=rng.choice(["bf16", "fp8", "mxfp4"]),
                    page=rng.choice([1, 8, 16, 64]), rope=rope)
    if op == "absorb_q":
        return dict(op="absorb_q", tokens=_log_int(rng, 1, 1024), heads=16, q=rng.choice(["bf16", "fp8"]),
                    rope=rope)
    if op == "absorb_out":
        return dict(op="absorb_out", tokens=_log_int(rng, 1, 1024), heads=16)
    bs = rng.randint(1, 9)
    q_hi = _log_int(rng, 1, 8192 // bs)
    past_hi = _log_int(rng, 1, 4096)
    if bs == 1 and q_hi <= 256:
        past_hi *= 8
    return dict(op="prefill", bs=bs, q_lo=max(1, q_hi // 8), q_hi=q_hi, past_lo=0,
                past_hi=past_hi if q_hi <= 2048 else 0, heads=rng.choice([4, 8, 16]),
                kv=rng.choice(["bf16", "fp8", "mxfp4"]), page=rng.choice([1, 8, 16, 64]), rope=rope,
                shape=rng.randint(0, 1 << 20))


def _lengths(case):
    """Request lengths of a case: they belong to the case, not to its inputs."""
    r = random.Random(case["shape"])
    n = case["bs"]
    if case["op"] == "step":
        return ([r.randint(case["old_lo"], case["old_hi"]) for _ in range(n)],
                [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)])
    return ([r.randint(case["past_lo"], case["past_hi"]) for _ in range(n)],
            [r.randint(case["q_lo"], case["q_hi"]) for _ in range(n)])


def _pages(n, page):
    return -(-n // page)


def _row_bytes(kv):
    return {"bf16": 2 * ROW, "fp8": ROW, "mxfp4": ROW // 2 + ROW // 32}[kv]


def work(case):
    op = case["op"]
    if op == "step":
        old, new = _lengths(case)
        pages = sum(_pages(a + b, case["page"]) for a, b in zip(old, new))
        need = pages - sum(_pages(a, case["page"]) for a in old)
        # lengths in; indptr, last page and table out; old table entries in, new ones from the free pages
        return {"bytes": 20 * case["bs"] + 8 * pages + 4 * need + 12 * sum(new), "flops": 0}
    if op == "write":
        t = case["tokens"]
        rows = 2 * ROW if case["kv"] == "mxfp4" else 0
        return {"bytes": t * (2 * ROW + _row_bytes(case["kv"]) + rows + 12 + 4 * ROPE) + 2 * LATENT,
                "flops": t * (5 * LATENT + 3 * ROPE)}
    if op == "absorb_q":
        t, h = case["tokens"], case["heads"]
        out = ROW * (1 if case["q"] == "fp8" else 2)
        return {"bytes": t * h * (2 * (NOPE + ROPE) + out) + t * (4 + 4 * ROPE) + h * NOPE * LATENT * 2,
                "flops": 2 * t * h * NOPE * LATENT}
    if op == "absorb_out":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * h * 2 * (LATENT + VDIM) + h * VDIM * LATENT * 2,
                "flops": 2 * t * h * VDIM * LATENT}
    past, q = _lengths(case)
    h = case["heads"]
    keys = sum(a + b for a, b in zip(past, q))
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(past, q))
    nq = sum(q)
    return {"bytes": keys * _row_bytes(case["kv"]) + 4 * sum(_pages(a + b, case["page"]) for a, b in zip(past, q))
            + nq * (h * 2 * (NOPE + ROPE + VDIM) + 4 + 4 * ROPE) + h * (NOPE + VDIM) * LATENT * 2,
            "flops": 2 * keys * h * (NOPE + VDIM) * LATENT + 2 * pairs * h * (NOPE + ROPE + VDIM)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rotation_table(n):
    pos = torch.arange(n, dtype=torch.float64, device="cuda")
    freq = 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device="cuda") / (ROPE // 2))
    a = pos[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _weights(g, heads):
    return (torch.randn(heads, NOPE + VDIM, LATENT, generator=g, device="cuda")
            / math.sqrt(LATENT)).bfloat16()


def _e2m1_codes(v):
    """Nearest e2m1 code (ties to the even code) of values already divided by their block's scale."""
    m = v.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int()
            + (m > 2.5).int() + (m >= 3.5).int() + (m > 5.0).int())
    return code | (torch.signbit(v).int() << 3)


def _mx_encode(y):
    """(codes [t,576], biased block exponents [t,18]) of values in y's own precision."""
    b = y.reshape(y.shape[0], ROW // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1].int() + 124, 0).clamp(0, 254)
    v = torch.ldexp(b, (127 - e)[..., None].to(b.dtype))
    return _e2m1_codes(v).reshape(y.shape), e


def _mx_values(codes, e):
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=codes.device)
    v = lut[codes.long()].reshape(codes.shape[0], ROW // 32, 32)
    return torch.ldexp(v, (e.int() - 127)[..., None].float()).reshape(codes.shape)


def _mx_pack(codes):
    c = codes.to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _mx_unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], ROW)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "step":
        old, new = _lengths(case)
        page, bs = case["page"], case["bs"]
        have = [_pages(a, page) for a in old]
        pages = [_pages(a + b, page) for a, b in zip(old, new)]
        pool = torch.randperm(sum(pages) + 17, generator=g, device="cuda").int()
        width = max(max(pages), 1) + 3
        table = torch.zeros(bs, width, dtype=torch.int32, device="cuda")
        have_t = torch.tensor(have, device="cuda")
        filled = torch.arange(width, device="cuda")[None] < have_t[:, None]
        table[filled] = pool[: sum(have)]
        i32 = dict(dtype=torch.int32, device="cuda")
        s.update(old=torch.tensor(old, **i32), new=torch.tensor(new, **i32), table=table,
                 free=pool[sum(have):].contiguous(),
                 kv_indptr=torch.empty(bs + 1, **i32), last=torch.empty(bs, **i32),
                 kv_indices=torch.empty(sum(pages), **i32), qo_indptr=torch.empty(bs + 1, **i32),
                 slots=torch.empty(sum(new), dtype=torch.int64, device="cuda"),
                 positions=torch.empty(sum(new), **i32), used=torch.empty(1, **i32),
                 err=torch.zeros(1, **i32))
        return s
    if op == "write":
        t, page = case["tokens"], case["page"]
        proj = torch.randn(t, ROW, generator=g, device="cuda").bfloat16()     # one projection's output
        rows = _pages(t, page) * page + page
        perm = torch.randperm(rows // page, generator=g, device="cuda")
        tok = torch.arange(t, device="cuda")
        s.update(latent=proj[:, :LATENT], k_rope=proj[:, LATENT:],
                 weight=(1 + 0.1 * torch.randn(LATENT, generator=g, device="cuda")).bfloat16(),
                 cos_sin=_rotation_table(32768),
                 positions=torch.randint(0, 32768, (t,), generator=g, device="cuda").int(),
                 slots=(perm[tok // page] * page + tok % page).long(),
                 err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if case["kv"] == "bf16":
            s["pool"] = torch.zeros(rows, ROW, dtype=torch.bfloat16, device="cuda")
        elif case["kv"] == "fp8":
            s["pool"] = torch.zeros(rows, ROW, dtype=torch.uint8, device="cuda")
            s["kv_scale"] = torch.full((1,), 6.0 / FP8_MAX, device="cuda")
        else:
            s["pool"] = torch.zeros(rows, ROW // 2, dtype=torch.uint8, device="cuda")
            s["e8m0"] = torch.zeros(rows, ROW // 32, dtype=torch.uint8, device="cuda")
            s["rows"] = torch.empty(t, ROW, dtype=torch.bfloat16, device="cuda")
        return s
    if op == "absorb_q":
        t, h = case["tokens"], case["heads"]
        s.update(q=torch.randn(t, h, NOPE + ROPE, generator=g, device="cuda").bfloat16(),
                 w=_weights(g, h), cos_sin=_rotation_table(32768),
                 positions=torch.randint(0, 32768, (t,), generator=g, device="cuda").int(),
                 err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if case["q"] == "fp8":
            s["q_scale"] = torch.full((1,), 6.0 / FP8_MAX, device="cuda")
            s["out"] = torch.empty(t, h, ROW, dtype=torch.uint8, device="cuda")
        else:
            s["out"] = torch.empty(t, h, ROW, dtype=torch.bfloat16, device="cuda")
        return s
    if op == "absorb_out":
        t, h = case["tokens"], case["heads"]
        # decode outputs are means of many latent rows
        s.update(o=(0.1 * torch.randn(t, h, LATENT, generator=g, device="cuda")).bfloat16(),
                 w=_weights(g, h), out=torch.empty(t, h, VDIM, dtype=torch.bfloat16, device="cuda"))
        return s
    past, q = _lengths(case)
    page, h = case["page"], case["heads"]
    n = [a + b for a, b in zip(past, q)]
    pages = [_pages(x, page) for x in n]
    kv_indptr, qo_indptr, positions = [0], [0], []
    for x, p, a, b in zip(n, pages, past, q):
        kv_indptr.append(kv_indptr[-1] + p)
        qo_indptr.append(qo_indptr[-1] + b)
        positions += range(a, a + b)
    total = sum(pages)
    rows = (total + 2) * page
    kv = torch.randn(rows, ROW, generator=g, device="cuda")
    s.update(q=torch.randn(sum(q), h, NOPE + ROPE, generator=g, device="cuda").bfloat16(),
             w=_weights(g, h), cos_sin=_rotation_table(max(n)),
             positions=torch.tensor(positions, dtype=torch.int32, device="cuda"),
             kv_indices=torch.randperm(total + 2, generator=g, device="cuda")[:total].int(),
             kv_indptr=kv_indptr, qo_indptr=qo_indptr,
             last=[x - (p - 1) * page for x, p in zip(n, pages)], lens=n,
             out=torch.empty(sum(q), h, VDIM, dtype=torch.bfloat16, device="cuda"))
    if case["kv"] == "bf16":
        s["pool"] = kv.bfloat16()
    elif case["kv"] == "fp8":
        s["kv_scale"] = torch.full((1,), 6.0 / FP8_MAX, device="cuda")
        s["pool"] = (kv / s["kv_scale"]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes, e = _mx_encode(kv)
        s["pool"], s["e8m0"] = _mx_pack(codes), e.to(torch.uint8)
    del kv
    if own:
        import mla_decode_stage1_gb300 as mla
        s["plan"] = mla.mla_prefill_plan(qo_indptr, kv_indptr, s["last"], page_size=page, heads=h,
                                         kv_dtype=case["kv"])
        s["workspace"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------- run
def _own(s):
    import mla_decode_stage1_gb300 as mla
    case = s["case"]
    op = case["op"]
    if op == "step":
        mla.mla_cache_step(s["old"], s["new"], s["table"], s["free"], page_size=case["page"],
                           kv_indptr=s["kv_indptr"], kv_last_page_len=s["last"],
                           kv_indices=s["kv_indices"], qo_indptr=s["qo_indptr"], slots=s["slots"],
                           positions=s["positions"], pages_used=s["used"], err=s["err"])
        return _step_outputs(s)
    if op == "write":
        mla.mla_cache_write(s["latent"], s["k_rope"], s["pool"], s["slots"], kv_dtype=case["kv"],
                            norm_weight=s["weight"], eps=EPS, positions=s["positions"],
                            cos_sin=s["cos_sin"], rope=case["rope"], kv_scale=s.get("kv_scale"),
                            kv_e8m0=s.get("e8m0"), rows=s.get("rows"), err=s["err"])
        return _write_outputs(s)
    if op == "absorb_q":
        mla.mla_absorb_q(s["q"], s["w"], s["out"], sm_scale=SM_SCALE, positions=s["positions"],
                         cos_sin=s["cos_sin"], rope=case["rope"], q_scale=s.get("q_scale"),
                         err=s["err"])
        return s["out"].view(torch.float8_e4m3fn) if case["q"] == "fp8" else s["out"]
    if op == "absorb_out":
        mla.mla_absorb_out(s["o"], s["w"], s["out"])
        return s["out"]
    mla.mla_prefill_run(s["plan"], s["q"], s["pool"], s["w"], s["out"], workspace=s["workspace"],
                        sm_scale=SM_SCALE, positions=s["positions"], cos_sin=s["cos_sin"],
                        rope=case["rope"], kv_scale=s.get("kv_scale"), kv_e8m0=s.get("e8m0"),
                        kv_indices=s["kv_indices"])
    return s["out"]


def _step_outputs(s):
    return {k: s[k] for k in ("table", "kv_indptr", "last", "kv_indices", "qo_indptr", "slots",
                              "positions", "used")}


def _write_outputs(s):
    # fp8 as the type itself; MXFP4 as the values that its codes stand for
    kv = s["case"]["kv"]
    return s["rows"] if kv == "mxfp4" else s["pool"].view(torch.float8_e4m3fn) if kv == "fp8" else s["pool"]


def _rotate(x, cos_sin, positions, rope):
    """x [t, ..., 64] rotated by its token's angles, in x's own precision."""
    cs = cos_sin[positions.long()].to(x.dtype)
    cs = cs.reshape(cs.shape[0], *([1] * (x.dim() - 2)), ROPE)
    c, n = cs[..., : ROPE // 2], cs[..., ROPE // 2:]
    if rope == "half":
        a, b = x[..., : ROPE // 2], x[..., ROPE // 2:]
        return torch.cat([a * c - b * n, b * c + a * n], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)


def _plain_step(s):
    old, new, table, page = s["old"].long(), s["new"].long(), s["table"], s["case"]["page"]
    have, pages = (old + page - 1) // page, (old + new + page - 1) // page
    need = pages - have
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device="cuda")[None]
    take = (col >= have[:, None]) & (col < pages[:, None])
    where = (first[:, None] + col - have[:, None]).clamp(0, len(s["free"]) - 1)
    table = torch.where(take, s["free"][where], table)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    b = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new)
    qo = torch.cat([zero, torch.cumsum(new, 0)])
    pos = torch.arange(len(b), device="cuda") - qo[b] + old[b]
    return dict(table=table, kv_indptr=torch.cat([zero, torch.cumsum(pages, 0)]).int(),
                last=(old + new - (pages - 1).clamp(min=0) * page).int(),
                kv_indices=table[col < pages[:, None]], qo_indptr=qo.int(),
                slots=table[b, pos // page].long() * page + pos % page, positions=pos.int(),
                used=need.sum().int().reshape(1))


def _plain_write(s):
    case = s["case"]
    x = s["latent"].float()
    # the mean in 64 bits: a value next to a rounding border of the storage
    # type must not depend on the order of a 32-bit sum
    ms = (x.double() * x.double()).mean(-1, keepdim=True).float()
    y = x * (1.0 / torch.sqrt(ms + EPS)) * s["weight"].float()
    y = torch.cat([y, _rotate(s["k_rope"].float(), s["cos_sin"], s["positions"], case["rope"])], 1)
    if case["kv"] == "bf16":
        s["pool"][s["slots"]] = y.bfloat16()
    elif case["kv"] == "fp8":
        q = (y / s["kv_scale"]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s["pool"][s["slots"]] = q.view(torch.uint8)
    else:
        codes, e = _mx_encode(y)
        s["pool"][s["slots"]] = _mx_pack(codes)
        s["e8m0"][s["slots"]] = e.to(torch.uint8)
        s["rows"] = _mx_values(codes, e).bfloat16()
    return _write_outputs(s)


def _plain_absorb_q(s):
    q = s["q"].float()
    lat = torch.bmm(q[..., :NOPE].transpose(0, 1), s["w"][:, :NOPE].float()).transpose(0, 1)
    rot = _rotate(q[..., NOPE:], s["cos_sin"], s["positions"], s["case"]["rope"])
    y = torch.cat([lat, rot], -1) * (SM_SCALE / DECODE_SCALE)
    if s["case"]["q"] == "fp8":
        return (y / s["q_scale"]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return y.bfloat16()


def _plain_absorb_out(s):
    y = torch.bmm(s["o"].float().transpose(0, 1), s["w"][:, NOPE:].float().transpose(1, 2))
    return y.transpose(0, 1).contiguous().bfloat16()


def _cached_rows(s, b, dtype):
    """The rows of request b as stored values, [n, 576]."""
    case, page = s["case"], s["case"]["page"]
    table = s["kv_indices"][s["kv_indptr"][b]: s["kv_indptr"][b + 1]].long()
    at = (table[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[: s["lens"][b]]
    if case["kv"] == "bf16":
        return s["pool"][at].to(dtype)
    if case["kv"] == "fp8":
        return s["pool"][at].view(torch.float8_e4m3fn).to(dtype) * s["kv_scale"].to(dtype)
    return _mx_values(_mx_unpack(s["pool"][at]), s["e8m0"][at]).to(dtype)


def _plain_prefill(s):
    case = s["case"]
    q = s["q"].float()
    q = torch.cat([q[..., :NOPE], _rotate(q[..., NOPE:], s["cos_sin"], s["positions"], case["rope"])], -1)
    w = s["w"].float()
    outs = []
    for b in range(case["bs"]):
        rows = _cached_rows(s, b, torch.float32)
        qb = q[s["qo_indptr"][b]: s["qo_indptr"][b + 1]]
        m, n = len(qb), len(rows)
        masked = torch.arange(n, device="cuda")[None] > torch.arange(n - m, n, device="cuda")[:, None]
        kv = torch.matmul(rows[:, :LATENT], w.transpose(1, 2))             # [heads, n, 256]
        k = torch.cat([kv[..., :NOPE], rows[:, LATENT:].expand(len(kv), -1, -1)], -1)
        sc = (qb.transpose(0, 1) @ k.transpose(1, 2)).mul_(SM_SCALE).masked_fill_(masked, -math.inf)
        p = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
        outs.append(((p @ kv[..., NOPE:]) / p.sum(-1, keepdim=True)).transpose(0, 1))
    return torch.cat(outs).bfloat16()


def run(state):
    if own:
        return _own(state)
    return {"step": _plain_step, "write": _plain_write, "absorb_q": _plain_absorb_q,
            "absorb_out": _plain_absorb_out, "prefill": _plain_prefill}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact
def _turn(x, table, positions, rope):
    """Rotation as a product of complex numbers, in 64 bits."""
    t = table[positions.long()].double()
    z = torch.complex(t[:, :32], t[:, 32:])
    while z.dim() < x.dim():
        z = z[:, None]
    if rope == "half":
        r = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * z
        return torch.cat([r.real, r.imag], -1)
    return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous()) * z).flatten(-2)


def exact(case, seed):
    op = case["op"]
    if op == "step":
        return None                                   # whole numbers: compared as they are
    s = prepare(case, seed)
    if op == "write":
        x = s["latent"].double()
        y = x / (x.square().sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
        y = torch.cat([y, _turn(s["k_rope"].double(), s["cos_sin"], s["positions"], case["rope"])], 1)
        if case["kv"] == "mxfp4":
            blk = y.view(-1, 18, 32)
            step = torch.exp2((blk.abs().amax(-1, keepdim=True).log2().floor() - 2).clamp(-127, 127))
            grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
            near = ((blk.abs() / step)[..., None] - grid).abs().argmin(-1)
            return (grid[near] * step * blk.sign()).reshape(y.shape)
        pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
        if case["kv"] == "fp8":
            y = (y / s["kv_scale"].double()).clamp(-FP8_MAX, FP8_MAX)
        pool[s["slots"]] = y
        return pool
    if op == "absorb_q":
        q, w = s["q"].double(), s["w"].double()
        lat = torch.einsum("thd,hdc->thc", q[..., :NOPE], w[:, :NOPE])
        y = torch.cat([lat, _turn(q[..., NOPE:], s["cos_sin"], s["positions"], case["rope"])], -1)
        y = y * math.sqrt(ROW / (NOPE + ROPE))
        return (y / s["q_scale"].double()).clamp(-FP8_MAX, FP8_MAX) if case["q"] == "fp8" else y
    if op == "absorb_out":
        return torch.einsum("thc,hvc->thv", s["o"].double(), s["w"][:, NOPE:].double())
    q, w = s["q"].double(), s["w"].double()
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    rot = _turn(q[..., NOPE:], s["cos_sin"], s["positions"], case["rope"])
    for b in range(case["bs"]):
        i0, i1, n = s["qo_indptr"][b], s["qo_indptr"][b + 1], s["lens"][b]
        rows = _cached_rows(s, b, torch.float64)
        for h in range(case["heads"]):
            k_lat = rows[:, :LATENT] @ w[h, :NOPE].T
            for r in range(i0, i1, 2048):
                e = min(r + 2048, i1)
                last = n - (i1 - e)                   # keys the last of these rows sees
                z = (q[r:e, h, :NOPE] @ k_lat[:last].T + rot[r:e, h] @ rows[:last, LATENT:].T) * SM_SCALE
                see = torch.ones(e - r, last, device="cuda", dtype=torch.bool).tril(last - (e - r))
                z = torch.where(see, z, -math.inf)
                out[r:e, h] = torch.softmax(z, 1) @ rows[:last, :LATENT] @ w[h, NOPE:].T
    return out
