#!/usr/bin/env python3
"""One MLA attention layer served with the library: prompts, then single tokens.

Each step hands out cache pages on the GPU (mla_cache_step), projects the new
tokens, writes their rows into the paged cache (mla_cache_write) and attends:
prompts in the expanded form (mla_prefill_run), single tokens in the absorbed
form (mla_absorb_q, mla_decode_run, mla_absorb_out).  At the end the layer's
outputs are compared with attention computed in 32 bits from the same tokens.

  python examples/attention_layer.py [--prompts 300,17,1200] [--tokens 5] [--kv fp8]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mla_decode_stage1_gb300 as mla  # noqa: E402

HIDDEN, HEADS, PAGE, SCALE = 1024, 16, 8, 1 / math.sqrt(192)


class Layer:
    """Random weights of one layer: hidden -> queries, latent and rotated key."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / math.sqrt(shape[-1])).bfloat16()

        self.q, self.kv = w(HEADS * 192, HIDDEN), w(576, HIDDEN)
        self.norm = torch.ones(512, dtype=torch.bfloat16, device="cuda")
        self.up = w(HEADS, 256, 512)              # key rows, then value rows, per head
        pos = torch.arange(8192, dtype=torch.float64, device="cuda")
        angle = pos[:, None] * 10000.0 ** (-torch.arange(32, device="cuda").double() / 32)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    def project(self, hidden):
        kv = hidden @ self.kv.T
        return (hidden @ self.q.T).view(-1, HEADS, 192), kv[:, :512], kv[:, 512:]


class Cache:
    """A paged latent cache: pool, block table, free pages."""

    def __init__(self, requests, capacity, kv):
        pages = requests * -(-capacity // PAGE)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.kv, rows = kv, pages * PAGE
        width = {"bf16": 576, "fp8": 576, "mxfp4": 288}[kv]
        self.pool = torch.zeros(rows, width, device="cuda",
                                dtype=torch.bfloat16 if kv == "bf16" else torch.uint8)
        self.scale = torch.full((1,), 6 / 448, device="cuda") if kv == "fp8" else None
        self.e8m0 = (torch.zeros(rows, 18, dtype=torch.uint8, device="cuda") if kv == "mxfp4"
                     else None)
        self.table = torch.zeros(requests, -(-capacity // PAGE), **i32)
        self.free = torch.randperm(pages, device="cuda").int()
        self.lens = [0] * requests                # the scheduler's own copy
        self.err = torch.zeros(1, **i32)

    def format(self):
        return dict(kv_scale=self.scale, kv_e8m0=self.e8m0)

    def step(self, new):
        """Pages, slots and positions for new[b] more tokens of request b."""
        bs, total = len(new), sum(new)
        i32 = dict(dtype=torch.int32, device="cuda")
        pages = [-(-(a + b) // PAGE) for a, b in zip(self.lens, new)]
        s = dict(kv_indptr=torch.empty(bs + 1, **i32), kv_last_page_len=torch.empty(bs, **i32),
                 kv_indices=torch.empty(sum(pages), **i32), qo_indptr=torch.empty(bs + 1, **i32),
                 slots=torch.empty(total, dtype=torch.int64, device="cuda"),
                 positions=torch.empty(total, **i32), pages_used=torch.empty(1, **i32))
        mla.mla_cache_step(torch.tensor(self.lens, **i32), torch.tensor(new, **i32), self.table,
                           self.free, page_size=PAGE, err=self.err, **s)
        used = sum(pages) - sum(-(-a // PAGE) for a in self.lens)
        self.free = self.free[used:]
        self.lens = [a + b for a, b in zip(self.lens, new)]
        indptr = [0]
        for p in pages:
            indptr.append(indptr[-1] + p)
        last = [n - (p - 1) * PAGE for n, p in zip(self.lens, pages)]
        return s, indptr, last                    # the plans read host arrays


def write(layer, cache, s, latent, k_rope):
    mla.mla_cache_write(latent, k_rope, cache.pool, s["slots"], kv_dtype=cache.kv,
                        norm_weight=layer.norm, positions=s["positions"], cos_sin=layer.cos_sin,
                        err=cache.err, **cache.format())


def prompts(layer, cache, hidden, lengths):
    """hidden [sum(lengths), HIDDEN] -> attention output [sum(lengths), HEADS, 128]."""
    s, indptr, last = cache.step(lengths)
    q, latent, k_rope = layer.project(hidden)
    write(layer, cache, s, latent, k_rope)
    qo = [0]
    for n in lengths:
        qo.append(qo[-1] + n)
    attend = mla.MlaPrefill(qo, indptr, last, page_size=PAGE, kv_dtype=cache.kv, heads=HEADS)
    out = torch.empty(qo[-1], HEADS, 128, dtype=torch.bfloat16, device="cuda")
    attend(q, cache.pool, layer.up, out, sm_scale=SCALE, positions=s["positions"],
           cos_sin=layer.cos_sin, kv_indices=s["kv_indices"], **cache.format())
    mla.mla_prefill_check(attend.plan, attend.workspace)
    return out


def tokens(layer, cache, hidden):
    """hidden [requests, HIDDEN], one token each -> [requests, HEADS, 128]."""
    bs = hidden.shape[0]
    s, indptr, last = cache.step([1] * bs)
    q, latent, k_rope = layer.project(hidden)
    write(layer, cache, s, latent, k_rope)
    decode = mla.MlaDecoder(torch.tensor(indptr), torch.tensor(last), page_size=PAGE,
                            q_dtype="bf16", kv_dtype=cache.kv)
    q_lat = torch.empty(bs, HEADS, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_q(q, layer.up, q_lat, sm_scale=SCALE, positions=s["positions"],
                     cos_sin=layer.cos_sin, err=cache.err)
    o = torch.empty(bs, HEADS, 512, dtype=torch.bfloat16, device="cuda")
    decode(q_lat, cache.pool, o, kv_indices=s["kv_indices"], **cache.format())
    mla.mla_decode_check(decode.plan, decode.workspace)
    out = torch.empty(bs, HEADS, 128, dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_out(o, layer.up, out, err=cache.err)
    return out


def plain(layer, hidden):
    """Causal attention of one sequence in 32 bits, from its hidden states."""
    q, latent, k_rope = (x.float() for x in layer.project(hidden))
    latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + 1e-6)
    cos, sin = layer.cos_sin[: len(q)].split(32, 1)

    def turn(x, c, s):
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)

    kv = torch.einsum("nc,hdc->hnd", latent, layer.up.float())
    k = torch.cat([kv[..., :128], turn(k_rope, cos, sin).expand(HEADS, -1, -1)], -1)
    q = torch.cat([q[..., :128], turn(q[..., 128:], cos[:, None], sin[:, None])], -1)
    s = torch.einsum("mhd,hnd->hmn", q, k) * SCALE
    hidden_keys = torch.ones(s.shape[1:], dtype=torch.bool, device="cuda").triu(1)
    return torch.einsum("hmn,hnd->mhd", s.masked_fill(hidden_keys, -math.inf).softmax(-1),
                        kv[..., 128:])


def main(lengths=(300, 17, 1200), new_tokens=5, kv="bf16", seed=0):
    """Serves the prompts and new_tokens single tokens; returns the relative
    error (2-norm) of the prompts' and of the single tokens' outputs."""
    lengths = list(lengths)
    layer, cache = Layer(seed), Cache(len(lengths), max(lengths) + new_tokens, kv)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    seqs = [torch.randn(n + new_tokens, HIDDEN, generator=g, device="cuda").bfloat16()
            for n in lengths]
    out = prompts(layer, cache, torch.cat([x[:n] for x, n in zip(seqs, lengths)]), lengths)
    single = [tokens(layer, cache, torch.stack([x[n + i] for x, n in zip(seqs, lengths)]))
              for i in range(new_tokens)]
    mla.mla_error_check(cache.err)
    ref = [plain(layer, x) for x in seqs]
    ref_out = torch.cat([r[:n] for r, n in zip(ref, lengths)])
    errors = [float((out.float() - ref_out).norm() / ref_out.norm())]
    if new_tokens:
        ref_one = torch.stack([torch.stack([r[n + i] for r, n in zip(ref, lengths)])
                               for i in range(new_tokens)])
        errors.append(float((torch.stack(single).float() - ref_one).norm() / ref_one.norm()))
    return errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", default="300,17,1200")
    ap.add_argument("--tokens", type=int, default=5)
    ap.add_argument("--kv", choices=["bf16", "fp8", "mxfp4"], default="bf16")
    a = ap.parse_args()
    e = main([int(x) for x in a.prompts.split(",")], a.tokens, a.kv)
    print(f"{a.kv} cache: relative error of the prompts' outputs {e[0]:.2e}"
          + (f", of the single tokens' {e[1]:.2e}" if len(e) > 1 else ""))
