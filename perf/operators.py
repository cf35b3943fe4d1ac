"""Serving over a paged KV cache held in 8 bits: what is timed, and against what.

Three operators, in the order in which a serving step runs them:

  plan    block tables, used lengths, token offsets and slot maps from the requests' lengths
  write   new K and V rows rounded to 8 bits into the pages, one scale per page and head
  attend  attention of the new query tokens over the pages (every row, a window, selected
          blocks, or selected rows of a shared latent row)

`run` with `own` false computes them with elementary torch operations, with `own` true
through the package's entry points.  Shapes follow the repository's own workloads: heads
and head sizes of gen/configs.py (64 / 4 heads at 192 / 128 with 16 blocks of 64, 64 / 8 at
128, 128 heads over a shared row of 576 / 512 with 2048 rows selected, 4 / 1 at 64), lengths
up to those of its decode and long-sequence cases.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
# the largest code, as frexp sees it: mantissa in [0.5, 1) and exponent
TOP = {"e4m3": (0.875, 9, 448.0), "int8": (127 / 128, 7, 127.0)}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attend(name, B, n_new, lo, hi, Hq, Hkv, dqk, dv, **kw):
    c = dict(name=name, op="attend", B=B, n_new=n_new, len_lo=lo, len_hi=hi, Hq=Hq, Hkv=Hkv, d_qk=dqk, d_v=dv,
             shared=False, page=64, fmt="e4m3", dtype="bf16", block=0, topk=0, window=-1, sinks=False)
    c.update(kw)
    return c


def _write(name, B, n_lo, n_hi, old_hi, Hkv, dqk, dv, **kw):
    c = dict(name=name, op="write", B=B, n_lo=n_lo, n_hi=n_hi, old_hi=old_hi, Hkv=Hkv, d_qk=dqk, d_v=dv,
             shared=False, page=64, fmt="e4m3", dtype="bf16")
    c.update(kw)
    return c


def _plan(name, B, n_lo, n_hi, old_hi, page):
    return dict(name=name, op="plan", B=B, n_lo=n_lo, n_hi=n_hi, old_hi=old_hi, page=page)


def listed():
    return [
        # one short request, one token: the latency of a call
        _attend("attend_one_short", 1, 1, 1000, 1000, 4, 1, 64, 64),
        # an ordinary decode step: ragged lengths from a new request to 8k
        _attend("attend_decode", 16, 1, 1, 8192, 64, 8, 128, 128),
        # long contexts, the cache far larger than L2
        _attend("attend_decode_long", 32, 1, 8192, 32768, 64, 8, 128, 128),
        # one long request alone: few rows, the work split over its length
        _attend("attend_one_long", 1, 1, 65536, 65536, 64, 4, 192, 128, fmt="int8"),
        # block selection, 16 blocks of 64 per token and KV head, a few tokens per request
        _attend("attend_blocks", 64, 2, 900, 8192, 64, 4, 192, 128, block=64, topk=16),
        # a sliding window of 128 with sinks, four tokens per request (drafts to verify)
        _attend("attend_window_sinks", 48, 4, 3, 4096, 64, 8, 128, 128, window=127, sinks=True, dtype="fp16",
                page=32),
        # rows of a shared latent selected one by one: 2048 per token, 128 heads
        _attend("attend_latent_rows", 48, 1, 1500, 32768, 128, 1, 576, 512, shared=True, block=1, topk=2048),
        # a decode step's one row per request
        _write("write_decode", 64, 1, 1, 8192, 8, 128, 128),
        # prompts: whole pages, the first behind rows that are already there
        _write("write_prompts", 7, 300, 2600, 500, 4, 192, 128),
        # the latent row, chunks of prompts, integers
        _write("write_latent", 24, 17, 200, 4096, 1, 576, 512, shared=True, fmt="int8"),
        # a decode step's plan
        _plan("plan_decode", 64, 1, 1, 8192, 64),
        # many requests, prompts among them
        _plan("plan_many", 1500, 0, 40, 4096, 32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend"] * 6 + ["write"] * 3 + ["plan"])
    if kind == "plan":
        hi = _log(rng, 1, 64)
        c = _plan("", _log(rng, 1, 1500), rng.choice([0, 1, hi]) if hi > 1 else rng.choice([0, 1]), hi,
                  _log(rng, 1, 8192), rng.choice([16, 32, 64, 128]))
        c["n_lo"] = min(c["n_lo"], c["n_hi"])
    elif kind == "write":
        Hkv, dqk, dv, shared = rng.choice([(8, 128, 128, False), (4, 192, 128, False), (1, 64, 64, False),
                                           (2, 128, 128, False), (1, 576, 512, True)])
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, 16000 // B))
        c = _write("", B, rng.randint(1, hi), hi, _log(rng, 1, 8192), Hkv, dqk, dv, shared=shared,
                   page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                   dtype=rng.choice(["bf16", "bf16", "fp16"]))
    else:
        mode = rng.choice(["all", "all", "window", "blocks", "blocks", "latent"])
        most = 640_000 * 8 * 256
        while True:
            B = _log(rng, 1, 128)
            hi = _log(rng, 1, 65536)
            lo = rng.choice([1, hi, rng.randint(1, hi)])
            n = rng.choice([1, 1, 1, 2, 3, 4, 8])
            G = rng.choice([1, 4, 7, 8, 16])
            Hkv, dqk, dv = rng.choice([(8, 128, 128), (4, 192, 128), (1, 64, 64), (2, 128, 128), (3, 192, 128)])
            kw = dict(page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                      dtype=rng.choice(["bf16", "bf16", "fp16"]), sinks=rng.random() < 0.3)
            if mode == "window":
                kw["window"] = _log(rng, 8, 1024) - 1
            elif mode == "blocks":
                kw.update(block=rng.choice([16, 32, 64]), topk=rng.randint(1, 24))
            elif mode == "latent":
                Hkv, dqk, dv, G = 1, 576, 512, rng.choice([16, 64, 128])
                kw.update(shared=True, block=1, topk=_log(rng, 16, 2048))
                n = rng.choice([1, 1, 2])
            # what the pages and the plain form's copies take
            rows = B * (hi + lo) / 2
            if rows * Hkv * (dqk + dv) > most or (mode == "latent" and (B * n * kw["topk"] > 48 * 2048 or
                                                                        rows > 32 * 20480)):
                continue
            if mode == "blocks" and B * n * Hkv * kw["topk"] * kw["block"] > 128 * 4 * 1024:
                continue
            if B * n * hi * Hkv * (4 * (dqk + dv) + 16 * G) > 40e9 * (n if mode == "all" else 1):
                continue
            break
        c = _attend("", B, n, lo, hi, Hkv * G, Hkv, dqk, dv, **kw)
    del c["name"]
    return c


def _spread(lo, hi, n, shift=0.0):
    """n lengths over [lo, hi], in no order."""
    return [lo + int((hi - lo + 1) * ((0.5 + shift + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lens(c):
    """(rows already there, new tokens) of each request."""
    if c["op"] == "attend":
        total = _spread(c["len_lo"], c["len_hi"], c["B"])
        new = [c["n_new"]] * c["B"]
        return [max(t - c["n_new"], 0) for t in total], new
    return _spread(0, c["old_hi"], c["B"], 0.25), _spread(c["n_lo"], c["n_hi"], c["B"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _fill_codes(shape, fmt, g):
    """Codes as the rounding of normal values leaves them: the page's largest near the top code."""
    out = torch.empty(shape, dtype=CODES[fmt], device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 28) // max(1, flat.shape[1]))
    for i in range(0, shape[0], step):
        x = torch.randn(flat[i:i + step].shape, generator=g, device=DEV, dtype=torch.bfloat16)
        if fmt == "e4m3":
            flat[i:i + step] = (x * 72).clamp_(-448, 448).to(CODES[fmt])
        else:
            flat[i:i + step] = (x * 24).round_().clamp_(-127, 127).to(CODES[fmt])
    return out


def _fill_scales(shape, fmt, g):
    """Powers of two around the scale that brings the codes back to unit variance."""
    mid = 2.0 ** -6 if fmt == "e4m3" else 2.0 ** -5
    return torch.tensor([mid / 2, mid, mid * 2], device=DEV)[torch.randint(0, 3, shape, generator=g, device=DEV)]


def prepare(c, seed):
    g = _gen(seed)
    old, new = _lens(c)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    B, page = c["B"], c["page"]
    if c["op"] == "plan":
        max_pages = -(-(max(old) + max(new)) // page) + 3
        held = [-(-o // page) for o in old]
        more = [-(-(o + n) // page) - h for o, n, h in zip(old, new, held)]
        n_pages = sum(held) + sum(more) + 5
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        h = i32(held)
        j = torch.arange(max_pages, device=DEV)
        at = (torch.cumsum(h, 0) - h)[:, None] + j
        table = torch.where(j < h[:, None], order[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
        free[:n_pages - sum(held)] = order[sum(held):]
        return dict(case=c, old=i32(old), new=i32(new), table=table, free=free, n_free=i32([n_pages - sum(held)]),
                    T=sum(new))
    Hkv, dqk, dv = c["Hkv"], c["d_qk"], c["d_v"]
    total = [max(o + n, 1) if c["op"] == "write" else max(o, 0) + n for o, n in zip(old, new)]
    if c["op"] == "attend":
        total = _spread(c["len_lo"], c["len_hi"], B)  # a request may hold fewer rows than it asks tokens
    used = [-(-t // page) for t in total]
    max_pages = max(used)
    n_pages = sum(used) + 4
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    u = i32(used)
    j = torch.arange(max_pages, device=DEV)
    at = (torch.cumsum(u, 0) - u)[:, None] + j
    table = torch.where(j < u[:, None], order[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
    dt = TYPES[c["dtype"]]
    T = sum(new)
    s = dict(case=c, table=table, lens=i32(total), cu=i32([sum(new[:b]) for b in range(B + 1)]), T=T,
             k=_fill_codes((n_pages, page, Hkv, dqk), c["fmt"], g), k_scale=_fill_scales((n_pages, Hkv), c["fmt"], g))
    s["v"] = None if c["shared"] else _fill_codes((n_pages, page, Hkv, dv), c["fmt"], g)
    s["v_scale"] = None if c["shared"] else _fill_scales((n_pages, Hkv), c["fmt"], g)
    if c["op"] == "write":
        # most rows stay under their page's scale; some heads' rows are four times as large
        loud = 1 + 3 * (torch.rand((T, Hkv, 1), generator=g, device=DEV) < 0.05)
        s["new_k"] = (torch.randn((T, Hkv, dqk), generator=g, device=DEV) * loud).to(dt)
        s["new_v"] = None if c["shared"] else torch.randn((T, Hkv, dv), generator=g, device=DEV).to(dt)
    else:
        s["q"] = torch.randn((T, c["Hq"], dqk), generator=g, device=DEV).to(dt)
        s["sinks"] = torch.randn(c["Hq"], generator=g, device=DEV) if c["sinks"] else None
        s["idx"] = _draw_idx(c, total, new, g) if c["topk"] else None
    if own:
        from top_sparse_attention_attn_b200 import Kv8Cache
        s["cache"] = Kv8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], d_v=dv)
    return s


def _draw_idx(c, total, new, g):
    """Per token and KV head: distinct blocks (or rows) at or before the token, its own block
    first, -1 behind them."""
    B, n, bs, Hkv, topk = c["B"], c["n_new"], c["block"], c["Hkv"], c["topk"]
    ta = torch.tensor([[t - n + i for i in range(n)] for t in total], device=DEV).view(B * n, 1, 1)
    own_block = torch.div(ta, bs, rounding_mode="floor").expand(-1, Hkv, 1)
    out = torch.full((B * n, Hkv, topk), -1, dtype=torch.int32, device=DEV)
    nb = max(t for t in total) // bs + 1
    step = max(1, (1 << 26) // (nb * Hkv))
    for i in range(0, B * n, step):
        key = torch.rand((own_block[i:i + step].shape[0], Hkv, nb), generator=g, device=DEV)
        j = torch.arange(nb, device=DEV)
        d = own_block[i:i + step]
        key = torch.where(j == d, 2.0, torch.where(j < d, key, -1.0))
        v, at = key.topk(min(topk, nb), dim=-1)
        out[i:i + step, :, :at.shape[-1]] = torch.where(v >= 0, at, -1).to(torch.int32)
    return out


# ---------------------------------------------------------------------------
# the pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if c["op"] == "plan":
        return _run_plan(s)
    if c["op"] == "write":
        return _run_write(s)
    return _run_attend(s)


def _run_plan(s):
    if own:
        from top_sparse_attention_attn_b200 import plan_pages
        p = plan_pages(s["old"], s["new"], s["table"], s["free"], s["n_free"], page_size=s["case"]["page"],
                       n_tokens=s["T"])
        return dict(table=s["table"], seq_lens=p.seq_lens, cu=p.cu_seqlens_q, slots=p.slots, n_free=p.n_free,
                    n_served=p.n_served)
    old, new, table, page, T = s["old"].long(), s["new"].long(), s["table"], s["case"]["page"], s["T"]
    held = (old + page - 1) // page
    pages = (old + new + page - 1) // page
    need = pages - held
    take = torch.cumsum(need, 0)
    fits = (take <= s["n_free"]) & (pages <= table.shape[1]) & (torch.cumsum(new, 0) <= T) & (old >= 0) & (new >= 0)
    served = torch.cumprod(fits.long(), 0)
    n = new * served
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(n, 0)])
    # page j of a request is new when it lies past the pages held: the next ones off the stack's end
    j = torch.arange(table.shape[1], device=DEV)
    rank = (take - need)[:, None] + j - held[:, None]
    fresh = (j >= held[:, None]) & (j < pages[:, None]) & (served[:, None] > 0)
    src = (s["n_free"].long() - 1 - rank).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][src], table))
    t = torch.arange(T, device=DEV)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=old.numel() - 1)
    pos = old[b] + t - cu[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return dict(table=table, seq_lens=(old + n).int(), cu=cu.int(), slots=torch.where(t < cu[-1], slot, -1),
                n_free=(s["n_free"] - (need * served).sum()).int(), n_served=served.sum().int().view(1))


def _scale_for(a, fmt):
    """The power of two 2^e, e in [-60, 60], with a <= top * 2^e; 2^-60 for a = 0."""
    m_top, e_top, _ = TOP[fmt]
    m, e = torch.frexp(a)
    e = torch.where(m <= m_top, e - e_top, e - e_top + 1)
    e = torch.where(a > 0, e, -60).clamp(-60, 60)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _power_at_least(a):
    """The power of two at or above a scale that is already there."""
    m, e = torch.frexp(a)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(a > 0, e, -60).clamp(-60, 60)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _round_to(x, fmt):
    top = TOP[fmt][2]
    x = x.clamp(-top, top)
    return x.to(CODES[fmt]) if fmt == "e4m3" else torch.nan_to_num(x).round().to(CODES[fmt])


def _write_plain(x, codes, scale, page_of, off, fmt):
    """x [T, H, d] into codes [pages, page, H, d] at (page_of, off); scale [pages, H]."""
    xf = x.float()
    size = torch.where(xf.isfinite(), xf.abs(), 0.0).amax(-1)
    at, which = torch.unique(page_of, return_inverse=True)
    amax = torch.zeros((at.numel(), x.shape[1]), device=DEV)
    amax.scatter_reduce_(0, which[:, None].expand_as(size), size, "amax")
    first = torch.full((at.numel(),), codes.shape[1], dtype=off.dtype, device=DEV)
    first.scatter_reduce_(0, which, off, "amin")
    need = _scale_for(amax, fmt)
    before = scale[at]
    after = torch.where((first > 0)[:, None], torch.maximum(_power_at_least(before), need), need)
    # rows of the page that were there before, in the new scale
    there = (torch.arange(codes.shape[1], device=DEV)[None] < first[:, None]) & True
    raw = codes.view(torch.uint8)
    kept = raw[at].view(codes.dtype).float()
    again = _round_to(kept * (before / after)[:, None, :, None], fmt).view(torch.uint8)
    same = (before == after)[:, None, :, None]
    raw[at] = torch.where(there[:, :, None, None] & ~same, again, raw[at])
    raw[page_of, off] = _round_to(xf / after[which][:, :, None], fmt).view(torch.uint8)
    scale[at] = after


def _run_write(s):
    c = s["case"]
    if own:
        s["cache"].write(s["new_k"], s["new_v"], s["table"], s["lens"], cu_seqlens_q=s["cu"])
    else:
        t = torch.arange(s["T"], device=DEV)
        b = torch.searchsorted(s["cu"], t, right=True) - 1
        pos = (s["lens"] - s["cu"].diff())[b] + t - s["cu"][b]
        page_of, off = s["table"][b, pos // c["page"]].long(), pos % c["page"]
        _write_plain(s["new_k"], s["k"], s["k_scale"], page_of, off, c["fmt"])
        if not c["shared"]:
            _write_plain(s["new_v"], s["v"], s["v_scale"], page_of, off, c["fmt"])
    out = dict(k=s["k"], k_scale=s["k_scale"])
    if not c["shared"]:
        out.update(v=s["v"], v_scale=s["v_scale"])
    return out


def _run_attend(s):
    c = s["case"]
    if own:
        o, lse = s["cache"].attend(s["q"], s["table"], s["lens"], cu_seqlens_q=s["cu"], idx=s["idx"],
                                   block_size=max(c["block"], 1), window=c["window"] if c["window"] >= 0 else None,
                                   sinks=s["sinks"], scale=c["d_qk"] ** -0.5)
        return dict(o=o, lse=lse)
    B, n, Hq, Hkv, dqk, dv, page = c["B"], c["n_new"], c["Hq"], c["Hkv"], c["d_qk"], c["d_v"], c["page"]
    G = Hq // Hkv
    ta = (s["lens"][:, None] - n + torch.arange(n, device=DEV)).long()                     # [B, n]
    if c["topk"]:
        # the rows each token and head selects: [B * n, Hkv, R]
        R = c["topk"] * c["block"]
        idx = s["idx"].long()
        pos = (idx[..., None] * c["block"] + torch.arange(c["block"], device=DEV)).view(B * n, Hkv, R)
        ok = (idx >= 0).repeat_interleave(c["block"], -1) & (pos <= ta.view(-1, 1, 1))
        req = torch.arange(B, device=DEV).repeat_interleave(n).view(-1, 1, 1)
        head = torch.arange(Hkv, device=DEV).view(1, -1, 1)
        q = s["q"].float().view(B * n, Hkv, G, dqk)
    else:
        # every row, the query tokens of a request together: [B, Hkv, R]
        R = int(s["table"].shape[1]) * page
        if c["window"] >= 0:  # no row before the window of the first token
            R = min(R, c["window"] + n)
        pos = (torch.arange(R, device=DEV) + (s["lens"].long() - R).clamp(min=0)[:, None] * (c["window"] >= 0)
               ).view(B, 1, R)
        ok = torch.ones((B, 1, R), dtype=torch.bool, device=DEV)
        req = torch.arange(B, device=DEV).view(-1, 1, 1)
        head = torch.arange(Hkv, device=DEV).view(1, -1, 1)
        q = s["q"].float().view(B, n, Hkv, G, dqk).transpose(1, 2).reshape(B, Hkv, n * G, dqk)
    safe = torch.where(ok & (pos < s["lens"].long().view(-1, 1, 1)[req.flatten()]), pos, 0)
    at = s["table"][req, safe // page].long().clamp(min=0)
    row = at * page + safe % page
    k = s["k"].view(-1, Hkv, dqk)[row, head].float() * s["k_scale"][at, head][..., None]
    score = (q @ k.transpose(-1, -2)) * dqk ** -0.5
    if c["shared"]:
        v = k[..., :dv]
    else:
        del k
        v = s["v"].view(-1, Hkv, dv)[row, head].float() * s["v_scale"][at, head][..., None]
    if c["topk"]:
        see = ok.view(B * n, Hkv, 1, R)
    else:
        t = ta.repeat_interleave(G, 1).view(B, 1, n * G, 1)
        p4 = pos.view(B, 1, 1, R)
        see = (p4 <= t) & (p4 >= 0)
        if c["window"] >= 0:
            see = see & (p4 >= t - c["window"])
    score = torch.where(see, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, 1, G).expand(score.shape[0], -1, score.shape[2] // G, -1)
        sink = sink.reshape(score.shape[0], Hkv, -1, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    den = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + torch.exp(sink - top)
    o = torch.where(den > 0, (p @ v) / den, 0.0)
    lse = torch.where(den > 0, top + torch.log(den), math.inf)
    if c["topk"]:
        o, lse = o.view(B * n, Hq, dv), lse.view(B * n, Hq)
    else:
        o = o.view(B, Hkv, n, G, dv).transpose(1, 2).reshape(B * n, Hq, dv)
        lse = lse.view(B, Hkv, n, G).transpose(1, 2).reshape(B * n, Hq)
    return dict(o=o.to(s["q"].dtype), lse=lse)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(c):
    old, new = _lens(c)
    page, B, T = c["page"], c["B"], sum(new)
    if c["op"] == "plan":
        held = sum(-(-o // page) for o in old)
        fresh = sum(-(-(o + n) // page) for o, n in zip(old, new)) - held
        # lengths in, offsets and lengths out, a slot per token with the page it lies on, the new pages
        touched = sum(-(-(o + n) // page) - o // page for o, n in zip(old, new) if n)
        return {"bytes": B * 16 + T * 8 + 8 * fresh + 4 * touched, "flops": 4 * B + 2 * T}
    Hkv, dqk, dv = c["Hkv"], c["d_qk"], c["d_v"]
    row = Hkv * (dqk + (0 if c["shared"] else dv))
    kinds = 1 if c["shared"] else 2
    if c["op"] == "write":
        touched = sum(-(-(o + n) // page) - o // page for o, n in zip(old, new) if n)
        return {"bytes": T * row * 3 + touched * (4 + 8 * Hkv * kinds), "flops": 3 * T * row}
    total = _spread(c["len_lo"], c["len_hi"], B)
    G, n = c["Hq"] // Hkv, c["n_new"]
    rows, pairs, pages = 0, 0, 0
    for L in total:
        unseen = 1.0  # the share of a request's rows that none of its tokens selects, on average
        for i in range(n):
            ta = L - n + i
            if ta < 0:
                continue
            if c["topk"]:
                bs = c["block"]
                seen = min(c["topk"], ta // bs + 1) * bs - (bs - 1 - ta % bs)
                unseen *= 1 - seen / L
            else:
                seen = ta + 1 if c["window"] < 0 else min(ta, c["window"]) + 1
            pairs += seen
        if not c["topk"]:
            held = L if c["window"] < 0 else min(L, c["window"] + n)
            rows += held
            pages += -(-held // page)
        elif L:
            rows += L * (1 - unseen)
            pages += min(-(-L // page), c["topk"] * max(1, c["block"] // page))
    b = rows * row + pages * (4 + 4 * Hkv * kinds) + T * c["Hq"] * (2 * dqk + 2 * dv + 4) + 8 * B
    b += 4 * T * Hkv * c["topk"] + (4 * c["Hq"] if c["sinks"] else 0)
    return {"bytes": b, "flops": 2 * pairs * Hkv * G * (dqk + dv)}


# ---------------------------------------------------------------------------
# the definition in 64 bits, request by request
# ---------------------------------------------------------------------------

def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers alone
    s = prepare(c, seed)
    if c["op"] == "write":
        out = {}
        for kind in ("k",) if c["shared"] else ("k", "v"):
            codes, scale = _exact_write(s, kind)
            out[kind] = codes if c["fmt"] == "e4m3" else None
            out[kind + "_scale"] = scale
        return out
    total, n = s["lens"].tolist(), c["n_new"]
    if sum(total) * c["Hq"] * n * (c["d_qk"] + c["d_v"]) > 4e12:
        return None
    o = torch.zeros((s["T"], c["Hq"], c["d_v"]), dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], c["Hq"]), math.inf, dtype=torch.float64, device=DEV)
    G, page = c["Hq"] // c["Hkv"], c["page"]
    for b, L in enumerate(total):
        mine = s["table"][b, :-(-L // page)].long()
        for h in range(c["Hkv"]):
            def rows(codes, scale):
                x = codes[mine, :, h].double() * scale[mine, h].double()[:, None, None]
                return x.reshape(-1, x.shape[-1])[:L]
            k = rows(s["k"], s["k_scale"])
            v = k[:, :c["d_v"]] if c["shared"] else rows(s["v"], s["v_scale"])
            for i in range(n):
                t, ta = b * n + i, L - n + i
                if ta < 0:
                    keep = torch.zeros(0, dtype=torch.long, device=DEV)
                elif c["topk"]:
                    x = s["idx"][t, h].long()
                    x = x[x >= 0]
                    keep = (x[:, None] * c["block"] + torch.arange(c["block"], device=DEV)).flatten()
                    keep = keep[keep <= ta]
                else:
                    keep = torch.arange(0 if c["window"] < 0 else max(0, ta - c["window"]), ta + 1, device=DEV)
                q = s["q"][t, h * G:(h + 1) * G].double()
                z = q @ k[keep].T / math.sqrt(c["d_qk"])
                if s["sinks"] is not None:
                    z = torch.cat([z, s["sinks"][h * G:(h + 1) * G].double()[:, None]], 1)
                if z.shape[1] == 0:
                    continue
                e = torch.logsumexp(z, 1)
                o[t, h * G:(h + 1) * G] = torch.exp(z - e[:, None])[:, :keep.numel()] @ v[keep]
                lse[t, h * G:(h + 1) * G] = e
    return dict(o=o, lse=lse)


def _exact_write(s, kind):
    """Codes (as the numbers that they are) and scales of the whole cache after the write."""
    c = s["case"]
    top, page = TOP[c["fmt"]][2], c["page"]
    codes, scale = s[kind].double(), s[kind + "_scale"].double().cpu().numpy()
    x = s["new_" + kind].double().cpu().numpy()

    def near(v):  # 4 significant bits, in steps of 2^-9 at the least
        if c["fmt"] == "int8":
            return np.clip(np.rint(v), -top, top)
        e = np.maximum(np.frexp(v)[1], -5) - 4
        return np.clip(np.ldexp(np.rint(np.ldexp(v, -e)), e), -top, top)

    def power(a):  # the least power of two that is no less
        m, e = np.frexp(np.maximum(a, 2.0 ** -60))
        return np.ldexp(1.0, np.where(m == 0.5, e - 1, e))

    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].cpu()
    for b in range(c["B"]):
        at = lens[b] - (cu[b + 1] - cu[b])
        t = cu[b]
        while t < cu[b + 1]:
            p, off = int(table[b, at // page]), at % page
            m = min(page - off, cu[b + 1] - t)
            part = x[t:t + m]
            new = power(np.abs(part).max((0, 2)) / top)
            if off:
                new = np.maximum(new, power(scale[p]))
                again = near(codes[p, :off].cpu().numpy() * (scale[p] / new)[None, :, None])
                codes[p, :off] = torch.from_numpy(again).to(DEV)
            codes[p, off:off + m] = torch.from_numpy(near(part / new[None, :, None])).to(DEV)
            scale[p] = new
            t, at = t + m, at + m
    return codes, torch.from_numpy(scale)
