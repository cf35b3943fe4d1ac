"""Serving over an 8-bit paged KV cache on the GPU against the float64 definition:
page plans and written caches exactly, attention within bounds derived from its roundings.

Bounds of the attention.  With d_z the error of a score, an element of O is off by at most
  sum_j p_j |v_j| (2 d_z + 2^-11 + n 2^-23)   (p_j moves by a factor e^(+-2 d_z) after the
        normalisation; the probabilities enter the product rounded to 11 bits; n fp32 sums)
  + |O| eps / 2                             (the output's own rounding)
and lse by d_z + 2^-22 (1 + |lse|), where d_z covers fp32 sums of d products, (d + 8) 2^-24
times scale sum |q||k|, plus 2^-20 for the exponential and the query held as fp16 times a
power of two (11 bits hold bf16 and fp16 values; what is lost lies 2^-30 below the largest)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8_ref as R
from top_sparse_attention_attn_b200 import Kv8Cache, SparseAttention, plan_pages
from top_sparse_attention_attn_b200 import _lib as L

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def make_cache(rng, lens, *, page, H, dqk, dv, shared=False, fmt="e4m3", spare=3, power=True, table_pad=0):
    """A cache whose pages lie in shuffled order, rows of random codes (NaN in e4m3 everywhere
    that no sequence's row lies), and its block table (-1 behind the used pages)."""
    B = len(lens)
    used = [-(-n // page) for n in lens]
    mp = max(max(used), 1)
    P = sum(used) + spare
    order = rng.permutation(P)
    table = np.full((B, mp + table_pad), -1)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    live = np.zeros((P, page), bool)
    for b in range(B):
        for r in range(lens[b]):
            live[table[b, r // page], r % page] = True

    def codes(d):
        if fmt == "int8":
            return rng.integers(-127, 128, (P, page, H, d)).astype(np.int8).view(np.uint8)
        c = R.round_codes(rng.standard_normal((P, page, H, d)) * 72, "e4m3")
        c[~live] = np.where(rng.random(c[~live].shape) < 0.5, 127, 255)
        return c

    def scales():
        e = rng.integers(-8, -4, (P, H)).astype(np.float64)
        return (2.0 ** (e if power else e + rng.random((P, H)))).astype(np.float32)

    k, ks = codes(dqk), scales()
    v, vs = (None, None) if shared else (codes(dv), scales())
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    to = lambda c: torch.from_numpy(c).cuda().view(dt)  # noqa: E731
    cache = Kv8Cache(to(k), None if shared else to(v), torch.from_numpy(ks).cuda(),
                     None if shared else torch.from_numpy(vs).cuda(), d_v=dv)
    kf = R.values(k, fmt) * R.read_scale(ks.astype(np.float64))[:, None, :, None]
    vf = kf[..., :dv] if shared else R.values(v, fmt) * R.read_scale(vs.astype(np.float64))[:, None, :, None]
    return cache, table[:, :mp + table_pad], kf, vf


def make_idx(rng, lens, new, H, block, topk):
    """Distinct blocks at or before each token in random slots, its own among them, -1 elsewhere."""
    idx = []
    for n, L_ in zip(new, lens):
        for i in range(n):
            ta = L_ - n + i
            for _ in range(H):
                row = np.full(topk, -1)
                if ta >= 0:
                    own = ta // block
                    sel = np.concatenate([[own], rng.permutation(own)])[:topk]
                    row[rng.permutation(topk)[:len(sel)]] = sel
                idx.append(row)
    return np.array(idx).reshape(-1, H, topk)


def check(name, o, lse, ref, dtype, d, n):
    """The module's bounds, row by row (o, lse on the device; ref = R.attend's)."""
    ro, rl, spread, big = ref
    o, lse = o.double().cpu().numpy().reshape(ro.shape), lse.double().cpu().numpy().reshape(rl.shape)
    dz = (d + 8) * 2.0 ** -24 * big + 2.0 ** -20
    eps = torch.finfo(dtype).eps
    tol = spread * (2 * dz + 2.0 ** -11 + n * 2.0 ** -23)[..., None] + np.abs(ro) * eps / 2 + 2.0 ** -24
    assert np.isfinite(o).all(), name
    worst = (np.abs(o - ro) / tol).max() if o.size else 0
    assert worst <= 1, f"{name}: O off by {worst:.3g} times its bound"
    assert np.array_equal(np.isinf(rl), np.isinf(lse)) and (lse[np.isinf(lse)] > 0).all(), name
    f = np.isfinite(rl)
    if f.any():
        e = np.abs(lse - rl)[f] / (dz + 2.0 ** -22 * (1 + np.abs(np.where(f, rl, 0))))[f]
        assert e.max() <= 1, f"{name}: lse off by {e.max():.3g} times its bound"


CASES = {
    # a new request of one row, an empty one, whole and broken pages; every head count in a tile
    "ragged": dict(lens=[1, 0, 16, 17, 63, 64, 65, 200, 777], new=[1] * 9, G=8, H=2, dqk=128, dv=128),
    "one": dict(lens=[1], new=[1], G=1, H=1, dqk=64, dv=64),
    "one_long": dict(lens=[9001], new=[1], G=4, H=1, dqk=64, dv=64, page=32),
    "wide": dict(lens=[300, 5, 1025], new=[2, 0, 3], G=16, H=3, dqk=192, dv=128, fmt="int8"),
    "heads20": dict(lens=[129, 400], new=[1, 2], G=20, H=2, dqk=128, dv=128, sinks=True),
    "heads7": dict(lens=[129, 400, 33], new=[3, 9, 5], G=7, H=1, dqk=128, dv=128, dtype="fp16"),
    "mha": dict(lens=[50, 513], new=[1, 1], G=1, H=5, dqk=64, dv=64, fmt="int8", sinks=True),
    # a chunk of a prompt, the first tokens of a request, more tokens than rows (those see nothing)
    "chunk": dict(lens=[150, 40, 3], new=[70, 40, 6], G=4, H=2, dqk=128, dv=128),
    "empty_rows": dict(lens=[2, 0, 5], new=[4, 3, 5], G=4, H=2, dqk=64, dv=64, sinks=True),
    # pages that a tile does not divide
    "page7": dict(lens=[100, 33, 250], new=[1, 2, 3], G=4, H=2, dqk=128, dv=128, page=7),
    "page48": dict(lens=[100, 33, 500], new=[2, 2, 2], G=8, H=2, dqk=192, dv=128, page=48),
    "page1": dict(lens=[37], new=[2], G=4, H=1, dqk=64, dv=64, page=1),
    "window": dict(lens=[1, 30, 128, 129, 900], new=[1, 4, 4, 2, 4], G=8, H=2, dqk=128, dv=128, window=127),
    "window0": dict(lens=[5, 70], new=[5, 3], G=2, H=1, dqk=64, dv=64, window=0, sinks=True, fmt="int8"),
    "blocks": dict(lens=[900, 64, 1, 333], new=[2, 2, 1, 1], G=16, H=2, dqk=192, dv=128, block=64, topk=5),
    "blocks16": dict(lens=[300, 50, 17], new=[3, 2, 1], G=4, H=2, dqk=64, dv=64, block=16, topk=7, page=32,
                     fmt="int8", sinks=True),
    "blocks_window": dict(lens=[700, 90], new=[2, 2], G=8, H=2, dqk=128, dv=128, block=32, topk=9, window=100),
    "blocks24": dict(lens=[300, 50], new=[2, 1], G=4, H=2, dqk=128, dv=128, block=24, topk=4),
    "rows": dict(lens=[300, 50, 7], new=[2, 1, 1], G=4, H=2, dqk=128, dv=128, block=1, topk=33),
    "blocks_large": dict(lens=[1000, 260], new=[1, 1], G=8, H=1, dqk=128, dv=128, block=128, topk=3, page=16),
    "scales": dict(lens=[500, 90], new=[1, 1], G=8, H=2, dqk=128, dv=128, power=False),
    "latent_rows": dict(lens=[600, 70, 1, 0], new=[2, 1, 1, 1], G=128, H=1, dqk=576, dv=512, shared=True, block=1,
                        topk=130),
    "latent_16": dict(lens=[333, 2], new=[1, 2], G=16, H=1, dqk=576, dv=512, shared=True, block=1, topk=64,
                      fmt="int8", page=16, sinks=True),
    "latent_all": dict(lens=[333, 64, 129], new=[1, 3, 1], G=64, H=1, dqk=576, dv=512, shared=True),
    "latent_24": dict(lens=[100, 41], new=[1, 1], G=24, H=2, dqk=576, dv=512, shared=True, window=50),
    "latent_64_int8": dict(lens=[700, 300, 20], new=[1, 1, 2], G=64, H=2, dqk=576, dv=512, shared=True, block=1, topk=200,
                           fmt="int8", sinks=True),
    "latent_50": dict(lens=[400, 129, 1], new=[1, 2, 1], G=50, H=1, dqk=576, dv=512, shared=True, dtype="fp16",
                      window=200),
    # tokens enough for the tensor-memory kernel
    "latents_rows": dict(lens=[600, 70, 1, 0, 333], new=[9, 7, 1, 1, 8], G=128, H=1, dqk=576, dv=512, shared=True, block=1,
                         topk=130),
    "latents_all": dict(lens=[333, 64, 129], new=[10, 6, 9], G=64, H=1, dqk=576, dv=512, shared=True, power=False),
    "latents_64_int8": dict(lens=[700, 300, 20], new=[4, 5, 9], G=64, H=2, dqk=576, dv=512, shared=True, block=1,
                            topk=200, fmt="int8", sinks=True),
    "latents_50": dict(lens=[400, 129, 1], new=[9, 12, 1], G=50, H=1, dqk=576, dv=512, shared=True, dtype="fp16",
                       window=200),
    "latents_blocks": dict(lens=[500, 77], new=[14, 14], G=33, H=1, dqk=576, dv=512, shared=True, block=16, topk=13,
                           page=16, fmt="int8"),
    # the last of several parts of the heads is a small one; pages and windows that cut the chunks of both kernels
    "latent_40": dict(lens=[90, 300], new=[1, 2], G=40, H=1, dqk=576, dv=512, shared=True, page=7),
    "latents_100": dict(lens=[500, 77], new=[9, 9], G=100, H=1, dqk=576, dv=512, shared=True, page=7, sinks=True),
    "latents_rows_window": dict(lens=[500, 77, 260], new=[12, 9, 4], G=64, H=1, dqk=576, dv=512, shared=True, block=1,
                                topk=300, window=131, dtype="fp16"),
    "latent_rows_window": dict(lens=[500, 77, 2], new=[2, 1, 2], G=8, H=2, dqk=576, dv=512, shared=True, block=4,
                               topk=60, window=131, page=16),
    # whole prompts beside a long request's one token
    "prompts": dict(lens=[300, 17, 2000], new=[300, 17, 1], G=8, H=1, dqk=128, dv=128),
    "prompts_mha": dict(lens=[150, 333], new=[150, 33], G=1, H=3, dqk=64, dv=64, fmt="int8", window=64, sinks=True),
    "prompts_latent": dict(lens=[120, 40], new=[120, 40], G=16, H=1, dqk=576, dv=512, shared=True),
    "shared_128": dict(lens=[500, 33, 8], new=[2, 1, 8], G=32, H=1, dqk=128, dv=128, shared=True, dtype="fp16"),
    "shared_128_blocks": dict(lens=[500, 33], new=[2, 1], G=6, H=2, dqk=128, dv=128, shared=True, block=16, topk=6),
}


def _problem(name):
    c = dict(page=64, fmt="e4m3", dtype="bf16", window=None, sinks=False, block=1, topk=0, shared=False, power=True)
    c.update(CASES[name])
    rng = np.random.default_rng(sum(map(ord, name)))
    lens, new, H, G = c["lens"], c["new"], c["H"], c["G"]
    cache, table, kf, vf = make_cache(rng, lens, page=c["page"], H=H, dqk=c["dqk"], dv=c["dv"], shared=c["shared"],
                                      fmt=c["fmt"], power=c["power"])
    T = sum(new)
    q = torch.from_numpy(rng.standard_normal((T, H * G, c["dqk"]))).to(TYPES[c["dtype"]]).cuda()
    idx = make_idx(rng, lens, new, H, c["block"], c["topk"]) if c["topk"] else None
    sinks = rng.standard_normal(H * G).astype(np.float32) if c["sinks"] else None
    cu = np.concatenate([[0], np.cumsum(new)])
    return c, cache, table, kf, vf, q, idx, sinks, cu


@pytest.mark.parametrize("name", list(CASES))
def test_attend(name):
    c, cache, table, kf, vf, q, idx, sinks, cu = _problem(name)
    scale = c["dqk"] ** -0.5
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, c["lens"], cu, c["page"], scale, idx=idx,
                   block_size=c["block"], window=c["window"], sinks=sinks)
    o, lse = cache.attend(q, _i32(table), _i32(c["lens"]), cu_seqlens_q=_i32(cu), idx=None if idx is None else _i32(idx),
                          block_size=c["block"], window=c["window"],
                          sinks=None if sinks is None else torch.from_numpy(sinks).cuda())
    torch.cuda.synchronize()
    assert cache.read_status() == L.SA_OK
    check(name, o, lse, ref, q.dtype, c["dqk"], max(c["lens"]))


def test_many_requests_share_the_ctas():
    """More units than CTAs, of every length: whole ones, cut ones, several in a CTA."""
    rng = np.random.default_rng(51)
    lens = np.concatenate([rng.integers(1, 60, 150), rng.integers(300, 900, 40), [4000, 0, 128, 129, 2500]]).tolist()
    rng.shuffle(lens)
    H, G, d, page = 3, 5, 64, 16
    cache, table, kf, vf = make_cache(rng, lens, page=page, H=H, dqk=d, dv=d)
    cu = np.arange(len(lens) + 1)
    q = torch.randn((len(lens), H * G, d), device="cuda").to(torch.bfloat16)
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu))
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, page, d ** -0.5)
    check("many", o, lse, ref, q.dtype, d, 4000)


@pytest.mark.parametrize("topk", [40, 300])
def test_many_latent_tokens_share_the_ctas(topk):
    rng = np.random.default_rng(52)
    lens, new = [400, 35, 700], [60, 35, 20]
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=1, dqk=576, dv=512, shared=True)
    cu = np.concatenate([[0], np.cumsum(new)])
    idx = make_idx(rng, lens, new, 1, 1, topk)
    q = torch.randn((cu[-1], 128, 576), device="cuda").to(torch.bfloat16)
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), idx=_i32(idx))
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 64, 576 ** -0.5, idx=idx)
    check("latent many", o, lse, ref, q.dtype, 576, 700)


def test_latent_codes_that_begin_between_32_bytes():
    """A cache 16 bytes into its buffer: the kernel that reads 32 at a time cannot take it."""
    rng = np.random.default_rng(53)
    lens, cu = [150, 40], [0, 1, 2]
    cache, table, kf, vf = make_cache(rng, lens, page=16, H=1, dqk=576, dv=512, shared=True)
    buf = torch.empty(cache.k.numel() + 16, dtype=torch.uint8, device="cuda")
    k = buf[16:].view(cache.k.dtype).view(cache.k.shape)
    k.view(torch.uint8).copy_(cache.k.view(torch.uint8))
    assert k.data_ptr() % 32 == 16
    q = torch.randn((2, 64, 576), device="cuda").to(torch.bfloat16)
    moved = Kv8Cache(k, None, cache.k_scale, None, d_v=512)
    o, lse = moved.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu))
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 16, 576 ** -0.5)
    check("moved", o, lse, ref, q.dtype, 576, 150)


@pytest.mark.parametrize("topk", [0, 200])
def test_many_latent_codes_that_begin_between_32_bytes(topk):
    """The same with tokens enough for that kernel, so that the alignment alone keeps the call off it."""
    rng = np.random.default_rng(56)
    lens, new = [333, 64, 129], [10, 6, 9]
    cu = np.concatenate([[0], np.cumsum(new)])
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=1, dqk=576, dv=512, shared=True)
    buf = torch.empty(cache.k.numel() + 16, dtype=torch.uint8, device="cuda")
    k = buf[16:].view(cache.k.dtype).view(cache.k.shape)
    k.view(torch.uint8).copy_(cache.k.view(torch.uint8))
    assert k.data_ptr() % 32 == 16
    q = torch.randn((25, 64, 576), device="cuda").to(torch.bfloat16)
    idx = make_idx(rng, lens, new, 1, 1, topk) if topk else None
    moved = Kv8Cache(k, None, cache.k_scale, None, d_v=512)
    o, lse = moved.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), idx=_i32(idx) if topk else None)
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 64, 576 ** -0.5, idx=idx)
    check("moved", o, lse, ref, q.dtype, 576, 333)


def test_attend_bsnd_strided_inputs_and_given_outputs():
    rng = np.random.default_rng(5)
    lens, s, H, G, d = [90, 200, 33], 2, 2, 4, 128
    cache, table, kf, vf = make_cache(rng, lens, page=32, H=H, dqk=d, dv=d, table_pad=5)
    fused = torch.randn((3, s, H * G + 2 * H, d), device="cuda").to(torch.bfloat16)
    q = fused[:, :, :H * G]                               # a slice of a fused projection
    o = torch.full((3, s, H * G, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, s, H * G), 7.0, device="cuda")
    # the first columns of a wider table
    got = cache.attend(q, _i32(table)[:, :7], _i32(lens), o=o, lse=lse)
    assert got[0] is o and got[1] is lse
    ref = R.attend(q.reshape(6, H * G, d).double().cpu().numpy(), kf, vf, table[:, :7], lens, [0, 2, 4, 6], 32, d ** -0.5)
    check("bsnd", o, lse, ref, q.dtype, d, 200)


@pytest.mark.parametrize("topk", [0, 4])
def test_rows_behind_the_last_sequence_stay(topk):
    rng = np.random.default_rng(6)
    lens, cu, T = [100, 40], [0, 2, 3], 8
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=1, dqk=128, dv=128)
    q = torch.randn((T, 8, 128), device="cuda").to(torch.bfloat16)
    q[3:] = float("nan")
    o = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 8), 7.0, device="cuda")
    idx = np.full((T, 1, topk), 1 << 30) if topk else None    # read behind the last sequence, these would raise the bit
    if topk:
        idx[:3] = make_idx(rng, lens, [2, 1], 1, 32, topk)
    cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), o=o, lse=lse, idx=None if idx is None else _i32(idx),
                 block_size=32)
    ref = R.attend(q[:3].double().cpu().numpy(), kf, vf, table, lens, cu, 64, 128 ** -0.5,
                   idx=None if idx is None else idx[:3], block_size=32)
    check("padded", o[:3], lse[:3], ref, q.dtype, 128, 100)
    assert (o[3:] == 7).all() and (lse[3:] == 7).all() and cache.read_status() == L.SA_OK


@pytest.mark.parametrize("heads,T,topk", [(16, 8, 300), (128, 8, 300), (64, 40, 200), (16, 200, 100), (128, 9, 40)])
def test_latent_rows_behind_the_last_sequence_stay(heads, T, topk):
    """The CTAs are shared out for T tokens, three of which there are."""
    rng = np.random.default_rng(61)
    lens, cu = [400, 90], [0, 2, 3]
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=1, dqk=576, dv=512, shared=True)
    q = torch.randn((T, heads, 576), device="cuda").to(torch.bfloat16)
    q[3:] = float("nan")
    o = torch.full((T, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), 7.0, device="cuda")
    idx = np.full((T, 1, topk), 1 << 30)
    idx[:3] = make_idx(rng, lens, [2, 1], 1, 1, topk)
    cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), o=o, lse=lse, idx=_i32(idx))
    ref = R.attend(q[:3].double().cpu().numpy(), kf, vf, table, lens, cu, 64, 576 ** -0.5, idx=idx[:3])
    check("latent padded", o[:3], lse[:3], ref, q.dtype, 576, 400)
    assert (o[3:] == 7).all() and (lse[3:] == 7).all() and cache.read_status() == L.SA_OK


@pytest.mark.parametrize("name", ["chunk", "window", "blocks", "latent_rows", "latents_rows", "latents_all",
                                  "page7"])
def test_rows_that_are_not_seen_may_hold_anything(name):
    """NaN codes and scales of rows behind a token (or before its window) leave it alone."""
    c, cache, table, kf, vf, q, idx, sinks, cu = _problem(name)
    fmt_nan = 127
    page, lens, new = c["page"], c["lens"], c["new"]
    hurt = 0
    # the last row of each sequence with several tokens: only its last token sees it
    for b, L_ in enumerate(lens):
        if new[b] > 1 and L_ > 1:
            p, r = table[b, (L_ - 1) // page], (L_ - 1) % page
            cache.k.view(torch.uint8)[p, r, :, 5] = fmt_nan
            if not c["shared"]:
                cache.v.view(torch.uint8)[p, r, :, 3] = fmt_nan
            kf[p, r, :, 5] = np.nan
            vf[p, r, :, 3 if not c["shared"] else 5] = np.nan
            hurt += 1
    assert hurt
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), idx=None if idx is None else _i32(idx),
                          block_size=c["block"], window=c["window"])
    keep = np.array([i + 1 < n or n == 1 or lens[b] <= 1 for b, n in enumerate(new) for i in range(n)])
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, page, c["dqk"] ** -0.5, idx=idx,
                   block_size=c["block"], window=c["window"])
    k = torch.from_numpy(keep).cuda()
    check(name, o[k], lse[k], tuple(x[keep] for x in ref), q.dtype, c["dqk"], max(lens))
    # and the tokens that see the row say so
    assert torch.isnan(lse[~k]).all()
    nan_ref = np.isnan(ref[0][~keep])
    assert np.array_equal(torch.isnan(o[~k]).cpu().numpy() | ~nan_ref, np.ones_like(nan_ref))


def test_nan_in_v_alone_reaches_the_tokens_that_see_it():
    rng = np.random.default_rng(8)
    lens, new, cu = [70], [5], [0, 5]
    cache, table, kf, vf = make_cache(rng, lens, page=16, H=1, dqk=128, dv=128)
    p, r = table[0, 67 // 16], 67 % 16                    # row 67: tokens at rows 65, 66 do not see it
    cache.v.view(torch.uint8)[p, r, 0, 9] = 255
    vf[p, r, 0, 9] = np.nan
    q = torch.randn((5, 4, 128), device="cuda").to(torch.bfloat16)
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu))
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 16, 128 ** -0.5)
    got = torch.isnan(o).cpu().numpy()
    want = np.zeros_like(got)
    want[2:, :, 9] = True
    assert np.array_equal(got, want)
    o2 = o.clone()
    o2[:, :, 9] = 0
    for x in ref[0], ref[2]:
        x[:, :, 9] = 0
    check("nan_v", o2, lse, ref, q.dtype, 128, 70)


def test_bad_pages_and_indices_select_nothing_and_raise_the_bit():
    rng = np.random.default_rng(9)
    lens, cu = [200, 120], [0, 1, 2]
    for bad in (-1, 10 ** 6):
        cache, table, kf, vf = make_cache(rng, lens, page=64, H=2, dqk=128, dv=128)
        table[0, 1] = bad
        q = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
        o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu))
        ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 64, 128 ** -0.5)
        check("bad page", o, lse, ref, q.dtype, 128, 200)
        assert cache.read_status() == L.SA_ERR_INDEX
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=2, dqk=128, dv=128)
    idx = make_idx(rng, lens, [1, 1], 2, 16, 6)
    idx[0, 0, 2], idx[1, 1, 0] = 2 ** 31 - 1, 8           # 8 * 16 = 128 lies behind row 119
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), idx=_i32(idx), block_size=16)
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 64, 128 ** -0.5, idx=idx, block_size=16)
    check("bad index", o, lse, ref, q.dtype, 128, 200)
    assert cache.read_status() == L.SA_ERR_INDEX


@pytest.mark.parametrize("given", [None, 0, "side"])
def test_the_status_word_is_sticky_until_it_is_cleared(given):
    rng = np.random.default_rng(55)
    lens, cu = [200, 120], [0, 1, 2]
    cache, table, _, _ = make_cache(rng, lens, page=64, H=2, dqk=128, dv=128)
    bad = table.copy()
    bad[0, 1] = -1
    q = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if given == "side" else given
    args = [(q, _i32(t), _i32(lens)) for t in (table, bad)]
    cu = _i32(cu)
    torch.cuda.synchronize()
    for clear in (False, True):
        cache.attend(*args[1], cu_seqlens_q=cu, stream=stream)
        if clear:
            cache.clear_status(stream)
        cache.attend(*args[0], cu_seqlens_q=cu, stream=stream)
        assert cache.read_status(stream) == (L.SA_OK if clear else L.SA_ERR_INDEX)
    torch.cuda.synchronize()


def test_duplicate_indices_count_twice_and_topk_len_cuts():
    rng = np.random.default_rng(10)
    lens, cu = [300], [0, 2]
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=2, dqk=192, dv=128)
    idx = np.array([[[3, 3, 0, -1], [4, 1, 4, 4]], [[0, 2, 3, 4], [1, 1, 1, 1]]])
    tl = np.array([[4, 3], [0, 2]])
    q = torch.randn((2, 32, 192), device="cuda").to(torch.float16)
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), idx=_i32(idx), block_size=64,
                          topk_len=_i32(tl))
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 64, 192 ** -0.5, idx=idx, block_size=64,
                   topk_len=tl)
    check("duplicates", o, lse, ref, q.dtype, 192, 300)


def test_extreme_scales_and_queries():
    """Scales read clamped, pages of very different scale in one row, large and tiny queries."""
    rng = np.random.default_rng(11)
    lens, cu = [400, 130], [0, 1, 2]
    cache, table, kf, vf = make_cache(rng, lens, page=16, H=1, dqk=128, dv=128)
    kf, vf = kf / cache.k_scale.double().cpu().numpy()[:, None, :, None], vf / cache.v_scale.double().cpu().numpy()[:, None, :, None]
    e = rng.integers(-14, 14, cache.v_scale.shape)
    cache.v_scale.copy_(torch.from_numpy((2.0 ** e).astype(np.float32)))
    cache.v_scale[int(table[0, 3])] = float("nan")
    cache.v_scale[int(table[0, 5])] = 0.0
    cache.k_scale.fill_(2.0 ** -9)
    kf = kf * 2.0 ** -9
    vf = vf * R.read_scale(cache.v_scale.double().cpu().numpy())[:, None, :, None]
    q = torch.randn((2, 4, 128), device="cuda")
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, 1:] *= 2.0 ** -12
    q = q.to(torch.bfloat16)
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 16, 1.0)
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu), scale=1.0)
    keep = [1, 2, 3]
    check("extreme", o[:, keep], lse[:, keep], tuple(x[:, keep] for x in ref), q.dtype, 128, 400)
    check("extreme", o[1:], lse[1:], tuple(x[1:] for x in ref), q.dtype, 128, 400)
    # scores of 1e30: one row takes all, and its scores' rounding decides nothing here
    assert torch.isfinite(o[0, 0]).all()
    assert abs(float(lse[0, 0]) / ref[1][0, 0] - 1) < 1e-4


def test_offsets_past_32_bits():
    H, d, page, P = 8, 128, 128, 36000                     # 36000 * 128 * 8 * 128 = 4.7e9 codes
    cache = Kv8Cache.empty(P, page, H, d, d, fmt="int8")
    lens, cu = [300, 129], [0, 2, 3]
    table = np.array([[P - 1, 0, 35000, -1], [34000, P - 2, -1, -1]])
    rng = np.random.default_rng(12)
    small_k = rng.standard_normal((429 - 126, H, d)).astype(np.float32)
    # sequences written whole through the write, read back through the attention
    n0, n1 = 300, 129
    x = torch.randn((n0 + n1, H, d), device="cuda").to(torch.bfloat16)
    y = torch.randn((n0 + n1, H, d), device="cuda").to(torch.bfloat16)
    del small_k
    cache.write(x, y, _i32(table), _i32(lens), cu_seqlens_q=_i32([0, n0, n0 + n1]))
    pages = [P - 1, 0, 35000, 34000, P - 2]
    sub = torch.tensor(pages, device="cuda")
    local = np.array([[0, 1, 2, -1], [3, 4, -1, -1]])
    kf = (cache.k[sub].double() * cache.k_scale[sub].double()[:, None, :, None]).cpu().numpy()
    vf = (cache.v[sub].double() * cache.v_scale[sub].double()[:, None, :, None]).cpu().numpy()
    want = np.zeros((5, page, H, d))
    for b, (t0, n) in enumerate([(0, n0), (n0, n1)]):
        for r in range(n):
            want[local[b, r // page], r % page] = x[t0 + r].double().cpu().numpy()
    assert np.abs(kf - want).max() <= np.abs(want).max() / 64 and np.abs(kf).max() > 1
    q = torch.randn((3, 16, d), device="cuda").to(torch.bfloat16)
    o, lse = cache.attend(q, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu))
    ref = R.attend(q.double().cpu().numpy(), kf, vf, local, lens, cu, page, d ** -0.5)
    check("far pages", o, lse, ref, q.dtype, d, 300)


@pytest.mark.parametrize("warp,wait,chunk", [(8, 0, 0), (8, 1, 0), (8, 2, 0), (8, 0, 3), (8, 1, 2), (8, 2, 1), (3, 3, 1),
                                             (0, 4, 2), (7, 5, 3), (5, 6, 1), (1, 7, 0), (6, 7, 3), (2, 8, 1), (7, 8, 3)])
def test_a_wait_that_gave_up_makes_its_units_nan(warp, wait, chunk):
    """The tensor-memory kernel: whichever warp's wait it was, the unit at hand and the share's later ones are NaN,
    and all others as ever."""
    rng = np.random.default_rng(54)
    lens, new, topk = [400, 200, 700], [60, 60, 40], 130
    T, n_cta, ch = sum(new), 148, 2                        # a unit: 64 heads of a token, 130 rows in chunks of 128
    cache, table, _, _ = make_cache(rng, lens, page=64, H=1, dqk=576, dv=512, shared=True)
    idx = _i32(make_idx(rng, lens, new, 1, 1, topk))
    tab, ln, cu = _i32(table), _i32(lens), _i32(np.concatenate([[0], np.cumsum(new)]))
    q = torch.randn((T, 128, 576), device="cuda").to(torch.bfloat16)
    o, lse = cache.attend(q, tab, ln, cu_seqlens_q=cu, idx=idx)
    c, a = L.SaKv8Cache.from_buffer_copy(cache._c), L.SaKv8Query()
    c.layout, c.t_q, c.batch, c.max_pages, c.table_stride = L.SA_LAYOUT_TND, T, 3, table.shape[1], table.shape[1]
    c.block_table, c.seq_lens, c.cu_seqlens_q = tab.data_ptr(), ln.data_ptr(), cu.data_ptr()
    a.dtype, a.n_heads_q, a.block_size, a.topk, a.win_left, a.scale = L.SA_DTYPE_BF16, 128, 1, topk, -1, 576 ** -0.5
    a.q, a.q_stride, a.idx = q.data_ptr(), 128 * 576, idx.data_ptr()
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    a.o, a.lse = o2.data_ptr(), lse2.data_ptr()
    r, n = ctypes.byref, ctypes.c_size_t(0)
    assert L.lib().sa_kv8_fwd_get_workspace_size(r(c), r(a), r(n)) == L.SA_OK
    ws = torch.zeros(n.value, dtype=torch.uint8, device="cuda")
    assert L.lib().sa_selftest_kv8_give_up(r(c), r(a), warp, wait, chunk, ws.data_ptr(), n.value, None) == L.SA_OK
    torch.cuda.synchronize()
    assert cache.read_status() == L.SA_ERR_TIMEOUT
    # the line of units, cut evenly: what each CTA holds from that chunk on (wait 8: if a part ends with it)
    base, rem = divmod(2 * T * ch, n_cta)
    ends = [base * i + min(i, rem) for i in range(n_cta + 1)]
    lost = np.zeros(2 * T, bool)
    for w0, w1 in zip(ends, ends[1:]):
        at = w0 + chunk
        if at < w1 and (wait < 8 or at % ch == ch - 1 or at == w1 - 1):
            lost[[w // ch for w in range(at, w1)]] = True
    assert lost.any() and (chunk < 2) >= lost.all()        # from chunk 2 on, some units come before
    lost = torch.from_numpy(lost).view(T, 2).repeat_interleave(64, 1).cuda()
    assert bool((torch.isnan(o2) == lost[..., None]).all()) and bool((torch.isnan(lse2) == lost).all())
    assert bool((o2[~lost] == o[~lost]).all()) and bool((lse2[~lost] == lse[~lost]).all())


@pytest.mark.parametrize("B", [0, 2])
@pytest.mark.parametrize("shared,dqk,dv", [(False, 128, 128), (True, 128, 128), (True, 576, 512)])
@pytest.mark.parametrize("topk", [0, 64])
def test_a_step_without_tokens(shared, dqk, dv, topk, B):
    cache = Kv8Cache.empty(4, 16, 1, dqk, dv, shared=shared)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, cu = z(B, 2), z(B), z(B + 1)
    q = torch.empty((0, 64, dqk), dtype=torch.bfloat16, device="cuda")
    idx = z(0, 1, topk) if topk else None
    o, lse = cache.attend(q, table, lens, cu_seqlens_q=cu, idx=idx)
    assert o.shape == (0, 64, dv) and lse.shape == (0, 64)
    cache.write(q[:, :1], None if shared else q[:, :1, :dv].contiguous(), table, lens, cu_seqlens_q=cu)
    # sequences without tokens, one layout after the other
    o, lse = cache.attend(q.view(B, 0, 64, dqk), table, lens, idx=None if idx is None else idx.view(B, 0, 1, topk))
    assert o.shape == (B, 0, 64, dv)
    torch.cuda.synchronize()
    assert cache.read_status() == L.SA_OK and int(cache.k.view(torch.uint8).max()) == 0


LATER = [(False, 8, 128, 128, 0), (False, 8, 192, 128, 3), (True, 16, 576, 512, 40), (True, 128, 576, 512, 40),
         (True, 64, 576, 512, 0)]


@pytest.mark.parametrize("shared,G,dqk,dv,topk", LATER)
def test_a_captured_step_replays_whatever_its_requests_bring(shared, G, dqk, dv, topk):
    """Plan, write and attention in one graph, replayed with other lengths each time, none at all among them."""
    rng = np.random.default_rng(61)
    B, T, page, mp = 4, 24, 16, 9
    cache = Kv8Cache.empty(40, page, 1, dqk, dv, shared=shared)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    old, new, table, free, n_free = z(B), z(B), z(B, mp) - 1, _i32(np.arange(40)), _i32([40])
    k, v, q = (torch.zeros((T, h, d), dtype=torch.bfloat16, device="cuda") for h, d in ((1, dqk), (1, dv), (G, dqk)))
    o, lse = torch.zeros((T, G, dv), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, G), device="cuda")
    idx = z(T, 1, topk) if topk else None
    block = 1 if shared else 16

    def step():
        p = plan_pages(old, new, table, free, n_free, page_size=page, n_tokens=T)
        cache.write(k, None if shared else v, table, p.seq_lens, cu_seqlens_q=p.cu_seqlens_q)
        cache.attend(q, table, p.seq_lens, cu_seqlens_q=p.cu_seqlens_q, idx=idx, block_size=block, o=o, lse=lse)
        old.copy_(p.seq_lens)
        n_free.copy_(p.n_free)
        return p

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = step()
    lens = np.zeros(B, int)
    for n in ([9, 0, 14, 1], [0, 0, 0, 0], [1, 1, 1, 1], [0, 22, 0, 0], [6, 6, 6, 6]):
        lens += n
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape))
        new.copy_(_i32(n))
        if topk:
            at = np.full((T, 1, topk), 1 << 30)
            at[:sum(n)] = make_idx(rng, lens.tolist(), n, 1, block, topk)
            idx.copy_(_i32(at))
        o.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        t = sum(n)
        cu = np.concatenate([[0], np.cumsum(n)])
        assert p.cu_seqlens_q.tolist() == cu.tolist() and old.tolist() == lens.tolist() and int(p.n_served) == B
        kf, vf = (None if x is None else x.double().cpu().numpy() for x in cache.dequantize())
        ref = R.attend(q[:t].double().cpu().numpy(), kf, kf[..., :dv] if shared else vf, table.cpu().numpy(), lens, cu, page,
                       dqk ** -0.5, idx=at[:t] if topk else None, block_size=block)
        check("step", o[:t], lse[:t], ref, q.dtype, dqk, 200)
        assert (o[t:] == 7).all() and (lse[t:] == 7).all() and cache.read_status() == L.SA_OK


@pytest.mark.parametrize("shared,G,dqk,dv,topk", LATER)
def test_lengths_beyond_the_table_are_cut_to_it(shared, G, dqk, dv, topk):
    """seq_lens past max_pages * page_size: the rows that the table holds, in the attention and in the write."""
    rng = np.random.default_rng(62)
    lens, n, page = [64, 48], [20, 17], 16
    cache, table, kf, vf = make_cache(rng, lens, page=page, H=1, dqk=dqk, dv=dv, shared=shared)
    table, cu = table[:1].repeat(2, 0), _i32(np.concatenate([[0], np.cumsum(n)]))
    q = torch.randn((sum(n), G, dqk), device="cuda").to(torch.bfloat16)
    block = 1 if shared else 16
    idx = make_idx(rng, [64, 64], n, 1, block, topk) if topk else None
    far = _i32([65, 2 ** 31 - 1])
    o, lse = cache.attend(q, _i32(table), far, cu_seqlens_q=cu, idx=None if idx is None else _i32(idx), block_size=block)
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, [64, 64], cu.tolist(), page, dqk ** -0.5, idx=idx,
                   block_size=block)
    check("far", o, lse, ref, q.dtype, dqk, 64)
    c = dict(lens=[64], new=[20], H=1, dqk=dqk, dv=dv, fmt="e4m3", shared=shared)
    k, v = (torch.from_numpy(rng.standard_normal((20, 1, d))).to(torch.bfloat16) for d in (dqk, dv))
    kd, vd = k.cuda(), None if shared else v.cuda()
    _check_write(c, cache, table[:1], k, v, [0, 20],
                 lambda: cache.write(kd, vd, _i32(table[:1]), far[1:], cu_seqlens_q=_i32([0, 20])))


@pytest.mark.parametrize("shared,G,dqk,dv,topk", LATER)
def test_calls_on_two_streams_repeat_each_other(shared, G, dqk, dv, topk):
    """The order of every sum is fixed: the same bits from each call, whatever runs beside it."""
    rng = np.random.default_rng(63)
    lens, new = [900, 33, 350, 1, 620], [5, 6, 7, 1, 6]
    cache, table, _, _ = make_cache(rng, lens, page=16, H=1, dqk=dqk, dv=dv, shared=shared)
    tab, ln, cu = _i32(table), _i32(lens), _i32(np.concatenate([[0], np.cumsum(new)]))
    block = 1 if shared else 16
    idx = _i32(make_idx(rng, lens, new, 1, block, topk)) if topk else None
    q = torch.randn((sum(new), G, dqk), device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(cache.attend(q, tab, ln, cu_seqlens_q=cu, idx=idx, block_size=block))
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs[1:])
    assert cache.read_status() == L.SA_OK


# ---- write --------------------------------------------------------------------

WRITES = {
    "decode": dict(lens=[1, 17, 64, 65, 200], new=[1] * 5, H=4, dqk=128, dv=128),
    "prompt": dict(lens=[130, 40, 5], new=[130, 33, 0], H=2, dqk=192, dv=128, fmt="int8", page=32),
    "chunk": dict(lens=[100, 300, 9], new=[70, 3, 9], H=2, dqk=64, dv=64, page=48, dtype="fp16"),
    "latent": dict(lens=[100, 300, 77], new=[1, 40, 77], H=1, dqk=576, dv=512, shared=True),
    "latent_int8": dict(lens=[100, 300, 77], new=[1, 40, 77], H=2, dqk=576, dv=512, shared=True, fmt="int8", page=16),
    "page7": dict(lens=[30, 8], new=[20, 2], H=3, dqk=128, dv=128, page=7),
    "page256": dict(lens=[600], new=[599], H=1, dqk=128, dv=128, page=256),
    "more_tokens_than_rows": dict(lens=[3, 0, 20], new=[6, 2, 20], H=2, dqk=64, dv=64, page=16),
    "many": dict(lens=[33] * 300, new=[1] * 300, H=8, dqk=128, dv=128, page=16),
}


def _write_problem(name):
    c = dict(page=64, fmt="e4m3", dtype="bf16", shared=False)
    c.update(WRITES[name])
    rng = np.random.default_rng(sum(map(ord, name)))
    cache, table, _, _ = make_cache(rng, c["lens"], page=c["page"], H=c["H"], dqk=c["dqk"], dv=c["dv"],
                                    shared=c["shared"], fmt=c["fmt"], power=name != "page7")
    T = sum(c["new"])
    dt = TYPES[c["dtype"]]
    # magnitudes over many pages' scales: some rows raise theirs, some do not, some heads are silent
    k = torch.from_numpy(rng.standard_normal((T, c["H"], c["dqk"])) * 2.0 ** rng.integers(-9, 6, (T, c["H"], 1))).to(dt)
    v = torch.from_numpy(rng.standard_normal((T, c["H"], c["dv"])) * 2.0 ** rng.integers(-9, 6, (T, c["H"], 1))).to(dt)
    k[::5, 0] = 0
    v[::3, -1] = 0
    return c, cache, table, k, v, np.concatenate([[0], np.cumsum(c["new"])])


def _check_write(c, cache, table, k, v, cu, call):
    parts = [("k", k)] + ([] if c["shared"] else [("v", v)])
    want = {}
    for name, x in parts:
        codes, scale = _bytes(getattr(cache, name)).copy(), getattr(cache, name + "_scale").double().cpu().numpy()
        want[name] = R.write(x.double().numpy(), codes, scale, table, c["lens"], cu, c["fmt"])
    call()
    torch.cuda.synchronize()
    for name, _ in parts:
        got, codes = _bytes(getattr(cache, name)), want[name][0]
        if c["fmt"] == "e4m3":  # the sign of a NaN says nothing
            got, codes = (np.where((a & 127) == 127, 127, a) for a in (got, codes))
        assert np.array_equal(got, codes), f"{name}: {(got != codes).sum()} codes differ"
        s = getattr(cache, name + "_scale").double().cpu().numpy()
        assert np.array_equal(s, want[name][1])


@pytest.mark.parametrize("name", list(WRITES))
def test_write(name):
    c, cache, table, k, v, cu = _write_problem(name)
    kd, vd = k.cuda(), None if c["shared"] else v.cuda()
    _check_write(c, cache, table, k, v, cu,
                 lambda: cache.write(kd, vd, _i32(table), _i32(c["lens"]), cu_seqlens_q=_i32(cu)))
    assert cache.read_status() == L.SA_OK


def test_write_bsnd_strided_and_padded():
    rng = np.random.default_rng(21)
    c = dict(lens=[40, 70], new=[3, 3], H=2, dqk=128, dv=128, fmt="e4m3", shared=False)
    cache, table, _, _ = make_cache(rng, c["lens"], page=16, H=2, dqk=128, dv=128)
    fused = torch.randn((2, 3, 8, 128)).to(torch.bfloat16).cuda()
    k, v = fused[:, :, 4:6], fused[:, :, 6:]
    _check_write(c, cache, table, k.reshape(6, 2, 128).cpu(), v.reshape(6, 2, 128).cpu(), [0, 3, 6],
                 lambda: cache.write(k, v, _i32(table), _i32(c["lens"])))
    # rows behind the last sequence are not written anywhere
    cache, table, _, _ = make_cache(rng, c["lens"], page=16, H=2, dqk=128, dv=128)
    k = torch.randn((50, 2, 128)).to(torch.bfloat16)
    kd = k.cuda()
    _check_write({**c, "new": [1, 2]}, cache, table, k, k, [0, 1, 3],
                 lambda: cache.write(kd, kd, _i32(table), _i32(c["lens"]), cu_seqlens_q=_i32([0, 1, 3])))


@pytest.mark.parametrize("first", [1, 3, 5, 300])
@pytest.mark.parametrize("B,lo,hi,H,d", [(5, 1, 3, 2, 128), (300, 5, 7, 8, 64), (300, 1, 9, 3, 64), (4, 20, 90, 2, 128)])
def test_write_of_a_slice_of_a_step(B, lo, hi, H, d, first):
    """Offsets that begin behind 0: a part of a larger step's sequences, with its packed tokens whole.  Few rows
    per request in windows of one and of several tokens, and many."""
    rng = np.random.default_rng(24 + first)
    new = rng.integers(lo, hi + 1, B)
    lens = (new + rng.integers(0, 40, B)).tolist()
    c = dict(lens=lens, new=new, H=H, dqk=d, dv=d, fmt="e4m3", shared=False)
    cache, table, _, _ = make_cache(rng, lens, page=16, H=H, dqk=d, dv=d)
    cu = first + np.concatenate([[0], np.cumsum(new)])
    k, v = (torch.from_numpy(rng.standard_normal((cu[-1] + 4, H, d))).to(torch.bfloat16) for _ in range(2))
    kd, vd = k.cuda(), v.cuda()
    _check_write(c, cache, table, k, v, cu,
                 lambda: cache.write(kd, vd, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu)))


def test_a_step_served_in_two_slices():
    """The plan of a step, written and attended to a part of its requests at a time: as in one call, bit by bit."""
    rng = np.random.default_rng(25)
    B, H, d, page, cut = 600, 8, 64, 16, 217
    new = rng.integers(1, 8, B)
    T = int(new.sum())
    k, v, q = (torch.from_numpy(rng.standard_normal((T, h, d))).to(torch.bfloat16).cuda() for h in (H, H, 2 * H))
    out = []
    for parts in ([(0, B)], [(0, cut), (cut, B)]):
        cache = Kv8Cache.empty(B, page, H, d, d)
        table = _i32(np.full((B, 1), -1))
        p = plan_pages(_i32([0] * B), _i32(new), table, _i32(np.arange(B)), _i32([B]), page_size=page, n_tokens=T)
        o, lse = torch.zeros_like(q), torch.zeros((T, 2 * H), device="cuda")
        for a, b in parts:
            s = dict(block_table=table[a:b], seq_lens=p.seq_lens[a:b], cu_seqlens_q=p.cu_seqlens_q[a:b + 1])
            cache.write(k, v, **s)
            cache.attend(q, **s, o=o, lse=lse)
        out.append((o, lse, cache))
    (o, lse, one), (o2, lse2, two) = out
    same = {n: torch.equal(getattr(one, n).view(torch.uint8), getattr(two, n).view(torch.uint8))
            for n in ("k", "v", "k_scale", "v_scale")}
    assert all(same.values()), same
    assert int(p.n_served) == B and torch.equal(o, o2) and torch.equal(lse, lse2) and lse.all()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("n", [2, 12])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_behind_rows_with_any_scale(fmt, n, shared):
    """Scales that no write leaves: the earlier rows are rounded again from what the attention reads them as."""
    rng = np.random.default_rng(26)
    odd = [0.0, -1.0, float("nan"), float("inf"), float("-inf"), 2.0 ** -70, 2.0 ** 70, 3.0, 0.25]
    H, (dqk, dv) = len(odd), (576, 512) if shared else (64, 64)
    lens, new = [20 + n, 40 + n], [n, n]
    c = dict(lens=lens, new=new, H=H, dqk=dqk, dv=dv, fmt=fmt, shared=shared)
    cache, table, _, _ = make_cache(rng, lens, page=64, H=H, dqk=dqk, dv=dv, fmt=fmt, shared=shared)
    for s in (cache.k_scale,) if shared else (cache.k_scale, cache.v_scale):
        s[torch.from_numpy(table[:, 0]).cuda()] = torch.tensor(odd, device="cuda")
    k, v = (torch.from_numpy(rng.standard_normal((2 * n, H, d))).to(torch.bfloat16) for d in (dqk, dv))
    k[n:] = 0                                              # rows that need no scale
    kd, vd, cu = k.cuda(), None if shared else v.cuda(), [0, n, 2 * n]
    _check_write(c, cache, table, k, v, cu,
                 lambda: cache.write(kd, vd, _i32(table), _i32(lens), cu_seqlens_q=_i32(cu)))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_of_infinities_nan_and_extremes(fmt):
    rng = np.random.default_rng(22)
    c = dict(lens=[20, 21], new=[4, 5], H=2, dqk=64, dv=64, fmt=fmt, shared=False)
    cache, table, _, _ = make_cache(rng, c["lens"], page=16, H=2, dqk=64, dv=64, fmt=fmt)
    k, v = torch.randn((9, 2, 64)).to(torch.bfloat16), torch.randn((9, 2, 64)).to(torch.bfloat16)
    k[0, 0, 3], k[1, 0, 4], k[2, 1, 5] = float("inf"), float("-inf"), float("nan")
    k[5] = 3e38                                            # above the largest scale: saturates
    v[4:, 0] = 1e-38                                       # below the smallest: zeros
    v[0, 1] = float("inf")
    kd, vd = k.cuda(), v.cuda()
    _check_write(c, cache, table, k, v, [0, 4, 9],
                 lambda: cache.write(kd, vd, _i32(table), _i32(c["lens"]), cu_seqlens_q=_i32([0, 4, 9])))


def test_write_through_a_bad_page_writes_nothing():
    rng = np.random.default_rng(23)
    c = dict(lens=[40, 70], new=[20, 3], H=2, dqk=128, dv=128, fmt="e4m3", shared=False)
    cache, table, _, _ = make_cache(rng, c["lens"], page=16, H=2, dqk=128, dv=128)
    table[0, 2], table[1, 4] = -1, 10 ** 6
    k = torch.randn((23, 2, 128)).to(torch.bfloat16)
    kd = k.cuda()
    _check_write(c, cache, table, k, k, [0, 20, 23],
                 lambda: cache.write(kd, kd, _i32(table), _i32(c["lens"]), cu_seqlens_q=_i32([0, 20, 23])))
    assert cache.read_status() == L.SA_ERR_INDEX


# ---- plan ---------------------------------------------------------------------

@pytest.mark.parametrize("B,page,lo,hi,old_hi,short", [
    (1, 16, 1, 1, 0, 0), (7, 16, 0, 40, 100, 0), (7, 16, 0, 40, 100, 3), (300, 64, 1, 1, 500, 0),
    (700, 32, 0, 9, 300, 40), (2000, 1, 0, 3, 5, 0), (5000, 64, 1, 1, 300, 0), (24576, 16, 0, 2, 60, 100),
    (3, 64, 5000, 9000, 70000, 0), (40, 16, 0, 0, 30, 0),
])
def test_plan(B, page, lo, hi, old_hi, short):
    rng = np.random.default_rng(B + page)
    old, new = rng.integers(0, old_hi + 1, B), rng.integers(lo, hi + 1, B)
    held = -(-old // page)
    more = -(-(old + new) // page) - held
    P = int(held.sum() + more.sum()) + 2
    order = rng.permutation(P)
    mp = int((held + more).max()) + 1
    table = np.full((B, mp), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.concatenate([order[at:], np.full(3, -7)])
    n_free = P - at - short
    T = int(new.sum()) + 3
    want = R.plan(old, new, table, free, n_free, page, T)
    dt = _i32(table)
    p = plan_pages(_i32(old), _i32(new), dt, _i32(free), _i32([n_free]), page_size=page, n_tokens=T)
    for got, ref in zip((dt, p.seq_lens, p.cu_seqlens_q, p.slots), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert int(p.n_free) == want[4] and int(p.n_served) == want[5]
    assert (want[5] < B) == (short > 0)


@pytest.mark.parametrize("B,T", [(0, 0), (0, 5), (3, 0), (3, 300)])
def test_plan_of_nothing(B, T):
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table = z(B, 2) - 1
    for free, n in ((z(0), 0), (z(4) + 1, 3)):
        p = plan_pages(z(B) + 7, z(B), table, free, z(1) + n, page_size=16, n_tokens=T)
        assert p.seq_lens.tolist() == [7] * B and p.cu_seqlens_q.tolist() == [0] * (B + 1)
        assert p.slots.tolist() == [-1] * T and p.n_free.tolist() == [n] and p.n_served.tolist() == [B]
        assert (table == -1).all()


@pytest.mark.parametrize("what", ["negative_old", "negative_new", "tokens", "max_pages", "huge", "no_free"])
def test_plan_stops_at_the_first_request_that_does_not_fit(what):
    old, new = np.array([5, 20, 3, 30, 0]), np.array([4, 1, 9, 2, 6])
    table = np.arange(15).reshape(5, 3)
    free, n_free, T = np.arange(50, 60), 10, 22
    if what == "negative_old":
        old[2] = -1
    if what == "negative_new":
        new[3] = -5
    if what == "tokens":
        T = 13
    if what == "max_pages":
        new[1] = 29                                        # 49 rows: a fourth page of 16
    if what == "huge":
        old[2], new[2] = 2 ** 31 - 1, 2 ** 31 - 1
    if what == "no_free":
        n_free = -3
    want = R.plan(old, new, table, free, n_free, 16, T)
    dt = _i32(table)
    p = plan_pages(_i32(old), _i32(new), dt, _i32(free), _i32([n_free]), page_size=16, n_tokens=T)
    for got, ref in zip((dt, p.seq_lens, p.cu_seqlens_q, p.slots), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert int(p.n_free) == max(want[4], 0) and int(p.n_served) == want[5] < 5


# ---- a run of them ---------------------------------------------------------------

@pytest.mark.parametrize("fmt,shared", [("e4m3", False), ("int8", False), ("e4m3", True)])
def test_serving_steps(fmt, shared):
    """Prompt, then decode steps: plan, write, attend; the cache against the definition's and the
    attention against exact attention over it, and against the 16-bit paged cache that the same
    slots fill."""
    rng = np.random.default_rng(31)
    H, G, dqk, dv, page = (1, 16, 576, 512, 16) if shared else (2, 8, 128, 128, 16)
    B, mp = 3, 6
    cache = Kv8Cache.empty(20, page, H, dqk, dv, shared=shared, fmt=fmt)
    table, free = _i32(np.full((B, mp), -1)), _i32(np.arange(20))
    n_free, lens = _i32([20]), _i32([0] * B)
    codes = {n: (_bytes(getattr(cache, n)).copy(), getattr(cache, n + "_scale").double().cpu().numpy())
             for n in (("k",) if shared else ("k", "v"))}
    rows16 = {n: torch.zeros((20 * page, H, d), dtype=torch.bfloat16, device="cuda")
              for n, d in (("k", dqk), ("v", dv))}
    for step, new in enumerate([[37, 5, 16], [1, 1, 1], [1, 0, 4], [1, 1, 1]]):
        T = sum(new) + 2                                   # a padded token axis
        k = (torch.randn((T, H, dqk)) * 1.3 ** step).to(torch.bfloat16)
        v = torch.randn((T, H, dv)).to(torch.bfloat16)
        q = torch.randn((T, H * G, dqk), device="cuda").to(torch.bfloat16)
        p = plan_pages(lens, _i32(new), table, free, n_free, page_size=page, n_tokens=T)
        cache.write(k.cuda(), None if shared else v.cuda(), table, p.seq_lens, cu_seqlens_q=p.cu_seqlens_q)
        o, lse = cache.attend(q, table, p.seq_lens, cu_seqlens_q=p.cu_seqlens_q)
        tab, ln, cu = (x.cpu().numpy() for x in (table, p.seq_lens, p.cu_seqlens_q))
        n = int(cu[-1])
        assert int(p.n_served) == B and n == sum(new)
        for name, x in (("k", k), ("v", v)):
            if name in codes:
                R.write(x.double().numpy(), *codes[name], tab, ln, cu, fmt)
                assert np.array_equal(_bytes(getattr(cache, name)), codes[name][0])
                assert np.array_equal(getattr(cache, name + "_scale").double().cpu().numpy(), codes[name][1])
            rows16[name].index_copy_(0, p.slots[:n], x[:n].cuda())
        kf, vf = cache.dequantize()
        vf = kf[..., :dv] if shared else vf
        ref = R.attend(q[:n].double().cpu().numpy(), kf.double().cpu().numpy(), vf.double().cpu().numpy(), tab, ln, cu,
                       page, dqk ** -0.5)
        check(f"step {step}", o[:n], lse[:n], ref, q.dtype, dqk, int(ln.max()))
        lens, n_free = p.seq_lens, p.n_free
    if not shared:
        # the 16-bit cache, through the same table and slots, as sa_fwd reads it (one token each)
        sa = SparseAttention(layout="BSND", Hq=H * G, Hkv=H, d_qk=dqk, d_v=dv, scale=dqk ** -0.5,
                             q=q[:3].reshape(3, 1, H * G, dqk), k=rows16["k"], v=rows16["v"], batch=3, s_q=1,
                             s_kv=mp * page, t_kv=20 * page, seqused_kv=lens, block_table=table, page_size=page)
        o16, lse16 = sa.forward()
        # 8-bit K and V against 16-bit ones: half a step of a 4-bit mantissa (or 1/127) per element
        assert (o16.reshape(3, -1).float() - o[:3].reshape(3, -1).float()).abs().max() < 0.25
        assert (lse16.flatten() - lse[:3].flatten()).abs().max() < 0.25
    assert cache.read_status() == L.SA_OK


def test_given_stream():
    """A call on a stream that is not the current one: its workspace belongs to that stream."""
    rng = np.random.default_rng(42)
    lens, cu = [3000, 129], [0, 1, 2]
    cache, table, kf, vf = make_cache(rng, lens, page=64, H=2, dqk=128, dv=128)
    q = torch.randn((2, 16, 128), device="cuda").to(torch.bfloat16)
    tab, ln, cu_d = _i32(table), _i32(lens), _i32(cu)
    ref = R.attend(q.double().cpu().numpy(), kf, vf, table, lens, cu, 64, 128 ** -0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for raw in (side.cuda_stream, 0):
        outs = []
        for _ in range(10):
            outs.append(cache.attend(q, tab, ln, cu_seqlens_q=cu_d, stream=raw))
            torch.full((4 << 20,), 7, dtype=torch.int32, device="cuda")   # takes freed memory of the current stream
        torch.cuda.synchronize()
        for o, lse in outs:
            check("stream", o, lse, ref, q.dtype, 128, 3000)
    p = plan_pages(_i32([0, 5]), _i32([3, 1]), _i32([[-1], [4]]), _i32([1, 2]), _i32([2]), page_size=16, n_tokens=4,
                   stream=side.cuda_stream)
    side.synchronize()
    assert p.slots.tolist() == [32, 33, 34, 69] and int(p.n_free) == 1
    k = torch.randn((2, 2, 128), device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    cache.write(k, k, tab, ln, cu_seqlens_q=cu_d, stream=side.cuda_stream)
    side.synchronize()
    got = cache.k[int(table[1, 2]), 0].float() * cache.k_scale[int(table[1, 2])][:, None]
    assert (got - k[1].float()).abs().max() <= k[1].float().abs().max() / 16
    assert cache.read_status() == L.SA_OK


def test_graph_replay_and_two_streams():
    """A step captured and replayed with new contents in the same buffers; two steps on two
    streams at once, a workspace each."""
    rng = np.random.default_rng(41)
    H, G, d, page, lens = 2, 8, 128, 16, [700, 33, 350]
    cache, table, kf, vf = make_cache(rng, lens, page=page, H=H, dqk=d, dv=d)
    tab, cu = _i32(table), _i32([0, 1, 2, 3])
    ln = _i32(lens)
    q = torch.randn((3, H * G, d), device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attend(q, tab, ln, cu_seqlens_q=cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = cache.attend(q, tab, ln, cu_seqlens_q=cu)
    for cut in ([700, 33, 350], [5, 1, 333], [690, 0, 16]):
        q.copy_(torch.randn((3, H * G, d), device="cuda"))
        ln.copy_(_i32(cut))
        graph.replay()
        torch.cuda.synchronize()
        ref = R.attend(q.double().cpu().numpy(), kf, vf, table, cut, [0, 1, 2, 3], page, d ** -0.5)
        check("replay", o, lse, ref, q.dtype, d, 700)
    ln.copy_(_i32(lens))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for rep in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(cache.attend(q, tab, ln, cu_seqlens_q=cu))
    torch.cuda.synchronize()
    for o2, lse2 in outs[1:]:
        assert torch.equal(o2, outs[0][0]) and torch.equal(lse2, outs[0][1])
