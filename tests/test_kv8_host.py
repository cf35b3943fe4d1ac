"""Serving over an 8-bit paged KV cache, without a GPU: the float64 definition pinned
against independent computations, and the refusals of the C ABI and of the wrapper."""

import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv8_ref as R
from top_sparse_attention_attn_b200 import Kv8Cache, plan_pages
from top_sparse_attention_attn_b200 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: these calls fail validation first


# ---- the definition ---------------------------------------------------------

def test_e4m3_values_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = R.values(np.arange(256, dtype=np.uint8), "e4m3")
    assert np.array_equal(np.isnan(want), np.isnan(got))
    assert np.array_equal(want[~np.isnan(want)], got[~np.isnan(got)])
    pos = got[:127]
    mid = (pos[1:] + pos[:-1]) / 2                       # the ties, and both sides of them
    x = np.concatenate([mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(-1)).astype(np.float64),
                        np.random.default_rng(1).standard_normal(4000) * 40, [0.0, -0.0, 448, -448]])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.round_codes(x, "e4m3"), want)
    assert R.values(R.round_codes(np.array([1e9, -np.inf]), "e4m3"), "e4m3").tolist() == [448, -448]


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_scale_is_the_least_power_of_two_that_holds(fmt):
    top = R.TOP[fmt]
    for a in [0.0, 1e-30, 0.1, 1.0, top, np.nextafter(top, 1e9), 3.5 * top, 1e5]:
        s = R.scale_for(a, fmt)
        assert a <= top * s and (s == 2.0 ** -60 or a > top * s / 2)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("scale", [0.0, -3.0, np.nan, np.inf, 2.0 ** -70, 2.0 ** 70, 2.0 ** -60, 3.0])
def test_an_append_keeps_what_the_earlier_rows_are_read_as(scale, fmt):
    rng = np.random.default_rng(3)
    codes = R.round_codes(rng.standard_normal((1, 8, 1, 16)) * 40, fmt)
    was = R.values(codes[0, :5], fmt) * R.read_scale(scale)
    sc = np.array([[scale]])
    R.write(np.zeros((1, 1, 16)), codes, sc, np.array([[0]]), [6], [0, 1], fmt)
    now = R.values(codes[0, :5], fmt) * R.read_scale(sc[0, 0])
    # 3.0 is raised to 4.0: half a step of a code, or half of e4m3's smallest
    err = np.maximum(np.abs(was) * 2.0 ** -4, 2.0 ** -10 * sc[0, 0]) if fmt == "e4m3" else sc[0, 0] / 2
    assert (np.abs(now - was) <= (err if scale == 3.0 else 0)).all() and (codes[0, 5] == 0).all()


def test_plan_serves_a_prefix_and_takes_pages_off_the_stack():
    table = np.full((4, 3), -1)
    table[0, 0] = 9
    free = np.array([4, 5, 6, 7, 1, 1])
    t, lens, cu, slots, left, served = R.plan([3, 0, 0, 0], [3, 4, 1, 9], table, free, 4, 4, 20)
    assert served == 3 and left == 1 and lens.tolist() == [6, 4, 1, 0] and cu.tolist() == [0, 3, 7, 8, 8]
    assert t[0].tolist() == [9, 7, -1] and t[1, 0] == 6 and t[2, 0] == 5 and t[3, 0] == -1
    assert slots.tolist() == [39, 28, 29, 24, 25, 26, 27, 20] + [-1] * 12


def test_attend_is_a_masked_softmax():
    rng = np.random.default_rng(2)
    P, ps, H, d, G = 5, 4, 2, 8, 2
    k, v = rng.standard_normal((P, ps, H, d)), rng.standard_normal((P, ps, H, d))
    table = np.array([[3, 1, 4], [0, 2, -1]])
    q = rng.standard_normal((3, H * G, d))
    o, lse, *_ = R.attend(q, k, v, table, [11, 6], [0, 2, 3], ps, 0.3, window=6)
    for b, t, ta in [(0, 0, 9), (0, 1, 10), (1, 2, 5)]:
        kk = torch.from_numpy(k[table[b][table[b] >= 0]].reshape(-1, H, d))
        vv = torch.from_numpy(v[table[b][table[b] >= 0]].reshape(-1, H, d))
        pos = torch.arange(kk.shape[0])
        for h in range(H * G):
            z = 0.3 * kk[:, h // G] @ torch.from_numpy(q[t, h])
            z[(pos > ta) | (pos < ta - 6)] = -torch.inf
            assert np.allclose(torch.softmax(z, 0) @ vv[:, h // G], o[t, h], atol=1e-12)
            assert np.isclose(torch.logsumexp(z, 0), lse[t, h])


# ---- refusals: the C ABI ------------------------------------------------------

def _cache(**kw):
    c = L.SaKv8Cache()
    c.format, c.n_heads_kv, c.d_qk, c.d_v = L.SA_KV8_E4M3, 2, 128, 128
    c.page_size, c.n_pages, c.batch, c.max_pages, c.table_stride = 16, 8, 2, 4, 4
    c.layout, c.t_q = L.SA_LAYOUT_TND, 5
    c.k = c.v = c.k_scale = c.v_scale = c.block_table = c.seq_lens = c.cu_seqlens_q = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _query(**kw):
    q = L.SaKv8Query()
    q.dtype, q.n_heads_q, q.block_size, q.topk, q.win_left, q.scale = L.SA_DTYPE_BF16, 8, 1, 0, -1, 0.1
    q.q_stride = 8 * 128
    q.q = q.o = q.lse = FAKE
    for k, v in kw.items():
        setattr(q, k, v)
    return q


BAD_CACHE = [
    (dict(format=2), L.SA_ERR_PARAM), (dict(layout=3), L.SA_ERR_PARAM), (dict(n_heads_kv=0), L.SA_ERR_PARAM),
    (dict(d_qk=100), L.SA_ERR_PARAM), (dict(d_qk=96, d_v=96), L.SA_ERR_UNSUPPORTED),
    (dict(kv_shared=1, d_qk=64, d_v=64), L.SA_ERR_UNSUPPORTED), (dict(page_size=0), L.SA_ERR_PARAM),
    (dict(n_pages=0), L.SA_ERR_PARAM), (dict(max_pages=0), L.SA_ERR_PARAM), (dict(table_stride=3), L.SA_ERR_PARAM),
    (dict(page_size=1 << 16, n_pages=1 << 15), L.SA_ERR_PARAM), (dict(batch=-1), L.SA_ERR_PARAM),
    (dict(page_size=1 << 20, max_pages=1 << 11, table_stride=1 << 11), L.SA_ERR_PARAM),
    (dict(page_size=1 << 10, max_pages=(1 << 20) + 1, table_stride=1 << 21), L.SA_ERR_PARAM),
    (dict(t_q=-1), L.SA_ERR_PARAM), (dict(layout=0, s_q=1 << 30), L.SA_ERR_PARAM), (dict(k=None), L.SA_ERR_NULLPTR),
    (dict(v=None), L.SA_ERR_NULLPTR), (dict(v_scale=None), L.SA_ERR_NULLPTR), (dict(seq_lens=None), L.SA_ERR_NULLPTR),
    (dict(cu_seqlens_q=None), L.SA_ERR_NULLPTR), (dict(block_table=None), L.SA_ERR_NULLPTR),
    (dict(k=FAKE + 8), L.SA_ERR_PARAM),
]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches_are_refused_by_both_calls(kw, status):
    n = ctypes.c_size_t(0)
    lib = L.lib()
    assert lib.sa_kv8_fwd_get_workspace_size(ctypes.byref(_cache(**kw)), ctypes.byref(_query()),
                                             ctypes.byref(n)) == status
    r = L.SaKv8Rows(dtype=0, k=FAKE, v=FAKE, k_stride=256, v_stride=256)
    assert lib.sa_kv8_write(ctypes.byref(_cache(**kw)), ctypes.byref(r), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), L.SA_ERR_PARAM), (dict(n_heads_q=7), L.SA_ERR_PARAM), (dict(n_heads_q=0), L.SA_ERR_PARAM),
    (dict(block_size=0), L.SA_ERR_PARAM), (dict(topk=-1), L.SA_ERR_PARAM), (dict(topk=4), L.SA_ERR_NULLPTR),
    (dict(win_left=-2), L.SA_ERR_PARAM), (dict(flags=1), L.SA_ERR_PARAM), (dict(scale=float("inf")), L.SA_ERR_PARAM),
    (dict(q_stride=8 * 128 - 8), L.SA_ERR_PARAM), (dict(q_stride=8 * 128 + 4), L.SA_ERR_PARAM),
    (dict(topk=1 << 20, block_size=1 << 10, idx=FAKE), L.SA_ERR_PARAM),
    (dict(q=None), L.SA_ERR_NULLPTR), (dict(o=None), L.SA_ERR_NULLPTR), (dict(lse=None), L.SA_ERR_NULLPTR),
    (dict(q=FAKE + 2), L.SA_ERR_PARAM), (dict(o=FAKE + 2), L.SA_ERR_PARAM), (dict(), L.SA_OK),
])
def test_bad_queries_are_refused(kw, status):
    n = ctypes.c_size_t(0)
    assert L.lib().sa_kv8_fwd_get_workspace_size(ctypes.byref(_cache()), ctypes.byref(_query(**kw)),
                                                 ctypes.byref(n)) == status


@pytest.mark.parametrize("t_q,max_pages,heads,takes", [
    (25, 6, 64, True),        # 25 tokens x 2 x 6 shares of 32 heads x 64 rows: more than SMs
    (2, 3, 64, False),        # 12 shares: the kernel with mma.sync at any alignment
    (25, 6, 32, False),       # up to 32 heads: likewise
])
def test_codes_between_32_bytes_take_the_kernel_that_can_read_them(t_q, max_pages, heads, takes):
    """The tensor-memory kernel reads 32 bytes of codes at a time.  Which kernel a call takes shows in its
    workspace: a part of a unit is 64 heads there, 32 at most in the other."""
    size = {}
    for off in (0, 16, 32):
        c = _cache(kv_shared=1, d_qk=576, d_v=512, n_heads_kv=1, page_size=64, n_pages=40, max_pages=max_pages,
                   table_stride=max_pages, t_q=t_q, k=FAKE + off)
        n = ctypes.c_size_t(0)
        q = _query(n_heads_q=heads, q_stride=heads * 576)
        assert L.lib().sa_kv8_fwd_get_workspace_size(ctypes.byref(c), ctypes.byref(q), ctypes.byref(n)) == L.SA_OK
        size[off] = n.value
    assert size[32] == size[0] and (size[16] != size[0]) == takes
    units = t_q * -(-heads // 32)                          # of 32 heads; chunks of 64 rows
    n_cta = min(148, units * max_pages)
    assert size[16] == -(-n_cta * 2 * 24 // 256) * 256 + n_cta * 2 * 32 * (2 + 512) * 4


def test_workspace_and_null_arguments_are_refused():
    lib, n = L.lib(), ctypes.c_size_t(0)
    assert lib.sa_kv8_fwd_get_workspace_size(None, ctypes.byref(_query()), ctypes.byref(n)) == L.SA_ERR_NULLPTR
    assert lib.sa_kv8_fwd_get_workspace_size(ctypes.byref(_cache()), None, ctypes.byref(n)) == L.SA_ERR_NULLPTR
    assert lib.sa_kv8_fwd_get_workspace_size(ctypes.byref(_cache()), ctypes.byref(_query()), None) == L.SA_ERR_NULLPTR
    assert lib.sa_kv8_write(ctypes.byref(_cache()), None, None) == L.SA_ERR_NULLPTR
    assert lib.sa_page_plan(None, None) == L.SA_ERR_NULLPTR
    # a step without tokens launches nothing
    assert lib.sa_kv8_fwd(ctypes.byref(_cache(t_q=0)), ctypes.byref(_query()), None, 0, None) == L.SA_OK
    assert lib.sa_kv8_write(ctypes.byref(_cache(t_q=0)), ctypes.byref(L.SaKv8Rows(k_stride=256, v_stride=256)),
                            None) == L.SA_OK


EMPTY_STEPS = """
import ctypes
from tests.test_kv8_host import FAKE, L, _cache, _query
r, lib = ctypes.byref, L.lib()
for shared, d, dv in [(0, 64, 64), (0, 128, 128), (0, 192, 128), (1, 128, 128), (1, 576, 512)]:
    for empty in [dict(t_q=0), dict(batch=0), dict(layout=0, s_q=0), dict(layout=0, s_q=3, batch=0)]:
        for topk in [0, 64]:
            print(shared, d, dv, empty, topk, flush=True)
            c = _cache(kv_shared=shared, d_qk=d, d_v=dv, **empty)
            q, n = _query(q_stride=8 * d, topk=topk, idx=FAKE), ctypes.c_size_t(7)
            assert lib.sa_kv8_fwd_get_workspace_size(r(c), r(q), r(n)) == L.SA_OK and n.value == 0
            assert lib.sa_kv8_fwd(r(c), r(q), None, 0, None) == L.SA_OK
            w = L.SaKv8Rows(k_stride=2 * d, v_stride=2 * dv)
            assert lib.sa_kv8_write(r(c), r(w), None) == L.SA_OK
"""


def test_a_step_without_tokens_or_requests_asks_for_nothing():
    """In a process of its own: arithmetic on a count of zero ends the process that it happens in."""
    r = subprocess.run([sys.executable, "-c", EMPTY_STEPS], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout[-200:], r.stderr[-500:])


@pytest.mark.parametrize("args,kw,status", [
    ((9, 0, 0), {}, L.SA_ERR_PARAM), ((8, 3, 0), {}, L.SA_ERR_PARAM), ((7, 2, 0), {}, L.SA_ERR_PARAM),
    ((0, 9, 0), {}, L.SA_ERR_PARAM), ((8, 0, -1), {}, L.SA_ERR_PARAM), ((8, 0, 0), dict(t_q=-1), L.SA_ERR_PARAM),
    ((8, 0, 0), dict(t_q=0), L.SA_ERR_UNSUPPORTED),
])
def test_bad_give_up_checks_are_refused(args, kw, status):
    c, q = _cache(kv_shared=1, d_qk=576, d_v=512, n_heads_kv=1, **kw), _query(n_heads_q=64, q_stride=64 * 576)
    assert L.lib().sa_selftest_kv8_give_up(ctypes.byref(c), ctypes.byref(q), *args, FAKE, 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), L.SA_ERR_PARAM), (dict(k=None), L.SA_ERR_NULLPTR), (dict(v=None), L.SA_ERR_NULLPTR),
    (dict(k_stride=248), L.SA_ERR_PARAM), (dict(v_stride=260), L.SA_ERR_PARAM), (dict(k=FAKE + 4), L.SA_ERR_PARAM),
])
def test_bad_rows_are_refused(kw, status):
    r = L.SaKv8Rows(dtype=0, k=FAKE, v=FAKE, k_stride=256, v_stride=256)
    for k, v in kw.items():
        setattr(r, k, v)
    assert L.lib().sa_kv8_write(ctypes.byref(_cache()), ctypes.byref(r), None) == status


@pytest.mark.parametrize("kw", [dict(page_size=1 << 25, n_pages=3), dict(page_size=(1 << 30) // 72 + 1, n_pages=1)])
def test_pages_of_more_pieces_than_32_bits_count_are_not_written(kw):
    """33 M rows of 576 are 2.4e9 pieces of 8: counted in 32 bits, none of them would be written."""
    r = L.SaKv8Rows(dtype=0, k=FAKE, k_stride=576)
    c = _cache(kv_shared=1, d_qk=576, d_v=512, n_heads_kv=1, max_pages=1, **kw)
    assert L.lib().sa_kv8_write(ctypes.byref(c), ctypes.byref(r), None) == L.SA_ERR_PARAM
    c.page_size, c.t_q = (1 << 30) // 72, 0                # the largest that is taken, and nothing to launch
    assert L.lib().sa_kv8_write(ctypes.byref(c), ctypes.byref(r), None) == L.SA_OK


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), L.SA_ERR_PARAM), (dict(batch=24577), L.SA_ERR_PARAM), (dict(page_size=0), L.SA_ERR_PARAM),
    (dict(max_pages=0), L.SA_ERR_PARAM), (dict(n_tokens=-1), L.SA_ERR_PARAM), (dict(table_stride=3), L.SA_ERR_PARAM),
    (dict(free_capacity=-1), L.SA_ERR_PARAM), (dict(max_pages=1 << 16, page_size=1 << 15, table_stride=1 << 16),
                                               L.SA_ERR_PARAM),
    (dict(old_lens=None), L.SA_ERR_NULLPTR), (dict(slots=None), L.SA_ERR_NULLPTR),
    (dict(free_pages=None), L.SA_ERR_NULLPTR), (dict(n_served=None), L.SA_ERR_NULLPTR),
    (dict(seq_lens=FAKE), L.SA_ERR_PARAM), (dict(n_free_out=FAKE + 192), L.SA_ERR_PARAM),
])
def test_bad_plans_are_refused(kw, status):
    a = L.SaPagePlanArgs()
    a.batch, a.max_pages, a.page_size, a.n_tokens, a.free_capacity, a.table_stride = 2, 4, 16, 9, 5, 4
    for i, name in enumerate(["old_lens", "new_lens", "free_pages", "n_free", "block_table", "seq_lens",
                              "cu_seqlens_q", "slots", "n_free_out", "n_served"]):
        setattr(a, name, FAKE + 64 * i)
    for k, v in kw.items():
        setattr(a, k, v)
    assert L.lib().sa_page_plan(ctypes.byref(a), None) == status


def test_kernels_that_start_early_read_with_ordinary_loads():
    """The kernels begin behind a programmatic dependency, so that what they read may have been written while they
    lived: no load through the read-only path, nor a pointer that lets the compiler choose it."""
    csrc = os.path.join(ROOT, "top_sparse_attention_attn_b200", "csrc")
    files = [f for f in os.listdir(csrc) if f.startswith("sa_kv8")]
    assert len(files) == 5
    for f in files:
        with open(os.path.join(csrc, f)) as src:
            code = re.sub(r"//[^\n]*|/\*.*?\*/", "", src.read(), flags=re.S)
        for word in ("__ldg", ".nc", "__restrict__"):
            assert word not in code, (f, word)


# ---- refusals: the wrapper ------------------------------------------------------

def _cpu_cache(shared=False, **kw):
    return Kv8Cache.empty(6, 16, 2, *((576, 512) if shared else (128, 128)), shared=shared, device="cpu", **kw)


def _step(T=5, B=2):
    return dict(block_table=torch.zeros((B, 4), dtype=torch.int32), seq_lens=torch.full((B,), 9, dtype=torch.int32),
                cu_seqlens_q=torch.tensor([0, 2, T], dtype=torch.int32))


def test_wrapper_refuses_wrong_types_shapes_and_strides():
    c, s = _cpu_cache(), _step()
    q = torch.zeros((5, 8, 128), dtype=torch.bfloat16)
    k = torch.zeros((5, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        c.attend(q.float(), **s)
    with pytest.raises(TypeError):
        c.attend(q, **{**s, "seq_lens": s["seq_lens"].long()})
    with pytest.raises(TypeError):
        c.attend(q, **{**s, "block_table": s["block_table"].long()})
    with pytest.raises(ValueError):
        c.attend(q, **{**s, "cu_seqlens_q": s["cu_seqlens_q"][:2]})
    with pytest.raises(ValueError):
        c.attend(q[..., :64], **s)
    with pytest.raises(ValueError):
        c.attend(q.transpose(0, 1).contiguous().transpose(0, 1), **s)
    with pytest.raises(ValueError):
        c.attend(q, **s, window=-1)
    with pytest.raises(ValueError):
        c.attend(q, **s, topk_len=torch.zeros((5, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        c.attend(q, **s, idx=torch.zeros((5, 3, 4), dtype=torch.int32))
    with pytest.raises(TypeError):
        c.attend(q, **s, idx=torch.zeros((5, 2, 4), dtype=torch.int64))
    with pytest.raises(ValueError):
        c.attend(q, **s, sinks=torch.zeros(4))
    with pytest.raises(TypeError):
        c.attend(q, **s, o=torch.zeros((5, 8, 128), dtype=torch.float16))
    with pytest.raises(ValueError):
        c.attend(q, s["block_table"], s["seq_lens"])     # [T, ..] without offsets
    with pytest.raises(ValueError):
        c.write(k, None, **s)
    with pytest.raises(TypeError):
        c.write(k, k.half(), **s)
    with pytest.raises(ValueError):
        _cpu_cache(shared=True).write(k, k, **s)
    # every check passes, but nothing here is on a GPU
    with pytest.raises(ValueError, match="CUDA"):
        c.attend(q, **s)
    with pytest.raises(ValueError, match="CUDA"):
        c.write(k, k, **s)


def test_the_status_word_can_be_cleared():
    c = _cpu_cache()
    c.status.fill_(3)
    c.clear_status()
    assert int(c.status) == 0


@pytest.mark.parametrize("shared", [False, True])
def test_dequantize_reads_scales_as_the_attention_does(shared):
    c = _cpu_cache(shared, fmt="int8")
    odd = torch.tensor([[0.0, -1.0], [float("nan"), float("inf")], [-float("inf"), 2.0 ** -70], [2.0 ** 70, 3.0],
                        [0.25, 2.0 ** 60], [1.0, 2.0 ** -60]])
    for x, s in ((c.k, c.k_scale),) if shared else ((c.k, c.k_scale), (c.v, c.v_scale)):
        x.copy_(torch.arange(x.numel()).remainder(255).sub(127).view(x.shape))
        s.copy_(odd)
    k, v = c.dequantize()
    assert (v is None) == shared
    for x, got in ((c.k, k),) if shared else ((c.k, k), (c.v, v)):
        want = x.numpy().astype(np.float64) * R.read_scale(odd.numpy().astype(np.float64))[:, None, :, None]
        assert np.array_equal(got.numpy(), want)


def test_empty_tensors_may_have_any_strides():
    """Without elements a tensor is contiguous whatever its strides: the checks pass, up to the one for a GPU."""
    c = _cpu_cache()
    none = torch.zeros(0, dtype=torch.int32)
    table = torch.tensor(np.zeros((0, 4)), dtype=torch.int32)
    assert table.stride() == (0, 0)
    s = dict(block_table=table, seq_lens=none, cu_seqlens_q=torch.zeros(1, dtype=torch.int32))
    x = torch.tensor(np.zeros((0, 2, 128)), dtype=torch.bfloat16)
    q = torch.zeros((128, 8, 5), dtype=torch.bfloat16).transpose(0, 2)[:0]
    for cols in (table, torch.zeros((3, 8), dtype=torch.int32).t()[:0, :3]):
        with pytest.raises(ValueError, match="CUDA"):
            c.attend(q, **{**s, "block_table": cols})
        with pytest.raises(ValueError, match="CUDA"):
            c.write(x, x, **{**s, "block_table": cols})
        with pytest.raises(ValueError, match="CUDA"):
            plan_pages(none, none, cols, none, torch.zeros(1, dtype=torch.int32), page_size=16, n_tokens=0)


def test_cache_refuses_tensors_that_do_not_fit():
    k = torch.zeros((6, 16, 2, 128), dtype=torch.int8)
    sc = torch.zeros((6, 2))
    with pytest.raises(TypeError):
        Kv8Cache(k.float(), k.float(), sc, sc)
    with pytest.raises(TypeError):
        Kv8Cache(k, k.view(torch.float8_e4m3fn), sc, sc)
    with pytest.raises(ValueError):
        Kv8Cache(k, k[:5], sc, sc)
    with pytest.raises(ValueError):
        Kv8Cache(k, k, sc[:, :1], sc)
    with pytest.raises(ValueError):
        Kv8Cache(k.transpose(1, 2), k, sc, sc)
    with pytest.raises(ValueError):
        Kv8Cache(k, k, sc, sc, d_v=64)


def test_plan_refuses_wrong_types_and_shapes():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(page_size=16, n_tokens=4)
    with pytest.raises(TypeError):
        plan_pages(i(2).long(), i(2), i(2, 4), i(9), i(1), **ok)
    with pytest.raises(ValueError):
        plan_pages(i(2), i(3), i(2, 4), i(9), i(1), **ok)
    with pytest.raises(ValueError):
        plan_pages(i(2), i(2), i(3, 4), i(9), i(1), **ok)
    with pytest.raises(ValueError):
        plan_pages(i(2), i(2), i(2, 4), i(9), i(2), **ok)
    with pytest.raises(ValueError, match="CUDA"):
        plan_pages(i(2), i(2), i(2, 4), i(9), i(1), **ok)
