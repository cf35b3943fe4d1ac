// sa_kv8_fwd.cu -- attention over a paged KV cache held in 8 bits (sa_kv8_fwd).
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "sa_kv8_device.cuh"
#include "sa_launch.h"
#include "sa_tc.cuh"

namespace sa {

bool k8_built(int dqk, int dv, bool shared) {
  if (shared) return (dqk == 128 && dv == 128) || (dqk == 576 && dv == 512);
  return (dqk == 64 && dv == 64) || (dqk == 128 && dv == 128) || (dqk == 192 && dv == 128);
}

// ---------------------------------------------------------------------------
// rows of up to 192 columns: split over the rows
// ---------------------------------------------------------------------------
// Work.  A unit is up to 16 query rows of one KV head: the G heads of 16 / G tokens
// of a sequence, or 16 of a token's heads where G > 16, or the heads of one token where
// each token selects its own blocks.  A unit's rows are cut into chunks of 128, and the
// chunks of all units lie on one line that is cut evenly over the CTAs, wherever a unit
// begins or ends: ragged lengths balance by themselves.  A unit that lies inside one
// CTA is finished there; the others leave (maximum, sum, O) of each part in the
// workspace for k8_join_kernel.
// A warp takes 32 rows of a chunk per step (two halves of 16, each within one page and
// one block, so with one scale) through a pipeline of its own (TMA boxes, no block
// barrier), keeps its own running maximum, sum and O, and the four warps meet once per
// unit.
// Codes become halves in registers right before the MMA (m16n8k16; exact): K from 16-byte
// reads of its rows, with the head dimension permuted alike in Q; V through transposed
// ldmatrix of byte pairs, two output columns per 16-bit element.  (The fp8 m16n8k32 on
// the codes themselves, with Q and P as sums of e5m2 terms, measured 1.8 times slower:
// 499 against 273 us on 645 k rows of 8 heads at 128 / 128.)
// Scales.  Q is held times a power of two per row (what lies 2^-30 below the row's
// largest is lost).  V's scale goes into the exponent: with w_j = s_j + log2 vs_j the
// products use p'_j = 2^(w_j - max w), and the sum gets p'_j / vs_j.  So P needs one
// exponential, and its 11 bits sit where the products are largest whatever the pages'
// scales are.  p' <= 2^15: the maximum is held at 2^7 and let grow by up to 2^8 before O is
// rescaled; halves reach 2^-31 of the held one.
// Measured: 32 requests of 8 k to 32 k rows, 64 / 8 heads of 128 / 128, 1.32 GB: 273 to 278 us,
// 4.8 TB/s of a copy's 6.55; bound by the issue slots close behind memory.  16 requests of
// up to 8 k rows: 43 us, of which start and join are 16.  One of 65536 rows, 4 heads of 192 / 128: 31.
constexpr int kK8Warps = 4;
constexpr int kK8Chunk = 32 * kK8Warps;
constexpr float kK8Grow = 8.f, kK8Top = 7.f;

// A unit, or a share's part of it, as its warps know it.
struct alignas(16) K8Unit {
  const int* idx;    // the token's indices (where it selects)
  const int* table;  // the sequence's pages
  long long begin;   // of the whole unit on the line
  int slots, L;      // usable indices; rows of the sequence
  int start, lo, hi; // the unit's first step, and the rows that any of its tokens sees
  int h, t0, ntok, ta0, head0, rows;  // KV head, first token, tokens, its row, first query head, query rows
  int c0, c1, ch;    // chunks of this part, and of the unit
};

template <int DK, int DV, bool ROWS, int FMT>
struct K8Split {
  static constexpr int kData = 32 * (DK + DV);
  static constexpr int kMeta = ROWS ? 384 : 32;  // rows and scales of a step
  static constexpr int kStages = DK + DV <= 128 ? 3 : 2;
  static constexpr int kOcc = DK + DV <= 128 ? 4 : (DK <= 128 ? 3 : 2);
  static constexpr int kRing = 8;         // units a warp may be ahead: kStages + 2 steps, and one in hand
  static constexpr int kQ = DK / 16 * 512;  // Q in the MMA's order: 16 bytes per lane and k step
  static constexpr int kQAt = kK8Warps * kStages * kData;
  static constexpr int kMetaAt = kQAt + kQ;
  static constexpr int kUnitAt = kMetaAt + kK8Warps * kStages * kMeta;
  static constexpr int kBarAt = kUnitAt + kK8Warps * kRing * (int)sizeof(K8Unit);
  static constexpr int kSmem = kBarAt + kK8Warps * kStages * 8 + 1024;  // the swizzles want 1024-byte alignment
  static_assert(16 * DV * 4 <= kData, "a warp's O must fit in a stage");
  static_assert(kStages + 3 <= kRing, "");
};
struct K8Maps {
  CUtensorMap k, k2, v;  // columns 0 .. 127 (or 63) of K, columns 128 .. 191, V
};

// Byte of 16-byte piece p of row r in a half step's 16 rows, as the TMA swizzles lay them.
template <int D>
__device__ __forceinline__ int k8_at(int r, int p) {
  if (D == 64) return r * 64 + ((p ^ ((r >> 1) & 3)) << 4);
  if (D == 128) return r * 128 + ((p ^ (r & 7)) << 4);
  return p < 8 ? r * 128 + ((p ^ (r & 7)) << 4) : 2048 + r * 64 + (((p - 8) ^ ((r >> 1) & 3)) << 4);
}
// The MMA's row n of 8 is row k8_row(n) of the step, so that the 16-byte reads of two
// rows' four neighbouring pieces fall on different banks: rows r and r + 4 of 128
// bytes, rows r and r + 1 of 64.
template <int DK>
__device__ __forceinline__ int k8_row(int n) {
  return DK == 64 ? n : (n >> 1) | ((n & 1) << 2);
}

__device__ __forceinline__ float2 k8_two(uint32_t v, int f16) {
  return f16 ? __half22float2(*reinterpret_cast<const __half2*>(&v))
             : make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint32_t k8_halves(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t k8_hsub2(uint32_t x, uint32_t y) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A word of four codes as halves: bytes (0, 1) and (2, 3).  e4m3 by conversion; int8 as 1024 +
// (code + 128), which is the byte under 0x64, less 1152 (exact).
template <int FMT>
__device__ __forceinline__ void k8_pair(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kFmtE4M3) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    lo = k8_hsub2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = k8_hsub2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  }
}
template <int FMT>
__device__ __forceinline__ void k8_pair_t(uint32_t w, uint32_t& even, uint32_t& odd) {  // bytes (0, 2) and (1, 3)
  if (FMT == kFmtE4M3) {
    k8_pair<FMT>(__byte_perm(w, 0, 0x3120), even, odd);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    even = k8_hsub2(__byte_perm(u, 0x64646464u, 0x4240), 0x64806480u);
    odd = k8_hsub2(__byte_perm(u, 0x64646464u, 0x4341), 0x64806480u);
  }
}
__device__ __forceinline__ void k8_mma(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void k8_cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void k8_cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ float k8_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float k8_log2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void k8_box(uint32_t dst, const CUtensorMap* map, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
// 16 rows of which lane (from + r) holds the row of the cache (negative: zeros)
template <int D>
__device__ __forceinline__ void k8_copy_rows(uint32_t dst, const uint8_t* src, int rs, int rr, int from, int lane) {
#pragma unroll
  for (int it = 0; it < D / 32; ++it) {
    const int i = it * 32 + lane, r = i / (D / 16), pc = i - r * (D / 16);
    const int at = __shfl_sync(~0u, rr, from + r);
    cp_async16(dst + k8_at<D>(r, pc), src + (long long)(at >= 0 ? at : 0) * rs + pc * 16, at >= 0);
  }
}

// A unit that spans several CTAs, as each of them notes it.  Output row r is token
// t + r / gdiv, head head + r % gdiv.
struct K8Join {
  int n;      // CTAs that hold a part of the unit; 0: nothing to join
  int first;  // the first of them
  int t, head, rows, gdiv;
};
// The workspace: two K8Join per CTA (the unit in whose midst its share begins; the unit
// that begins in its share and ends behind it), then these units' parts, two per CTA:
// maxima and sums of a unit's rows (16, or 16 MT), and O [rows][DV].
__host__ __device__ inline size_t k8_parts_at(int n_cta) {
  return ((size_t)n_cta * 2 * sizeof(K8Join) + 255) / 256 * 256;
}
__host__ __device__ inline size_t k8_part_floats(int rows, int dv) { return (size_t)rows * (2 + dv); }
__device__ __forceinline__ float* k8_part(float* ws, int n_cta, int i, int rows, int dv) {
  return reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + k8_parts_at(n_cta)) + i * k8_part_floats(rows, dv);
}

// n chunks shared evenly over CTAs: the first `rem` of them have one more.  Or, with a.per_unit,
// units of a.sel_ch chunks (fewer than 2^28 in all) over that many CTAs each.
struct K8Share {
  long long base;
  int rem;
  __device__ long long at(const K8Fwd& a, int i) const {
    if (a.per_unit) {
      const int u = k8_quot(a.by_per, i);
      return u * a.sel_ch + k8_quot(a.by_per, (i - u * a.per_unit) * a.sel_ch);
    }
    return base * i + min(i, rem);
  }
  __device__ int of(const K8Fwd& a, long long w) const {
    if (a.per_unit) {
      const int u = k8_quot(a.by_ch, (int)w);
      return u * a.per_unit + k8_quot(a.by_ch, ((int)w - u * a.sel_ch + 1) * a.per_unit - 1);
    }
    const long long head = (base + 1) * rem;
    return (int)(w < head ? w / (base + 1) : rem + (w - head) / base);
  }
};

// sink: a head's sink logit times log2(e), -inf for none.
__device__ __forceinline__ float k8_sink(const K8Fwd& a, int head) {
  return a.sinks ? k8_read(a.sinks + head) * 1.4426950408889634f : -INFINITY;
}
// What an output row's O is multiplied by, from its maximum, sum and sink; and its lse.
__device__ __forceinline__ float k8_norm(float sink, float m, float l, float* lse) {
  float base = m == -INFINITY ? m : m - kK8Top, f = 1.f;
  if (sink != -INFINITY) {
    const float top = fmaxf(base, sink);
    f = ex2_approx(base - top);
    l = l * f + ex2_approx(sink - top);
    base = top;
  }
  *lse = l == 0.f ? INFINITY : 0.6931471805599453f * (base + log2f(l));
  return l == 0.f ? 0.f : f / l;
}
__device__ __forceinline__ void k8_store(const K8Fwd& a, int t, int head, int d, float f, float4 o) {
  uint2 out;
  if (a.f16) {
    const __half2 x = __floats2half2_rn(o.x * f, o.y * f), y = __floats2half2_rn(o.z * f, o.w * f);
    out = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    out = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
  }
  *reinterpret_cast<uint2*>(static_cast<char*>(a.o) + (((long long)t * a.Hq + head) * a.c.dv + d) * 2) = out;
}

// units and chunks per unit of a sequence
struct K8Span {
  K8Seq s;
  int units, ch;
  int per_h;  // units of a KV head
  int len;    // a unit on the line: its chunks, and a.over for what a unit costs besides
};
__device__ __forceinline__ K8Span k8_span(const K8Fwd& a, int b) {
  K8Span r;
  r.s = k8_seq(a.c, b);
  r.per_h = k8_quot(a.by_tpt, r.s.n + a.tpt - 1) * a.hs;
  r.units = r.per_h * a.c.Hkv;
  if (a.sel_ch) {
    r.ch = a.sel_ch;
  } else {
    r.ch = max((r.s.L + a.chunk - 1) / a.chunk, 1);
    // a window: from the step of 16 that its first row lies in
    if (a.win < (1 << 29)) r.ch = min(r.ch, (a.win + a.tpt + 15 + a.chunk - 1) / a.chunk);
  }
  r.len = r.ch + a.over;
  return r;
}

// a / b for 0 <= a < 2^31, 1 <= b: an approximate quotient, then put right (an exact division is a chain
// of some hundred dependent instructions, in front of everything else here).
__device__ __forceinline__ uint32_t k8_udiv(uint32_t a, uint32_t b) {
  uint32_t q = (uint32_t)__fdividef((float)a, (float)b);
  while (q * (unsigned long long)b > a) --q;
  while ((q + 1ull) * b <= a) ++q;
  return q;
}

// Where a CTA stands on the line.
struct K8Cursor {
  long long w0, w1;  // its share
  K8Share share;
  long long seq_at;  // where the sequence begins
  int b, h, ut, c0;  // sequence, KV head, unit of the head, first chunk of the unit
  K8Span sp;
};
struct K8Found {
  long long sum[8];
  long long at, w0, w1;
  int b, h, ut, c0;
  K8Span sp;
};
// The line's length, this CTA's share and the unit that it begins in; false: it has none.
// NT threads look at the sequences; threads behind them come along.
template <int NT>
__device__ __forceinline__ bool k8_begin(const K8Fwd& a, float* ws, int tid, K8Found& f, K8Cursor& cur) {
  const int lane = tid & 31, warp = tid >> 5, B = a.c.B;
  const int per = (B + NT - 1) / NT, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long mine = 0;
  K8Span sp = {};
  for (int b = b0; b < b1; ++b) {
    sp = k8_span(a, b);
    mine += (long long)sp.units * sp.len;
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31 && warp < NT / 32) f.sum[warp] = inc;
  __syncthreads();
  long long W = 0, at = inc - mine;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    W += f.sum[x];
    if (x < warp) at += f.sum[x];
  }
  int n_cta = (int)min(W, (long long)gridDim.x);  // a share is empty only in CTAs behind these
  if (a.per_unit) n_cta = min(k8_quot(a.by_ch, (int)min(W, 148ll * a.sel_ch)) * a.per_unit, (int)gridDim.x);
  if (tid < 2) (reinterpret_cast<K8Join*>(ws) + 2 * blockIdx.x)[tid].n = 0;
  if (blockIdx.x >= n_cta) return false;
  if (a.per_unit) {
    cur.share.base = cur.share.rem = 0;
  } else if (W <= 0x7fffffff) {
    cur.share.base = k8_udiv((uint32_t)W, (uint32_t)n_cta);
    cur.share.rem = (int)((uint32_t)W - (uint32_t)cur.share.base * (uint32_t)n_cta);
  } else {
    cur.share.base = W / n_cta;
    cur.share.rem = (int)(W % n_cta);
  }
  // This share's two ends, each put where a unit can be cut: not within its first a.over, and not at
  // all in a unit of up to a.keep chunks while a CTA has such a unit or more.  (Both CTAs at
  // an end see it alike.)
  const long long ends[2] = {cur.share.at(a, blockIdx.x), cur.share.at(a, blockIdx.x + 1)};
  if (tid == 0 && ends[1] >= W) f.w1 = W;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (!(at <= ends[e] && ends[e] < at + mine)) continue;
    long long from = at;
    for (int b = b0;; ++b) {
      if (b1 - b0 > 1) sp = k8_span(a, b);
      const long long n = (long long)sp.units * sp.len;
      if (ends[e] >= from + n) {
        from += n;
        continue;
      }
      const long long off = ends[e] - from;
      const int unit = off <= 0x7fffffff ? (int)k8_udiv((uint32_t)off, (uint32_t)sp.len) : (int)(off / sp.len);
      int pos = (int)(off - (long long)unit * sp.len);
      if (sp.ch <= a.keep && cur.share.base >= sp.len) pos = 2 * pos < sp.len ? 0 : sp.len;
      else if (pos <= a.over) pos = 0;
      (e ? f.w1 : f.w0) = from + (long long)unit * sp.len + pos;
      if (e == 0) {
        f.at = from;
        f.sp = sp;
        f.b = b;
        f.h = (int)k8_udiv((uint32_t)unit, (uint32_t)sp.per_h);
        f.ut = unit - f.h * sp.per_h;
        f.c0 = pos == 0 || pos == sp.len ? 0 : pos - a.over;
        if (pos == sp.len && ++f.ut == sp.per_h) {
          f.ut = 0;
          ++f.h;
        }
      }
      break;
    }
  }
  __syncthreads();
  cur.w0 = f.w0;
  cur.w1 = f.w1;
  cur.seq_at = f.at;
  cur.sp = f.sp;
  cur.b = f.b;
  cur.h = f.h;
  cur.ut = f.ut;
  cur.c0 = f.c0;
  return cur.w0 < cur.w1;
}
__device__ __forceinline__ void k8_settle(const K8Fwd& a, K8Cursor& c) {  // to the next sequence with work
  while (c.h >= a.c.Hkv || c.sp.units == 0) {
    c.seq_at += (long long)c.sp.units * c.sp.len;
    c.sp = k8_span(a, ++c.b);
    c.h = 0;
  }
}
__device__ __forceinline__ void k8_next(K8Cursor& c) {
  c.c0 = 0;
  if (++c.ut == c.sp.per_h) {
    c.ut = 0;
    ++c.h;
  }
}
// Notes that this CTA leaves a part of a unit of length len that begins at `begin`; c0: the part's first chunk.
__device__ __forceinline__ void k8_note(const K8Fwd& a, float* ws, const K8Share& share, long long begin, int c0, int len,
                                        int t, int head, int rows, int gdiv) {
  K8Join jn;
  jn.first = c0 == 0 ? (int)blockIdx.x : share.of(a, begin + a.over);
  jn.n = share.of(a, begin + len - 1) - jn.first + 1;
  jn.t = t;
  jn.head = head;
  jn.rows = rows;
  jn.gdiv = gdiv;
  (reinterpret_cast<K8Join*>(ws) + 2 * blockIdx.x)[c0 == 0] = jn;
}
// The unit at the cursor, which moves on.
__device__ __forceinline__ K8Unit k8_take(const K8Fwd& a, K8Cursor& cur) {
  k8_settle(a, cur);
  const K8Span& sp = cur.sp;
  K8Unit u;
  u.h = cur.h;
  u.c0 = cur.c0;
  u.ch = sp.ch;
  u.c1 = (int)min((long long)sp.ch, cur.c0 + (cur.w1 - cur.w0) - (cur.c0 ? 0 : a.over));
  u.begin = cur.seq_at + ((long long)cur.h * sp.per_h + cur.ut) * sp.len;
  // a KV head's units lie together, a token's parts of the heads innermost
  const int tile = a.hs == 1 ? cur.ut : cur.ut / a.hs, hp = cur.ut - tile * a.hs;
  u.t0 = sp.s.t0 + tile * a.tpt;
  u.ntok = min(a.tpt, sp.s.n - tile * a.tpt);
  u.head0 = cur.h * a.G + hp * a.unit_rows;
  u.rows = a.hs > 1 ? min(a.unit_rows, a.G - hp * a.unit_rows) : u.ntok * a.G;
  u.ta0 = sp.s.first + tile * a.tpt;
  const int ta1 = u.ta0 + u.ntok - 1;  // rows of the first and last token
  u.L = sp.s.L;
  u.lo = a.win >= u.ta0 ? 0 : u.ta0 - a.win;
  u.hi = min(ta1 + 1, u.L);
  u.start = u.lo & ~15;
  const long long iu = (long long)u.t0 * a.c.Hkv + u.h;
  u.idx = a.topk ? a.idx + iu * a.topk : nullptr;
  u.slots = a.topk;
  if (a.topk && a.topk_len) u.slots = min(u.slots, max(0, k8_read(a.topk_len + iu)));
  u.table = a.c.table + cur.b * a.c.tstride;
  cur.w0 += u.c1 - u.c0 + (u.c0 ? 0 : a.over);
  k8_next(cur);
  return u;
}

template <int DK, int DV, bool ROWS, int FMT>
__global__ void __launch_bounds__(128, K8Split<DK, DV, ROWS, FMT>::kOcc)
    k8_split_kernel(const __grid_constant__ K8Fwd a, const __grid_constant__ K8Maps maps, float* ws) {
  using P = K8Split<DK, DV, ROWS, FMT>;
  constexpr int S = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  __shared__ int dead_word;
  __shared__ float q_scale[16];
  __shared__ float meet[kK8Warps][32];  // maxima and sums of a unit's rows
  const K8Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, q4 = lane & 3;
  if (tid == 0) dead_word = 0;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + P::kBarAt) + warp * S;
  if (!ROWS) {
    if (lane < S) mbar_init(bars + lane, 1);
    mbar_fence_init();
  }
  pdl_trigger();  // the join waits for this kernel's end, but need not be launched after it
  pdl_wait();

  __shared__ K8Found found;
  K8Cursor cur;
  if (!k8_begin<128>(a, ws, tid, found, cur)) return;
  long long left = cur.w1 - cur.w0;  // of the share

  uint8_t* const wsm = smem + warp * S * P::kData;
  uint32_t* const sq = reinterpret_cast<uint32_t*>(smem + P::kQAt);
  uint8_t* const wmeta = smem + P::kMetaAt + warp * S * P::kMeta;
  const K8Unit* const units = reinterpret_cast<const K8Unit*>(smem + P::kUnitAt) + warp * P::kRing;
  const uint32_t sbase = smem_u32(wsm), mbase = smem_u32(wmeta), bar0 = smem_u32(bars);
  uint32_t phases = 0;  // of this warp's barriers
  int dead = 0;         // a wait gave up: no more copies, and NaN for a result
  const int krs = c.Hkv * DK, vrs = c.Hkv * DV;  // bytes from row to row of the cache

  // --- The warp's fetching runs ahead of its computing, over the units of the share: a step's
  // index is asked for two steps before its rows, and its page one.  Lane x of 32 (ROWS) or
  // of 2 resolves row (or half) x of a step. ---
  const int lane_row = warp * 32 + (ROWS ? lane : (lane & 1) * 16);
  int fu = P::kRing - 1, fk = 0, fn = 0;  // the fetch's unit (ring slot), step of it, steps of it
  auto advance = [&]() {                  // to the next step; fn = 0: none is left
    if (++fk < fn) return;
    fk = fn = 0;
    if (cur.w0 >= cur.w1) return;
    fu = (fu + 1) & (P::kRing - 1);
    const K8Unit u = k8_take(a, cur);
    if (lane == 0) const_cast<K8Unit*>(units)[fu] = u;
    fn = u.c1 - u.c0;
    __syncwarp();
  };
  auto fetch_idx = [&](int un, int k) -> int {  // of step k of unit un; un < 0: no step
    if (!a.topk || un < 0) return 0;
    const K8Unit& u = units[un];
    const int slot = k8_quot(a.by_bs, (u.c0 + k) * kK8Chunk + lane_row);
    return slot < u.slots ? k8_read(u.idx + slot) : -1;
  };
  auto resolve = [&](int un, int k, int x) -> int {  // its (first) row, -1: none
    if (un < 0) return -1;
    const K8Unit& u = units[un];
    const int p = (u.c0 + k) * kK8Chunk + lane_row;
    int row = u.start + p;
    if (a.topk) {
      if (x < 0) return -1;
      if ((long long)x * a.bs >= u.L) {
        if (c.status) atomicOr(c.status, kStatusIndexRange);
        return -1;
      }
      row = x * a.bs + k8_rem(a.by_bs, p);
    }
    const int last = ROWS ? row : row + 15;
    return row < u.hi && last >= u.lo ? row : -1;
  };
  auto fetch_page = [&](int un, int row) -> int {
    return row >= 0 ? k8_read(units[un].table + k8_quot(c.by_ps, row)) : 0;
  };
  int fx = 0, f_row = -1, f_page = 0, f_head = 0;
  // the page of the step that the fetch stands at, then the index of the one behind it
  auto look = [&]() {
    const int un = fn ? fu : -1;
    f_row = resolve(un, fk, fx);
    f_page = fetch_page(un, f_row);
    if (fn) f_head = units[fu].h;
    advance();
    fx = fetch_idx(fn ? fu : -1, fk);
  };
  auto issue = [&](int st, int row, int page, int head) {  // into stage st
    if (row >= 0 && (page < 0 || page >= c.n_pages)) {
      if (c.status) atomicOr(c.status, kStatusIndexRange);
      row = -1;
    }
    const uint32_t dst = sbase + st * P::kData, meta = mbase + st * P::kMeta;
    int* im = reinterpret_cast<int*>(wmeta + st * P::kMeta);
    const int rr = row >= 0 ? page * c.ps + k8_rem(c.by_ps, row) : -1;  // row of the cache
    const long long sc = (long long)page * c.Hkv + head;
    if (ROWS) {
      im[lane] = row;
      if (row >= 0) {
        k8_cp4(meta + 128 + 4 * lane, c.ks + sc);
        k8_cp4(meta + 256 + 4 * lane, c.vs + sc);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        k8_copy_rows<DK>(dst + x * 16 * DK, c.k + head * DK, krs, rr, 16 * x, lane);
        k8_copy_rows<DV>(dst + 32 * DK + x * 16 * DV, c.v + head * DV, vrs, rr, 16 * x, lane);
      }
    } else {
      const int both = (row >= 0) + __shfl_xor_sync(~0u, row >= 0, 1);
      if (lane == 0 && both) mbar_arrive_tx(bars + st, both * 16 * (DK + DV));
      __syncwarp();
      if (lane < 2) {
        im[lane] = row;
        if (row >= 0) {
          k8_cp4(meta + 8 + 4 * lane, c.ks + sc);
          k8_cp4(meta + 16 + 4 * lane, c.vs + sc);
          const uint32_t bar = bar0 + st * 8, kd = dst + lane * 16 * DK;
          k8_box(kd, &maps.k, head, rr, bar);
          if (DK == 192) k8_box(kd + 2048, &maps.k2, head, rr, bar);
          k8_box(dst + 32 * DK + lane * 16 * DV, &maps.v, head, rr, bar);
        }
      }
    }
  };

  // --- Q of a unit: warp w brings rows 4 w .. 4 w + 3, 8 lanes a row ---
  constexpr int kQw = DK / 64;  // 16-byte pieces of a lane: piece qp + 8 i of the row
  const int qrow = warp * 4 + (lane >> 3), qp = lane & 7;
  uint4 raw[kQw];
  auto load_q = [&](const K8Unit& u) {
    const int tok = k8_quot(a.by_gdiv, qrow);
    const char* src = static_cast<const char*>(a.q) +
                      ((long long)(u.t0 + tok) * a.qstride + (long long)(u.head0 + qrow - tok * a.gdiv) * DK) * 2;
#pragma unroll
    for (int i = 0; i < kQw; ++i)
      raw[i] = qrow < u.rows ? k8_read(reinterpret_cast<const uint4*>(src + (qp + 8 * i) * 16)) : make_uint4(0, 0, 0, 0);
  };
  auto lay_q = [&]() {
    // halves times 2^(14 - E), E the exponent of the row's largest, in the MMA's order
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < kQw; ++i) {
      const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = k8_two(v[j], a.f16);
        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
    const int E = big > 0.f ? max((int)(__float_as_uint(big) >> 23) - 127, -110) : 14;
    const float mul = __uint_as_float((uint32_t)(14 - E + 127) << 23);
    if (qp == 0) q_scale[qrow] = a.scale_log2 * __uint_as_float((uint32_t)(E - 14 + 127) << 23);
#pragma unroll
    for (int i = 0; i < kQw; ++i) {
      // columns 64 i + 8 qp .. + 7, that is 16 q4' + 8 x with q4' = qp / 2, x = qp % 2
      const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t hh[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = k8_two(v[j], a.f16);
        hh[j] = k8_halves(f.x * mul, f.y * mul);
      }
      // the lane that holds row qrow % 8 and columns q4' of the MMA; register r (+ 2 for the upper k);
      // 4 columns are k 2 q4' + {0, 1 | 8, 9} of k step 4 i + 2 x + {0, 1}
      const int to = (qrow & 7) * 4 + (qp >> 1), r = qrow >> 3;
      uint32_t* dst = sq + ((4 * i + 2 * (qp & 1)) * 32 + to) * 4 + r;
      dst[0] = hh[0];
      dst[2] = hh[1];
      dst[128] = hh[2];
      dst[130] = hh[3];
    }
  };

  {
    // the first S steps, their indices and then their pages asked for together
    int us[S + 2], ks[S + 2], xs[S + 2], rw[S + 1], pg[S + 1], hd[S + 1];
#pragma unroll
    for (int k = 0; k < S + 2; ++k) {
      advance();
      us[k] = fn ? fu : -1;
      ks[k] = fk;
      xs[k] = fetch_idx(us[k], fk);
      if (k == 0) load_q(units[fu]);
    }
#pragma unroll
    for (int k = 0; k < S + 1; ++k) {
      rw[k] = resolve(us[k], ks[k], xs[k]);
      pg[k] = fetch_page(us[k], rw[k]);
      hd[k] = us[k] >= 0 ? units[us[k]].h : 0;
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      issue(k, rw[k], pg[k], hd[k]);
      cp_async_commit();
    }
    f_row = rw[S];
    f_page = pg[S];
    f_head = hd[S];
    fx = xs[S + 1];
  }
  lay_q();
  __syncthreads();

  int at = 0;
  for (int un = 0; left > 0; un = (un + 1) & (P::kRing - 1)) {
    const K8Unit& u = units[un];
    const int n_steps = u.c1 - u.c0, ta0 = u.ta0;
    left -= n_steps + (u.c0 ? 0 : a.over);
    const int lo_last = max(0, ta0 + u.ntok - 1 - a.win);
    int ta[2], lo[2];  // of this thread's rows gr and gr + 8
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ta[r] = ta0 + min(k8_quot(a.by_gdiv, gr + 8 * r), u.ntok - 1);
      lo[r] = max(0, ta[r] - a.win);
    }
    const float sink = (tid >> 3) < u.rows ? k8_sink(a, u.head0 + k8_rem(a.by_gdiv, tid >> 3)) : -INFINITY;
    const float fr[2] = {q_scale[gr], q_scale[gr + 8]};

    float o[DV / 16][2][4];
#pragma unroll
    for (int i = 0; i < DV / 16; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][e][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float base[2] = {0.f, 0.f}, limit[2] = {-INFINITY, -INFINITY};  // m - kK8Top, and how far above it w may lie

    for (int k = 0; k < n_steps; ++k) {
      k8_cp_wait<S - 1>();
      __syncwarp();
      uint8_t* const st = wsm + at * P::kData;
      uint8_t* const stv = st + 32 * DK;
      const uint32_t sv = sbase + at * P::kData + 32 * DK;
      const int* im = reinterpret_cast<const int*>(wmeta + at * P::kMeta);
      int row0[2] = {ROWS ? 0 : im[0], ROWS ? 0 : im[1]};
      bool any = !dead && (ROWS ? __any_sync(~0u, im[lane] >= 0) : row0[0] >= 0 || row0[1] >= 0);
      if (!ROWS && any) {
        const uint32_t parity = (phases >> at) & 1;
        if (!__all_sync(~0u, mbar_try_wait(bars + at, parity)) &&
            !__all_sync(~0u, mbar_wait(bars + at, parity, &dead_word, c.status))) {
          dead = 1;
          any = false;
        }
        phases ^= (uint32_t)any << at;
      }
      if (any) {
        // --- scores of 32 rows: tiles 0, 1 of the first half, 2, 3 of the second ---
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        const uint4* q = reinterpret_cast<const uint4*>(sq) + lane;
#pragma unroll
        for (int ch = 0; ch < DK / 64; ++ch) {
          uint4 kw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            kw[j] = *reinterpret_cast<const uint4*>(st + (j >> 1) * 16 * DK +
                                                    k8_at<DK>(8 * (j & 1) + k8_row<DK>(gr), ch * 4 + q4));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 qa = q[(4 * ch + e) * 32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b0, b1;
              k8_pair<FMT>(e == 0 ? kw[j].x : e == 1 ? kw[j].y : e == 2 ? kw[j].z : kw[j].w, b0, b1);
              k8_mma(s[j], qa, b0, b1);
            }
          }
        }

        // --- w = score + log2 of V's scale, less what the exponential's argument starts from;
        // what a row does not see becomes -inf ---
        float iv[4][2];  // 1 / V's scale: per half, or per row
        bool full = !ROWS;
        if (!ROWS) {
          const float* fm = reinterpret_cast<const float*>(im);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float ks = k8_scale(fm[2 + x]), vs = k8_scale(fm[4 + x]);
            const float f0 = fr[0] * ks, f1 = fr[1] * ks, lv = k8_log2(vs), a0 = lv - base[0], a1 = lv - base[1];
            iv[x][0] = k8_rcp(vs);
#pragma unroll
            for (int j = 2 * x; j < 2 * x + 2; ++j) {
              s[j][0] = fmaf(s[j][0], f0, a0);
              s[j][1] = fmaf(s[j][1], f0, a0);
              s[j][2] = fmaf(s[j][2], f1, a1);
              s[j][3] = fmaf(s[j][3], f1, a1);
            }
            full = full && row0[x] >= lo_last && row0[x] + 15 <= ta0;
          }
          if (!full) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int pos = row0[j >> 1] + 8 * (j & 1) + k8_row<DK>(2 * q4 + (e & 1));
                if (row0[j >> 1] < 0 || pos > ta[e >> 1] || pos < lo[e >> 1]) s[j][e] = -INFINITY;
              }
          }
        } else {
          const float* fm = reinterpret_cast<const float*>(im);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = 8 * j + k8_row<DK>(2 * q4 + e), pos = im[col];
              const float ks = k8_scale(fm[32 + col]), vs = k8_scale(fm[64 + col]), lv = k8_log2(vs);
              iv[j][e] = k8_rcp(vs);
              s[j][e] = pos >= 0 && pos <= ta[0] && pos >= lo[0] ? fmaf(s[j][e], fr[0] * ks, lv - base[0]) : -INFINITY;
              s[j][e + 2] =
                  pos >= 0 && pos <= ta[1] && pos >= lo[1] ? fmaf(s[j][e + 2], fr[1] * ks, lv - base[1]) : -INFINITY;
            }
        }
        if (FMT == kFmtE4M3 && !full) {
          // A NaN in a V row that some of the unit's rows do not see (a stale row of the page,
          // a later token's): the product would carry it (0 * NaN) to all of them.  It is set
          // into the rows that see it here, and out of the tile.  (A half without rows, which
          // holds whatever the stage did before, becomes zeros.)
          if (!ROWS && (row0[0] < 0 || row0[1] < 0)) {
            for (int i = lane; i < DV; i += 32)
              *reinterpret_cast<uint4*>(stv + (row0[0] < 0 ? 0 : 16 * DV) + i * 16) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
          }
          uint32_t nan = 0;
#pragma unroll
          for (int i = 0; i < DV / 16; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(stv + (i * 32 + lane) * 16);
            nan |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                   ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
          }
          if (__any_sync(~0u, nan & 0x80808080u)) {
#pragma unroll 1
            for (int r = 0; r < 32; ++r) {
              const int first = r < 16 ? row0[0] : row0[1];
              const int pos = ROWS ? im[r] : first < 0 ? -1 : first + (r & 15);
              const bool see[2] = {pos >= 0 && pos <= ta[0] && pos >= lo[0], pos >= 0 && pos <= ta[1] && pos >= lo[1]};
#pragma unroll
              for (int pc = 0; pc < DV / 16; ++pc) {
                const uint32_t v =
                    *reinterpret_cast<const uint32_t*>(stv + (r >> 4) * 16 * DV + k8_at<DV>(r & 15, pc) + 4 * q4);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  if (((v >> (8 * x)) & 0x7f) != 0x7f) continue;
                  if (see[0]) o[pc][x & 1][x >> 1] = __int_as_float(0x7fffffff);
                  if (see[1]) o[pc][x & 1][2 + (x >> 1)] = __int_as_float(0x7fffffff);
                }
              }
            }
            __syncwarp();
            for (int i = lane; i < 8 * DV; i += 32) {
              uint32_t* v = reinterpret_cast<uint32_t*>(stv) + i;
              *v &= ~__vcmpeq4(*v & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
            fence_async_smem();  // the next copy into this stage comes behind these writes
            __syncwarp();
          }
        }

        // --- the running maximum; O is rescaled only when it grew by more than 2^kK8Grow ---
        float mx[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
          for (int j = 1; j < 4; ++j) mx[r] = fmaxf(mx[r], fmaxf(s[j][2 * r], s[j][2 * r + 1]));
        }
        if (__any_sync(~0u, mx[0] > limit[0] || mx[1] > limit[1])) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
            const float mn = fmaxf(m[r], mx[r] + base[r]);
            if (mn == -INFINITY) continue;
            const float al = ex2_approx(m[r] - mn), shift = base[r] - (mn - kK8Top);
            m[r] = mn;
            base[r] = mn - kK8Top;
            limit[r] = kK8Top + kK8Grow;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[j][2 * r] += shift;
              s[j][2 * r + 1] += shift;
            }
            l[r] *= al;
#pragma unroll
            for (int i = 0; i < DV / 16; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                o[i][e][2 * r] *= al;
                o[i][e][2 * r + 1] *= al;
              }
          }
        }
        uint32_t ph[4][2];  // p' as halves: rows gr, gr + 8 of each tile
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = ex2_approx(s[j][e]);
          ph[j][0] = k8_halves(s[j][0], s[j][1]);
          ph[j][1] = k8_halves(s[j][2], s[j][3]);
          if (ROWS) {
            l[0] = fmaf(s[j][0], iv[j][0], fmaf(s[j][1], iv[j][1], l[0]));
            l[1] = fmaf(s[j][2], iv[j][0], fmaf(s[j][3], iv[j][1], l[1]));
          }
        }
        if (!ROWS) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            l[0] = fmaf((s[2 * x][0] + s[2 * x][1]) + (s[2 * x + 1][0] + s[2 * x + 1][1]), iv[x][0], l[0]);
            l[1] = fmaf((s[2 * x][2] + s[2 * x][3]) + (s[2 * x + 1][2] + s[2 * x + 1][3]), iv[x][0], l[1]);
          }
        }

        // --- O += P V, a piece of 16 columns at a time ---
        const uint4 pt[2] = {make_uint4(ph[0][0], ph[0][1], ph[1][0], ph[1][1]),
                             make_uint4(ph[2][0], ph[2][1], ph[3][0], ph[3][1])};
#pragma unroll
        for (int pc = 0; pc < DV / 16; ++pc) {
          uint32_t v[4];  // tiles 0 .. 3
          ldsm_x4_t(v, sv + (lane >> 4) * 16 * DV + k8_at<DV>(k8_row<DK>(lane & 7) + (lane & 8), pc));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t e0, o0, e1, o1;
            k8_pair_t<FMT>(v[2 * x], e0, o0);
            k8_pair_t<FMT>(v[2 * x + 1], e1, o1);
            k8_mma(o[pc][0], pt[x], e0, e1);
            k8_mma(o[pc][1], pt[x], o0, o1);
          }
        }
      }
      if (k + 1 == n_steps) break;  // the last stage takes this warp's O first
      __syncwarp();                 // the stage has been read
      if (!dead) issue(at, f_row, f_page, f_head);
      cp_async_commit();
      look();
      at = at + 1 == S ? 0 : at + 1;
    }
    if (dead) l[0] = l[1] = __int_as_float(0x7fffffff);

    // --- the warps' results meet: maximum, sum, O (rows of DV floats, odd rows' 64-byte halves swapped) ---
    float* const fo = reinterpret_cast<float*>(wsm + at * P::kData);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
      const int row = gr + 8 * r;
      if (q4 == 0) {
        meet[warp][row] = m[r];
        meet[warp][16 + row] = l[r];
      }
#pragma unroll
      for (int i = 0; i < DV / 16; ++i)
        *reinterpret_cast<float4*>(fo + row * DV + 4 * ((4 * i + q4) ^ ((row & 1) << 2))) =
            make_float4(o[i][0][2 * r], o[i][1][2 * r], o[i][0][2 * r + 1], o[i][1][2 * r + 1]);
    }
    if (left > 0) load_q(units[(un + 1) & (P::kRing - 1)]);
    __syncthreads();
    {
      const int row = tid >> 3, part = tid & 7;
      // all warps have taken the same number of steps: the same stage holds their O
      const float* f0 = reinterpret_cast<const float*>(smem + at * P::kData);
      constexpr int kW = S * P::kData / 4;
      float mw[kK8Warps], top = -INFINITY, total = 0.f;
#pragma unroll
      for (int x = 0; x < kK8Warps; ++x) {
        mw[x] = meet[x][row];
        top = fmaxf(top, mw[x]);
      }
#pragma unroll
      for (int x = 0; x < kK8Warps; ++x) {
        mw[x] = top == -INFINITY ? 1.f : ex2_approx(mw[x] - top);
        total = fmaf(meet[x][16 + row], mw[x], total);
      }
      const bool whole = u.c0 == 0 && u.c1 == u.ch;
      float* const part_out = k8_part(ws, gridDim.x, 2 * blockIdx.x + (u.c0 == 0), 16, DV);
      if (row < u.rows) {
        const int tok = k8_quot(a.by_gdiv, row), t = u.t0 + tok, head = u.head0 + row - tok * a.gdiv;
        float lse, norm = 0.f;
        if (whole) norm = k8_norm(sink, top, total, &lse);
        if (whole && part == 0) a.lse[(long long)t * a.Hq + head] = lse;
#pragma unroll
        for (int i = 0; i < DV / 32; ++i) {
          const int col = part + 8 * i;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < kK8Warps; ++x) {
            const float4 y = *reinterpret_cast<const float4*>(f0 + x * kW + row * DV + 4 * (col ^ ((row & 1) << 2)));
            v.x = fmaf(y.x, mw[x], v.x);
            v.y = fmaf(y.y, mw[x], v.y);
            v.z = fmaf(y.z, mw[x], v.z);
            v.w = fmaf(y.w, mw[x], v.w);
          }
          if (whole) k8_store(a, t, head, 4 * col, norm, v);
          else *reinterpret_cast<float4*>(part_out + 32 + row * DV + 4 * col) = v;
        }
        if (!whole && part == 0) {
          part_out[row] = top;
          part_out[16 + row] = total;
        }
      }
      if (!whole && tid == 0)
        k8_note(a, ws, cur.share, u.begin, u.c0, u.ch + a.over, u.t0, u.head0, u.rows, a.gdiv);
    }
    if (left > 0) lay_q();  // every warp has taken the scores of this unit
    fence_async_smem();     // the copies that fill the stage again come behind these accesses
    __syncthreads();
    if (!dead) issue(at, f_row, f_page, f_head);
    cp_async_commit();
    look();
    at = at + 1 == S ? 0 : at + 1;
  }
  k8_cp_wait<0>();
  if (dead && !ROWS)
    for (int i = 0; i < S; ++i) mbar_wait_drain(bars + i, (phases >> i) & 1);
}

// The units that span several CTAs.  The n blocks that held a part of a unit share its
// rows: block x of them takes rows x, x + n, ...  Up to 8 parts, a warp sums a row's;
// more, the 8 warps take an eighth of a row's parts each.  The order is fixed.
template <int R, int DV>
__global__ void __launch_bounds__(256) k8_join_kernel(const K8Fwd a, float* ws, int n_grid) {
  constexpr int NV = DV < 128 ? 1 : DV / 128, kLanes = DV < 128 ? DV / 4 : 32;  // float4 of a lane, lanes
  __shared__ float sl[8];
  __shared__ float4 so[8][NV * kLanes];
  // No early launch of what comes behind: another attention's CTAs, placed while these still run, end up
  // unevenly on the SMs (381 instead of 272 us a call, one long decode step behind the other; 59 instead of 43,
  // one decode step).
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const K8Join jn = reinterpret_cast<const K8Join*>(ws)[2 * blockIdx.x + which];
    if (jn.n == 0) continue;
    const int step = jn.n <= 8 ? 1 : 8, mine = blockIdx.x - jn.first;
    auto part = [&](int x) { return k8_part(ws, n_grid, 2 * (jn.first + x) + (x == 0), R, DV); };
    for (int row = mine + (step == 1 ? warp * jn.n : 0); row < jn.rows; row += step == 1 ? 8 * jn.n : jn.n) {
      const int head = jn.head + row % jn.gdiv;
      const float sink = k8_sink(a, head);
      float top = -INFINITY, sum = 0.f;
      float4 v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = lane; x < jn.n; x += 32) top = fmaxf(top, __ldcg(part(x) + row));
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
#pragma unroll 4
      for (int x = step == 1 ? 0 : warp; x < jn.n; x += step) {
        const float* p = part(x);
        const float f = top == -INFINITY ? 1.f : ex2_approx(__ldcg(p + row) - top);
        sum = fmaf(__ldcg(p + R + row), f, sum);
        if (lane < kLanes) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(p + 2 * R + row * DV) + lane + 32 * i);
            v[i].x = fmaf(y.x, f, v[i].x);
            v[i].y = fmaf(y.y, f, v[i].y);
            v[i].z = fmaf(y.z, f, v[i].z);
            v[i].w = fmaf(y.w, f, v[i].w);
          }
        }
      }
      if (step == 8) {
        if (lane == 0) sl[warp] = sum;
        if (lane < kLanes)
#pragma unroll
          for (int i = 0; i < NV; ++i) so[warp][lane + 32 * i] = v[i];
        __syncthreads();
        if (warp == 0) {
#pragma unroll 1
          for (int x = 1; x < 8; ++x) {
            sum += sl[x];
            if (lane < kLanes) {
#pragma unroll
              for (int i = 0; i < NV; ++i) {
                const float4 y = so[x][lane + 32 * i];
                v[i].x += y.x;
                v[i].y += y.y;
                v[i].z += y.z;
                v[i].w += y.w;
              }
            }
          }
        }
      }
      if (step == 1 || warp == 0) {
        const int t = jn.t + row / jn.gdiv;
        float lse;
        const float norm = k8_norm(sink, top, sum, &lse);
        if (lane == 0) a.lse[(long long)t * a.Hq + head] = lse;
        if (lane < kLanes)
#pragma unroll
          for (int i = 0; i < NV; ++i) k8_store(a, t, head, 4 * (lane + 32 * i), norm, v[i]);
      }
      if (step == 8) __syncthreads();  // sl, so
    }
  }
}

static bool k8_latent(const K8Fwd& a) { return a.c.dqk > 192; }

// CTAs: all that the SMs hold at once, or as many as the longest possible line has chunks.
static int k8_ctas(const K8Fwd& a) {
  if (a.per_unit) return a.c.T * a.hs * a.c.Hkv * a.per_unit;
  const int occ = k8_latent(a) ? 1 : a.c.dqk + a.c.dv <= 128 ? 4 : (a.c.dqk <= 128 ? 3 : 2);
  const long long units = ((long long)(a.c.T + a.tpt - 1) / a.tpt + (a.tpt > 1 ? min(a.c.B, a.c.T) : 0)) * a.hs * a.c.Hkv;
  long long ch = a.sel_ch;
  if (!ch) {
    ch = ((long long)a.c.max_pages * a.c.ps + a.chunk - 1) / a.chunk;
    if (a.win < (1 << 29)) ch = min(ch, (long long)(a.win + a.tpt + 15 + a.chunk - 1) / a.chunk);
  }
  return (int)min((long long)148 * occ, units * max(ch, 1ll));
}

template <int DK, int DV, bool ROWS, int FMT>
static cudaError_t split_t(const K8Fwd& a, void* ws, cudaStream_t st) {
  using P = K8Split<DK, DV, ROWS, FMT>;
  auto k = k8_split_kernel<DK, DV, ROWS, FMT>;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(k, P::kSmem, done);
  if (e != cudaSuccess) return e;
  K8Maps maps;
  memset(&maps, 0, sizeof(maps));
  if (!ROWS) {
    const uint64_t rows = (uint64_t)a.c.n_pages * a.c.ps, heads = a.c.Hkv;
    if (!make_tmap_codes(&maps.k, a.c.k, rows, heads, DK, DK == 64 ? 64 : 128, 16) ||
        !make_tmap_codes(&maps.v, a.c.v, rows, heads, DV, DV, 16) ||
        (DK == 192 && !make_tmap_codes(&maps.k2, a.c.k + 128, rows, heads, 192, 64, 16)))
      return cudaErrorInvalidValue;
  }
  const int n = k8_ctas(a);
  count_launch();
  e = launch_pdl(k, (unsigned)n, 128, P::kSmem, st, a, maps, static_cast<float*>(ws));
  if (e != cudaSuccess || n == 1) return e;
  count_launch();
  return launch_pdl(k8_join_kernel<16, DV>, (unsigned)n, 256, 0, st, a, static_cast<float*>(ws), n);
}

template <int DK, int DV>
static cudaError_t split_d(const K8Fwd& a, void* ws, cudaStream_t st) {
  // steps of 16 rows lie in one page, and in one block, unless these sizes break them
  const bool rows = a.c.ps % 16 != 0 || (a.topk && a.bs % 16 != 0);
  if (a.c.fmt == kFmtE4M3)
    return rows ? split_t<DK, DV, true, kFmtE4M3>(a, ws, st) : split_t<DK, DV, false, kFmtE4M3>(a, ws, st);
  return rows ? split_t<DK, DV, true, kFmtInt8>(a, ws, st) : split_t<DK, DV, false, kFmtInt8>(a, ws, st);
}

// ---------------------------------------------------------------------------
// a shared row of 576 columns, V its first 512
// ---------------------------------------------------------------------------
// Up to 32 heads at a time (more than 32, where there is work for it: the next section).  A unit
// is one token and 16 MT of its heads, MT = 1 or 2; 64 rows per chunk and one CTA of 8 warps per
// SM, on the same line of chunks as above.  The rows, selected one by one, are copied whole
// (cp.async, three stages), and serve as K and V.  For the scores warp (mg, tg) takes 16 of the
// heads against its share of the rows; for O a warp takes all heads against 64 of the columns.  P
// goes through shared memory between the two.  The running maximum is shared by the CTA and
// looked at with the barrier that the stages need anyway; it is exchanged only when some row's
// grew by more than 2^kK8Grow.
// Measured: 48 tokens x 16 heads x 2048 rows 37 us, a token x 128 heads x 2048 rows 16.5.  Bound by
// a chunk's dependent steps (stage, scores, P, O) in the one CTA that fits an SM.
constexpr int kLatRows = 64, kLatDK = 576, kLatDV = 512;

template <int MT>
struct K8Lat {
  static constexpr int kStages = 3;
  static constexpr int kStage = kLatRows * kLatDK;
  static constexpr int kQAt = kStages * kStage;
  static constexpr int kQ = kLatDK / 16 * MT * 512;
  static constexpr int kPAt = kQAt + kQ;
  static constexpr int kP = MT * 16 * 128;
  static constexpr int kMetaAt = kPAt + kP;
  static constexpr int kMeta = kLatRows * 8;  // row, scale
  static constexpr int kRedAt = kMetaAt + kStages * kMeta;
  static constexpr int kSmem = kRedAt + 8 * MT * 16 * 4 + MT * 16 * 8;
  // scores: warps along the heads and along the rows, row tiles of heads and of rows of a warp
  static constexpr int kMG = MT == 1 ? 1 : 2, kTG = 8 / kMG, kMT = MT / kMG, kNT = kLatRows / 8 / kTG;
};
// piece p of row r (rows of 36 pieces, 64 bytes out of step with 128): 8 rows' same piece,
// and two rows' four neighbouring pieces, on different banks
__device__ __forceinline__ int lat_at(int r, int p) { return r * kLatDK + ((p ^ ((r >> 1) & 3)) << 4); }

template <int MT, int FMT>
__global__ void __launch_bounds__(256, 1) k8_latent_kernel(const __grid_constant__ K8Fwd a, float* ws) {
  using P = K8Lat<MT>;
  constexpr int S = P::kStages, R = MT * 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ K8Found found;
  const K8Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, q4 = lane & 3;
  const int mg = P::kMG == 1 ? 0 : warp & 1, tg = P::kMG == 1 ? warp : warp >> 1;
  float* const red = reinterpret_cast<float*>(smem + P::kRedAt);  // [kTG][R]
  float* const q_scale = red + 8 * R;                             // [R]
  uint32_t* const sq = reinterpret_cast<uint32_t*>(smem + P::kQAt);
  const uint32_t sp_at = smem_u32(smem + P::kPAt);
  pdl_trigger();
  pdl_wait();
  K8Cursor cur;
  if (!k8_begin<256>(a, ws, tid, found, cur)) return;
  const int krs = c.Hkv * kLatDK;

  for (long long w = cur.w0; w < cur.w1;) {
    k8_settle(a, cur);
    const K8Span& sp = cur.sp;
    const int b = cur.b, h = cur.h, ut = cur.ut, c0 = cur.c0, c1 = (int)min((long long)sp.ch, c0 + (cur.w1 - w));
    const int tile = a.hs == 1 ? ut : ut / a.hs, hp = ut - tile * a.hs;
    const int t = sp.s.t0 + tile, ta = sp.s.first + tile;
    const int head0 = h * a.G + hp * R, rows = min(R, a.G - hp * R);
    const int lo = a.win >= ta ? 0 : ta - a.win, hi = min(ta + 1, sp.s.L), start = lo & ~15;
    const long long iu = (long long)t * c.Hkv + h;
    const int* idx = a.topk ? a.idx + iu * a.topk : nullptr;
    int slots = a.topk;
    if (a.topk && a.topk_len) slots = min(slots, max(0, k8_read(a.topk_len + iu)));
    const int* table = c.table + b * c.tstride;

    // warp w resolves and copies rows 8 w .. 8 w + 7 of a chunk (lane x: row x % 8)
    const int n_steps = c1 - c0, p0 = c0 * kLatRows + warp * 8 + (lane & 7);
    auto fetch_idx = [&](int k) -> int {
      if (!a.topk) return 0;
      const int slot = k8_quot(a.by_bs, p0 + k * kLatRows);
      return k < n_steps && slot < slots ? k8_read(idx + slot) : -1;
    };
    auto resolve = [&](int k, int x) -> int {
      if (k >= n_steps) return -1;
      const int p = p0 + k * kLatRows;
      int row = start + p;
      if (a.topk) {
        if (x < 0) return -1;
        if ((long long)x * a.bs >= sp.s.L) {
          if (c.status) atomicOr(c.status, kStatusIndexRange);
          return -1;
        }
        row = x * a.bs + k8_rem(a.by_bs, p);
      }
      return row < hi && row >= lo ? row : -1;
    };
    auto fetch_page = [&](int row) -> int { return row >= 0 ? k8_read(table + k8_quot(c.by_ps, row)) : 0; };
    auto issue = [&](int st, int row, int page) {
      if (row >= 0 && (page < 0 || page >= c.n_pages)) {
        if (c.status) atomicOr(c.status, kStatusIndexRange);
        row = -1;
      }
      const int rr = row >= 0 ? page * c.ps + k8_rem(c.by_ps, row) : -1;
      uint8_t* meta = smem + P::kMetaAt + st * P::kMeta;
      if (lane < 8) {
        reinterpret_cast<int*>(meta)[warp * 8 + lane] = row;
        if (row >= 0) k8_cp4(smem_u32(meta) + 256 + 4 * (warp * 8 + lane), c.ks + (long long)page * c.Hkv + h);
      }
      const uint32_t dst = smem_u32(smem) + st * P::kStage;
      const uint8_t* src = c.k + h * kLatDK;
#pragma unroll
      for (int it = 0; it < 9; ++it) {
        const int i = it * 32 + lane, r = i / 36, pc = i - r * 36;
        const int at = __shfl_sync(~0u, rr, r);
        cp_async16(dst + lat_at(warp * 8 + r, pc), src + (long long)(at >= 0 ? at : 0) * krs + pc * 16, at >= 0);
      }
    };
    int xs[S + 1], rw[S], pg[S];
#pragma unroll
    for (int k = 0; k <= S; ++k) xs[k] = fetch_idx(k);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      rw[k] = resolve(k, xs[k]);
      pg[k] = fetch_page(rw[k]);
    }
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
      issue(k, rw[k], pg[k]);
      cp_async_commit();
    }
    int next_row = rw[S - 1], next_page = pg[S - 1], next_x = xs[S];

    // Q, 8 lanes a row, as halves times 2^(14 - E) in the MMA's order
#pragma unroll 1
    for (int r0 = 0; r0 < R; r0 += 32) {
      const int row = r0 + warp * 4 + (lane >> 3), qp = lane & 7;
      if (R < 32 && row >= R) break;  // whole warps
      const char* src = static_cast<const char*>(a.q) + ((long long)t * a.qstride + (long long)(head0 + row) * kLatDK) * 2;
      uint4 raw[9];
#pragma unroll
      for (int i = 0; i < 9; ++i)
        raw[i] = row < rows ? k8_read(reinterpret_cast<const uint4*>(src + (qp + 8 * i) * 16)) : make_uint4(0, 0, 0, 0);
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = k8_two(v[j], a.f16);
          big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
      const int E = big > 0.f ? max((int)(__float_as_uint(big) >> 23) - 127, -110) : 14;
      const float mul = __uint_as_float((uint32_t)(14 - E + 127) << 23);
      if (qp == 0) q_scale[row] = a.scale_log2 * __uint_as_float((uint32_t)(E - 14 + 127) << 23);
      const int mt = row >> 4, to = (row & 7) * 4 + (qp >> 1), r = (row >> 3) & 1;
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t hh[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = k8_two(v[j], a.f16);
          hh[j] = k8_halves(f.x * mul, f.y * mul);
        }
        uint32_t* dst = sq + (((4 * i + 2 * (qp & 1)) * MT + mt) * 32 + to) * 4 + r;
        dst[0] = hh[0];
        dst[2] = hh[1];
        dst[MT * 128] = hh[2];
        dst[MT * 128 + 2] = hh[3];
      }
    }
    __syncthreads();

    float o[MT][4][2][4];  // heads x four pieces of 16 columns
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[x][i][e][j] = 0.f;
    // of the score rows mg * kMT * 16 + 16 x + gr (+ 8)
    float l[P::kMT][2], base[P::kMT][2], fr[P::kMT][2], limit = -INFINITY;
#pragma unroll
    for (int x = 0; x < P::kMT; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[x][r] = base[x][r] = 0.f;
        fr[x][r] = q_scale[(mg * P::kMT + x) * 16 + gr + 8 * r];
      }
    bool first = true;  // nothing seen yet: base is no maximum

    int at = 0, fill = S - 1;
    for (int k = 0; k < n_steps; ++k) {
      k8_cp_wait<S - 2>();
      __syncthreads();  // the chunk is there; the one before has been read (and P)
      issue(fill, next_row, next_page);
      cp_async_commit();
      next_row = resolve(k + S, next_x);
      next_page = fetch_page(next_row);
      next_x = fetch_idx(k + S + 1);
      const uint8_t* const st = smem + at * P::kStage;
      const int* im = reinterpret_cast<const int*>(smem + P::kMetaAt + at * P::kMeta);
      const float* fm = reinterpret_cast<const float*>(im) + 64;
      fill = at;
      at = at + 1 == S ? 0 : at + 1;
      if (!__any_sync(~0u, im[lane] >= 0 || im[lane + 32] >= 0)) continue;  // no row in it, as all warps see

      // --- scores ---
      float s[P::kMT][P::kNT][4];
#pragma unroll
      for (int x = 0; x < P::kMT; ++x)
#pragma unroll
        for (int j = 0; j < P::kNT; ++j) s[x][j][0] = s[x][j][1] = s[x][j][2] = s[x][j][3] = 0.f;
      const uint4* q = reinterpret_cast<const uint4*>(sq) + mg * P::kMT * 32 + lane;
#pragma unroll 3
      for (int ch = 0; ch < kLatDK / 64; ++ch) {
        uint4 kw[P::kNT];
#pragma unroll
        for (int j = 0; j < P::kNT; ++j)
          kw[j] = *reinterpret_cast<const uint4*>(st + lat_at((tg * P::kNT + j) * 8 + gr, ch * 4 + q4));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 qa[P::kMT];
#pragma unroll
          for (int x = 0; x < P::kMT; ++x) qa[x] = q[((4 * ch + e) * MT + x) * 32];
#pragma unroll
          for (int j = 0; j < P::kNT; ++j) {
            uint32_t b0, b1;
            k8_pair<FMT>(e == 0 ? kw[j].x : e == 1 ? kw[j].y : e == 2 ? kw[j].z : kw[j].w, b0, b1);
#pragma unroll
            for (int x = 0; x < P::kMT; ++x) k8_mma(s[x][j], qa[x], b0, b1);
          }
        }
      }
      float iv[P::kNT][2], mx[P::kMT][2];
      bool grew = false;
#pragma unroll
      for (int x = 0; x < P::kMT; ++x) mx[x][0] = mx[x][1] = -INFINITY;
#pragma unroll
      for (int j = 0; j < P::kNT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = (tg * P::kNT + j) * 8 + 2 * q4 + e;
          const bool see = im[col] >= 0;
          const float ks = k8_scale(fm[col]), lv = k8_log2(ks);
          iv[j][e] = k8_rcp(ks);
#pragma unroll
          for (int x = 0; x < P::kMT; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& v = s[x][j][2 * r + e];
              v = see ? fmaf(v, fr[x][r] * ks, lv - base[x][r]) : -INFINITY;
              mx[x][r] = fmaxf(mx[x][r], v);
            }
        }
#pragma unroll
      for (int x = 0; x < P::kMT; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r) grew = grew || mx[x][r] > limit;
      if (__syncthreads_or(grew)) {
        // the chunk's maxima over the warps that share the heads; those that grew move their base
#pragma unroll
        for (int x = 0; x < P::kMT; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float v = fmaxf(mx[x][r], __shfl_xor_sync(~0u, mx[x][r], 1));
            v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
            if (q4 == 0) red[tg * R + (mg * P::kMT + x) * 16 + gr + 8 * r] = v;
          }
        __syncthreads();
        // a row's shift of its base (in units of log2): by how much its scores and O scale down
        if (tid < R) {
          float v = -INFINITY;
#pragma unroll
          for (int g = 0; g < P::kTG; ++g) v = fmaxf(v, red[g * R + tid]);
          // from the old base (0 before the first chunk with rows) to maximum - kK8Top
          red[tid] = v > limit ? v - kK8Top : 0.f;
          if (first && v == -INFINITY) red[tid] = 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < P::kMT; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float d = red[(mg * P::kMT + x) * 16 + gr + 8 * r];
            base[x][r] += d;
            l[x][r] *= first ? 1.f : ex2_approx(-d);
#pragma unroll
            for (int j = 0; j < P::kNT; ++j) {
              s[x][j][2 * r] -= d;
              s[x][j][2 * r + 1] -= d;
            }
          }
        if (!first) {
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float f = ex2_approx(-red[x * 16 + gr + 8 * r]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  o[x][i][e][2 * r] *= f;
                  o[x][i][e][2 * r + 1] *= f;
                }
            }
        }
        first = false;
        limit = kK8Top + kK8Grow;
        __syncthreads();  // red is written again by the next exchange
      }
      // --- P ---
#pragma unroll
      for (int x = 0; x < P::kMT; ++x)
#pragma unroll
        for (int j = 0; j < P::kNT; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0v = ex2_approx(s[x][j][2 * r]), p1v = ex2_approx(s[x][j][2 * r + 1]);
            l[x][r] = fmaf(p0v, iv[j][0], fmaf(p1v, iv[j][1], l[x][r]));
            const int row = (mg * P::kMT + x) * 16 + gr + 8 * r, col = (tg * P::kNT + j) * 8 + 2 * q4;
            *reinterpret_cast<uint32_t*>(smem + P::kPAt + row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2) =
                k8_halves(p0v, p1v);
          }
      __syncthreads();
      // --- O += P V: this warp's 64 columns ---
      const uint32_t sv = smem_u32(st);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint4 pa[MT];
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          const int row = x * 16 + (lane & 15), pc = kk * 2 + (lane >> 4);
          uint32_t v[4];
          ldsm_x4(v, sp_at + row * 128 + ((pc ^ (row & 7)) << 4));
          pa[x] = make_uint4(v[0], v[1], v[2], v[3]);
        }
#pragma unroll
        for (int pc = 0; pc < 4; pc += 2) {
          uint32_t v[4];
          ldsm_x4_t(v, sv + lat_at(kk * 16 + (lane & 15), warp * 4 + pc + (lane >> 4)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t e0, o0, e1, o1;
            k8_pair_t<FMT>(v[2 * i], e0, o0);
            k8_pair_t<FMT>(v[2 * i + 1], e1, o1);
#pragma unroll
            for (int x = 0; x < MT; ++x) {
              k8_mma(o[x][pc + i][0], pa[x], e0, e1);
              k8_mma(o[x][pc + i][1], pa[x], o0, o1);
            }
          }
        }
      }
    }
    k8_cp_wait<0>();

    // --- sums over the warps that share the heads; out ---
    __syncthreads();
#pragma unroll
    for (int x = 0; x < P::kMT; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[x][r] += __shfl_xor_sync(~0u, l[x][r], 1);
        l[x][r] += __shfl_xor_sync(~0u, l[x][r], 2);
        const int row = (mg * P::kMT + x) * 16 + gr + 8 * r;
        if (q4 == 0) red[tg * R + row] = l[x][r];
        if (q4 == 0 && tg == 0) q_scale[row] = base[x][r];
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == sp.ch;
    float* const part_out = k8_part(ws, gridDim.x, 2 * blockIdx.x + (c0 == 0), R, kLatDV);
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = x * 16 + gr + 8 * r;
        if (row >= rows) continue;
        float total = 0.f;
#pragma unroll
        for (int g = 0; g < P::kTG; ++g) total += red[g * R + row];
        const float m = first ? -INFINITY : q_scale[row] + kK8Top;
        float lse, norm = 0.f;
        if (whole) norm = k8_norm(k8_sink(a, head0 + row), m, total, &lse);
        if (warp == 0 && q4 == 0) {
          if (whole) {
            a.lse[(long long)t * a.Hq + head0 + row] = lse;
          } else {
            part_out[row] = m;
            part_out[R + row] = total;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = warp * 64 + i * 16 + 4 * q4;
          const float4 v = make_float4(o[x][i][0][2 * r], o[x][i][1][2 * r], o[x][i][0][2 * r + 1], o[x][i][1][2 * r + 1]);
          if (whole) k8_store(a, t, head0 + row, d, norm, v);
          else *reinterpret_cast<float4*>(part_out + 2 * R + row * kLatDV + d) = v;
        }
      }
    if (!whole && tid == 0)
      k8_note(a, ws, cur.share, cur.seq_at + ((long long)cur.h * sp.per_h + cur.ut) * sp.len, c0, sp.len, t, head0, rows,
              a.gdiv);
    __syncthreads();  // red, q_scale, the stages and Q are written again
    w += c1 - c0;
    k8_next(cur);
  }
}

// ---------------------------------------------------------------------------
// the same with more than 32 heads: tcgen05
// ---------------------------------------------------------------------------
// A unit is one token and 64 of its heads; 128 rows per chunk, one CTA per SM.  The rows
// lie along the MMA's M:
//   S^T [128 rows x 64 heads] = K [128 x 576] Q^T       (K and Q K-major)
//   O^T [4 x 128 columns x 64 heads] += V^T P^T         (V the first 8 slabs of K, MN-major)
// so that K is converted once and serves both products, O stays in TMEM (256 columns) and a
// thread holds a row's scores.  Shared memory holds one chunk as halves (147 KB, 9 slabs of
// 64 columns) and Q (74 KB); P^T takes the slab of the last 64 columns, which only the scores
// need.  Eight warps convert a chunk's codes from registers, slab by slab as the MMAs of the
// chunk before let go of the slabs, ask for the next chunk's in their place, and do the softmax;
// a ninth issues (of a third warpgroup, which gives its registers to the other two).
// Measured: 48 tokens x 128 heads x 2048 rows 96 us, of which a part's start (lookups of four
// dependent loads, Q, the first conversions) is 10 and its end 5.  A chunk takes some 7600 cycles:
// conversion 3600 (its stores of 147 KB and the operands of the 68 MMAs, 6 KB each at N = 64, share
// shared memory's 128 bytes a cycle), the last scores 2100, softmax 1600, of which only
// O and the first scores overlap with the conversion.  The conversion's arithmetic is 4 % of it all.
constexpr int kTcRows = 128, kTcSlab = kTcRows * 128, kTcSlabs = 9;
struct K8Tc {
  static constexpr int kQAt = kTcSlabs * kTcSlab;
  static constexpr int kMetaAt = kQAt + 9 * 64 * 128;       // [2][128] rows seen, [2][128] scales
  static constexpr int kHeadAt = kMetaAt + 2 * kTcRows * 8;  // [64] (fr, base)
  static constexpr int kRedAt = kHeadAt + 64 * 8;            // [4][64]
  static constexpr int kBarAt = kRedAt + 4 * 64 * 4;         // full [2], p_full, s_done, free [4], drained
  static constexpr int kSmem = kBarAt + 16 * 8 + 1024;
  static constexpr uint32_t kTmemS = 256;  // column of S^T behind the four blocks of O^T
};
__host__ __device__ constexpr uint32_t k8_idesc(int M, int N, bool a_mn, bool b_mn) {  // halves, fp32 sums
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Of the eight converting warps: a barrier, and whether any thread says yes.
__device__ __forceinline__ void tc_bar() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
__device__ __forceinline__ bool tc_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, 1, 256, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

struct K8Codes {
  uint32_t w[8];
};
// hi: the upper half of both operands' descriptors; one thread of the warp issues (tc_elect)
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(id), "r"(acc));
}
__device__ __forceinline__ bool tc_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ K8Codes tc_ld32(const uint8_t* p) {  // 32 codes, 32-byte aligned; none: zeros
  K8Codes r;
  if (p) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = 0;
  }
  return r;
}
// GIVE_UP, for the test of what a wait that gave up leaves behind: a wait of one warp at one chunk completes and
// counts as given up; all others are made as ever, so that nothing runs out of turn.
template <int FMT, bool GIVE_UP>
__global__ void __launch_bounds__(384, 1) k8_tc_kernel(const __grid_constant__ K8Fwd a, float* ws) {
  using P = K8Tc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  __shared__ K8Found found;
  __shared__ uint32_t tmem_at;
  // abort_word: a wait of this CTA gave up.  Whichever warp it was (the one that issues goes on with operands that
  // are not all there, and what it commits lets the others' waits complete), the unit at hand and the share's
  // later ones become NaN.  fresh: the chunk begins a part, O^T is overwritten.
  __shared__ int abort_word, fresh;
  const K8Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto wait = [&](int which, long long chunk, uint64_t* bar, uint32_t parity) -> bool {
    if (!GIVE_UP) return mbar_wait(bar, parity, &abort_word, c.status);
    mbar_wait_drain(bar, parity);
    if (warp != a.give_up_warp || which != a.give_up_wait || chunk != a.give_up_chunk) return true;
    abort_word = 1;
    if (c.status) atomicOr(c.status, kStatusTimeout);
    return false;
  };
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + P::kBarAt);
  uint64_t *const p_full = full + 2, *const s_done = full + 3, *const blk_free = full + 4, *const drained = full + 8;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(full + i, 8);
    for (int i = 3; i < 9; ++i) mbar_init(full + i, 1);
    mbar_fence_init();
    abort_word = 0;
  }
  if (warp == 8) {
    tmem_alloc(&tmem_at, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  pdl_trigger();
  pdl_wait();
  K8Cursor cur;
  const bool some = k8_begin<256>(a, ws, tid, found, cur);
  const long long n_chunks = some ? cur.w1 - cur.w0 : 0;

  // 384 threads launch with 168 registers: 2 x 128 x 232 + 128 x 40 are as many
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    // --- the MMAs ---
    if (warp == 8 && some) {
      const uint32_t kat = smem_u32(smem), qat = kat + P::kQAt, pat = kat + 8 * kTcSlab;
      const uint32_t dk = (uint32_t)sdesc(kat, 0, 1024), dq = (uint32_t)sdesc(qat, 0, 1024);
      const uint32_t dv = (uint32_t)sdesc(kat, kTcSlab, 1024), dp = (uint32_t)sdesc(pat, kTcSlab, 1024);
      const uint32_t hi = (uint32_t)(sdesc(0, 0, 1024) >> 32);
      constexpr uint32_t id_s = k8_idesc(128, 64, false, false), id_o = k8_idesc(128, 64, true, true);
      // A wait that gave up changes nothing here (abort_word keeps the products out of the result): the warp stays
      // together, as electing asks for.
      for (long long n = 0; n < n_chunks; ++n) {
        const uint32_t ph = (uint32_t)(n & 1);
        // Unrolled with constant offsets from bases that the compiler sees to be alike in the whole warp, so that
        // a descriptor takes one addition in the warp's own registers; 32 bits of it, the others never change.
        // (Additions carried from MMA to MMA took 120 to 170 cycles each, one thread's registers 2 % of the call.)
#pragma unroll
        for (int sl = 0; sl < kTcSlabs; ++sl) {
          if ((sl & 3) == 0 && sl < 8) {  // four slabs, then five: a wait and its fence cost 300 to 500 cycles
            wait(sl >> 2, n, full + (sl >> 2), ph);
            fence_async_smem();  // the converting warps' stores, seen through the barrier, before the MMAs' reads
            tc_fence_after();
          }
          if (tc_elect()) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tc_mma(tmem + P::kTmemS, dk + ((sl * kTcSlab + 32 * e) >> 4), dq + ((sl * 8192 + 32 * e) >> 4), hi, id_s,
                     sl || e);
            if (sl == kTcSlabs - 1) mma_commit(s_done);
          }
        }
        wait(2, n, p_full, ph);
        fence_async_smem();
        tc_fence_after();
        const uint32_t over = *(volatile int*)&fresh;
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
          if (tc_elect()) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              tc_mma(tmem + mb * 64, dv + ((mb * 2 * kTcSlab + 2048 * e) >> 4), dp + ((2048 * e) >> 4), hi, id_o,
                     !over || e);
            mma_commit(blk_free + mb);
          }
        }
      }
      if (tc_elect()) mma_commit(drained);  // the workers that gave up did not wait for the last products
      mbar_wait_drain(drained, 0);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
    uint32_t* const see_of = reinterpret_cast<uint32_t*>(smem + P::kMetaAt);         // [2][128]
    float* const scale_of = reinterpret_cast<float*>(smem + P::kMetaAt) + 2 * kTcRows;  // [2][128]
    float2* const head_of = reinterpret_cast<float2*>(smem + P::kHeadAt);            // [64] fr, base
    float* const red = reinterpret_cast<float*>(smem + P::kRedAt);                   // [4][64]
    const uint32_t tm_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int hh = warp >> 2, row_j = 32 * (warp & 3) + lane;  // this thread's heads and row in the softmax
    const int krs = c.Hkv * kLatDK;
    bool dead = false;
    long long n = 0;  // chunks done
    while (n < n_chunks) {
      const K8Unit u = k8_take(a, cur);
      const int n_steps = u.c1 - u.c0;
      // rows of a chunk: warp w looks up and converts rows 16 w .. 16 w + 15 (lane x: row x % 16)
      const int p0 = u.c0 * kTcRows + warp * 16 + (lane & 15);
      auto fetch_idx = [&](int k) -> int {
        if (!a.topk) return 0;
        const int slot = k8_quot(a.by_bs, p0 + k * kTcRows);
        return k < n_steps && slot < u.slots ? k8_read(u.idx + slot) : -1;
      };
      auto resolve = [&](int k, int x) -> int {
        if (k >= n_steps) return -1;
        const int p = p0 + k * kTcRows;
        int row = u.start + p;
        if (a.topk) {
          if (x < 0) return -1;
          if ((long long)x * a.bs >= u.L) {
            if (c.status) atomicOr(c.status, kStatusIndexRange);
            return -1;
          }
          row = x * a.bs + k8_rem(a.by_bs, p);
        }
        return row < u.hi && row >= u.lo ? row : -1;
      };
      auto fetch_page = [&](int row) -> int { return row >= 0 ? k8_read(u.table + k8_quot(c.by_ps, row)) : 0; };
      // the lane's row of the cache, from what was looked up (-1: none), and its scale
      float ks_next = 0.f;
      auto place = [&](int row, int page) -> int {
        if (row >= 0 && (page < 0 || page >= c.n_pages)) {
          if (c.status) atomicOr(c.status, kStatusIndexRange);
          row = -1;
        }
        if (row < 0) return -1;
        ks_next = k8_read(c.ks + (long long)page * c.Hkv + u.h);
        return page * c.ps + k8_rem(c.by_ps, row);
      };
      auto note = [&](uint32_t ph, int rr) {  // for the softmax
        if (lane < 16) {
          see_of[ph * kTcRows + warp * 16 + lane] = rr >= 0;
          scale_of[ph * kTcRows + warp * 16 + lane] = ks_next;
        }
      };
      // the lane's pieces of the codes.  Pairs of slabs: rows 8 j + lane / 4, 32 codes of 128; the ninth: row lane / 2
      const uint8_t* ptr[3];
      auto point = [&](int rr) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const int at = __shfl_sync(~0u, rr, j < 2 ? 8 * j + (lane >> 2) : lane >> 1);
          const int col = j < 2 ? (lane & 3) * 32 : 512 + (lane & 1) * 32;
          ptr[j] = at >= 0 ? c.k + (long long)at * krs + u.h * kLatDK + col : nullptr;
        }
      };
      auto prefetch = [&](int rr) {  // 8 rows of 576 bytes: 4 lanes a row, 128 bytes apart, and the last 64
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = __shfl_sync(~0u, rr, 8 * j + (lane >> 2));
          if (at < 0) continue;
          const uint8_t* const p = c.k + (long long)at * krs + u.h * kLatDK + (lane & 3) * 128;
          asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p));
          if ((lane & 3) == 3) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p + 128));
        }
      };
      int x0 = fetch_idx(0), x1 = fetch_idx(1), x2 = fetch_idx(2), next_x = fetch_idx(3);
      // --- Q, 8 lanes a row, as halves times 2^(14 - E); the scores of the unit before have been taken ---
      uint4 qr[2][9];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = 32 * y + warp * 4 + (lane >> 3);
        const char* src = static_cast<const char*>(a.q) + ((long long)u.t0 * a.qstride + (long long)(u.head0 + row) * kLatDK) * 2;
#pragma unroll
        for (int i = 0; i < 9; ++i)
          qr[y][i] = row < u.rows ? k8_read(reinterpret_cast<const uint4*>(src + ((lane & 7) + 8 * i) * 16)) : make_uint4(0, 0, 0, 0);
      }
      const int row0 = resolve(0, x0), pg0 = fetch_page(row0), row1 = resolve(1, x1), pg1 = fetch_page(row1);
      int next_row = resolve(2, x2), next_page = fetch_page(next_row);
      K8Codes raw[9];  // pair g, row j: 2 g + j
      auto load = [&](int g) {  // pair g of slabs, the ninth with the last
#pragma unroll
        for (int j = 0; j < 2; ++j) raw[2 * g + j] = tc_ld32(ptr[j] ? ptr[j] + g * 128 : nullptr);
        if (g == 3) raw[8] = tc_ld32(ptr[2]);
      };
      int rr = place(row0, pg0);
      point(rr);
#pragma unroll
      for (int g = 0; g < 4; ++g) load(g);
      note((uint32_t)(n & 1), rr);
      rr = place(row1, pg1);
      prefetch(rr);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = 32 * y + warp * 4 + (lane >> 3), qp = lane & 7;
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 9; ++i) {
          const uint32_t v[4] = {qr[y][i].x, qr[y][i].y, qr[y][i].z, qr[y][i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = k8_two(v[j], a.f16);
            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
        const int E = big > 0.f ? max((int)(__float_as_uint(big) >> 23) - 127, -110) : 14;
        const float mul = __uint_as_float((uint32_t)(14 - E + 127) << 23);
        if (qp == 0) head_of[row] = make_float2(a.scale_log2 * __uint_as_float((uint32_t)(E - 14 + 127) << 23), 0.f);
#pragma unroll
        for (int i = 0; i < 9; ++i) {
          const uint32_t v[4] = {qr[y][i].x, qr[y][i].y, qr[y][i].z, qr[y][i].w};
          uint32_t hv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = k8_two(v[j], a.f16);
            hv[j] = k8_halves(f.x * mul, f.y * mul);
          }
          *reinterpret_cast<uint4*>(smem + P::kQAt + i * 8192 + row * 128 + ((qp ^ (row & 7)) << 4)) =
              make_uint4(hv[0], hv[1], hv[2], hv[3]);
        }
      }

      float l[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) l[i] = 0.f;
      bool first = true;
      for (int k = 0; k < n_steps; ++k, ++n) {
        const uint32_t ph = (uint32_t)(n & 1);
        // --- codes to halves, slab by slab; the next chunk's take their place ---
        point(k + 1 < n_steps ? rr : -1);
        // 32 codes to 64 bytes of slab `sl`, row r, from its 16-byte piece ch0 on.  The order of the pieces
        // keeps eight lanes' stores (two rows, two slabs) on different banks.
        auto put = [&](const K8Codes& x, int sl, int r, int ch0, int turn) {
          uint8_t* dst = smem + sl * kTcSlab + r * 128;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int i = y ^ turn;  // 0 or 2: the words below are picked by selects
            uint32_t w[4];
            k8_pair<FMT>(turn ? x.w[2 * (y ^ 2)] : x.w[2 * y], w[0], w[1]);
            k8_pair<FMT>(turn ? x.w[2 * (y ^ 2) + 1] : x.w[2 * y + 1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + (((ch0 + i) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        };
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (n > 0 && (GIVE_UP || !dead)) dead |= !wait(3 + g, n, blk_free + g, ph ^ 1);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            put(raw[2 * g + j], 2 * g + ((lane >> 1) & 1), warp * 16 + 8 * j + (lane >> 2), 4 * (lane & 1), lane & 2);
          if (g == 3) put(raw[8], 8, warp * 16 + (lane >> 1), 4 * (lane & 1), 0);
          // (the thread that issues the MMAs has the fence between these stores and their reads; here it would
          // wait for the loads under way, 300 to 900 cycles)
          if (g & 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(full + (g >> 1));
          }
          if (k + 1 < n_steps) load(g);
        }
        if (k + 1 < n_steps) {  // the lookups of the chunks behind it, while the last scores are computed
          note(ph ^ 1, rr);
          rr = place(next_row, next_page);
          prefetch(rr);
          next_row = resolve(k + 3, next_x);
          next_page = fetch_page(next_row);
          next_x = fetch_idx(k + 4);
        }
        tc_bar();  // the chunk's rows and scales, and Q's factors, are there for all

        // --- softmax: this thread's row against 32 heads ---
        const bool see = see_of[ph * kTcRows + row_j] != 0;
        const float ks = k8_scale(scale_of[ph * kTcRows + row_j]), lv = k8_log2(ks), iv = k8_rcp(ks);
        if (GIVE_UP || !dead) dead |= !wait(7, n, s_done, ph);
        tc_fence_after();
        float s[32];
        {
          uint32_t r0[16], r1[16];
          tmem_ld16(tm_lane + P::kTmemS + 32 * hh, r0);
          tmem_ld16(tm_lane + P::kTmemS + 32 * hh + 16, r1);
          tmem_wait_ld();
          reg_dep16(r0);
          reg_dep16(r1);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[i] = __uint_as_float(r0[i]);
            s[16 + i] = __uint_as_float(r1[i]);
          }
        }
        const float4* hf = reinterpret_cast<const float4*>(head_of + 32 * hh);
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 f = hf[i];
          s[2 * i] = see ? fmaf(s[2 * i], f.x * ks, lv - f.y) : -INFINITY;
          s[2 * i + 1] = see ? fmaf(s[2 * i + 1], f.z * ks, lv - f.w) : -INFINITY;
          mx = fmaxf(mx, fmaxf(s[2 * i], s[2 * i + 1]));
        }
        if (tc_any(mx > (first ? -INFINITY : kK8Top + kK8Grow))) {
          // the chunk's maxima per head: over the warp's rows, then over the four warps
          float mine = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            // floats in the order of signed integers; NaN as -inf
            const int b = __float_as_int(s[i]), key = b >= 0 ? b : b ^ 0x7fffffff;
            const int top = __reduce_max_sync(~0u, s[i] == s[i] ? key : (int)0x807fffff);
            if (lane == i) mine = __int_as_float(top >= 0 ? top : top ^ 0x7fffffff);
          }
          red[(warp & 3) * 64 + 32 * hh + lane] = mine;
          tc_bar();
          if (tid < 64) {
            const float v = fmaxf(fmaxf(red[tid], red[64 + tid]), fmaxf(red[128 + tid], red[192 + tid]));
            const float d = v > (first ? -INFINITY : kK8Top + kK8Grow) ? v - kK8Top : 0.f;
            red[tid] = d;
            head_of[tid].y += d;
          }
          tc_bar();
          const float* shift = red + 32 * hh;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float d = shift[i];
            s[i] -= d;
            if (!first) l[i] *= ex2_approx(-d);
          }
          if (!first) {
            // O^T's blocks 2 hh and 2 hh + 1, 16 columns (heads) at a time
            const unsigned long long moved = __ballot_sync(~0u, red[lane] != 0.f) |
                                             (unsigned long long)__ballot_sync(~0u, red[32 + lane] != 0.f) << 32;
#pragma unroll 1
            for (int cb = 0; cb < 128; cb += 16) {
              if (!((moved >> (cb & 63)) & 0xffff)) continue;  // none of these heads grew
              uint32_t r[16];
              const uint32_t at = tm_lane + hh * 128 + cb;
              tmem_ld16(at, r);
              tmem_wait_ld();
              reg_dep16(r);
#pragma unroll
              for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * ex2_approx(-red[(cb + i) & 63]));
              tmem_st16(at, r);
            }
            tmem_wait_st();
          }
          first = false;
          tc_bar();  // red is written again by the next exchange
        }
        if (tid == 0) fresh = k == 0;
        // --- P^T: row j of the last slab, 64 heads of 2 bytes ---
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e0 = ex2_approx(s[8 * i + 2 * j]), e1 = ex2_approx(s[8 * i + 2 * j + 1]);
            l[8 * i + 2 * j] = fmaf(e0, iv, l[8 * i + 2 * j]);
            l[8 * i + 2 * j + 1] = fmaf(e1, iv, l[8 * i + 2 * j + 1]);
            w[j] = k8_halves(e0, e1);
          }
          *reinterpret_cast<uint4*>(smem + 8 * kTcSlab + row_j * 128 + (((4 * hh + i) ^ (row_j & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }

      // --- the part's sums, and O^T out ---
      if (GIVE_UP || !dead) dead |= !wait(8, n - 1, blk_free + 3, (uint32_t)((n - 1) & 1));
      tc_fence_after();
#pragma unroll
      for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < d; ++i) {
          const float keep = lane & d ? l[i + d] : l[i], give = lane & d ? l[i] : l[i + d];
          l[i] = keep + __shfl_xor_sync(~0u, give, d);
        }
      red[(warp & 3) * 64 + 32 * hh + lane] = l[0];  // lane x holds head x's
      const bool lost = tc_any(*(volatile int*)&abort_word != 0);
      const bool whole = u.c0 == 0 && u.c1 == u.ch;
      float* const part_out = k8_part(ws, gridDim.x, 2 * blockIdx.x + (u.c0 == 0), 64, kLatDV);
      float norm = 0.f;
      if (tid < u.rows) {
        const float m = first ? -INFINITY : head_of[tid].y + kK8Top;
        const float total =
            lost ? __int_as_float(0x7fffffff) : red[tid] + red[64 + tid] + red[128 + tid] + red[192 + tid];
        if (whole) {
          float lse;
          norm = k8_norm(k8_sink(a, u.head0 + tid), m, total, &lse);
          a.lse[(long long)u.t0 * a.Hq + u.head0 + tid] = lse;
        } else {
          part_out[tid] = m;
          part_out[64 + tid] = total;
        }
      }
      tc_bar();
      if (tid < 64) red[tid] = norm;
      tc_bar();
#pragma unroll 1
      for (int mb = 2 * hh; mb < 2 * hh + 2; ++mb) {
        const int d = mb * 128 + row_j;
        char* const out = static_cast<char*>(a.o) + (((long long)u.t0 * a.Hq + u.head0) * kLatDV + d) * 2;
        float* const part = part_out + 128 + d;
#pragma unroll 1
        for (int h0 = 0; h0 < u.rows; h0 += 32) {
          uint32_t r0[16], r1[16];
          tmem_ld16(tm_lane + mb * 64 + h0, r0);
          tmem_ld16(tm_lane + mb * 64 + h0 + 16, r1);
          tmem_wait_ld();
          reg_dep16(r0);
          reg_dep16(r1);
          if (whole) {
            // two heads at a time: even lanes store columns d, d + 1 of the first, odd ones d - 1, d of the second
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float f0 = red[h0 + i], f1 = red[h0 + i + 1];
              const float v0 = __uint_as_float(i < 16 ? r0[i & 15] : r1[i & 15]);
              const float v1 = __uint_as_float(i < 16 ? r0[(i + 1) & 15] : r1[(i + 1) & 15]);
              const float y0 = f0 == 0.f ? 0.f : v0 * f0, y1 = f1 == 0.f ? 0.f : v1 * f1;
              const bool odd = lane & 1;
              const float got = __shfl_xor_sync(~0u, odd ? y0 : y1, 1), lo = odd ? got : y0, hi = odd ? y1 : got;
              const int head = h0 + i + odd;
              if (head < u.rows)
                *reinterpret_cast<uint32_t*>(out + (head * kLatDV - odd) * 2) = a.f16 ? k8_halves(lo, hi) : pack_bf16(lo, hi);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (h0 + i < u.rows) part[(h0 + i) * kLatDV] = __uint_as_float(i < 16 ? r0[i & 15] : r1[i & 15]);
          }
        }
      }
      tc_fence_before();
      if (!whole && tid == 0) k8_note(a, ws, cur.share, u.begin, u.c0, u.ch, u.t0, u.head0, u.rows, a.gdiv);
      tc_bar();  // red and Q's factors are written again
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int MT, int FMT>
static cudaError_t latent_t(const K8Fwd& a, void* ws, cudaStream_t st) {
  using P = K8Lat<MT>;
  auto k = k8_latent_kernel<MT, FMT>;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(k, P::kSmem, done);
  if (e != cudaSuccess) return e;
  const int n = k8_ctas(a);
  count_launch();
  e = launch_pdl(k, (unsigned)n, 256, P::kSmem, st, a, static_cast<float*>(ws));
  if (e != cudaSuccess || n == 1 || a.per_unit == 1) return e;
  count_launch();
  return launch_pdl(k8_join_kernel<MT * 16, kLatDV>, (unsigned)n, 256, 0, st, a, static_cast<float*>(ws), n);
}
template <int FMT, bool GIVE_UP>
static cudaError_t tc_t(const K8Fwd& a, void* ws, cudaStream_t st) {
  auto k = k8_tc_kernel<FMT, GIVE_UP>;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(k, K8Tc::kSmem, done);
  if (e != cudaSuccess) return e;
  const int n = k8_ctas(a);
  count_launch();
  e = launch_pdl(k, (unsigned)n, 384, K8Tc::kSmem, st, a, static_cast<float*>(ws));
  if (e != cudaSuccess || n == 1 || a.per_unit == 1) return e;
  count_launch();
  return launch_pdl(k8_join_kernel<64, kLatDV>, (unsigned)n, 256, 0, st, a, static_cast<float*>(ws), n);
}
template <int FMT>
static cudaError_t latent_f(const K8Fwd& a, void* ws, cudaStream_t st) {
  if (a.unit_rows == 16) return latent_t<1, FMT>(a, ws, st);
  if (a.unit_rows == 32) return latent_t<2, FMT>(a, ws, st);
  return tc_t<FMT, false>(a, ws, st);
}

static void k8_geometry(K8Fwd& a) {
  const bool lat = k8_latent(a);
  // More than 32 heads of a shared row go to the tcgen05 kernel (64 heads x 128 rows a step; it reads codes
  // 32 bytes at a time), but not where shares of 32 heads x 64 rows leave SMs idle: its start and end cost
  // 13 us more.  There mma.sync took 16.5 us against 29 (a token, 2048 rows, 128 heads), 11.7 against 20.5
  // (4 tokens, 36 rows); beyond, 142 against 96 (48 tokens, 2048 rows), 30 against 26.4 (8 tokens, 1024).
  const long long small = (long long)a.c.T * a.c.Hkv * ((a.G + 31) / 32) *
                          (a.topk ? ((long long)a.topk * a.bs + 63) / 64 : ((long long)a.c.max_pages * a.c.ps + 63) / 64);
  const bool tc = a.G > 32 && small > 148 && ((uintptr_t)a.c.k & 31) == 0;
  a.unit_rows = !lat || a.G <= 16 ? 16 : tc ? 64 : 32;
  a.chunk = !lat ? kK8Chunk : a.unit_rows == 64 ? kTcRows : kLatRows;
  a.gdiv = min(a.G, a.unit_rows);
  a.hs = (a.G + a.unit_rows - 1) / a.unit_rows;
  a.tpt = lat || a.topk || a.G > 16 ? 1 : 16 / a.G;
  a.sel_ch = a.topk ? (int)(((long long)a.topk * a.bs + a.chunk - 1) / a.chunk) : 0;
  a.by_tpt = k8_div_of(a.tpt);
  a.by_gdiv = k8_div_of(a.gdiv);
  // Units of one length, and no more than SMs: as many CTAs each as there are, of which none has parts of two
  // units.  A part's start, end and join (131 KB of 64 heads x 512) cost as much as 5 chunks of 64 heads.  With 2048 rows:
  // 37 against 45 us of the even cut (48 tokens, 16 heads), 59 against 71 (40, 64), 96 against 106 (48, 128).  Only
  // 2048 rows were measured: with many more, a whole unit's chunks on one CTA outweigh what a part costs.
  const long long units = (long long)a.c.T * a.hs * a.c.Hkv;
  a.per_unit = lat && a.topk && units <= 148 && a.sel_ch < 1 << 20 ? min(148 / (int)units, a.sel_ch) : 0;
  a.by_ch = k8_div_of(max(a.sel_ch, 1));
  a.by_per = k8_div_of(max(a.per_unit, 1));
  // of a unit, what it costs beside its chunks, in chunks; the most chunks that are not worth cutting
  a.over = lat ? 0 : 1;
  a.keep = lat ? 0 : 4;
}

size_t k8_fwd_workspace(K8Fwd a) {
  if (a.c.T == 0 || a.c.B == 0) return 0;  // nothing is launched, and there is no unit to share the CTAs out to
  k8_geometry(a);
  const int n = k8_ctas(a);
  return k8_parts_at(n) + (size_t)n * 2 * k8_part_floats(a.unit_rows, a.c.dv) * sizeof(float);
}

cudaError_t launch_kv8_fwd(K8Fwd a, void* ws, cudaStream_t st) {
  if (a.c.T == 0 || a.c.B == 0) return cudaSuccess;
  k8_geometry(a);
  if (k8_latent(a)) return a.c.fmt == kFmtE4M3 ? latent_f<kFmtE4M3>(a, ws, st) : latent_f<kFmtInt8>(a, ws, st);
  if (a.c.dqk == 64) return split_d<64, 64>(a, ws, st);
  if (a.c.dqk == 128) return split_d<128, 128>(a, ws, st);
  return split_d<192, 128>(a, ws, st);
}

cudaError_t launch_kv8_give_up(K8Fwd a, void* ws, cudaStream_t st) {
  if (a.c.T == 0 || a.c.B == 0 || !k8_latent(a) || a.c.fmt != kFmtE4M3) return cudaErrorNotSupported;
  k8_geometry(a);
  return a.unit_rows == 64 ? tc_t<kFmtE4M3, true>(a, ws, st) : cudaErrorNotSupported;
}

}  // namespace sa
