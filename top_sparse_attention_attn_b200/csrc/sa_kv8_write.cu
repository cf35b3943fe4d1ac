// sa_kv8_write.cu -- the page plan of a serving step and the write that rounds
// new K / V rows to 8 bits into the pages (sa_page_plan, sa_kv8_write).
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_kv8_device.cuh"
#include "sa_launch.h"

namespace sa {

// ---------------------------------------------------------------------------
// page plan
// ---------------------------------------------------------------------------
// One launch.  Every block scans the requests' lengths itself (8 bytes a request,
// from L2) into two prefix arrays in shared memory, tokens and new pages, and then
// looks up its share of the tokens and new pages there by bisection; block 0 writes
// the per-request outputs.  The scan repeated per block costs less than a second
// launch that would wait for it.  Bound by latency: 6.4 us for 64 requests, 7.3 for 1500.
__device__ __forceinline__ int plan_upper(const int* a, int n, int x) {  // largest b < n with a[b] <= x
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void page_plan_kernel(PagePlan p) {
  extern __shared__ int sm[];
  int* cu = sm;                // [B + 1]
  int* pg = sm + p.B + 1;      // [B + 1]
  __shared__ long long wtok[32], wpage[32];
  __shared__ int fail;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int n_free = min(max(k8_read(p.n_free), 0), p.free_cap);
  if (tid == 0) fail = p.B;
  const int per = (p.B + nt - 1) / nt, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  // sums of this thread's requests (64 bits: the lengths are the caller's)
  long long tok = 0, page = 0;
  for (int b = b0; b < b1; ++b) {
    const long long o = k8_read(p.old_lens + b), n = k8_read(p.new_lens + b);
    if (o < 0 || n < 0) continue;
    tok += n;
    page += (o + n + p.ps - 1) / p.ps - (o + p.ps - 1) / p.ps;
  }
  long long it = tok, ip = page;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long a = __shfl_up_sync(~0u, it, d), b = __shfl_up_sync(~0u, ip, d);
    if (lane >= d) { it += a; ip += b; }
  }
  if (lane == 31) { wtok[warp] = it; wpage[warp] = ip; }
  __syncthreads();
  if (warp == 0) {
    long long a = lane < (nt >> 5) ? wtok[lane] : 0, b = lane < (nt >> 5) ? wpage[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(~0u, a, d), y = __shfl_up_sync(~0u, b, d);
      if (lane >= d) { a += x; b += y; }
    }
    wtok[lane] = a;
    wpage[lane] = b;
  }
  __syncthreads();
  long long ct = it - tok + (warp ? wtok[warp - 1] : 0), cp = ip - page + (warp ? wpage[warp - 1] : 0);
  int bad = p.B;
  for (int b = b0; b < b1; ++b) {
    const long long o = k8_read(p.old_lens + b), n = k8_read(p.new_lens + b);
    // sums behind the first request that fails are never used; they only need to stay in range
    cu[b] = (int)min(ct, (long long)p.T);
    pg[b] = (int)min(cp, (long long)n_free);
    const bool valid = o >= 0 && n >= 0;
    const long long pages = valid ? (o + n + p.ps - 1) / p.ps : 0;
    if (valid) {
      ct += n;
      cp += pages - (o + p.ps - 1) / p.ps;
    }
    if ((!valid || pages > p.max_pages || ct > p.T || cp > n_free) && bad == p.B) bad = b;
  }
  if (tid == nt - 1) {
    cu[p.B] = (int)min(ct, (long long)p.T);
    pg[p.B] = (int)min(cp, (long long)n_free);
  }
  if (bad < p.B) atomicMin(&fail, bad);
  __syncthreads();
  const int served = fail;
  const int n_tok = cu[served], n_new = pg[served];
  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.B; b += nt) p.cu[b] = b < served ? cu[b] : n_tok;
    for (int b = tid; b < p.B; b += nt) p.seq_lens[b] = k8_read(p.old_lens + b) + (b < served ? k8_read(p.new_lens + b) : 0);
    if (tid == 0) {
      *p.n_free_out = n_free - n_new;
      *p.n_served = served;
    }
  }
  const int gid = blockIdx.x * nt + tid, gn = gridDim.x * nt;
  for (int i = gid; i < n_new; i += gn) {
    const int b = plan_upper(pg, served, i);
    const int held = (int)(((long long)k8_read(p.old_lens + b) + p.ps - 1) / p.ps);
    p.table[b * p.tstride + held + i - pg[b]] = k8_read(p.free_pages + (n_free - 1 - i));
  }
  for (int t = gid; t < p.T; t += gn) {
    long long slot = -1;
    if (t < n_tok) {
      const int b = plan_upper(cu, served, t);
      const int o = k8_read(p.old_lens + b), pos = o + t - cu[b];
      const int held = (int)(((long long)o + p.ps - 1) / p.ps), j = pos / p.ps;
      // entries below `held` are read here and entries from `held` on written above: never the same one
      const int id = j < held ? p.table[b * p.tstride + j] : k8_read(p.free_pages + (n_free - 1 - (pg[b] + j - held)));
      if (id >= 0) slot = (long long)id * p.ps + (pos - j * p.ps);
    }
    p.slots[t] = slot;
  }
}

cudaError_t launch_page_plan(const PagePlan& p, cudaStream_t st) {
  const unsigned block = p.B > 512 ? 1024 : 256;
  const size_t smem = (size_t)(p.B + 1) * 2 * sizeof(int);
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(page_plan_kernel, (kPlanMaxBatch + 1) * 2 * (int)sizeof(int), done);
  if (e != cudaSuccess) return e;
  const int grid = min(148, max(1, (int)((p.T + (long long)block - 1) / block)));
  count_launch();
  return launch_pdl(page_plan_kernel, (unsigned)grid, block, smem, st, p);
}

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------
// e of the least 2^e, in [-60, 60], with a <= top * 2^e, from the bits of a = 1.m 2^E:
// 448 = 1.75 * 2^8 and 127 = 1.984375 * 2^6 (a = 0 and subnormals: -60).
__device__ __forceinline__ int k8_exp_for(float a, int fmt) {
  const uint32_t u = __float_as_uint(a);
  const int E = (int)(u >> 23) - 127;
  const uint32_t m = u & 0x7fffffu;
  const int e = fmt == kFmtE4M3 ? E - (m <= 0x600000u ? 8 : 7) : E - (m <= 0x7e0000u ? 6 : 5);
  return min(max(e, -60), 60);
}
// e of the least power of two at or above a scale that is already there (in [2^-60, 2^60])
__device__ __forceinline__ int k8_exp_at_least(float a) {
  const uint32_t u = __float_as_uint(a);
  return (int)(u >> 23) - 127 + ((u & 0x7fffffu) ? 1 : 0);
}
__device__ __forceinline__ float k8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <bool F16>
__device__ __forceinline__ void k8_unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Of two pairs of 16-bit floats, the larger magnitudes (a magnitude of NaN is passed over).
template <bool F16>
__device__ __forceinline__ uint32_t k8_absmax2(uint32_t a, uint32_t b) {
  b &= 0x7fff7fffu;
  if (F16) {
    const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// m new rows (x, `stride` apart) of head h to rows [off, off + m) of the page that `table`
// names, none if it names none of the cache; NT threads, which meet at named barrier `bar`.
// The rows are fetched before the table's answer is looked at.  A thread keeps its first kHold pieces of 8 elements
// in registers between the maximum and the rounding, so that a page is read once; what a
// larger page has beyond them is read again (from L1 or L2).
template <bool F16, int NT>
__device__ __forceinline__ void k8_write_part(const char* x, long long stride, int m, int d, const K8Div& by_per,
                                              const K8Cache& cc, const int* table, uint8_t* cache, float* scales, int h,
                                              int off, int tid, int bar, float* red) {
  constexpr int kHold = NT == 512 ? 9 : NT == 128 ? 12 : 4;  // 64 rows of 576 or of 192; a few rows
  const int page = k8_read(table), fmt = cc.fmt;
  const int per = d >> 3, n8 = m * per;
  auto piece = [&](int i, int& r, int& c) {
    r = k8_quot(by_per, i);
    c = i - r * per;
  };
  uint4 hold[kHold];
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int i = tid + j * NT;
    int r, c;
    piece(i, r, c);
    if (i < n8) hold[j] = k8_read(reinterpret_cast<const uint4*>(x + r * stride * 2 + c * 16));
  }
  if (page < 0 || page >= cc.n_pages) {
    if (cc.status) atomicOr(cc.status, kStatusIndexRange);
    return;
  }
  float* const scale = scales + (long long)page * cc.Hkv + h;
  const long long row_bytes = (long long)cc.Hkv * d;
  uint8_t* const codes = cache + (long long)page * cc.ps * row_bytes + (long long)h * d;
  const float before = off ? k8_scale(*scale) : 0.f;  // as the attention reads it
  // The maximum, two elements at a time (NaN loses); once more, one by one, where it is infinite: infinities
  // and NaN set no scale.
  float a = 0.f;
  auto reduce = [&](auto&& most) {
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if (tid + j * NT < n8) most(hold[j]);
    for (int i = tid + kHold * NT; i < n8; i += NT) {
      int r, c;
      piece(i, r, c);
      most(k8_read(reinterpret_cast<const uint4*>(x + r * stride * 2 + c * 16)));
    }
  };
  auto meet = [&]() {
#pragma unroll
    for (int s = 16; s; s >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, s));
    if ((tid & 31) == 0) red[tid >> 5] = a;
    asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "n"(NT) : "memory");
    a = red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) a = fmaxf(a, red[w]);
  };
  uint32_t two = 0;
  reduce([&](const uint4& w) {
    two = k8_absmax2<F16>(two, w.x);
    two = k8_absmax2<F16>(two, w.y);
    two = k8_absmax2<F16>(two, w.z);
    two = k8_absmax2<F16>(two, w.w);
  });
  const float2 halves = F16 ? __half22float2(*reinterpret_cast<const __half2*>(&two))
                            : make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
  a = fmaxf(halves.x, halves.y);
  meet();
  if (!(a < INFINITY)) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "n"(NT) : "memory");  // red has been read
    a = 0.f;
    reduce([&](const uint4& w) {
      float v[8];
      k8_unpack8<F16>(w, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = fabsf(v[j]);
        a = fmaxf(a, s < INFINITY ? s : 0.f);
      }
    });
    meet();
  }
  int e = k8_exp_for(a, fmt);
  if (off) e = max(e, k8_exp_at_least(before));
  const float after = k8_pow2(e), inv = k8_pow2(-e);  // x * 2^-e is x / s exactly
  if (off && before != after) {
    // rows that were there before: their codes in the new scale
    const float ratio = before / after;
    for (int i = tid; i < off * per; i += NT) {
      int r, c;
      piece(i, r, c);
      uint2* at = reinterpret_cast<uint2*>(codes + r * row_bytes + c * 8);
      uint2 w = *at;
      uint32_t* u = &w.x;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = k8_code((uint8_t)(u[y] >> (8 * j)), fmt) * ratio;
        u[y] = k8_round2(v[0], v[1], fmt) | (k8_round2(v[2], v[3], fmt) << 16);
      }
      *at = w;
    }
  }
  auto put = [&](int i, const uint4& w) {
    int r, c;
    piece(i, r, c);
    float v[8];
    k8_unpack8<F16>(w, v);
    uint2 o;
    o.x = k8_round2(v[0] * inv, v[1] * inv, fmt) | (k8_round2(v[2] * inv, v[3] * inv, fmt) << 16);
    o.y = k8_round2(v[4] * inv, v[5] * inv, fmt) | (k8_round2(v[6] * inv, v[7] * inv, fmt) << 16);
    *reinterpret_cast<uint2*>(codes + (off + r) * row_bytes + c * 8) = o;
  };
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (tid + j * NT < n8) put(tid + j * NT, hold[j]);
  for (int i = tid + kHold * NT; i < n8; i += NT) {
    int r, c;
    piece(i, r, c);
    put(i, k8_read(reinterpret_cast<const uint4*>(x + r * stride * 2 + c * 16)));
  }
  asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "n"(NT) : "memory");  // red[] and the old scale have been read
  if (tid == 0) *scale = after;
}

// The sequence of token t, by a whole warp: a 32-way search of the offsets.
__device__ __forceinline__ int k8_find_warp(const K8Cache& c, int t, int lane) {
  if (!c.cu) return t / c.s_q;
  int lo = 0, n = c.B;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const int below = __popc(__ballot_sync(~0u, at < n && k8_read(c.cu + lo + at) <= t));
    const int k = max(below - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// A run is the new rows of one page; it has one writer, so the scale and the codes do too.
//
// Where requests bring many rows, a CTA takes a run, a head, and K or V: the first threads
// of the grid's x range find run x over the requests' page counts.  Bound by the bytes (2
// in, 1 out per element) and, a run at a time, by the chain offsets -> rows -> maximum ->
// codes; CTAs enough that an SM holds several.  10 k tokens of 7 prompts, 4 heads of 192 / 128:
// 13.2 us, 2.9 TB/s.
template <bool F16, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : 6) kv8_write_runs_kernel(const __grid_constant__ K8Write a) {
  __shared__ float red[NT / 32];
  __shared__ int sums[NT / 32];
  __shared__ int found[4];  // first token, rows, page of the sequence, offset
  __shared__ const int* found_table;
  pdl_trigger();
  pdl_wait();
  const K8Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y, half = blockIdx.z;
  const int per = (c.B + NT - 1) / NT, b0 = min(tid * per, c.B), b1 = min(b0 + per, c.B);
  K8Seq s = {};
  auto pages = [&](const K8Seq& q) {  // pages that get rows
    const int first = max(q.first, 0);
    return q.n > 0 && q.L > first ? k8_quot(c.by_ps, q.L - 1) - k8_quot(c.by_ps, first) + 1 : 0;
  };
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    s = k8_seq(c, b);
    mine += pages(s);
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int at = inc - mine, total = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    if (x < warp) at += sums[x];
    total += sums[x];
  }
  const int run = blockIdx.x;
  if (run >= total) return;
  if (at <= run && run < at + mine) {
    for (int b = b0;; ++b) {
      if (b1 - b0 > 1) s = k8_seq(c, b);
      const int n = pages(s);
      if (run < at + n) {
        const int first = max(s.first, 0), j = k8_quot(c.by_ps, first) + run - at, pos = max(first, j * c.ps);
        found[0] = s.t0 + pos - s.first;
        found[1] = min((j + 1) * c.ps, s.L) - pos;
        found[2] = j;
        found[3] = pos - j * c.ps;
        found_table = c.table + b * c.tstride + j;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int t = found[0], d = half ? c.dv : c.dqk;
  const char* x = half ? static_cast<const char*>(a.v) + (t * a.vstride + (long long)h * d) * 2
                       : static_cast<const char*>(a.k) + (t * a.kstride + (long long)h * d) * 2;
  k8_write_part<F16, NT>(x, half ? a.vstride : a.kstride, found[1], d, half ? a.by_v : a.by_k, c, found_table,
                         half ? c.v : c.k, half ? c.vs : c.ks, h, found[3], tid, 1, red);
}

// Where they bring a few rows each, a CTA takes the runs that begin in its window of
// tokens (one token, unless there are many), NT threads for K and as many for V.  Bound by
// the chain offsets -> length -> table -> scale: 3.3 us for 64 tokens of 8 heads of 128 / 128.
template <bool F16, int NT, bool SHARED>
__global__ void __launch_bounds__(SHARED ? NT : 2 * NT, 8) kv8_write_kernel(const __grid_constant__ K8Write a) {
  __shared__ float red[2][NT / 32];
  pdl_trigger();
  pdl_wait();
  const K8Cache& c = a.c;
  const int h = blockIdx.y, half = SHARED ? 0 : threadIdx.x / NT, tid = SHARED ? threadIdx.x : threadIdx.x % NT;
  int t = blockIdx.x * a.window;
  const int t_end = min(t + a.window, c.T);
  int b = k8_find_warp(c, t, threadIdx.x & 31);
  K8Seq s = k8_seq(c, b);
  t = max(t, s.t0);  // tokens before the first sequence are no sequence's
  while (t < t_end) {
    while (t >= s.t0 + s.n) {  // behind this sequence (or behind an empty one)
      if (++b >= c.B) return;
      s = k8_seq(c, b);
    }
    const int i = t - s.t0, pos = s.first + i;  // i >= 0: a sequence begins where the one before ends, or earlier
    if (pos < 0) {
      t -= pos;
      continue;
    }
    const int j = k8_quot(c.by_ps, pos), off = pos - j * c.ps, m = min(c.ps - off, s.n - i);
    const bool starts = i == 0 || off == 0 || pos == 0;
    if (starts) {
      const int d = half ? c.dv : c.dqk;
      const char* x = half ? static_cast<const char*>(a.v) + (t * a.vstride + (long long)h * d) * 2
                           : static_cast<const char*>(a.k) + (t * a.kstride + (long long)h * d) * 2;
      k8_write_part<F16, NT>(x, half ? a.vstride : a.kstride, m, d, half ? a.by_v : a.by_k, c, c.table + b * c.tstride + j,
                             half ? c.v : c.k, half ? c.vs : c.ks, h, off, tid, 1 + half, red[half]);
    }
    t += m;
  }
}

cudaError_t launch_kv8_write(K8Write a, cudaStream_t st) {
  const K8Cache& c = a.c;
  if (c.T == 0 || c.B == 0) return cudaSuccess;
  a.by_k = k8_div_of(c.dqk / 8);
  a.by_v = k8_div_of(c.dv / 8);
  // 8 rows per request on average: 10 k tokens of 7 prompts, 4 heads of 192 / 128, took 31 us
  // window by window, 13 run by run
  if (c.T >= 8ll * c.B) {
    const dim3 grid((unsigned)(c.T / c.ps + 2 * c.B), (unsigned)c.Hkv, c.shared ? 1 : 2);
    const auto k = c.dqk > 192 ? (a.f16 ? kv8_write_runs_kernel<true, 512> : kv8_write_runs_kernel<false, 512>)
                               : (a.f16 ? kv8_write_runs_kernel<true, 128> : kv8_write_runs_kernel<false, 128>);
    count_launch();
    return launch_pdl(k, grid, c.dqk > 192 ? 512u : 128u, 0, st, a);
  }
  a.window = (int)max(1ll, (long long)c.T * c.Hkv / (148 * 16));
  const dim3 grid((unsigned)((c.T + a.window - 1) / a.window), (unsigned)c.Hkv);
  const auto k = c.shared ? (a.f16 ? kv8_write_kernel<true, 64, true> : kv8_write_kernel<false, 64, true>)
                          : (a.f16 ? kv8_write_kernel<true, 32, false> : kv8_write_kernel<false, 32, false>);
  count_launch();
  return launch_pdl(k, grid, 64u, 0, st, a);
}

}  // namespace sa
