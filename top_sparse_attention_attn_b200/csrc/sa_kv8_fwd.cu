// sa_kv8_fwd.cu -- attention over a paged KV cache held in 8 bits (sa_kv8_fwd).
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_kv8_device.cuh"
#include "sa_launch.h"

namespace sa {

bool k8_built(int dqk, int dv, bool shared) {
  if (shared) return (dqk == 128 && dv == 128) || (dqk == 576 && dv == 512);
  return (dqk == 64 && dv == 64) || (dqk == 128 && dv == 128) || (dqk == 192 && dv == 128);
}

// One CTA per (token, query head): scores of 128 rows at a time, one per thread,
// an online softmax, then each thread sums its output columns over the rows.
__global__ void __launch_bounds__(128) k8_row_kernel(K8Fwd a) {
  __shared__ float q[576], p[128], red[4];
  __shared__ long long at[128];
  __shared__ float vsc[128];
  const K8Cache& c = a.c;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / a.G, tid = threadIdx.x;
  const int b = k8_find(c, t);
  const K8Seq s = k8_seq(c, b);
  const int i = t - s.t0;
  if (i < 0 || i >= s.n) return;
  const int ta = s.first + i;
  for (int d = tid; d < c.dqk; d += 128) q[d] = k8_in(a.q, t * a.qstride + (long long)hq * c.dqk + d, a.f16);
  const int lo = a.win >= ta ? 0 : ta - a.win;
  const long long unit = (long long)t * c.Hkv + h;
  int slots = a.topk;
  if (a.topk_len) slots = min(slots, max(0, __ldg(a.topk_len + unit)));
  const int first = a.topk ? 0 : lo, n_rows = ta < 0 ? 0 : a.topk ? slots * a.bs : ta + 1;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int n_o = (c.dv + 127) / 128;
  for (int r0 = first; r0 < n_rows; r0 += 128) {
    int row = r0 + tid;
    bool see = row < n_rows;
    if (see && a.topk) {
      const int x = __ldg(a.idx + unit * a.topk + row / a.bs);
      if (x >= 0 && (long long)x * a.bs >= s.L && c.status) atomicOr(c.status, kStatusIndexRange);
      see = x >= 0 && (long long)x * a.bs < s.L;
      row = see ? x * a.bs + row % a.bs : 0;
    }
    see = see && row >= lo && row <= ta;
    const int page = see ? k8_page(c, b, row) : -1;
    see = page >= 0;
    float z = -INFINITY;
    __syncthreads();
    at[tid] = -1;
    vsc[tid] = 0.f;
    if (see) {
      const long long rr = ((long long)page * c.ps + row % c.ps) * c.Hkv + h;
      const uint8_t* k = c.k + rr * c.dqk;
      float acc = 0.f;
      for (int d = 0; d < c.dqk; ++d) acc = fmaf(q[d], k8_code(k[d], c.fmt), acc);
      z = acc * k8_scale(c.ks[(long long)page * c.Hkv + h]) * a.scale_log2;
      at[tid] = rr * (c.shared ? c.dqk : c.dv);
      vsc[tid] = k8_scale((c.shared ? c.ks : c.vs)[(long long)page * c.Hkv + h]);
    }
    float mx = z;
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = mx == -INFINITY ? 0.f : mx, alpha = exp2f(m - base);
    m = mx;
    float pr = see ? exp2f(z - base) : 0.f;
    p[tid] = pr;
    __syncthreads();
#pragma unroll
    for (int d = 16; d; d >>= 1) pr += __shfl_xor_sync(~0u, pr, d);
    if ((tid & 31) == 0) red[tid >> 5] = pr;
    __syncthreads();
    l = l * alpha + (red[0] + red[1] + red[2] + red[3]);
    for (int j = 0; j < n_o; ++j) {
      const int d = tid + j * 128;
      if (d >= c.dv) break;
      float acc = o[j] * alpha;
      for (int r = 0; r < 128; ++r)
        if (at[r] >= 0) acc = fmaf(p[r], vsc[r] * k8_code((c.shared ? c.k : c.v)[at[r] + d], c.fmt), acc);
      o[j] = acc;
    }
  }
  if (a.sinks) {
    const float sink = __ldg(a.sinks + hq) * 1.4426950408889634f, mx = fmaxf(m, sink);
    const float base = mx == -INFINITY ? 0.f : mx, alpha = exp2f(m - base);
    l = l * alpha + exp2f(sink - base);
    for (int j = 0; j < n_o; ++j) o[j] *= alpha;
    m = mx;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int j = 0; j < n_o; ++j) {
    const int d = tid + j * 128;
    if (d >= c.dv) break;
    const float v = l == 0.f ? 0.f : o[j] * (l == l ? inv : l);
    const long long e = ((long long)t * a.Hq + hq) * c.dv + d;
    if (a.f16) static_cast<__half*>(a.o)[e] = __float2half_rn(v);
    else static_cast<bf16*>(a.o)[e] = __float2bfloat16_rn(v);
  }
  if (tid == 0) a.lse[(long long)t * a.Hq + hq] = l == 0.f ? INFINITY : 0.6931471805599453f * (m + log2f(l));
}

size_t k8_fwd_workspace(const K8Fwd&) { return 0; }

cudaError_t launch_kv8_fwd(const K8Fwd& a, void*, cudaStream_t st) {
  if (a.c.T == 0 || a.c.B == 0) return cudaSuccess;
  k8_row_kernel<<<dim3((unsigned)a.c.T, (unsigned)a.Hq), 128, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace sa
