// sa_kv8.h -- serving over a paged KV cache held in 8 bits: device-side
// descriptions and launchers (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sa {

enum { kFmtE4M3 = 0, kFmtInt8 = 1 };
constexpr int kPlanMaxBatch = 24576;  // two prefix arrays of 4 bytes in shared memory

// n / d for 0 <= n < 2^31 by a multiplication: with 2^s >= d and m = ceil(2^(31+s) / d),
// m d exceeds 2^(31+s) by less than 2^s, so n m / 2^(31+s) exceeds n / d by less than 1 / d.
struct K8Div {
  uint32_t m;
  int s, d;
};
inline K8Div k8_div_of(int d) {
  K8Div r;
  r.d = d;
  r.s = 0;
  while ((1ll << r.s) < d) ++r.s;
  r.m = (uint32_t)(((1ull << (31 + r.s)) + d - 1) / d);
  return r;
}

// The cache and the step's tokens (see sa_kv8_cache).
struct K8Cache {
  int fmt, Hkv, dqk, dv, shared, ps, n_pages, B, max_pages;
  K8Div by_ps;
  int s_q;  // tokens per sequence when cu is null
  int T;    // rows of the packed token axis
  long long tstride;
  uint8_t *k, *v;
  float *ks, *vs;
  const int *table, *lens, *cu;
  int* status;
};

struct K8Write {
  K8Cache c;
  int f16;
  const void *k, *v;
  long long kstride, vstride;
  int window;        // tokens per CTA
  K8Div by_k, by_v;  // 8-element pieces of a K or V row
};

struct K8Fwd {
  K8Cache c;
  int f16, Hq, G, bs, topk;
  K8Div by_bs;
  // the units of query rows that the kernels work on: rows per chunk, query rows of a unit at
  // most, tokens per unit, query rows of a token in a unit, units over a token's heads, and
  // chunks of a unit that selects (0: every row)
  int chunk, unit_rows, tpt, gdiv, hs, sel_ch;
  int over, keep;   // see k8_begin
  int per_unit;     // CTAs of a unit, with an even share of it each; 0: the line is cut evenly
  K8Div by_tpt, by_gdiv, by_ch, by_per;  // by_ch, by_per: sel_ch and per_unit
  int win;           // rows before the token's own that it sees (2^30: all)
  float scale_log2;  // scale * log2(e)
  const void* q;
  long long qstride;
  const int *idx, *topk_len;
  const float* sinks;
  void* o;
  float* lse;
  int give_up_warp, give_up_wait, give_up_chunk;  // launch_kv8_give_up
};

struct PagePlan {
  int B, max_pages, ps, T, free_cap;
  long long tstride;
  const int *old_lens, *new_lens, *free_pages, *n_free;
  int *table, *seq_lens, *cu;
  long long* slots;
  int *n_free_out, *n_served;
};

cudaError_t launch_page_plan(const PagePlan& p, cudaStream_t st);
cudaError_t launch_kv8_write(K8Write a, cudaStream_t st);
bool k8_built(int dqk, int dv, bool shared);
size_t k8_fwd_workspace(K8Fwd a);
cudaError_t launch_kv8_fwd(K8Fwd a, void* ws, cudaStream_t st);
// The tcgen05 kernel with one wait counted as given up; cudaErrorNotSupported where another kernel runs.
cudaError_t launch_kv8_give_up(K8Fwd a, void* ws, cudaStream_t st);

}  // namespace sa
