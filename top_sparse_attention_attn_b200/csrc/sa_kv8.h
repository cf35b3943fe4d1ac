// sa_kv8.h -- serving over a paged KV cache held in 8 bits: device-side
// descriptions and launchers (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sa {

enum { kFmtE4M3 = 0, kFmtInt8 = 1 };
constexpr int kPlanMaxBatch = 24576;  // two prefix arrays of 4 bytes in shared memory

// The cache and the step's tokens (see sa_kv8_cache).
struct K8Cache {
  int fmt, Hkv, dqk, dv, shared, ps, n_pages, B, max_pages;
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
  int window;  // tokens per CTA
};

struct K8Fwd {
  K8Cache c;
  int f16, Hq, G, bs, topk;
  int win;           // rows before the token's own that it sees (INT_MAX: all)
  float scale_log2;  // scale * log2(e)
  const void* q;
  long long qstride;
  const int *idx, *topk_len;
  const float* sinks;
  void* o;
  float* lse;
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
size_t k8_fwd_workspace(const K8Fwd& a);
cudaError_t launch_kv8_fwd(const K8Fwd& a, void* ws, cudaStream_t st);

}  // namespace sa
