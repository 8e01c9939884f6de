// Internal interface of the operators around the attention: norm + RoPE, the
// 4-bit key/value cache, attention over it and cross attention.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/ra.h"

namespace ra {

constexpr int kNumSMs = 148;  // B200: the split of a call is planned for this many SMs

// Kernels of these operators start while the kernel before them in the stream ends
// (programmatic stream serialisation): each waits for it, in every thread and before
// it touches memory, with grid_wait(), so that a call sees what the stream's order
// promises; grid_trigger() lets the next one start.  A launch's start and a block's
// set-up, 1 to 2 us, then lie under the end of the call before.  The trigger comes
// after the wait, so that a kernel starts only when the one before the one before it has
// ended: no line that that one left in an SM's first cache outlives the start.  Loads are
// ordinary ones (ld_global), which see what grid_wait() makes visible: the read-only path
// (__ldg) does not promise it for memory that is written after the kernel's start, and the
// compiler may move it ahead of the wait.
#ifdef __CUDACC__
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename T>
__device__ __forceinline__ T ld_global(const T* p) { return *p; }
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
#endif

// Heads of two tensors that a CTA of a row-wise kernel walks over, `ahead` at a time,
// for `tiles` token tiles and `per_sm` CTAs at once on an SM: the waves of CTAs times
// their length, a CTA's start counted as two heads, and groups of the larger tensor
// made even.  A grid of many waves ends as its last CTAs do, half a wave of waste.  (Over
// 14 shapes of norm + RoPE, 1 x 1560 to 1 x 32760 tokens, on average 1 % and at most 4 %
// above the best of nine group sizes, which are up to 1.5 times apart.)
inline int heads_per_cta(long long tiles, const int* heads, int per_sm, int ahead) {
  const long long slots = static_cast<long long>(per_sm) * kNumSMs;
  const int most = heads[0] > heads[1] ? heads[0] : heads[1];
  int best = 1;
  long long best_cost = -1;
  for (int n = 1; n <= 64; ++n) {
    const int groups = (most + n - 1) / n, g = (most + groups - 1) / groups;
    const long long ctas = tiles * ((heads[0] + g - 1) / g + (heads[1] + g - 1) / g);
    const long long waves16 = ctas <= 3 * slots ? (ctas + slots - 1) / slots * 16 : ctas * 16 / slots + 8;
    const long long cost = waves16 * ((g + ahead - 1) / ahead * ahead + 2);
    if (best_cost < 0 || cost <= best_cost) {  // of equal ones the fewest CTAs
      best = g;
      best_cost = cost;
    }
  }
  return best;
}

// ---------------------------------------------------------------- norm + RoPE
struct NormRopeCall {
  const void* x[2];  // q, k (NULL: absent)
  ra_strides st[2];
  const float* weight[2];
  const float* bias[2];
  void* out[2];
  int heads[2];
  int norm, dtype;
  float eps;
  const int32_t* pos;
  const float2* tab;
};
cudaError_t launch_norm_rope(const ra_problem& p, const NormRopeCall& c, cudaStream_t st);
cudaError_t read_norm_rope_status(uint32_t* out);

// ---------------------------------------------------------------- 4-bit cache
cudaError_t launch_kv4_append(const ra_kv4_cache& c, int dtype, int B, int T, const void* k, const ra_strides& ks,
                              const void* v, const ra_strides& vs, const int32_t* table, int max_pages,
                              const int32_t* start, const int32_t* n_new, cudaStream_t st);
cudaError_t launch_kv4_read(const ra_kv4_cache& c, int dtype, int B, int T, const int32_t* table, int max_pages,
                            const int32_t* start, const int32_t* n, void* k, void* v, cudaStream_t st);
cudaError_t read_kv4_status(uint32_t* out);

// Attention over the cache.  The rows of a key head, G = H / Hk query heads of
// Nq rows each, are one dense [R = G * Nq, D] block of q and out.
struct Kv4Plan {
  bool tiles;   // 128-row tensor-core tiles, or a few rows per CTA
  int nsplit;   // parts the keys of a row are split into
};
Kv4Plan kv4_plan(const ra_kv4_cache& c, const ra_kv4_attn& a);

// Split results, joined by launch_kv4_join: per part and row an fp32 output
// (normalised by the part's own sum) and the part's log2-sum-exp2.
struct Kv4Parts {
  float* o;     // [nsplit, B * Hk * R, D]
  float* lse2;  // [nsplit, B * Hk * R]
};
Kv4Parts kv4_parts(const ra_kv4_cache& c, const ra_kv4_attn& a, const Kv4Plan& plan, void* ws);
cudaError_t launch_kv4_rows(const ra_kv4_cache& c, const ra_kv4_attn& a, const Kv4Plan& plan, const void* q,
                            const int32_t* table, const int32_t* seq_lens, const int32_t* q_lens,
                            const Kv4Parts& parts, void* out, float* lse, cudaStream_t st);
cudaError_t launch_kv4_join(const ra_kv4_cache& c, const ra_kv4_attn& a, const Kv4Plan& plan,
                            const int32_t* q_lens, const Kv4Parts& parts, void* out, float* lse, cudaStream_t st);

// ---------------------------------------------------------------- 128-row tiles
cudaError_t launch_kv4_tiles(const ra_kv4_cache& c, const ra_kv4_attn& a, const Kv4Plan& plan, const void* q,
                             const int32_t* table, const int32_t* seq_lens, const int32_t* q_lens,
                             const Kv4Parts& parts, void* out, float* lse, cudaStream_t st);
cudaError_t launch_attn_cross(const ra_cross_problem& p, const void* q, const ra_strides& qs, const void* k,
                              const ra_strides& ks, const void* v, const ra_strides& vs, const int32_t* kv_lens,
                              void* out, const ra_strides& os, float* lse, cudaStream_t st);
cudaError_t read_tiles_status(uint32_t* out);

}  // namespace ra
