// C ABI of the operators around the attention: argument validation and
// dispatch.  See include/ra.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <utility>

#include "ra_block.h"
#include "ra_internal.h"

namespace {

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4_or_null(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16_or_null(const void* p) { return p == nullptr || aligned16(p); }

ra_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RA_OK : RA_ERR_CUDA; }

constexpr int kMaxGrid = 65535;          // CUDA's limit on grid y and z
constexpr int64_t kMaxStride = 1LL << 38;  // elements; a tensor map's byte strides end at 2^40

// a * b < limit for positive values whose product may not fit 64 bits.
bool below(int64_t a, int64_t b, int64_t limit) { return a < limit && b < limit && a * b < limit; }

// Strides of a [B, H, N, D] tensor with elements of `size` bytes.
bool valid_strides(const ra_strides* s, int B, int H, int N, int size) {
  if (!s) return false;
  const int64_t st[3] = {s->b, s->h, s->n};
  const int ext[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (ext[i] > 1 && (st[i] < 1 || st[i] >= kMaxStride || (st[i] * size) % 16 != 0)) return false;
  return true;
}

// Rows of D elements that lie clear of one another: of the axes with more than one entry,
// each steps over all that the ones of smaller strides span.
bool rows_apart(const ra_strides& s, int B, int H, int N, int D) {
  int64_t st[3] = {s.b, s.h, s.n};
  int ext[3] = {B, H, N};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (st[j] > st[j + 1]) {
        std::swap(st[j], st[j + 1]);
        std::swap(ext[j], ext[j + 1]);
      }
  int64_t span = D;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;
    if (st[i] < span || ext[i] - 1 > (1LL << 46) / st[i]) return false;  // 2^46 elements: no memory holds them
    span += (ext[i] - 1) * st[i];
  }
  return true;
}

bool valid_dim(int D) { return D == 64 || D == 128; }

bool valid_cache(const ra_kv4_cache* c) {
  if (!c || c->num_pages < 1 || c->Hk < 1 || c->Hk > kMaxGrid / 2 || !valid_dim(c->D)) return false;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return false;
  // The kernels count the cache's rows in 32 bits (2^32 of them are more than the memory holds).
  if (static_cast<int64_t>(c->num_pages) * c->Hk * c->page_size > (1LL << 32) - 1) return false;
  return aligned16(c->k4) && aligned16(c->sk) && aligned16(c->v4) && aligned16(c->sv);
}

// B sequences of T tokens over a block table of max_pages entries each.
bool valid_table(const ra_kv4_cache* c, int B, int T, const int32_t* table, int max_pages) {
  return B >= 1 && B <= kMaxGrid && T >= 1 && T <= (1 << 24) && max_pages >= 1 &&
         max_pages <= (1 << 30) / c->page_size && table && aligned4_or_null(table);
}

// The problem of ra_attn_kv4 without its pointers.
bool valid_kv4_attn(const ra_kv4_cache* c, const ra_kv4_attn* a) {
  if (!c || !a || c->Hk < 1 || !valid_dim(c->D)) return false;
  if (a->B < 1 || a->H < 1 || a->Nq < 1 || a->max_len < 0 || a->H % c->Hk != 0) return false;
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale) || (a->causal != 0 && a->causal != 1)) return false;
  return below(static_cast<int64_t>(a->B) * a->H, a->Nq, (1LL << 31) / c->D);
}

}  // namespace

extern "C" {

size_t ra_rope_table_bytes(const ra_problem* p) {
  if (ra_workspace_bytes(p) == 0) return 0;  // invalid
  return ra::rope_table_len(*p) * sizeof(float2);
}

ra_status ra_rope_table(const ra_problem* p, void* table, size_t bytes, void* stream) {
  const size_t need = ra_rope_table_bytes(p);
  if (need == 0 || !aligned16(table) || bytes < need) return RA_ERR_INVALID_ARG;
  const float2* at = nullptr;
  return from_cuda(ra::launch_rope_table(*p, table, &at, static_cast<cudaStream_t>(stream)));
}

ra_status ra_qk_norm_rope(const ra_problem* p, int Hk, int norm, float eps, int in_dtype, const void* q,
                          const ra_strides* q_st, const void* k, const ra_strides* k_st, const float* q_weight,
                          const float* k_weight, const float* q_bias, const float* k_bias, const int32_t* pos,
                          const void* table, size_t table_bytes, void* q_out, void* k_out, void* stream) {
  if (ra_workspace_bytes(p) == 0 || (in_dtype != RA_DT_F32 && in_dtype != RA_DT_BF16)) return RA_ERR_INVALID_ARG;
  if (norm != RA_NORM_RMS && norm != RA_NORM_LAYER) return RA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || Hk < 1) return RA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->B) * Hk * p->N * p->D >= (1LL << 31)) return RA_ERR_INVALID_ARG;
  if (p->B > kMaxGrid || static_cast<int64_t>(p->H) + Hk > kMaxGrid) return RA_ERR_UNSUPPORTED;
  if ((!q) != (!q_out) || (!k) != (!k_out) || (!q && !k)) return RA_ERR_INVALID_ARG;
  if ((!pos) != (!table) || !aligned4_or_null(pos) || !aligned16_or_null(table)) return RA_ERR_INVALID_ARG;
  if (table && table_bytes < ra_rope_table_bytes(p)) return RA_ERR_INVALID_ARG;
  const int size = in_dtype == RA_DT_BF16 ? 2 : 4;
  ra::NormRopeCall c{};
  const void* x[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const ra_strides* st[2] = {q_st, k_st};
  const float* weight[2] = {q_weight, k_weight};
  const float* bias[2] = {q_bias, k_bias};
  const int heads[2] = {p->H, Hk};
  for (int i = 0; i < 2; ++i) {
    if (!x[i]) continue;
    if (!aligned16(x[i]) || !aligned16(out[i]) || !valid_strides(st[i], p->B, heads[i], p->N, size))
      return RA_ERR_INVALID_ARG;
    if (!aligned4_or_null(weight[i]) || !aligned4_or_null(bias[i])) return RA_ERR_INVALID_ARG;
    c.x[i] = x[i];
    c.out[i] = out[i];
    c.st[i] = *st[i];
    c.weight[i] = weight[i];
    c.bias[i] = bias[i];
    c.heads[i] = heads[i];
  }
  c.norm = norm;
  c.dtype = in_dtype;
  c.eps = eps;
  c.pos = pos;
  c.tab = static_cast<const float2*>(table);
  return from_cuda(ra::launch_norm_rope(*p, c, static_cast<cudaStream_t>(stream)));
}

ra_status ra_kv4_append(const ra_kv4_cache* c, int in_dtype, int B, int T, const void* k, const ra_strides* k_st,
                        const void* v, const ra_strides* v_st, const int32_t* block_table, int max_pages,
                        const int32_t* start, const int32_t* n_new, void* stream) {
  if (!valid_cache(c) || (in_dtype != RA_DT_F32 && in_dtype != RA_DT_BF16)) return RA_ERR_INVALID_ARG;
  if (!valid_table(c, B, T, block_table, max_pages)) return RA_ERR_INVALID_ARG;
  const int size = in_dtype == RA_DT_BF16 ? 2 : 4;
  if (!aligned16(k) || !aligned16(v) || !valid_strides(k_st, B, c->Hk, T, size) ||
      !valid_strides(v_st, B, c->Hk, T, size) || !aligned4_or_null(start) || !aligned4_or_null(n_new))
    return RA_ERR_INVALID_ARG;
  return from_cuda(ra::launch_kv4_append(*c, in_dtype, B, T, k, *k_st, v, *v_st, block_table, max_pages, start, n_new,
                                         static_cast<cudaStream_t>(stream)));
}

ra_status ra_kv4_read(const ra_kv4_cache* c, int out_dtype, int B, int T, const int32_t* block_table, int max_pages,
                      const int32_t* start, const int32_t* n, void* k, void* v, void* stream) {
  if (!valid_cache(c) || (out_dtype != RA_DT_F32 && out_dtype != RA_DT_BF16)) return RA_ERR_INVALID_ARG;
  if (!valid_table(c, B, T, block_table, max_pages)) return RA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4_or_null(start) || !aligned4_or_null(n)) return RA_ERR_INVALID_ARG;
  return from_cuda(ra::launch_kv4_read(*c, out_dtype, B, T, block_table, max_pages, start, n, k, v,
                                       static_cast<cudaStream_t>(stream)));
}

size_t ra_attn_kv4_workspace_bytes(const ra_kv4_cache* c, const ra_kv4_attn* a) {
  if (!valid_kv4_attn(c, a)) return 0;
  const ra::Kv4Plan plan = ra::kv4_plan(*c, *a);
  if (plan.nsplit == 1) return 0;
  const size_t rows = static_cast<size_t>(a->B) * a->H * a->Nq;
  return plan.nsplit * rows * (c->D + 1) * sizeof(float);
}

ra_status ra_attn_kv4(const ra_kv4_cache* c, const ra_kv4_attn* a, const void* q, const int32_t* block_table,
                      const int32_t* seq_lens, const int32_t* q_lens, void* workspace, size_t ws_bytes, void* out,
                      float* lse, void* stream) {
  if (!valid_cache(c) || !valid_kv4_attn(c, a) || !valid_table(c, a->B, a->Nq, block_table, a->max_pages))
    return RA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned4_or_null(lse) || !seq_lens || !aligned4_or_null(seq_lens) ||
      !aligned4_or_null(q_lens))
    return RA_ERR_INVALID_ARG;
  const size_t need = ra_attn_kv4_workspace_bytes(c, a);
  if (need > 0 && (!aligned16(workspace) || ws_bytes < need)) return RA_ERR_INVALID_ARG;
  const ra::Kv4Plan plan = ra::kv4_plan(*c, *a);
  const ra::Kv4Parts parts = ra::kv4_parts(*c, *a, plan, workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = plan.tiles
                      ? ra::launch_kv4_tiles(*c, *a, plan, q, block_table, seq_lens, q_lens, parts, out, lse, st)
                      : ra::launch_kv4_rows(*c, *a, plan, q, block_table, seq_lens, q_lens, parts, out, lse, st);
  if (e == cudaSuccess && plan.nsplit > 1) e = ra::launch_kv4_join(*c, *a, plan, q_lens, parts, out, lse, st);
  return from_cuda(e);
}

ra_status ra_attn_cross(const ra_cross_problem* p, const void* q, const ra_strides* q_st, const void* k,
                        const ra_strides* k_st, const void* v, const ra_strides* v_st, const int32_t* kv_lens,
                        void* out, const ra_strides* out_st, float* lse, void* stream) {
  if (!p || p->B < 1 || p->H < 1 || p->Hk < 1 || p->H % p->Hk != 0 || p->Nq < 1 || p->Nk < 1 || !valid_dim(p->D))
    return RA_ERR_INVALID_ARG;
  if (p->Nq > (1 << 24) || p->Nk > (1 << 24) || !(p->scale > 0.0f) || !std::isfinite(p->scale))
    return RA_ERR_INVALID_ARG;
  if (!below(static_cast<int64_t>(p->B) * p->H, (p->Nq + 255) / 256, 1LL << 30)) return RA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4_or_null(lse) ||
      !aligned4_or_null(kv_lens))
    return RA_ERR_INVALID_ARG;
  if (!valid_strides(q_st, p->B, p->H, p->Nq, 2) || !valid_strides(k_st, p->B, p->Hk, p->Nk, 2) ||
      !valid_strides(v_st, p->B, p->Hk, p->Nk, 2) || !valid_strides(out_st, p->B, p->H, p->Nq, 2))
    return RA_ERR_INVALID_ARG;
  if (!rows_apart(*out_st, p->B, p->H, p->Nq, p->D)) return RA_ERR_INVALID_ARG;
  return from_cuda(ra::launch_attn_cross(*p, q, *q_st, k, *k_st, v, *v_st, kv_lens, out, *out_st, lse,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
