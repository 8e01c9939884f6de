// Norm of every head's query and key row, 3D RoPE and the RoPE-aware rotation
// in one pass (papernotes page, key design 1: R M q and R M k).  The norm is over
// the D channels of a head; a norm over all heads' channels of a token, which some
// video transformers have instead, is not this operator.
//
// For each row x of D channels, in fp32:
//   y = (x - mu) * rsqrt(mean((x - mu)^2) + eps) * w + b   (mu = 0 for RMS)
//   then the pair products with the RoPE table and the rotation of ra_rope.cuh,
//   rounded once to bf16.
//
// Bound: HBM (read each row once, write it once; about 10 operations a channel).
// D/8 lanes hold a row, eight channels each, so a row is one or two 16-byte
// loads per lane and its sums are four or three shuffles.  A thread stays with
// one token and walks over heads: positions and table entries are loaded once
// for all of them, and in token-major projections the heads of a token are
// neighbours in memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ra_common.cuh"
#include "ra_rope.cuh"
#include "ra_block.h"

namespace ra {
namespace {

__device__ uint32_t g_norm_status = 0;
std::atomic<bool> g_used{false};  // a program that has never called these does not read their status

constexpr int kThreads = 256;
// Heads whose loads travel while as many are worked on.
__host__ __device__ constexpr int ahead_of(bool bf16) { return bf16 ? 4 : 2; }

struct NormArgs {
  const void* x[2];
  ra_strides st[2];
  const float* weight[2];
  const float* bias[2];
  __nv_bfloat16* out[2];
  int heads[2];
  int groups_q;      // head groups of q; the groups of k follow
  int group;         // heads per group
  int N;
  float eps;
  const int32_t* pos;
  const float2* tab;
  SegInfo s;
};

__device__ __forceinline__ float group_sum(float v, int lpt) {
  for (int o = lpt >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Half rotation of the RoPE'd rows of a warp's tokens: outputs d and d + 1 are
// the sum and the difference, over sqrt(2), of channels u and u + Dj/2 of the row
// (RopePlan::hp), which other lanes hold.  They cross in shared memory in four planes,
// channel e in plane e mod 4 at e / 4: a lane's u advance by four from lane to lane,
// so that its reads are neighbours, and the tokens lie where neither reads nor writes
// meet in a bank (rows as they are met four at a time: 48 wavefronts a head, not 16).
template <int kD>
struct HalfRows {
  static constexpr int kTok = 256 / kD, kTokStride = kD / 4;
  static constexpr int kPlane = kTok * kTokStride + (kD == 64 ? 8 : 16);
  int put, get[4];  // get: the places of u and u + Dj/2
  static __device__ __forceinline__ int base(int tok) {
    return tok * kTokStride + (kD == 64 ? (tok >> 1) * 8 : tok * 16);
  }
  __device__ __forceinline__ void init(const RopePlan& rp, int tok, int c0) {
    put = base(tok) + (c0 >> 2);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int u = (rp.hp[p] & 0xFFFFu) >> 2, w = rp.hp[p] >> 18;
      get[p] = ((u & 3) * kPlane + base(tok) + (u >> 2)) | ((w & 3) * kPlane + base(tok) + (w >> 2)) << 16;
    }
  }
  __device__ __forceinline__ void apply(float* row, float* x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(row + i * kPlane + put) = make_float2(x[i], x[i + 4]);
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float u = row[get[p] & 0xFFFF], w = row[get[p] >> 16];
      x[2 * p] = __fmul_rn(__fadd_rn(u, w), 0.70710678118654752440f);
      x[2 * p + 1] = __fmul_rn(__fsub_rn(u, w), 0.70710678118654752440f);
    }
    __syncwarp();
  }
};

// kRot: the rotation, or -1 for the norm alone.
template <bool kBf16, int kD, int kRot, bool kLayer>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const NormArgs a) {
  constexpr int kLanes = kD / 8, kTok = 32 / kLanes;  // lanes per row, tokens per warp
  constexpr int kAhead = ahead_of(kBf16);
  constexpr bool kHalf = kRot == RA_ROT_HALF;
  __shared__ __align__(16) float rows[kHalf ? kThreads / 32 : 1][kHalf ? kAhead : 1][kHalf ? 4 * HalfRows<kD>::kPlane : 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok = lane / kLanes, c0 = (lane % kLanes) * 8;
  const int which = static_cast<int>(blockIdx.y) >= a.groups_q ? 1 : 0;
  const int h0 = (blockIdx.y - (which ? a.groups_q : 0)) * a.group;
  const int h1 = min(h0 + a.group, a.heads[which]);
  const int n = (blockIdx.x * (kThreads / 32) + warp) * kTok + tok;
  const bool in_range = n < a.N;
  const int nc = in_range ? n : a.N - 1;  // lanes past the end work on the last row and do not store
  const size_t src = blockIdx.z * a.st[which].b + nc * a.st[which].n + c0;
  grid_wait();
  grid_trigger();
  Raw8<kBf16> next[kAhead] = {};
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (h0 + i < h1) load_raw8<kBf16, false>(a.x[which], src + (h0 + i) * a.st[which].h, next[i]);
  RopePlan rp;
  HalfRows<kD> half;
  float2 cf[4];
  if constexpr (kRot >= 0) {
    rp.init(a.s, c0);
    if constexpr (kHalf) half.init(rp, tok, c0);
    int gp[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) gp[j] = ld_global(a.pos + 3 * nc + j);
    rope_coef8p<false>(a.s, rp, a.tab, gp, cf, &g_norm_status);
  }
  float w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = a.weight[which] ? ld_global(a.weight[which] + c0 + i) : 1.0f;
    b[i] = a.bias[which] ? ld_global(a.bias[which] + c0 + i) : 0.0f;
  }
  const size_t hn = static_cast<size_t>(a.N) * kD;
  __nv_bfloat16* dst = a.out[which] + blockIdx.z * hn * a.heads[which] + static_cast<size_t>(nc) * kD + c0;
  for (int hb = h0; hb < h1; hb += kAhead) {
    Raw8<kBf16> cur[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      cur[i] = next[i];
      if (hb + kAhead + i < h1) load_raw8<kBf16, false>(a.x[which], src + (hb + kAhead + i) * a.st[which].h, next[i]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {  // heads past the last one are worked on but not stored
      const int h = hb + u;
      float x[8];
      unpack8<kBf16>(cur[u], x);
      if constexpr (kLayer) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i];
        const float mu = group_sum(s, kLanes) * (1.0f / kD);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] -= mu;
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      const float r = rsqrtf(fmaf(group_sum(ss, kLanes), 1.0f / kD, a.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i] * r, w[i], b[i]);
      if constexpr (kRot >= 0) rope_apply8(a.s, rp, kHalf ? RA_ROT_NONE : kRot, cf, c0, x, nullptr);
      if constexpr (kHalf) half.apply(rows[warp][u], x);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      if (in_range && h < h1) *reinterpret_cast<uint4*>(dst + h * hn) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool kBf16, int kD, int kRot>
cudaError_t launch_norm(const NormArgs& a, bool layer, dim3 grid, cudaStream_t st) {
  return layer ? launch_early(norm_rope_kernel<kBf16, kD, kRot, true>, grid, kThreads, 0, st, a)
               : launch_early(norm_rope_kernel<kBf16, kD, kRot, false>, grid, kThreads, 0, st, a);
}

template <bool kBf16, int kD>
cudaError_t launch_rot(const NormArgs& a, int rot, bool layer, dim3 grid, cudaStream_t st) {
  switch (rot) {
    case RA_ROT_NONE: return launch_norm<kBf16, kD, RA_ROT_NONE>(a, layer, grid, st);
    case RA_ROT_INTERLEAVED: return launch_norm<kBf16, kD, RA_ROT_INTERLEAVED>(a, layer, grid, st);
    case RA_ROT_HALF: return launch_norm<kBf16, kD, RA_ROT_HALF>(a, layer, grid, st);
    case RA_ROT_FULL: return launch_norm<kBf16, kD, RA_ROT_FULL>(a, layer, grid, st);
    default: return launch_norm<kBf16, kD, -1>(a, layer, grid, st);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const ra_problem& p, const NormRopeCall& c, cudaStream_t st) {
  g_used.store(true, std::memory_order_relaxed);
  NormArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = c.x[i];
    a.st[i] = c.st[i];
    a.weight[i] = c.weight[i];
    a.bias[i] = c.bias[i];
    a.out[i] = static_cast<__nv_bfloat16*>(c.out[i]);
    a.heads[i] = c.x[i] ? c.heads[i] : 0;
  }
  a.N = p.N;
  a.eps = c.eps;
  a.pos = c.pos;
  a.tab = c.tab;
  a.s = seg_info(p);
  const int tok = (kThreads / 32) * (256 / p.D);  // tokens per CTA
  const int tiles = (p.N + tok - 1) / tok;
  // A CTA begins with a chain of loads (positions, table), which eight heads do not
  // pay for (32760 tokens x 80 heads: 285 us against 211).
  const int group = heads_per_cta(static_cast<long long>(tiles) * p.B, a.heads, 3, ahead_of(c.dtype == RA_DT_BF16));
  a.group = group;
  a.groups_q = (a.heads[0] + group - 1) / group;
  const dim3 grid(tiles, a.groups_q + (a.heads[1] + group - 1) / group, p.B);
  const int rot = c.pos ? p.rot : -1;
  const bool layer = c.norm == RA_NORM_LAYER;
  if (c.dtype == RA_DT_BF16)
    return p.D == 64 ? launch_rot<true, 64>(a, rot, layer, grid, st) : launch_rot<true, 128>(a, rot, layer, grid, st);
  return p.D == 64 ? launch_rot<false, 64>(a, rot, layer, grid, st) : launch_rot<false, 128>(a, rot, layer, grid, st);
}

cudaError_t read_norm_rope_status(uint32_t* out) {
  *out = 0;
  if (!g_used.load(std::memory_order_relaxed)) return cudaSuccess;
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_norm_status, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_norm_status, &zero, sizeof(uint32_t));
}

}  // namespace ra
