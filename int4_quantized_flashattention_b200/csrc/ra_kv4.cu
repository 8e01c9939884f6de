// The paged 4-bit key/value cache: quantising new tokens into it, reading
// tokens back, and attention of a few query rows per key head over it.
// Quantisation is the INT4 rule of the prologue's Q and K (per token and head,
// symmetric; gecl notes "Key Insight").
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ra_common.cuh"
#include "ra_rope.cuh"
#include "ra_block.h"
#include "ra_kv4.cuh"

namespace ra {
namespace {

__device__ uint32_t g_kv4_status = 0;
std::atomic<bool> g_used{false};  // a program that has never called these does not read their status

constexpr int kThreads = 256;
// CTAs at once on an SM (4680 tokens x 40 heads, append and read together: 65.4 us with
// 3 and 6, 65.6 with 4 and 4, 61.7 with 4 and 6, 66.8 with 5, whose registers spill, and 6).
constexpr int kAppendPerSm = 4, kReadPerSm = 6;
// Heads whose loads travel while as many are worked on.
__host__ __device__ constexpr int append_ahead(bool bf16) { return bf16 ? 4 : 2; }
constexpr int kReadAhead = 4;

// ---------------------------------------------------------------- append and read
struct CacheArgs {
  uint8_t* codes[2];      // k4, v4
  float* scale[2];        // sk, sv
  const void* x[2];       // append: k, v
  void* y[2];             // read: k, v
  ra_strides st[2];       // of x
  const int32_t* table;
  const int32_t* start;
  const int32_t* count;
  int num_pages, page_log2, max_pages, Hk, T;
  int groups, group;      // head groups per tensor, heads per group
};

// Tokens of this CTA's sequence that the call holds; 0 for a bad count (which is reported).
__device__ __forceinline__ int token_count(const CacheArgs& a) {
  if (!a.count) return a.T;
  const int cnt = ld_global(a.count + blockIdx.z);
  if (cnt >= 0 && cnt <= a.T) return cnt;
  atomicOr(&g_kv4_status, kStatusBadPosition);
  return 0;
}

// The cache row (page * Hk * page_size + slot, head 0) of token t of this CTA's sequence, which
// begins at s, or -1 when it has no valid place (which is reported).
__device__ __forceinline__ long long token_row(const CacheArgs& a, int s, int t) {
  const long long pos = static_cast<long long>(s) + t;
  const long long pi = pos >> a.page_log2;
  if (s < 0 || pi >= a.max_pages) {
    atomicOr(&g_kv4_status, kStatusBadPosition);
    return -1;
  }
  const int page = ld_global(a.table + static_cast<size_t>(blockIdx.z) * a.max_pages + pi);
  if (page < 0 || page >= a.num_pages) {
    atomicOr(&g_kv4_status, kStatusBadPosition);
    return -1;
  }
  return ((static_cast<long long>(page) * a.Hk) << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
}

// The largest magnitude among eight bf16, NaN if one of them is.
__device__ __forceinline__ float max_abs_bf16(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  auto mag = [](uint32_t w) {
    w &= 0x7FFF7FFFu;
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  };
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(mag(a), mag(b)), __hmax2_nan(mag(c), mag(d)));
  const float2 f = __bfloat1622float2(m);
  return max_nan(f.x, f.y);
}

// D/8 lanes per token row, eight channels each; a thread stays with kPer tokens
// and walks over heads, kAhead rows at a time, so its pages are looked up once, and
// the loads of the next rows travel while it works.  kPer is 1 unless there are fewer heads
// than rows at a time (one head of 64 channels, 12 x 3345 tokens, append and read together: 23.4
// us with one token a thread, 13.7 with four).  Bound: HBM.
template <bool kBf16, int kD, int kPer>
__global__ void __launch_bounds__(kThreads, kAppendPerSm) kv4_append_kernel(const CacheArgs a) {
  constexpr int kLanes = kD / 8, kTok = 32 / kLanes, kAhead = append_ahead(kBf16), kHeads = kAhead / kPer;
  constexpr int kNext = kThreads / kLanes;  // from one token of a thread to the next
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kNext * kPer + warp * kTok + lane / kLanes;
  const int c0 = (lane % kLanes) * 8;
  const int which = static_cast<int>(blockIdx.y) >= a.groups ? 1 : 0;
  const int h0 = (blockIdx.y - (which ? a.groups : 0)) * a.group, h1 = min(h0 + a.group, a.Hk);
  grid_wait();
  grid_trigger();
  const int cnt = token_count(a);
  const size_t src = blockIdx.z * a.st[which].b + static_cast<size_t>(t) * a.st[which].n + c0;
  // Row i of a batch: head i / kPer, token i % kPer.  Padding is worked on as zeros.
  Raw8<kBf16> next[kAhead];
  auto load = [&](int hb, int i, Raw8<kBf16>& r) {
    const int h = hb + i / kPer, n = (i % kPer) * kNext;
    if (h < h1 && t + n < cnt) load_raw8<kBf16, false>(a.x[which], src + h * a.st[which].h + n * a.st[which].n, r);
    else r = Raw8<kBf16>{};
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(h0, i, next[i]);
  long long row[kPer];  // -1: not stored
  const int s = a.start ? ld_global(a.start + blockIdx.z) : 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) row[i] = t + i * kNext < cnt ? token_row(a, s, t + i * kNext) : -1;
  // The maxima of kAhead rows are reduced together: each exchange halves the rows a
  // lane holds before it halves the lanes, so that a lane ends with one row's maximum,
  // and one division by and one of it serve all rows (9 exchanges and 2 divisions for
  // four rows, not 16 and 8: the kernel is bound by its instructions).
  constexpr int kTop = kLanes / 2, kLast = kAhead == 4 ? kTop / 2 : kTop;  // lane bits that select the row
  const bool second = (lane & kLast) != 0;
  const int mine = (kAhead == 4 && (lane & kTop) ? 2 : 0) + (second ? 1 : 0);
  long long my_row = row[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i)
    if (mine % kPer == i) my_row = row[i];
  for (int hb = h0; hb < h1; hb += kHeads) {
    Raw8<kBf16> cur[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      cur[i] = next[i];
      load(hb + kHeads, i, next[i]);
    }
    float m[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if constexpr (kBf16) {
        const uint4 w = cur[u].u[0];
        m[u] = max_abs_bf16(w.x, w.y, w.z, w.w);
      } else {
        float x[8];
        unpack8<kBf16>(cur[u], x);
        m[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[u] = max_nan(m[u], fabsf(x[i]));
      }
    }
    if constexpr (kAhead == 4) {
      const bool upper = (lane & kTop) != 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float got = __shfl_xor_sync(0xFFFFFFFFu, upper ? m[u] : m[u + 2], kTop);
        m[u] = max_nan(upper ? m[u + 2] : m[u], got);
      }
    }
    const float got = __shfl_xor_sync(0xFFFFFFFFu, second ? m[0] : m[1], kLast);
    float top = max_nan(second ? m[1] : m[0], got);
#pragma unroll
    for (int o = kLast >> 1; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    // What is not finite stays so: the row's scale is NaN, whatever its codes then are.  (Codes of zeros
    // took a test and a selection a row: 23.9 us against 21.9 for 40 heads x 4680 tokens.)
    if (top == INFINITY) top = NAN;
    if (top < kKv4Tiny) top = 0.0f;  // 7 / top would leave fp32's range
    const float inv = top == 0.0f ? 0.0f : __fdiv_rn(7.0f, top);
    const float scale = __fdiv_rn(top, 7.0f);
    const int my_head = hb + mine / kPer;
    if ((lane & (kLast - 1)) == 0 && my_head < h1 && my_row >= 0)
      a.scale[which][static_cast<size_t>(my_row) + (static_cast<size_t>(my_head) << a.page_log2)] = scale;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u / kPer;
      const int from = (kAhead == 4 && (u & 2) ? kTop : 0) + (u & 1 ? kLast : 0);
      const float f = __shfl_sync(0xFFFFFFFFu, inv, from, kLanes);
      float x[8];
      unpack8<kBf16>(cur[u], x);
      uint32_t bits[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) quant4_bits2(x[i], x[i + 1], f, f, bits + i);
      if (h < h1 && row[u % kPer] >= 0) {
        const size_t at = static_cast<size_t>(row[u % kPer]) + (static_cast<size_t>(h) << a.page_log2);
        *reinterpret_cast<uint32_t*>(a.codes[which] + at * (kD / 2) + (c0 >> 1)) = pack8_bits(bits);
      }
    }
  }
}

// The same walk the other way.  A lane writes 16 bytes of a row, so that a
// warp's stores are whole lines: eight bf16 channels, or four fp32 channels from
// one half of a code word.  Bound: HBM, the output most of it.
template <bool kBf16, int kD, int kPer>
__global__ void __launch_bounds__(kThreads, kReadPerSm) kv4_read_kernel(const CacheArgs a) {
  constexpr int kCh = kBf16 ? 8 : 4, kLanes = kD / kCh, kTok = 32 / kLanes, kHeads = kReadAhead / kPer;
  constexpr int kNext = kThreads / kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kNext * kPer + warp * kTok + lane / kLanes;
  const int c0 = (lane % kLanes) * kCh;
  const int which = static_cast<int>(blockIdx.y) >= a.groups ? 1 : 0;
  const int h0 = (blockIdx.y - (which ? a.groups : 0)) * a.group, h1 = min(h0 + a.group, a.Hk);
  grid_wait();
  grid_trigger();
  const int s = a.start ? ld_global(a.start + blockIdx.z) : 0;
  const int cnt = token_count(a);
  const uint8_t* codes[kPer];
  const float* scales[kPer];  // NULL: not read
  bool any = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long row = t + i * kNext < cnt ? token_row(a, s, t + i * kNext) : -1;
    codes[i] = a.codes[which] + row * (kD / 2) + ((c0 >> 1) & ~3);
    scales[i] = row < 0 ? nullptr : a.scale[which] + row;
    any = any || row >= 0;
  }
  if (!any) return;
  uint32_t next_w[kReadAhead];
  float next_s[kReadAhead];
  auto load = [&](int hb, int i, uint32_t& w, float& scale) {  // row i: head i / kPer, token i % kPer
    const int h = hb + i / kPer;
    w = 0;
    scale = 0.0f;
    if (h < h1 && (kPer == 1 || scales[i % kPer])) {
      const size_t at = static_cast<size_t>(h) << a.page_log2;
      w = ld_global(reinterpret_cast<const uint32_t*>(codes[i % kPer] + at * (kD / 2)));
      scale = ld_global(scales[i % kPer] + at);
    }
  };
#pragma unroll
  for (int i = 0; i < kReadAhead; ++i) load(h0, i, next_w[i], next_s[i]);
  for (int hb = h0; hb < h1; hb += kHeads) {
    uint32_t cur_w[kReadAhead];
    float cur_s[kReadAhead];
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
      cur_w[i] = next_w[i];
      cur_s[i] = next_s[i];
      load(hb + kHeads, i, next_w[i], next_s[i]);
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      const int h = hb + u / kPer;
      if (h >= h1) break;
      if (kPer > 1 && !scales[u % kPer]) continue;
      const uint32_t w = cur_w[u] >> (4 * (c0 & 4));
      float y[kCh];
#pragma unroll
      for (int i = 0; i < kCh; ++i)
        y[i] = static_cast<float>(static_cast<int>(w << (28 - 4 * i)) >> 28) * cur_s[u];
      const size_t o =
          ((static_cast<size_t>(blockIdx.z) * a.Hk + h) * a.T + t + (u % kPer) * kNext) * kD + c0;
      if constexpr (kBf16)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y[which]) + o) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(a.y[which]) + o) = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
}

// ---------------------------------------------------------------- attention, few rows
// A CTA takes the query rows of one key head, at most 8 * NT, and one part of its
// keys; its four warps take 32-key steps in turn, each with its own running
// maximum, sum and output, joined at the end.  Bound: HBM, the codes and
// scales of the keys read once ((D + 8) bytes a key and head).
//   * Codes and scales go to shared memory by 16-byte asynchronous copies, a
//     ring of kStages steps per warp; warps never wait for one another.
//   * S^T = K Q^T with mma.m16n8k16: 16 keys by 8 rows, so a single query row
//     costs half of what rows as M would.  tcgen05 (M >= 64) would spend 128
//     rows on one.  The channels of a k step are free to choose as long as Q
//     uses the same: a lane's 16 bytes of a key are its four words, and the
//     nibbles j and j + 4 of a word make an f16 pair (codes_f16_lo / _hi).
//   * Products run in f16, in which the codes are exact.  (As f16's subnormals
//     2^-24 (code + 8), with 8 times Q's sum taken off beforehand, they save an
//     operation a pair, 137 us against 144 at 16 x 40 heads x 8191 keys; but the sums
//     then lose bits: log-sum-exp 1.3e-6 off at nine keys, 4e-8 now.)  Each row of Q is
//     brought to a largest value of about 2^14 by a power of two of its own: f16's 11 bits
//     hold bf16's 8, and what lies 2^28 below the row's largest value loses bits.  (One
//     power of two for all rows of the CTA saved four multiplications a step and made rows
//     of zeros of those beside a much larger or an infinite one.)  The keys' scales
//     multiply S in fp32.  The values' scales multiply P in fp32, relative
//     to a power of two not below the largest that the row has seen so far, so that the one
//     rounding of P to f16 costs 2^-11 (bf16 cost 2^-8: 1.6 times the error of the
//     output's own rounding; now none that shows).  Below 2^-25 of it a product loses
//     bits.  Keys that a row does not see leave its reference alone, whatever they hold.
//   * O^T = V^T P^T, again 16 channels by 8 rows: P^T comes out of S^T by one
//     8x8 transpose per 8 keys, V^T by pairing the words of two keys.  The
//     pairs are keys x and x + 4 of each eight, which puts the rows that the
//     lanes read at the same time into different banks.
struct RowsArgs {
  const uint8_t* k4;
  const float* sk;
  const uint8_t* v4;
  const float* sv;
  const __nv_bfloat16* q;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* q_lens;
  __nv_bfloat16* out;
  float* lse;
  Kv4Parts parts;
  int num_pages, page_log2, max_pages, Hk, G, Nq, causal, nsplit;
  float scale_log2;  // scale * log2(e)
};

constexpr int kRowWarps = 4;
constexpr int kStep = 32;    // keys per warp and step
constexpr int kStages = 3;
// CTAs at once on an SM, as many as the registers allow without spilling (16 x 40 heads x 8191
// keys: D = 128, one row: 3, 4 and 5 take 147, 146 and 162 us, 16 rows: 2, 3 and 4 take 228, 235
// and 428; D = 64, one row: 4, 5 and 6 take 95, 98 and 100, 16 rows: 2, 3 and 4 take 152, 135 and 141).
template <int D, int NT> constexpr int kRowsPerSm = NT == 1 ? 4 : D == 128 ? 2 : 3;
constexpr float kLazy = 4.0f;  // the reference maximum moves when a score passes it by this (powers of two)
constexpr float kNone = -3e38f;  // reference of a row that has met no key: finite, so that -inf - kNone is -inf
constexpr float kPUp = 2048.0f;  // P goes to f16 times this: at most 2^(4 + 11), below 2^-25 it loses bits
constexpr uint32_t kPUpBits = (127u + 127 + 11) << 23;  // less the bits of a power of two: those of kPUp over it

template <int D>
struct RowsCfg {
  static constexpr int kRow = D / 2;                    // code bytes of a key
  static constexpr int kChunks = kRow / 16;             // 16-byte chunks of a key
  static constexpr int oV = kStep * kRow;
  static constexpr int oSk = 2 * kStep * kRow;
  static constexpr int oSv = oSk + kStep * 4;
  static constexpr int kStage = oSv + kStep * 4;
  static constexpr int kSmem = kRowWarps * kStages * kStage;
};

// Place of key x (0..15) of a 16-key group in the K tile, which the lanes of
// row group g read at places g and 8 + g: keys 8j + g/2 (g even) or 8j + 4 + g/2.
__device__ __forceinline__ int k_place(int x) { return (x & 8) | ((x & 3) << 1) | ((x >> 2) & 1); }
// Key of place g of eight.
__device__ __forceinline__ int key_of(int g) { return (g >> 1) | ((g & 1) << 2); }

template <int D, int NT>
__global__ void __launch_bounds__(kRowWarps * 32, kRowsPerSm<D, NT>) kv4_rows_kernel(const RowsArgs a) {
  using C = RowsCfg<D>;
  constexpr int kW = D / 32;        // code words of a key per lane (K)
  constexpr int kM = D / 16;        // 16-channel tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q4 = lane & 3;
  const int bh = blockIdx.x, b = bh / a.Hk, hk = bh % a.Hk;
  const int split = blockIdx.y;
  const int R = a.G * a.Nq;
  uint32_t bad = 0;
  grid_wait();
  const int len = clamp_len(ld_global(a.seq_lens + b), a.max_pages << a.page_log2, &bad);
  const int ql = a.q_lens ? clamp_len(ld_global(a.q_lens + b), a.Nq, &bad) : a.Nq;
  // Steps of this CTA: [t0, t1), every kRowWarps-th for this warp.
  const int nstep = (len + kStep - 1) / kStep;
  const int per = (nstep + a.nsplit - 1) / a.nsplit;
  const int t0 = min(split * per, nstep), t1 = min(t0 + per, nstep);

  // A step's copies: lane x copies the 16 bytes at 16 x of every 512 (of K and of
  // V), lanes 0-7 the scales.  Everything that does not change is computed here.
  constexpr int kCopies = 16 * C::kRow / 512;  // per 16 keys, and 8 keys apart where there are two
  const int x0 = lane / C::kChunks, ch0 = lane % C::kChunks;
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kStage;
  const uint32_t kdst = k_place(x0) * C::kRow + ch0 * 16;
  const uint32_t vdst = C::oV + x0 * C::kRow + (C::kChunks == 4 ? ch0 ^ (x0 & 2) : ch0) * 16;
  const uint32_t sdst = (lane < 4 ? C::oSk : C::oSv) + (lane & 3) * 16;
  const uint8_t* const ksrc = a.k4 + lane * 16;
  const uint8_t* const vsrc = a.v4 + lane * 16;
  const float* const ssrc = (lane < 4 ? a.sk : a.sv) + (lane & 3) * 4;
  const int32_t* const tb = a.table + static_cast<size_t>(b) * a.max_pages;
  const int page_mask = (1 << a.page_log2) - 1;
  // Rows of the cache fit 32 bits: 2^32 rows of 72 bytes and more exceed the memory.
  const uint32_t page_rows = static_cast<uint32_t>(a.Hk) << a.page_log2, head_row = static_cast<uint32_t>(hk) << a.page_log2;
  auto load = [&](int t, int stage) {
    const uint32_t st = ring + stage * C::kStage;
    const int left = t < t1 ? len - t * kStep : 0;  // keys of this step
    auto row_of = [&](int key0) -> uint32_t {
      uint32_t page = static_cast<uint32_t>(ld_global(tb + (key0 >> a.page_log2)));
      if (page >= static_cast<uint32_t>(a.num_pages)) {
        bad |= kStatusBadPosition;
        page = 0;
      }
      return page * page_rows + head_row + (key0 & page_mask);
    };
    auto copy = [&](int s, uint32_t row, uint32_t bytes) {  // bytes 0: the places are filled with zeros
      const uint8_t* const ks = ksrc + static_cast<uint64_t>(row) * C::kRow;
      const uint8_t* const vs = vsrc + static_cast<uint64_t>(row) * C::kRow;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        cp_async16(st + kdst + (16 * s + 8 * i) * C::kRow, ks + 512 * i, bytes);
        cp_async16(st + vdst + (16 * s + 8 * i) * C::kRow, vs + 512 * i, bytes);
      }
      if (lane < 8) cp_async16(st + sdst + 64 * s, ssrc + row, bytes);
    };
    const uint32_t row0 = left > 0 ? row_of(t * kStep) : 0u;
    uint32_t row1 = row0 + 16;  // the same page, but for pages of 16
    if (left <= 16) row1 = 0;
    else if (a.page_log2 == 4) row1 = row_of(t * kStep + 16);
    copy(0, row0, left > 0 ? 16u : 0u);
    copy(1, row1, left > 16 ? 16u : 0u);
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(t0 + warp + i * kRowWarps, i);

  // Q fragments: row 8j + g, the channels of this lane's words.
  uint32_t qf[NT][2 * kW][2];
  uint4 qraw[NT][kW];
  float most[NT];  // of row 8j + g
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    most[j] = 0.0f;
    const int r = 8 * j + g;
    const bool in_use = r < R && r % a.Nq < ql;
    const __nv_bfloat16* const src = a.q + (static_cast<size_t>(bh) * R + (in_use ? r : 0)) * D + q4 * (D / 4);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      qraw[j][w] = in_use ? ld_global(reinterpret_cast<const uint4*>(src + 8 * w)) : make_uint4(0, 0, 0, 0);
      const uint32_t x[4] = {qraw[j][w].x, qraw[j][w].y, qraw[j][w].z, qraw[j][w].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        most[j] = fmaxf(most[j], fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xFFFF0000u))));
    }
  }
  float q_down[NT][2];  // what the scores of rows 8j + 2 q4 + n are multiplied with: above zero, as -inf passes through it
  int lim[NT][2];
  int lim_min = len;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    most[j] = fmaxf(most[j], __shfl_xor_sync(0xFFFFFFFFu, most[j], 1));
    most[j] = fmaxf(most[j], __shfl_xor_sync(0xFFFFFFFFu, most[j], 2));
    // 2^(14 - exponent of the row's largest value), at most 2^100
    const int ex = max(static_cast<int>(__float_as_uint(most[j]) >> 23), 41);
    const float q_up = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
    const float down = fmaxf(a.scale_log2 / q_up, 1e-38f);
    q_down[j][0] = __shfl_sync(0xFFFFFFFFu, down, 8 * q4);
    q_down[j][1] = __shfl_sync(0xFFFFFFFFu, down, 8 * q4 + 4);
    auto pair = [&](uint32_t lo, uint32_t hi, bool odd) {  // channels c and c + 4
      const float x = __uint_as_float(odd ? lo & 0xFFFF0000u : lo << 16);
      const float y = __uint_as_float(odd ? hi & 0xFFFF0000u : hi << 16);
      return pack_f16(x * q_up, y * q_up);
    };
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const uint4 u = qraw[j][w];
      qf[j][2 * w][0] = pair(u.x, u.z, false);      // channels 0, 4
      qf[j][2 * w][1] = pair(u.x, u.z, true);       // 1, 5
      qf[j][2 * w + 1][0] = pair(u.y, u.w, false);  // 2, 6
      qf[j][2 * w + 1][1] = pair(u.y, u.w, true);   // 3, 7
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = 8 * j + 2 * q4 + e, i = rr % a.Nq;
      lim[j][e] = rr < R && i < ql ? (a.causal ? max(len - ql + i + 1, 0) : len) : 0;
    }
  }
  if (a.causal) lim_min = max(len - a.Nq, 0);

  float acc[NT][kM][4];
  float m[NT][2], l[NT][2];
  constexpr float kVStart = 9.8607613e-32f;  // 2^-103
  float vinv[NT][2];      // kPUp over each row's reference of the values' scales
  float vlim = kVStart;   // the smallest reference of this lane's rows
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    vinv[j][0] = vinv[j][1] = kPUp / kVStart;
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.0f;
    m[j][0] = m[j][1] = kNone;
    l[j][0] = l[j][1] = 0.0f;
  }
  int stage = 0;
  for (int t = t0 + warp; t < t1; t += kRowWarps) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    {
      int ns = stage + kStages - 1;
      if (ns >= kStages) ns -= kStages;
      load(t + (kStages - 1) * kRowWarps, ns);
    }
    const uint8_t* const st = smem + (warp * kStages + stage) * C::kStage;
    if (++stage == kStages) stage = 0;
    // ---- S^T of 2 x 16 keys
    float s[NT][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t w0[kW], w1[kW];
      load_words<kW>(st + (16 * u + g) * C::kRow + q4 * (C::kRow / 4), w0);
      load_words<kW>(st + (16 * u + 8 + g) * C::kRow + q4 * (C::kRow / 4), w1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        s[j][u][0] = s[j][u][1] = s[j][u][2] = s[j][u][3] = 0.0f;
      }
#pragma unroll
      for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t af[4];
          af[0] = codes_f16_lo(w0[w] >> (8 * k));
          af[1] = codes_f16_lo(w1[w] >> (8 * k));
          af[2] = codes_f16_hi(w0[w] >> (8 * k));
          af[3] = codes_f16_hi(w1[w] >> (8 * k));
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_f16(s[j][u], af, qf[j][2 * w + k][0], qf[j][2 * w + k][1]);
        }
    }
    // ---- the keys' and values' scales; masks where a row or the sequence ends in this step
    float fk[2][2], fv[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fk[u][e] = *reinterpret_cast<const float*>(st + C::oSk + (16 * u + 8 * e) * 4 + key_of(g) * 4);
        fv[u][e] = *reinterpret_cast<const float*>(st + C::oSv + (16 * u + 8 * e) * 4 + key_of(g) * 4);
      }
    if (t * kStep + kStep > lim_min) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = t * kStep + key_of(g) + 16 * u + 8 * e;
          // The key's scale goes into the scores here, of the rows that see it only: a
          // scale of zero or NaN would make NaN of the mask.
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) s[j][u][2 * e + n] = key < lim[j][n] ? s[j][u][2 * e + n] * fk[u][e] : -INFINITY;
          fk[u][e] = 1.0f;
          if (key >= len) fv[u][e] = 0.0f;  // slots behind the last key may hold anything: 0 * NaN is not 0
        }
    }
    // ---- scores beside the reference, in powers of two
    float z[NT][2][4];
    const float fv_top = max_nan(max_nan(fabsf(fv[0][0]), fabsf(fv[0][1])), max_nan(fabsf(fv[1][0]), fabsf(fv[1][1])));
    float over = fv_top <= vlim ? 0.0f : 1e30f;  // NaN and infinities too
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int n = 0; n < 2; ++n) z[j][u][2 * e + n] = fmaf(s[j][u][2 * e + n], fk[u][e] * q_down[j][n], -m[j][n]);
          over = max3(over, z[j][u][2 * e], z[j][u][2 * e + 1]);
        }
    if (__any_sync(0xFFFFFFFFu, over > kLazy)) {
      vlim = INFINITY;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float f[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float x = kNone;
#pragma unroll
          for (int u = 0; u < 2; ++u)
            x = fmaxf(x, fmaxf(__fmul_rn(s[j][u][n], fk[u][0] * q_down[j][n]),
                               __fmul_rn(s[j][u][2 + n], fk[u][1] * q_down[j][n])));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
          const float mn = fmaxf(m[j][n], x);
          f[n] = ex2_approx(m[j][n] - mn);
          m[j][n] = mn;
          l[j][n] *= f[n];
          // The same for the values' scales; a value that is not finite makes NaN of the
          // rows that see it, and is left out of the products.
          uint32_t v = 0;  // magnitudes compare like their bits, what is not finite above all others
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (s[j][u][2 * e + n] != -INFINITY) v = max(v, __float_as_uint(fv[u][e]) & 0x7FFFFFFFu);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
          const bool spoiled = v >= 0x7F800000u;
          const uint32_t was = kPUpBits - __float_as_uint(vinv[j][n]);  // powers of two: differences of bits
          const uint32_t now = spoiled ? was : max(was, min((v + 0x007FFFFFu) & 0x7F800000u, 0x7F000000u));
          vinv[j][n] = __uint_as_float(kPUpBits - now);
          vlim = fminf(vlim, __uint_as_float(now));
          f[n] *= spoiled ? NAN : __uint_as_float(was) * __uint_as_float(0x7F000000u - now);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 2; ++n)  // the product rounded as in the maximum: scores of 2^27 and more are off by powers
              z[j][u][2 * e + n] = __fmul_rn(s[j][u][2 * e + n], fk[u][e] * q_down[j][n]) - m[j][n];
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          acc[j][i][0] *= f[0];
          acc[j][i][1] *= f[1];
          acc[j][i][2] *= f[0];
          acc[j][i][3] *= f[1];
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) fv[u][e] = fabsf(fv[u][e]) < INFINITY ? fv[u][e] : 0.0f;
    }
    // ---- P^T (times the values' scales) and O^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float p0 = ex2_approx(z[j][u][2 * e]), p1 = ex2_approx(z[j][u][2 * e + 1]);
          l[j][0] += p0;
          l[j][1] += p1;
          // in this order: zero times the scale of a key that the row does not see stays zero
          pb[j][e] = transpose8(pack_f16(p0 * fv[u][e] * vinv[j][0], p1 * fv[u][e] * vinv[j][1]));
        }
      }
      constexpr int kVW = D / 64;  // code words of a key per lane (V)
      uint32_t x[4][kVW];          // keys q4, q4 + 4, 8 + q4, 12 + q4
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * u + 4 * i + q4;
        const int ch = kVW == 2 ? ((g >> 1) ^ (r & 2)) * 16 + (g & 1) * 8 : g * 4;
        load_words<kVW>(st + C::oV + r * C::kRow + ch, x[i]);
      }
      // Channels of this lane: its words' nibbles in order; tile i has nibble i
      // of the first half of them as row g and of the second as row g + 8.
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        uint32_t af[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int nib = i + (e & 1) * kM;              // 0 .. D/8 - 1
          const int w = nib >> 3, half = (nib >> 2) & 1, sh = 8 * ((nib >> 1) & 1);
          const uint32_t x0 = x[(e >> 1) * 2][w], x1 = x[(e >> 1) * 2 + 1][w];
          const uint32_t pw = __byte_perm(x0, x1, half ? 0x7632 : 0x5410) >> sh;
          af[e] = (nib & 1) ? codes_f16_hi(pw) : codes_f16_lo(pw);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_f16(acc[j][i], af, pb[j][0], pb[j][1]);
      }
    }
  }
  grid_trigger();
  cp_async_wait<0>();
  if (bad) atomicOr(&g_kv4_status, bad);

  // ---- join the warps' results
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[j][n] += __shfl_xor_sync(0xFFFFFFFFu, l[j][n], o);
  __syncthreads();
  constexpr int kRows = 8 * NT;
  float* const ro = reinterpret_cast<float*>(smem);                 // [warp][row][D]
  float* const rm = ro + kRowWarps * kRows * D;                     // [warp][row]
  float* const rl = rm + kRowWarps * kRows;
  static_assert((kRowWarps * kRows * (D + 2)) * 4 <= C::kSmem, "shared memory of the join");
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ro[(warp * kRows + 8 * j + 2 * q4 + (e & 1)) * D + g * (D / 8) + i + (e >> 1) * kM] = acc[j][i][e] * __uint_as_float(0x7F000000u - __float_as_uint(vinv[j][e & 1]));
    if (g == 0) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        rm[warp * kRows + 8 * j + 2 * q4 + n] = m[j][n];
        rl[warp * kRows + 8 * j + 2 * q4 + n] = l[j][n];
      }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < kRows * (D / 4); idx += kRowWarps * 32) {
    const int row = idx / (D / 4), c = (idx % (D / 4)) * 4;
    if (row >= R || row % a.Nq >= ql) continue;
    float top = kNone;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, rm[w * kRows + row]);
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const float mw = rm[w * kRows + row];
      const float f = mw == kNone ? 0.0f : ex2_approx(mw - top);
      const float4 v = *reinterpret_cast<const float4*>(ro + (w * kRows + row) * D + c);
      sum = fmaf(f, rl[w * kRows + row], sum);
      o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    }
    // Sums tell rows without keys (zero) from rows that are not finite (NaN).  Scores of minus
    // infinity alone, 0 / 0, leave a sum of zero too: such a row, or such a part of it, is NaN
    // with a log-sum-exp of -inf, which the join takes for NaN if the row has nothing else.
    const int i = row % a.Nq;
    const bool sees = t0 < t1 && (a.causal ? len - ql + i + 1 : len) > t0 * kStep;
    const float inv = sum != 0.0f ? 1.0f / sum : sees ? NAN : 0.0f;
    const float lse2 = sum != 0.0f ? top + log2f(sum) : -INFINITY;
    const size_t at = static_cast<size_t>(bh) * R + row;
    o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    if (a.nsplit == 1) {
      *reinterpret_cast<uint2*>(a.out + at * D + c) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      if (c == 0 && a.lse) a.lse[at] = lse2 * kLn2;
    } else {
      const size_t pr = static_cast<size_t>(split) * gridDim.x * R + at;
      *reinterpret_cast<float4*>(a.parts.o + pr * D + c) = o;
      if (c == 0) a.parts.lse2[pr] = lse2;
    }
  }
}

// Joins the parts of every row, one warp per row: weights 2^(lse2 - max).
template <int D>
__global__ void __launch_bounds__(128) kv4_join_kernel(Kv4Parts parts, int nsplit, long long rows, int Nq, int rows_b,
                                                       const int32_t* q_lens, __nv_bfloat16* out, float* lse) {
  constexpr int kC = D / 32;
  const int lane = threadIdx.x & 31;
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  grid_wait();
  grid_trigger();
  if (r >= rows) return;
  if (q_lens && static_cast<int>(r % Nq) >= ld_global(q_lens + r / rows_b)) return;
  float top = -INFINITY;
  for (int s = 0; s < nsplit; ++s) top = fmaxf(top, parts.lse2[s * rows + r]);
  float sum = 0.0f, none = 0.0f, o[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) o[i] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < nsplit; ++s) {
    const float x = parts.lse2[s * rows + r];
    const float* src = parts.o + (s * rows + r) * D + lane * kC;
    if (x == -INFINITY) {  // no keys (zeros), or weights that are all zero (NaN)
      none += src[0];
      continue;
    }
    const float w = ex2_approx(x - top);
    sum += w;
#pragma unroll
    for (int i = 0; i < kC; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + i);
      o[i] = fmaf(w, v.x, o[i]);
      o[i + 1] = fmaf(w, v.y, o[i + 1]);
    }
  }
  const float inv = sum != 0.0f ? 1.0f / sum : none;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + r * D + lane * kC);
#pragma unroll
  for (int i = 0; i < kC; i += 2) dst[i / 2] = pack_bf16(o[i] * inv, o[i + 1] * inv);
  if (lse && lane == 0) lse[r] = sum != 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

int log2_of(int x) { return __builtin_ctz(static_cast<unsigned>(x)); }

CacheArgs cache_args(const ra_kv4_cache& c, int B, int T, const int32_t* table, int max_pages, const int32_t* start,
                     const int32_t* count, int lanes, int per_sm, int ahead,
                     int tokens, dim3* grid) {
  CacheArgs a{};
  a.codes[0] = c.k4; a.codes[1] = c.v4;
  a.scale[0] = c.sk; a.scale[1] = c.sv;
  a.table = table; a.start = start; a.count = count;
  a.num_pages = c.num_pages; a.page_log2 = log2_of(c.page_size); a.max_pages = max_pages;
  a.Hk = c.Hk; a.T = T;
  const int tok = kThreads / lanes * tokens;  // tokens per CTA
  const int tiles = (T + tok - 1) / tok;
  const int heads[2] = {c.Hk, c.Hk};
  const int group = heads_per_cta(static_cast<long long>(tiles) * B, heads, per_sm, ahead / tokens);
  a.groups = (c.Hk + group - 1) / group;
  a.group = group;
  *grid = dim3(tiles, 2 * a.groups, B);
  return a;
}

template <int D, int NT>
cudaError_t launch_rows(const RowsArgs& a, dim3 grid, cudaStream_t st) {
  auto kern = kv4_rows_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(kern, grid, kRowWarps * 32, RowsCfg<D>::kSmem, st, a);
}

}  // namespace

namespace {

using CacheKernel = void (*)(CacheArgs);

// Tokens of a thread: as many as fill the rows it works on at a time.
int tokens_per_thread(int heads, int ahead) { return heads == 1 ? ahead : heads == 2 ? ahead / 2 : 1; }

template <bool kBf16, int kD>
CacheKernel append_kernel(int tokens) {
  if constexpr (append_ahead(kBf16) == 4)
    if (tokens == 4) return kv4_append_kernel<kBf16, kD, 4>;
  return tokens == 2 ? kv4_append_kernel<kBf16, kD, 2> : kv4_append_kernel<kBf16, kD, 1>;
}

template <bool kBf16, int kD>
CacheKernel read_kernel(int tokens) {
  return tokens == 4   ? kv4_read_kernel<kBf16, kD, 4>
         : tokens == 2 ? kv4_read_kernel<kBf16, kD, 2>
                       : kv4_read_kernel<kBf16, kD, 1>;
}

}  // namespace

cudaError_t launch_kv4_append(const ra_kv4_cache& c, int dtype, int B, int T, const void* k, const ra_strides& ks,
                              const void* v, const ra_strides& vs, const int32_t* table, int max_pages,
                              const int32_t* start, const int32_t* n_new, cudaStream_t st) {
  g_used.store(true, std::memory_order_relaxed);
  dim3 grid;
  const int tokens = tokens_per_thread(c.Hk, append_ahead(dtype == RA_DT_BF16));
  CacheArgs a = cache_args(c, B, T, table, max_pages, start, n_new, c.D / 8, kAppendPerSm,
                           append_ahead(dtype == RA_DT_BF16), tokens, &grid);
  a.x[0] = k; a.x[1] = v;
  a.st[0] = ks; a.st[1] = vs;
  auto* kern = dtype == RA_DT_BF16 ? (c.D == 64 ? append_kernel<true, 64>(tokens) : append_kernel<true, 128>(tokens))
                                   : (c.D == 64 ? append_kernel<false, 64>(tokens) : append_kernel<false, 128>(tokens));
  return launch_early(kern, grid, kThreads, 0, st, a);
}

cudaError_t launch_kv4_read(const ra_kv4_cache& c, int dtype, int B, int T, const int32_t* table, int max_pages,
                            const int32_t* start, const int32_t* n, void* k, void* v, cudaStream_t st) {
  g_used.store(true, std::memory_order_relaxed);
  dim3 grid;
  const int tokens = tokens_per_thread(c.Hk, kReadAhead);
  CacheArgs a = cache_args(c, B, T, table, max_pages, start, n, dtype == RA_DT_BF16 ? c.D / 8 : c.D / 4,
                           kReadPerSm, kReadAhead, tokens, &grid);
  a.y[0] = k; a.y[1] = v;
  auto* kern = dtype == RA_DT_BF16 ? (c.D == 64 ? read_kernel<true, 64>(tokens) : read_kernel<true, 128>(tokens))
                                   : (c.D == 64 ? read_kernel<false, 64>(tokens) : read_kernel<false, 128>(tokens));
  return launch_early(kern, grid, kThreads, 0, st, a);
}

Kv4Plan kv4_plan(const ra_kv4_cache& c, const ra_kv4_attn& a) {
  Kv4Plan plan{};
  const long long R = static_cast<long long>(a.H / c.Hk) * a.Nq, bh = static_cast<long long>(a.B) * c.Hk;
  // Up to 16 rows, which one CTA of the few-row kernel holds, that kernel; the tiles take the
  // same time for 1 row as for 128.  (640 heads x 8191 keys, D = 128: 146, 147, 150, 235 us at
  // 1, 4, 8, 16 rows against 790 to 800 in tiles, which take 800, 816, 840, 889 at 17, 32, 64,
  // 128; D = 64: 95 to 133 against 722.  8 heads x 32760 keys: 22 to 30 against 53.  4 x 8 heads x
  // 700 keys: 8 to 13 against 14.  Several CTAs of 16 rows for 17 to 48 rows, each reading the
  // keys by itself, measured 400 to 607 us, 46 to 48 and 13, which a later form could take up.)
  plan.tiles = R > 16;
  // The number of parts with the least estimated time, in keys of work of one SM:
  // an SM gets the ceiling of its share of CTAs, each of which costs its keys and a
  // fixed part (kFixed), and joining costs a launch and the parts' traffic.  Few-row
  // CTAs share an SM, whose rate one or two of them do not reach.  (Measured, one row
  // each: 640 heads x 8191 keys 162, 146, 146, 159, 175 us at 1, 2, 3, 5, 9 parts; 8 heads x
  // 32760 keys 55, 30, 21, 23, 30 us at 4, 9, 18, 28, 64.)
  const long long items = bh * (plan.tiles ? (R + 255) / 256 : 1);
  const double fixed = plan.tiles ? 256.0 : 350.0, join = plan.tiles ? 300.0 : 700.0;
  const int step = plan.tiles ? 64 : kRowWarps * kStep;
  double best = 0.0;
  for (int k = 1; k <= 64 && (k == 1 || (k - 1) * step < a.max_len); ++k) {
    const long long ctas = (items * k + kNumSMs - 1) / kNumSMs;
    const double rate = plan.tiles || ctas >= 3 ? 1.0 : ctas == 2 ? 0.9 : 0.75;
    double cost = ctas * (a.max_len / static_cast<double>(k) + fixed) / rate;
    if (k > 1) cost += join + (plan.tiles ? 0.015 : 0.06) * k * static_cast<double>(bh) * R * c.D / 128.0;
    if (k == 1 || cost < 0.98 * best) {
      best = cost;
      plan.nsplit = k;
    }
  }
  return plan;
}

Kv4Parts kv4_parts(const ra_kv4_cache& c, const ra_kv4_attn& a, const Kv4Plan& plan, void* ws) {
  Kv4Parts p{};
  if (plan.nsplit == 1) return p;
  const size_t rows = static_cast<size_t>(a.B) * a.H * a.Nq;
  p.o = static_cast<float*>(ws);
  p.lse2 = p.o + plan.nsplit * rows * c.D;
  return p;
}

cudaError_t launch_kv4_rows(const ra_kv4_cache& c, const ra_kv4_attn& at, const Kv4Plan& plan, const void* q,
                            const int32_t* table, const int32_t* seq_lens, const int32_t* q_lens,
                            const Kv4Parts& parts, void* out, float* lse, cudaStream_t st) {
  g_used.store(true, std::memory_order_relaxed);
  RowsArgs a{};
  a.k4 = c.k4; a.sk = c.sk; a.v4 = c.v4; a.sv = c.sv;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.table = table; a.seq_lens = seq_lens; a.q_lens = q_lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.parts = parts;
  a.num_pages = c.num_pages; a.page_log2 = log2_of(c.page_size); a.max_pages = at.max_pages;
  a.Hk = c.Hk; a.G = at.H / c.Hk; a.Nq = at.Nq; a.causal = at.causal; a.nsplit = plan.nsplit;
  a.scale_log2 = at.scale * kLog2e;
  const int R = a.G * a.Nq;
  const dim3 grid(at.B * c.Hk, plan.nsplit);
  if (R <= 8) return c.D == 64 ? launch_rows<64, 1>(a, grid, st) : launch_rows<128, 1>(a, grid, st);
  return c.D == 64 ? launch_rows<64, 2>(a, grid, st) : launch_rows<128, 2>(a, grid, st);
}

cudaError_t launch_kv4_join(const ra_kv4_cache& c, const ra_kv4_attn& a, const Kv4Plan& plan,
                            const int32_t* q_lens, const Kv4Parts& parts, void* out, float* lse, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.B) * a.H * a.Nq;
  const int rows_b = a.H * a.Nq;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  return launch_early(c.D == 64 ? kv4_join_kernel<64> : kv4_join_kernel<128>, grid, 128, 0, st, parts, plan.nsplit, rows,
                      a.Nq, rows_b, q_lens, o, lse);
}

cudaError_t read_kv4_status(uint32_t* out) {
  *out = 0;
  if (!g_used.load(std::memory_order_relaxed)) return cudaSuccess;
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_kv4_status, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_kv4_status, &zero, sizeof(uint32_t));
}

}  // namespace ra
