// Attention in 128-row tiles on the tensor cores: cross attention in bf16 to
// an encoder's states, and attention of many query rows over the 4-bit cache.
//   O = softmax(scale q k^T) v, fp32 scores, softmax and sums.
//
// One persistent CTA per SM takes two 128-row query tiles of one head (an
// item) and walks over 64-key blocks, which the tiles share.  S has two buffers
// per tile, so the tensor cores work on one block while the softmax is at the
// other: with 128-key blocks and one buffer a tile's products and its softmax
// took turns (890 TFLOP/s at 8192 x 8192, D = 128, softmax warps idle half of
// the time; 1333 now in single launches, 1200 back to back under the power cap).  What bounds it at D = 128: shared memory, 1280 of 1570 cycles
// a block (S with N = 64 reads Q again for every block, 48 cycles an MMA against 32 of
// arithmetic; P V 64 an MMA), and the exponentials, 1024 (8 cycles a warp
// instruction, 16384 of them a block and partition); at D = 64 the exponentials; the
// cache's kernel besides what the unpacking warps take of the issue slots and of shared
// memory.  Issuing an MMA costs 16 cycles only from a thread that the compiler knows to
// be alone (elect_one); under a test of the lane it cost 56 to 100, and the kernel was
// bound by it (1157 TFLOP/s).  Measured and left out, some of it under that bound:
// exponentials of every fourth pair by a polynomial on the FMA pipe (3 % slower at
// 8192 keys, 1 % faster at 512), P beside S so that S(g + 1) need not wait for
// P V(g - 1) (4 % slower), 16 softmax warps (6 % slower, 20 % for the cache), four warps
// of their own for the output (6 % slower at 8192 keys, 3 % faster at 512), two blocks' S by one
// product with N = 128, which reads Q half as often but waits for both P V (24 % slower),
// an item's output after the exponentials of the next one's first block (3 % slower at 512
// keys, 25 % at 128), one tile half an item behind the other (2 to 3 % slower).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ra_common.cuh"
#include "ra_tmem_row.cuh"
#include "ra_block.h"
#include "ra_kv4.cuh"

namespace ra {
namespace {

__device__ uint32_t g_tiles_status = 0;
std::atomic<bool> g_used{false};  // a program that has never called these does not read their status

constexpr int kRows = 128;   // query rows per tile = MMA M
constexpr int kTiles = 2;    // query tiles per CTA
constexpr int kKeys = 64;    // keys per block = MMA N of S
// The reference maximum moves when a score passes it by kLazy (powers of two).
template <bool KV4> constexpr float kLazy = KV4 ? 4.0f : 8.0f;
// A score is off by about 2^-24 of its size, and x = score - reference, taken in one operation,
// by half a unit of the reference, which P does not hold from some size on.  From 2^kFar on, a
// row's differences are halved until the reference is below it: where scores are off by whole
// powers of two, only what is within their error changes its weight.
template <bool KV4> constexpr int kFar = KV4 ? 23 : 28;
constexpr float kPUp = 11.0f;  // cache: P goes to f16 times 2^kPUp, at most 2^15
constexpr int kVUp = 12;       // and the values times 2^kVUp, at most 7 * 2^12: a scale keeps its bits down to
                               // 2^-26 of the largest of its 32 keys
// Under a causal mask, values of 32 keys whose scales are further apart than 2^kApart, or not
// finite, go to the products as codes, and their scales into P of each row, relative to the
// largest that the row sees: with one exponent for all rows, keys that a row does not see would
// take its bits.  A form of the kernel by itself, as what looks for such values costs where
// there are none (a frame of 1560 rows over 32760 keys, causal and not: 1433 and 1366 us at
// D = 128, 1310 and 1236 at D = 64).
constexpr int kApart = 8;
constexpr float kOdd = -200.0f, kUnseen = -150.0f;  // in place of an exponent (which is at least -100)
constexpr float kNoSum = 140.0f;                    // a shift whose inverse, 2^-140, is zero

template <int D, bool KV4>
struct CfgT {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kRows * 128;           // a 64-channel box of a Q tile
  static constexpr int kHalf = kKeys * 128;            // and of a K or V block
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kKVBytes = kKeys * D * 2;
  static constexpr int kStages = KV4 && D == 64 ? 8 : 4;  // of K, and of V (cache at D = 64: as many as there is room
                                                          // for, 1297 us with four, 1237 with eight)
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + kTiles * kQBytes;
  static constexpr int oV = oK + kStages * kKVBytes;
  static constexpr int oScale = oV + kStages * kKVBytes;      // [sk | log2 sv][stage][key], cache only
  static constexpr int oVExp = oScale + (KV4 ? 2 * kStages * kKeys * 4 : 0);   // [stage][half]: exponents, then masks
  static constexpr int oStage = oVExp + (KV4 ? 16 * kStages : 0);              // [softmax warp][row][kPiece]
  static constexpr int kPiece = KV4 ? 64 : 128;        // bytes of a row that leave at a time
  static constexpr int oBar = oStage + 8 * 32 * kPiece;
  static constexpr int kNumBars = 2 + 2 + 5 * kStages + 4 + 4 + 4 + 2;
  static constexpr int oMisc = oBar + kNumBars * 8;
  static constexpr int kSmem = oMisc + 16 + 1024;
  // Unpacking warps: at D = 128 four for the keys and four for the values (1380 us
  // against 1453 at 1560 x 32760 x 40 heads), at D = 64, where the softmax is the
  // slower side, four for both (with four stages 1340 us against 1357, causal 1402
  // against 1572).
  static constexpr bool kTwoUnpack = KV4 && D == 128;
  static constexpr int kFirstSoftmax = KV4 ? (kTwoUnpack ? 12 : 8) : 4;
  static constexpr int kThreads = (kFirstSoftmax + 8) * 32;
  static constexpr uint32_t kIdescQK = instr_desc(kCfmtF32, 1, 1, 0, 0, kRows, kKeys);
  static constexpr uint32_t kIdescPV = instr_desc(kCfmtF32, KV4 ? 0 : 1, KV4 ? 0 : 1, 0, 1, kRows, D);
  static_assert(kSmem <= 232448, "shared memory");
};

struct TileArgs {
  int heads;        // heads that items run over: query heads (cross) or key heads (cache)
  int group;        // cross: query heads per key head; cache: unused
  int R;            // query rows per head of an item
  int npairs, nsplit, nitems;
  float scale_log2;
  __nv_bfloat16* out;
  ra_strides os;
  float* lse;
  const int32_t* kv_lens;   // cross: may be NULL; cache: seq_lens
  // cross
  int Nk;
  // cache
  const int32_t* q_lens;
  const int32_t* table;
  const uint8_t* k4;
  const float* sk;
  const uint8_t* v4;
  const float* sv;
  int num_pages, page_log2, max_pages, Nq;
  Kv4Parts parts;
};

struct Item {
  int b, h, row0, split;
  int len, ql;      // keys and query rows of the sequence
  int k0, nb;       // first key and number of the item's key blocks
};

template <bool KV4, bool MASK>
__device__ __forceinline__ Item get_item(const TileArgs& a, int item, uint32_t* bad) {
  Item it;
  const int pair = item % a.npairs, rest = item / a.npairs;
  it.split = rest % a.nsplit;
  const int bh = rest / a.nsplit;
  it.b = bh / a.heads;
  it.h = bh % a.heads;
  it.row0 = pair * kTiles * kRows;
  it.ql = a.R;
  int end;
  if constexpr (KV4) {
    it.len = clamp_len(ld_global(a.kv_lens + it.b), a.max_pages << a.page_log2, bad);
    it.ql = a.q_lens ? clamp_len(ld_global(a.q_lens + it.b), a.Nq, bad) : a.Nq;
    end = it.len;
    if constexpr (MASK) {  // the furthest key that a row of the item sees
      const int last = min(it.row0 + kTiles * kRows, a.R) - 1;
      if (it.row0 / a.Nq == last / a.Nq) end = max(0, min(end, it.len - it.ql + last % a.Nq + 1));
    }
  } else {
    it.len = a.kv_lens ? clamp_len(ld_global(a.kv_lens + it.b), a.Nk, bad) : a.Nk;
    end = it.len;
  }
  const int blocks = (end + kKeys - 1) / kKeys;
  const int per = (blocks + a.nsplit - 1) / a.nsplit;
  const int first = min(it.split * per, blocks);
  it.k0 = first * kKeys;
  it.nb = min(per, blocks - first);
  return it;
}

// Waits for a phase with the blocking test (the hardware holds the warp until the
// phase completes or a short limit passes: three of these sit on the chain S, softmax, P V,
// where sleeping between polls measured 400 cycles each), at most kWaitLimitNs.
__device__ __forceinline__ bool wait_t(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 7u) == 0) {
      if (*abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        return false;
      }
    }
  }
}

// The same for a whole warp: every lane waits, and all of them go on or none (a
// wait that gave up must not part the warp before its collectives).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool got = wait_t(bar, parity, abort);
  return __all_sync(0xFFFFFFFFu, got);
}

__device__ __forceinline__ float max3t(float a, float b, float c) { return fmaxf(a, fmaxf(b, c)); }

// MASK: causal (cache only).
template <int D, bool KV4, bool MASK>
__global__ void __launch_bounds__(CfgT<D, KV4>::kThreads, 1)
attn_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const TileArgs a) {
  using C = CfgT<D, KV4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* b = reinterpret_cast<uint64_t*>(smem + C::oBar);
  uint64_t* const q_full = b; b += 2;              // [tile]
  uint64_t* const q_free = b; b += 2;
  uint64_t* const k_full = b; b += C::kStages;
  uint64_t* const k_empty = b; b += C::kStages;
  uint64_t* const v_full = b; b += C::kStages;     // cross: the copy has landed
  uint64_t* const v_ready = b; b += C::kStages;    // the MMA may read
  uint64_t* const v_empty = b; b += C::kStages;
  uint64_t* const s_full = b; b += 4;              // [tile][buffer]
  uint64_t* const p_full = b; b += 4;
  uint64_t* const pv_done = b; b += 4;
  uint64_t* const drain = b;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::oMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1); mbar_init(q_free + i, 1); mbar_init(drain + i, 1);
    }
    for (int i = 0; i < 4; ++i) { mbar_init(s_full + i, 1); mbar_init(p_full + i, 4); mbar_init(pv_done + i, 1); }
    for (int i = 0; i < C::kStages; ++i) {
      // cache: four unpacking warps fill a stage; the softmax warps read its scales
      mbar_init(k_full + i, KV4 ? 4 : 1); mbar_init(k_empty + i, KV4 ? 2 + 8 : 2);
      mbar_init(v_full + i, 1); mbar_init(v_ready + i, KV4 ? 4 : 1); mbar_init(v_empty + i, KV4 ? 2 + 8 : 2);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_q);
    if (!KV4) { prefetch_tmap(&tm_k); prefetch_tmap(&tm_v); }
  }
  // Before TMEM is taken: a block of the kernel before on this SM may still have to take its own.
  grid_wait();
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  float* const scales = reinterpret_cast<float*>(smem + C::oScale);  // cache: of the keys
  float* const v_log = scales + C::kStages * kKeys;                   // cache: log2 of the values' scales, kOdd only
  float* const v_exp = reinterpret_cast<float*>(smem + C::oVExp);     // cache: exponents of the values' scales
  uint32_t* const v_bad = reinterpret_cast<uint32_t*>(v_exp + 2 * C::kStages);  // keys not finite, kOdd only
  uint32_t bad = 0;
  bool ok = true;
  if (warp < 4) {
    if constexpr (KV4) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const bool one = elect_one();  // the thread that issues; ptxas knows it to be alone, a test of the lane it does not
    if (warp == 0 && one) {
      // ------------------------------------------------------------ TMA producer
      uint32_t g = 0, li = 0;
      for (int item = blockIdx.x; item < a.nitems && ok; item += gridDim.x) {
        const Item it = get_item<KV4, MASK>(a, item, &bad);
        if (it.nb == 0) continue;
        auto load_q = [&]() {
          for (int tt = 0; tt < kTiles && ok; ++tt) {
            if (!(ok = wait_t(q_free + tt, (li & 1) ^ 1, abort_flag))) return;
            mbar_arrive_expect_tx(q_full + tt, C::kQBytes);
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(smem + C::oQ + tt * C::kQBytes + h * C::kQHalf, &tm_q, q_full + tt, h * 64,
                          it.row0 + tt * kRows, it.h, it.b);
          }
          ++li;
        };
        if constexpr (KV4) {
          load_q();
        } else {
          const int hk = it.h / a.group;
          for (int t = 0; t < it.nb && ok; ++t, ++g) {
            const int s = g % C::kStages, key = it.k0 + t * kKeys;
            const uint32_t par = ((g / C::kStages) & 1) ^ 1;
            if (!(ok = wait_t(k_empty + s, par, abort_flag))) break;
            mbar_arrive_expect_tx(k_full + s, C::kKVBytes);
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(smem + C::oK + s * C::kKVBytes + h * C::kHalf, &tm_k, k_full + s, h * 64, key, hk, it.b);
            if (t == 0) {
              load_q();
              if (!ok) break;
            }
            if (!(ok = wait_t(v_empty + s, par, abort_flag))) break;
            mbar_arrive_expect_tx(v_full + s, C::kKVBytes);
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(smem + C::oV + s * C::kKVBytes + h * C::kHalf, &tm_v, v_full + s, h * 64, key, hk, it.b);
          }
        }
      }
      // Wait (bounded) for the copies of the last stages and of Q to land.
      uint32_t n = 0;
      if (!KV4)
        for (uint32_t k = (g > (uint32_t)C::kStages ? g - C::kStages : 0); k < g; ++k) {
          while (!mbar_try_wait(k_full + (k % C::kStages), (k / C::kStages) & 1) && ++n < kSpinLimit) {}
          while (!mbar_try_wait(v_full + (k % C::kStages), (k / C::kStages) & 1) && ++n < kSpinLimit) {}
        }
      if (li > 0)
        for (int tt = 0; tt < kTiles; ++tt)
          while (!mbar_try_wait(q_full + tt, (li - 1) & 1) && ++n < kSpinLimit) {}
    } else if ((warp == 1 || warp == 2) && one) {
      // ------------------------------------------------------------ MMA issuers
      // Per tile: P V(g), then S(g + 2) into the buffer whose P it has read (after
      // it has completed: products into different accumulators are not ordered).
      const int tt = warp - 1;
      const uint32_t dQ = desc_lo(smem_u32(smem + C::oQ) + tt * C::kQBytes, 16);
      const uint32_t dK = desc_lo(smem_u32(smem + C::oK), 16), dV = desc_lo(smem_u32(smem + C::oV), C::kHalf);
      const uint32_t tS0 = tbase + tt * 128, tO = tbase + 256 + tt * 128;
      uint32_t g0 = 0, li = 0;
      auto scores = [&](uint32_t g, bool last) -> bool {
        const int s = g % C::kStages;
        const uint32_t buf = g & 1;
        if (!wait_t(k_full + s, (g / C::kStages) & 1, abort_flag)) return false;
        if (g >= 2 && !wait_t(pv_done + tt * 2 + buf, ((g - 2) >> 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t k = dK + s * (C::kKVBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss<C::kIdescQK>(tS0 + buf * 64, dQ + (kk >> 2) * (C::kQHalf >> 4) + (kk & 3) * 2,
                              k + (kk >> 2) * (C::kHalf >> 4) + (kk & 3) * 2, kk > 0);
        mma_commit(s_full + tt * 2 + buf);
        mma_commit(k_empty + s);
        if (last) mma_commit(q_free + tt);
        return true;
      };
      for (int item = blockIdx.x; item < a.nitems && ok; item += gridDim.x) {
        const Item it = get_item<KV4, MASK>(a, item, &bad);
        if (it.nb == 0) continue;
        if (!(ok = wait_t(q_full + tt, li & 1, abort_flag))) break;
        ++li;
        for (int t = 0; t < 2 && t < it.nb && ok; ++t) ok = scores(g0 + t, t == it.nb - 1);
        for (int t = 0; t < it.nb && ok; ++t) {
          const uint32_t g = g0 + t, buf = g & 1;
          const int s = g % C::kStages;
          if (!(ok = wait_t(v_ready + s, (g / C::kStages) & 1, abort_flag))) break;
          if (!(ok = wait_t(p_full + tt * 2 + buf, (g >> 1) & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t v = dV + s * (C::kKVBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts<C::kIdescPV>(tO, tS0 + buf * 64 + kk * 8, v + kk * (16 * 128 >> 4), kk > 0 || t > 0);
          mma_commit(pv_done + tt * 2 + buf);
          mma_commit(v_empty + s);
          if (t + 2 < it.nb) ok = scores(g + 2, t + 2 == it.nb - 1);
        }
        g0 += it.nb;
      }
      mma_commit(drain + tt);
      uint32_t n = 0;
      while (!mbar_try_wait(drain + tt, 0) && ++n < kSpinLimit) {}
    } else if (warp == 3 && !KV4) {
      // ------------------------------------------------------------ value rows behind the last key
      uint32_t g = 0;
      for (int item = blockIdx.x; item < a.nitems && ok; item += gridDim.x) {
        const Item it = get_item<KV4, MASK>(a, item, &bad);
        for (int t = 0; t < it.nb; ++t, ++g) {
          const int s = g % C::kStages;
          if (!(ok = wait_warp(v_full + s, (g / C::kStages) & 1, abort_flag))) break;
          // Rows past Nk are zeros already (filled by the copy).
          const int first = it.len - (it.k0 + t * kKeys), last = min(kKeys, a.Nk - (it.k0 + t * kKeys));
          if (first < last) {
            for (int idx = lane; idx < (last - first) * C::kHalves * 8; idx += 32) {
              const int row = first + idx / (C::kHalves * 8), ch = idx % (C::kHalves * 8);
              *reinterpret_cast<uint4*>(smem + C::oV + s * C::kKVBytes + (ch >> 3) * C::kHalf + row * 128 +
                                        (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(v_ready + s);
        }
      }
    }
  } else if (KV4 && warp < C::kFirstSoftmax) {
    // -------------------------------------------------------------- unpacking warps
    if constexpr (C::kTwoUnpack) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");  // 72 and 192 for the softmax: 1340 us, not 1297
    if constexpr (KV4) {
      constexpr int kQ = D / 64;  // 16-byte pieces of a code row per thread: two threads per key
      const int row = threadIdx.x & 63, part = (threadIdx.x >> 6) & 1;
      // Place of this thread's key of block t, or -1 behind the last key.
      auto place = [&](const Item& it, int t) -> long long {
        const int key = it.k0 + t * kKeys + row;
        if (t >= it.nb || key >= it.len) return -1;
        int page = ld_global(a.table + static_cast<size_t>(it.b) * a.max_pages + (key >> a.page_log2));
        if (page < 0 || page >= a.num_pages) {
          bad |= kStatusBadPosition;
          page = 0;
        }
        return ((static_cast<long long>(page) * a.heads + it.h) << a.page_log2) + (key & ((1 << a.page_log2) - 1));
      };
      auto fetch = [&](const uint8_t* codes, const float* scale, long long at, uint4* w, float& s) {
        if (at >= 0) {
          const uint4* const p = reinterpret_cast<const uint4*>(codes + at * (D / 2)) + part * kQ;
#pragma unroll
          for (int i = 0; i < kQ; ++i) w[i] = ld_global(p + i);
          s = ld_global(scale + at);
        } else {
#pragma unroll
          for (int i = 0; i < kQ; ++i) w[i] = make_uint4(0, 0, 0, 0);
          s = 0.0f;
        }
      };
      // Keys of block g: bf16, eight channels in their order.
      auto put_keys = [&](const uint4* code, float scale, uint32_t g) -> bool {
        const int s = g % C::kStages;
        if (!wait_warp(k_empty + s, ((g / C::kStages) & 1) ^ 1, abort_flag)) return false;
        uint8_t* const kt = smem + C::oK + s * C::kKVBytes + row * 128;
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t p0 = codes_bf16(w[c]), p1 = codes_bf16(w[c] >> 4);
            const uint32_t p2 = codes_bf16(w[c] >> 8), p3 = codes_bf16(w[c] >> 12);
            const uint4 o = make_uint4(__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410),
                                       __byte_perm(p0, p1, 0x7632), __byte_perm(p2, p3, 0x7632));
            const int ch = (part * kQ + i) * 4 + c;
            *reinterpret_cast<uint4*>(kt + (ch >> 3) * C::kHalf + (((ch & 7) ^ (row & 7)) << 4)) = o;
          }
        }
        if (part == 0) scales[s * kKeys + row] = scale * a.scale_log2;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + s);
        return true;
      };
      // Values of block g: f16, with their scale, relative (2^kVUp) to the power of two not below
      // the largest scale of these 32 keys (whose exponent the softmax puts into P);
      // channels 0 4 1 5 2 6 3 7 of eight, which the output puts right.
      auto put_values = [&](const uint4* code, float scale, uint32_t g) -> bool {
        const int s = g % C::kStages;
        float vm = fabsf(scale);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) vm = max_nan(vm, __shfl_xor_sync(0xFFFFFFFFu, vm, o));
        const uint32_t ve = min(max((__float_as_uint(vm) + 0x007FFFFFu) >> 23, 27u), 253u);  // 2^(ve - 127)
        float v_up = scale * __uint_as_float((254u + kVUp - ve) << 23), e = static_cast<float>(ve) - 127.0f;
        if constexpr (MASK) {
          if (__any_sync(0xFFFFFFFFu, (scale != 0.0f && fabsf(scale) * (1 << kApart) < vm) || !(vm < INFINITY))) {
            v_up = copysignf(1 << kVUp, scale);
            e = kOdd;
          }
        }
        const __half2 v_scale = __float2half2_rn(v_up);
        auto times = [&](uint32_t x) {
          const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), v_scale);
          return *reinterpret_cast<const uint32_t*>(&r);
        };
        if (!wait_warp(v_empty + s, ((g / C::kStages) & 1) ^ 1, abort_flag)) return false;
        uint8_t* const vt = smem + C::oV + s * C::kKVBytes + row * 128;
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 o = make_uint4(times(codes_f16_lo(w[c])), times(codes_f16_hi(w[c])),
                                       times(codes_f16_lo(w[c] >> 8)), times(codes_f16_hi(w[c] >> 8)));
            const int ch = (part * kQ + i) * 4 + c;
            *reinterpret_cast<uint4*>(vt + (ch >> 3) * C::kHalf + (((ch & 7) ^ (row & 7)) << 4)) = o;
          }
        }
        if (part == 0 && lane == 0) v_exp[s * 2 + (row >> 5)] = e;
        if constexpr (MASK) {
          if (part == 0 && e == kOdd) {
            const bool finite = fabsf(scale) < INFINITY;
            v_log[s * kKeys + row] = finite ? __log2f(fabsf(scale)) : -INFINITY;
            const uint32_t bad_keys = ~__ballot_sync(0xFFFFFFFFu, finite);
            if (lane == 0) v_bad[s * 2 + (row >> 5)] = bad_keys;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready + s);
        return true;
      };
      uint32_t g = 0;
      for (int item = blockIdx.x; item < a.nitems && ok; item += gridDim.x) {
        const Item it = get_item<KV4, MASK>(a, item, &bad);
        // The codes of the next block travel while this one's are unpacked.
        if constexpr (C::kTwoUnpack) {
          const bool of_keys = warp < 8;  // warps 4-7 the keys, 8-11 the values
          const uint8_t* const codes = of_keys ? a.k4 : a.v4;
          const float* const from = of_keys ? a.sk : a.sv;
          uint4 next[kQ];
          float next_scale;
          fetch(codes, from, place(it, 0), next, next_scale);
          for (int t = 0; t < it.nb && ok; ++t, ++g) {
            uint4 cur[kQ];
#pragma unroll
            for (int i = 0; i < kQ; ++i) cur[i] = next[i];
            const float cur_scale = next_scale;
            fetch(codes, from, place(it, t + 1), next, next_scale);
            ok = of_keys ? put_keys(cur, cur_scale, g) : put_values(cur, cur_scale, g);
          }
        } else {
          long long at = place(it, 0);
          uint4 k[kQ], v[kQ];
          float ks, vs;
          fetch(a.k4, a.sk, at, k, ks);
          for (int t = 0; t < it.nb; ++t, ++g) {
            fetch(a.v4, a.sv, at, v, vs);
            if (!(ok = put_keys(k, ks, g))) break;
            at = place(it, t + 1);
            fetch(a.k4, a.sk, at, k, ks);
            if (!(ok = put_values(v, vs, g))) break;
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax, one row per thread
    if constexpr (C::kTwoUnpack) asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    else if constexpr (KV4) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int tt = (warp - C::kFirstSoftmax) >> 2;
    const int quad = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS0 = tbase + tt * 128 + lane_off, tO = tbase + 256 + tt * 128 + lane_off;
    uint32_t g = 0;
    for (int item = blockIdx.x; item < a.nitems && ok; item += gridDim.x) {
      const Item it = get_item<KV4, MASK>(a, item, &bad);
      const int r = it.row0 + tt * kRows + quad * 32 + lane;
      int lim = it.len;
      bool row_live = r < a.R;
      if constexpr (KV4) {
        const int i = r % a.Nq;
        row_live = row_live && i < it.ql;
        if constexpr (MASK) lim = max(0, it.len - it.ql + i + 1);
      }
      float m = -INFINITY, l = 0.0f;
      float small = 1.0f;  // what differences of scores are multiplied with: 1 below 2^kFar
      float ev = -100.0f;  // cache: O holds values times 2^(kPUp + kVUp - ev); NaN: the row saw one that is not finite
      for (int t = 0; t < it.nb; ++t, ++g) {
        const uint32_t buf = g & 1, tS = tS0 + buf * 64;
        if (!(ok = wait_warp(s_full + tt * 2 + buf, (g >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        const int stg = g % C::kStages;
        float e_lo = 0.0f, e_hi = 0.0f;
        if constexpr (KV4) {  // early: their way from shared memory is long while the MMA reads it
          if (!(ok = wait_warp(v_ready + stg, (g / C::kStages) & 1, abort_flag))) break;
          e_lo = v_exp[stg * 2];
          e_hi = v_exp[stg * 2 + 1];
        }
        uint32_t raw[kKeys];
        tmem_ld_row<kKeys>(tS, raw);
        float* const s = reinterpret_cast<float*>(raw);
        if constexpr (KV4) {
          const float4* const sc = reinterpret_cast<const float4*>(scales + stg * kKeys);
#pragma unroll
          for (int j = 0; j < kKeys / 4; ++j) {
            const float4 f = sc[j];
            const float2 lo = __fmul2_rn(make_float2(s[4 * j], s[4 * j + 1]), make_float2(f.x, f.y));
            const float2 hi = __fmul2_rn(make_float2(s[4 * j + 2], s[4 * j + 3]), make_float2(f.z, f.w));
            s[4 * j] = lo.x; s[4 * j + 1] = lo.y; s[4 * j + 2] = hi.x; s[4 * j + 3] = hi.y;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(k_empty + stg);
        }
        const int left = lim - (it.k0 + t * kKeys);  // keys of this block that the row sees
        if (left < kKeys) {
#pragma unroll
          for (int j = 0; j < kKeys; ++j)
            if (j >= left) s[j] = -INFINITY;
          if constexpr (MASK) {  // values that the row does not see leave its exponent alone
            if (left <= 0) e_lo = kUnseen;
            if (left <= 32) e_hi = kUnseen;
          }
        }
        float top[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          top[q] = s[q];
#pragma unroll
          for (int j = 4; j + 4 < kKeys; j += 8) top[q] = max3t(top[q], s[j + q], s[j + 4 + q]);
          top[q] = fmaxf(top[q], s[kKeys - 4 + q]);
        }
        float mb = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if constexpr (!KV4) mb *= a.scale_log2;
        // The reference moves on the first block and when passed by kLazy, the
        // exponent of the values when theirs is larger.
        const bool up = mb > m + kLazy<KV4>;
        float f = up ? ex2_approx(m - mb) : 1.0f;
        if (up) {
          m = mb;
          l *= f;
          const int far = static_cast<int>((__float_as_uint(m) >> 23) & 0xFFu) - (126 + kFar<KV4>);
          small = __uint_as_float((127u - max(far, 0)) << 23);
        }
        bool turned = up, odd = false;
        if constexpr (KV4) {
          const float et = fmaxf(e_lo, e_hi);
          if (et > ev) {
            f *= ex2_approx(ev - et);
            ev = et;
            turned = true;
          }
          if constexpr (MASK) {
            odd = fminf(e_lo, e_hi) == kOdd;
            turned = turned || odd;
          }
          e_lo = kPUp + fmaxf(e_lo - ev, -64.0f);  // values below 2^-64 of the largest do not count
          e_hi = kPUp + fmaxf(e_hi - ev, -64.0f);
        }
        const bool any_up = __any_sync(0xFFFFFFFFu, turned);
        if constexpr (MASK) {
          if (any_up) {
            if (odd) {
              float e[2] = {left > 0 ? v_exp[stg * 2] : kUnseen, left > 32 ? v_exp[stg * 2 + 1] : kUnseen};
              const float was = ev;
              bool spoiled = false;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (e[c] != kOdd) continue;
                const int n = min(left - 32 * c, 32);  // keys of these 32 that the row sees, at least one
                spoiled = spoiled || (v_bad[stg * 2 + c] << (32 - n)) != 0;
                float et = -100.0f;
                for (int j = 0; j < n; ++j) et = fmaxf(et, ceilf(v_log[stg * kKeys + 32 * c + j]));
                if (et > ev) ev = et;
              }
              if (ev > was) f *= ex2_approx(was - ev);
              if (spoiled) ev = NAN;
              // The sum is taken here; then the scores take the values' scales.
              const float mr = m == -INFINITY ? 0.0f : m, large = 1.0f / small;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (e[c] != kOdd) {
                  e[c] = kPUp + fmaxf(e[c] - ev, -64.0f);
                  continue;
                }
                e[c] = kNoSum;
                const float base = (kPUp - ev - kNoSum) * large;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  l += ex2_approx((s[32 * c + j] - mr) * small);
                  s[32 * c + j] += fmaf(v_log[stg * kKeys + 32 * c + j], large, base);
                }
                if (isnan(ev)) {
#pragma unroll
                  for (int j = 0; j < 32; ++j) s[32 * c + j] = -INFINITY;
                }
              }
              e_lo = e[0];
              e_hi = e[1];
            }
            __syncwarp();
          }
        }
        if (any_up && t > 0) {  // O holds the blocks before this one
          if (!(ok = wait_warp(pv_done + tt * 2 + (buf ^ 1), ((g - 1) >> 1) & 1, abort_flag))) break;
          tc_fence_after();
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld_row<32>(tO + c, o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = __fmul2_rn(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2);
              o[i] = __float_as_uint(x.x);
              o[i + 1] = __float_as_uint(x.y);
            }
            tmem_st_row_nw<32>(tO + c, o);
          }
        }
        const float mr = m == -INFINITY ? 0.0f : m * small;
        const float cr = KV4 ? small : a.scale_log2 * small;
        const float2 c2 = make_float2(cr, cr);
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) {
          const float shift = KV4 ? (c == 0 ? e_lo : e_hi) - mr : -mr;
          const float2 m2 = make_float2(shift, shift);
          float2 sum2 = make_float2(0.0f, 0.0f);
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float2 x = make_float2(s[c + j], s[c + j + 1]), y = make_float2(s[c + j + 2], s[c + j + 3]);
            x = __ffma2_rn(x, c2, m2);
            y = __ffma2_rn(y, c2, m2);
            x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            sum2 = __fadd2_rn(sum2, x);
            sum2 = __fadd2_rn(sum2, y);
            w[j / 2] = KV4 ? pack_f16(x.x, x.y) : pack_bf16(x.x, x.y);
            w[j / 2 + 1] = KV4 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
          }
          tmem_st_row_nw<16>(tS + c / 2, w);
          sum += (sum2.x + sum2.y) * (KV4 ? ex2_approx(c == 0 ? -e_lo : -e_hi) : 1.0f);
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_full + tt * 2 + buf);
          if constexpr (KV4) mbar_arrive(v_empty + stg);
        }
      }
      if (!ok) break;
      if (it.nb > 0) {
        if (!(ok = wait_warp(pv_done + tt * 2 + ((g - 1) & 1), ((g - 1) >> 1) & 1, abort_flag))) break;
        tc_fence_after();
      }
      // The sum tells a row without keys (zero) from one that is not finite (NaN).  Scores of
      // minus infinity alone, 0 / 0, leave a sum of zero too, and give NaN.
      const bool some = l != 0.0f || (it.nb > 0 && lim > it.k0);
      const float inv = some ? (KV4 ? ex2_approx(ev - kPUp - kVUp) : 1.0f) / l : 0.0f;
      const float lse2 = l != 0.0f ? m + log2f(l) : -INFINITY;
      const size_t bh = static_cast<size_t>(it.b) * a.heads + it.h;
      const size_t at = bh * a.R + r;
      const bool split = KV4 && a.nsplit > 1;
      const size_t prow = static_cast<size_t>(it.split) * (a.nitems / (a.npairs * a.nsplit)) * a.R + at;
      // Rows leave through shared memory, kPiece bytes of each at a time, neighbouring
      // lanes a piece together: a thread writing its own row touched 32 lines per
      // store, 7800 cycles an item at 512 keys against 2500.
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, row_live);
      constexpr int kChunks = C::kPiece / 16, kAtOnce = 32 / kChunks;  // chunks of a piece, rows per store
      auto place = [&](int row, int ch) {  // a row's chunks lie in other banks than its neighbours'
        return smem + C::oStage + ((warp - C::kFirstSoftmax) * 32 + row) * C::kPiece +
               ((ch ^ (row * C::kPiece >> 7 & (kChunks - 1))) << 4);
      };
      const int64_t rbase = it.row0 + tt * kRows + quad * 32;
      auto put = [&](const uint32_t* w, void* dst, int64_t row_bytes) {  // kPiece bytes of each row
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          *reinterpret_cast<uint4*>(place(lane, i)) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        __syncwarp();
        const int ch = lane % kChunks;
        uint8_t* p = static_cast<uint8_t*>(dst) + (lane / kChunks) * row_bytes + ch * 16;
#pragma unroll
        for (int row = lane / kChunks, i = 0; i < kChunks; ++i, row += kAtOnce, p += kAtOnce * row_bytes) {
          const uint4 v = *reinterpret_cast<const uint4*>(place(row, ch));
          if ((live >> row) & 1u) *reinterpret_cast<uint4*>(p) = v;
        }
        __syncwarp();
      };
      constexpr int kPass = C::kPiece / 2;  // channels
#pragma unroll
      for (int c = 0; c < D; c += kPass) {
        uint32_t o[kPass];
        if (it.nb > 0) {
          tmem_ld_row<kPass>(tO + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < kPass; ++i) o[i] = 0u;
        }
        float x[kPass];
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
          // cache: column 2i + e of eight holds channel i + 4e
          const int from = KV4 ? (i & ~7) + 2 * (i & 3) + ((i >> 2) & 1) : i;
          x[i] = some ? __uint_as_float(o[from]) * inv : 0.0f;
        }
        if (split) {
          float* const dst = a.parts.o + (prow - lane) * D + c;
          put(reinterpret_cast<const uint32_t*>(x), dst, D * 4);
          put(reinterpret_cast<const uint32_t*>(x + kPass / 2), dst + kPass / 2, D * 4);
        } else {
          uint32_t w[kPass / 2];
#pragma unroll
          for (int i = 0; i < kPass / 2; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
          put(w, a.out + it.b * a.os.b + it.h * a.os.h + rbase * a.os.n + c, a.os.n * 2);
        }
      }
      tc_fence_before();
      if (row_live) {
        if (split) a.parts.lse2[prow] = lse2;
        else if (a.lse) a.lse[at] = lse2 * kLn2;
      }
    }
  }
  if (!ok) bad |= kStatusTimeout;
  if (bad) atomicOr(&g_tiles_status, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 get_encoder_t() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// 4D map over bf16 [B, H, N, D] with strides; box = 64 channels x `rows`,
// 128-byte swizzle, zeros past N.
bool make_map(CUtensorMap* m, const void* base, int B, int H, int N, int D, const ra_strides& st, int rows) {
  auto enc = get_encoder_t();
  if (!enc) return false;
  // The stride of an extent of one is free; the map wants a valid one.
  const int64_t row = static_cast<int64_t>(D);
  const int64_t sn = N > 1 ? st.n : row, sh = H > 1 ? st.h : row, sb = B > 1 ? st.b : row;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(sn) * 2, static_cast<cuuint64_t>(sh) * 2,
                           static_cast<cuuint64_t>(sb) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool KV4, bool MASK>
cudaError_t launch_tiles(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TileArgs& a,
                         cudaStream_t st) {
  using C = CfgT<D, KV4>;
  auto kern = attn_tiles_kernel<D, KV4, MASK>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(a.nitems < kNumSMs ? a.nitems : kNumSMs), C::kThreads, C::kSmem, st, mq, mk, mv, a);
}

}  // namespace

cudaError_t launch_kv4_tiles(const ra_kv4_cache& c, const ra_kv4_attn& at, const Kv4Plan& plan, const void* q,
                             const int32_t* table, const int32_t* seq_lens, const int32_t* q_lens,
                             const Kv4Parts& parts, void* out, float* lse, cudaStream_t st) {
  g_used.store(true, std::memory_order_relaxed);
  TileArgs a{};
  a.heads = c.Hk; a.group = 1; a.R = at.H / c.Hk * at.Nq;
  a.npairs = (a.R + kTiles * kRows - 1) / (kTiles * kRows);
  a.nsplit = plan.nsplit;
  a.nitems = at.B * c.Hk * a.nsplit * a.npairs;
  a.scale_log2 = at.scale * kLog2e;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.os.n = c.D;
  a.os.h = static_cast<int64_t>(a.R) * c.D;
  a.os.b = a.os.h * c.Hk;
  a.lse = lse;
  a.kv_lens = seq_lens; a.q_lens = q_lens; a.table = table;
  a.k4 = c.k4; a.sk = c.sk; a.v4 = c.v4; a.sv = c.sv;
  a.num_pages = c.num_pages; a.page_log2 = __builtin_ctz(static_cast<unsigned>(c.page_size));
  a.max_pages = at.max_pages; a.Nq = at.Nq;
  a.parts = parts;
  CUtensorMap mq;
  if (!make_map(&mq, q, at.B, c.Hk, a.R, c.D, a.os, kRows)) return cudaErrorInvalidValue;
  if (at.causal)
    return c.D == 64 ? launch_tiles<64, true, true>(mq, mq, mq, a, st) : launch_tiles<128, true, true>(mq, mq, mq, a, st);
  return c.D == 64 ? launch_tiles<64, true, false>(mq, mq, mq, a, st) : launch_tiles<128, true, false>(mq, mq, mq, a, st);
}

cudaError_t launch_attn_cross(const ra_cross_problem& p, const void* q, const ra_strides& qs, const void* k,
                              const ra_strides& ks, const void* v, const ra_strides& vs, const int32_t* kv_lens,
                              void* out, const ra_strides& os, float* lse, cudaStream_t st) {
  g_used.store(true, std::memory_order_relaxed);
  TileArgs a{};
  a.heads = p.H; a.group = p.H / p.Hk; a.R = p.Nq;
  a.npairs = (a.R + kTiles * kRows - 1) / (kTiles * kRows);
  a.nsplit = 1;
  a.nitems = p.B * p.H * a.npairs;
  a.scale_log2 = p.scale * kLog2e;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.os = os;
  a.lse = lse;
  a.kv_lens = kv_lens;
  a.Nk = p.Nk;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, q, p.B, p.H, p.Nq, p.D, qs, kRows) || !make_map(&mk, k, p.B, p.Hk, p.Nk, p.D, ks, kKeys) ||
      !make_map(&mv, v, p.B, p.Hk, p.Nk, p.D, vs, kKeys))
    return cudaErrorInvalidValue;
  return p.D == 64 ? launch_tiles<64, false, false>(mq, mk, mv, a, st) : launch_tiles<128, false, false>(mq, mk, mv, a, st);
}

cudaError_t read_tiles_status(uint32_t* out) {
  *out = 0;
  if (!g_used.load(std::memory_order_relaxed)) return cudaSuccess;
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_tiles_status, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_tiles_status, &zero, sizeof(uint32_t));
}

}  // namespace ra
