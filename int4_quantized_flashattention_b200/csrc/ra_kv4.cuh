// Device helpers of the 4-bit key/value cache: code unpacking, mma.sync and
// asynchronous 16-byte copies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ra_common.cuh"

namespace ra {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kKv4Tiny = 2.350988701644575e-38f;  // 2^-125: rows below it are stored as zeros

// A length given by the caller, held to [0, most]; a value outside is noted.
__device__ __forceinline__ int clamp_len(int x, int most, uint32_t* bad) {
  if (x < 0 || x > most) *bad |= kStatusBadPosition;
  return min(max(x, 0), most);
}

// The two codes in bits 0-3 and 16-19 of w as a bf16 pair: two's complement
// XOR 8 is code + 8, in the low bits of a bf16 of exponent 7 it is 128 + 8 +
// code, and the subtraction of 136 is exact.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t x = (w & 0x000F000Fu) ^ 0x43084308u;
  const uint32_t k136 = 0x43084308u;  // 136 as bf16, twice
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   *reinterpret_cast<const __nv_bfloat162*>(&k136));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// (a & b) ^ c
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The codes as f16 pairs, from bits 0-3 and 16-19, and from bits 4-7 and 20-23.  That an
// integer in the low mantissa bits under the exponent of 1024 is the number 1024 + integer, so
// that one subtraction converts it, is a published method for quantised weights (Kim et al.,
// "Who Says Elephants Can't Run", 2022); the two's complement codes enter by an exclusive-or.
// f16 has ten mantissa bits, so the second pair needs no shift (1024 + 16 (code + 8),
// times 1/16 and minus 72 in one exact fused operation).  Shifts and masks are what
// bounds the kernels that unpack in registers: a word takes five of them, in bf16
// seven.
__device__ __forceinline__ uint32_t codes_f16_lo(uint32_t w) {
  const uint32_t x = and_xor(w, 0x000F000Fu, 0x64086408u);
  const uint32_t k1032 = 0x64086408u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&k1032));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t w) {
  const uint32_t x = and_xor(w, 0x00F000F0u, 0x64806480u);
  const uint32_t k16th = 0x2C002C00u, k72 = 0xD480D480u;  // 1/16 and -72, twice
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&k16th),
                            *reinterpret_cast<const __half2*>(&k72));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// N words from shared memory (aligned to their size) as one access.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
}

// c += a b, f16 in, fp32 out: a 16 x 16 (row), b 16 x 8 (column).
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes the warp's 8 x 8 matrix of 16-bit values.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes global -> shared without registers; `bytes` 0 fills with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace ra
