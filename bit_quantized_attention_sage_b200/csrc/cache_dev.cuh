// cache_dev.cuh -- device helpers that the attention kernels over the 8-bit
// cache share: code conversions and query rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"

namespace sage {

constexpr float kLog2e = 1.4426950408889634f;

// Swizzled tiles need 1024-byte aligned shared memory; a block that finds
// another base records it and leaves before any barrier or copy.
__device__ __forceinline__ bool smem_misaligned(const void* base, int* status) {
  if ((static_cast<uint32_t>(__cvta_generic_to_shared(base)) & 1023u) == 0) return false;
  if (threadIdx.x == 0 && atomicCAS(status, 0, 3 /* SAGE_ERR_CUDA */) == 0) atomicExch(status + 1, 0x20005);
  return true;
}

// Four int8 codes to two fp16 pairs: code + 128 becomes the low mantissa bits
// of 1024, and 1152 is taken off (exact).
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// The power e with amax 2^-e in [2^14, 2^15) (0 for amax = 0; clamped where
// 2^-e would not be a normal fp32 number).
__device__ __forceinline__ int row_power(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 0;
  return max(-126, min(static_cast<int>(u >> 23) - 127 - 14, 126));
}

__device__ __forceinline__ float load_q(const void* q, int type, size_t i) {
  return type == kTypeBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i])
                           : __half2float(static_cast<const __half*>(q)[i]);
}

// One query row as fp16 values through put(channel, x 2^-e), by a warp;
// returns the row's factor 2^e.  A row that is not there becomes zero.
template <int D, typename Put>
__device__ __forceinline__ float stage_row_as(const CacheAttnArgs& a, int b, int h, int r, int rows,
                                              int lane, Put put) {
  constexpr int PER = D / 32;
  float f[PER];
  float m = 0.0f;
  if (r < rows) {
    const size_t base = a.qb * b + a.qh * (static_cast<size_t>(h) * a.G + r % a.G) +
                        a.qn * (r / a.G) + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e++) {
      f[e] = load_q(a.q, a.type, base + e);
      m = fmaxf(m, fabsf(f[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < PER; e++) f[e] = 0.0f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int p = row_power(m);
  const float inv = pow2i(-p);
#pragma unroll
  for (int e = 0; e < PER; e++) put(lane * PER + e, f[e] * inv);
  return pow2i(p);
}
template <int D>
__device__ __forceinline__ float stage_row(const CacheAttnArgs& a, int b, int h, int r, int rows,
                                           __half* dst, int lane) {
  return stage_row_as<D>(a, b, h, r, rows, lane, [&](int ch, float x) { dst[ch] = __float2half_rn(x); });
}

__device__ __forceinline__ int query_len(const CacheAttnArgs& a, int b) {
  if (!a.q_lens) return a.Nq;
  const int n = __ldg(a.q_lens + b);
  if (n < 0 || n > a.Nq) {
    if (atomicCAS(a.c.status, 0, 1) == 0) atomicExch(a.c.status + 1, 0x20004);
    return n < 0 ? 0 : a.Nq;
  }
  return n;
}

}  // namespace sage
