// cache_dev.cuh -- device helpers that the attention kernels over the 8-bit
// cache share: code conversions and query rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "sm100.cuh"

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

// Two neighbouring channels of one output row.
__device__ __forceinline__ void store_o2(const CacheAttnArgs& a, size_t i, float x, float y) {
  if (a.type == kTypeBf16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.o) + i;
    p[0] = __float2bfloat16_rn(x);
    p[1] = __float2bfloat16_rn(y);
  } else {
    __half* p = static_cast<__half*>(a.o) + i;
    p[0] = __float2half_rn(x);
    p[1] = __float2half_rn(y);
  }
}

// ---------------------------------------------------------------- tcgen05 operands

// fp16 operand tiles: [D / 64][128 rows][128 bytes], 128-byte swizzle.  Byte
// offset of 16-byte chunk `ch` (8 channels) of row r.
__device__ __forceinline__ uint32_t op_off(int r, int ch) {
  return static_cast<uint32_t>((ch >> 3) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}
// Instruction descriptor of kind::f16 with f16 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// The fixed upper words of the operand descriptors (128-byte swizzle, 8-row
// groups 1024 bytes apart); the lower word holds the address / 16 and the
// leading offset: unused (1) for K-major tiles, from run to run of 64 channels
// (16 KB) for the MN-major V.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
constexpr uint32_t kDescLoK = 1u << 16, kDescLoV = (16384u >> 4) << 16;
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
  return d;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// D[tmem] = A B^T over D channels of two K-major operand tiles, given by the
// lower words of their descriptors.
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t tmem, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; kk++) {
    const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
    mma_f16_ss(tmem, desc_of(a + off), desc_of(b + off), idesc, kk > 0);
  }
}

// UN chunks of eight channels of the query, as they lie (at[u] < 0: zeros);
// all loads are on their way before the first is waited for.
template <int UN>
__device__ __forceinline__ void load_q8(const CacheAttnArgs& a, const long long (&at)[UN], uint4 (&r)[UN]) {
  const uint16_t* q = static_cast<const uint16_t*>(a.q);
  if (a.q_vec) {
#pragma unroll
    for (int u = 0; u < UN; u++)
      r[u] = at[u] < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4*>(q + at[u]));
  } else {
#pragma unroll
    for (int u = 0; u < UN; u++) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (at[u] >= 0) {
#pragma unroll
        for (int j = 0; j < 4; j++)
          w[j] = __ldg(q + at[u] + 2 * j) | static_cast<uint32_t>(__ldg(q + at[u] + 2 * j + 1)) << 16;
      }
      r[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}
__device__ __forceinline__ void q8_floats(const CacheAttnArgs& a, const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if (a.type == kTypeBf16) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      f[2 * j] = x.x;
      f[2 * j + 1] = x.y;
    }
  }
}
// Of head h of key heads, chunk c of query row r (token r / G, head r % G of the group).
__device__ __forceinline__ long long q8_at(const CacheAttnArgs& a, int b, int h, int r, int c) {
  const int tok = r / a.G;
  return static_cast<long long>(a.qb * b + a.qh * (static_cast<size_t>(h) * a.G + (r - tok * a.G)) + a.qn * tok +
                                c * 8);
}

// The largest magnitude of a row whose CH chunks lie in as many lanes.
template <int CH>
__device__ __forceinline__ float row_max(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
  for (int o = CH / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// Chunk c of operand row r: f 2^-p as fp16.
__device__ __forceinline__ void store_q8(uint8_t* tile, int r, int c, const float (&f)[8], int p) {
  const float inv = pow2i(-p);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const __half2 x = __floats2half2_rn(f[2 * j] * inv, f[2 * j + 1] * inv);
    w[j] = *reinterpret_cast<const uint32_t*>(&x);
  }
  *reinterpret_cast<uint4*>(tile + op_off(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Query rows r0 .. r0 + n - 1 (n <= 128; those from `rows` on become zero) to
// an fp16 operand tile; factor[i] = the row's power of two.  By NT threads,
// `tid` in [0, NT); n * D / 8 must be a multiple of 32.
template <int D, int NT>
__device__ __forceinline__ void stage_rows(const CacheAttnArgs& a, int b, int h, int r0, int rows, int n,
                                           uint8_t* tile, float* factor, int tid) {
  constexpr int CH = D / 8, UN = 4;
  for (int i0 = tid; i0 < n * CH; i0 += NT * UN) {
    long long at[UN];
    uint4 raw[UN];
#pragma unroll
    for (int u = 0; u < UN; u++) {
      const int i = i0 + u * NT, r = r0 + i / CH;
      at[u] = i < n * CH && r < rows ? q8_at(a, b, h, r, i % CH) : -1;
    }
    load_q8(a, at, raw);
#pragma unroll
    for (int u = 0; u < UN; u++) {
      const int i = i0 + u * NT;
      if (i - (tid & 31) >= n * CH) break;  // whole warps
      float f[8];
      q8_floats(a, raw[u], f);
      const int p = row_power(row_max<CH>(f));
      store_q8(tile, i / CH, i % CH, f, p);
      if (i % CH == 0) factor[i / CH] = pow2i(p);
    }
  }
}

// ---------------------------------------------------------------- sums of weights
//
// y = 2^(t + e - M + 7) of a key with score t on a page of value exponent e; a
// row's sum adds y 2^-e.  Exponents lie up to 160 apart, so y may be below every
// fp32 number (2^-126) where y 2^-e is what the sum consists of.  Pages kFar
// or more below E, the largest exponent so far, therefore take
// 2^(t + f - M + 7) 2^-f for the sum, f = E - kFar.  Nothing is lost then: with
// M = t' + e' of a key that was seen, e' <= E, that power is 2^(t - t' - 53) at
// least, and as t + e <= M + 8 it is 2^(15 + 160 - kFar) at most.  (The product
// with the values keeps y: against 2^(t' + e') it is nothing.)
constexpr int kFar = 60;
__device__ __forceinline__ int sum_exp(int e, int top) { return max(e, top - kFar); }
__device__ __forceinline__ float sum_unit(int f) { return pow2i(min(-f, 127)); }

// s + x 2^d, d <= 0, al = 2^d (0 below 2^-126): a sum x of pages far below the
// new reference is scaled in two steps.
__device__ __forceinline__ float add_scaled(float s, float x, float d, float al) {
  if (d >= -100.0f) return fmaf(al, x, s);
  const float h = ex2_approx(0.5f * d);
  return s + x * h * h;
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

// ---------------------------------------------------------------- shares of the work
//
// The work of a call is a line of pages: sequences in order, in each the key
// heads, in each head the pages its rows visit.  Block c of C takes the c-th
// of C equal stretches of it, so uneven sequences cost no tail and a block's
// start (its first dependent loads and tile, some 4 us) is paid once, not
// once for every range of a fixed length.  A stretch cuts at most two heads:
// the partial result of a head begun by an earlier block goes to slot 2 c,
// that of one a later block finishes to slot 2 c + 1.

// Pages of sequence b that count (0: nothing to do; at least 1 where rows
// have to be written).
template <bool WEIGHTS>
__device__ __forceinline__ PageRuns seq_runs(const CacheAttnArgs& a, int b, int len, int qn) {
  PageRuns r;
  if constexpr (WEIGHTS) {  // every page: those that no row sees get 0
    r.n = r.ns = (len + kPage - 1) / kPage;
    r.gap = 0;
  } else {
    const long long off = static_cast<long long>(len) - qn;
    r = page_runs(a.mask, off, off + max(qn - 1, 0), len);
  }
  return r;
}
template <bool WEIGHTS>
__device__ __forceinline__ int seq_work(const CacheAttnArgs& a, int b) {
  const int len = seq_length(a.c, b), qn = query_len(a, b);
  if (WEIGHTS) return seq_runs<WEIGHTS>(a, b, len, qn).n;
  return qn == 0 ? 0 : max(1, seq_runs<WEIGHTS>(a, b, len, qn).n);
}

__device__ __forceinline__ long long share_start(long long work, int c, int n) { return work * c / n; }
// The block whose stretch holds position x.
__device__ __forceinline__ int share_of(long long work, long long x, int n) {
  return static_cast<int>(((x + 1) * n - 1) / work);
}

struct Place {
  long long work;    // of the whole call, pages
  long long before;  // pages of one head before sequence b
  int b;
};
template <int W>
struct PlaceSmem {
  long long sum[W];
  long long before;
  int b;
};
// By a block of W warps: the whole work, and the sequence that position x (a
// function of the work) lies in.
template <int W, bool WEIGHTS, typename X>
__device__ __forceinline__ Place locate(PlaceSmem<W>& s, const CacheAttnArgs& a, X x) {
  constexpr int NT = W * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Every warp by itself, one barrier instead of five (weights of 2 x 32 tokens
  // 41.0 -> 40.0 us, of 16 tokens 27.5 -> 26.8, attention of 32 113.4 -> 112.9).
  if (a.c.B <= 32) {
    const int n = lane < a.c.B ? seq_work<WEIGHTS>(a, lane) : 0;
    int run = n;  // (at most 2^24 pages a sequence)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    Place p;
    p.work = static_cast<long long>(__shfl_sync(0xffffffffu, run, 31)) * a.c.Hkv;
    const long long at = x(p.work);
    const uint32_t here = __ballot_sync(0xffffffffu, static_cast<long long>(run - n) * a.c.Hkv <= at &&
                                                         at < static_cast<long long>(run) * a.c.Hkv);
    p.b = here ? __ffs(here) - 1 : a.c.B;
    p.before = __shfl_sync(0xffffffffu, run - n, p.b & 31);
    __syncthreads();
    return p;
  }
  const int first = tid < a.c.B ? seq_work<WEIGHTS>(a, tid) : 0;
  long long mine = first;
  for (int b = tid + NT; b < a.c.B; b += NT) mine += seq_work<WEIGHTS>(a, b);
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s.sum[warp] = mine;
  if (tid == 0) s.b = a.c.B;
  __syncthreads();
  Place p{0, 0, 0};
#pragma unroll
  for (int w = 0; w < W; w++) p.work += s.sum[w];
  p.work *= a.c.Hkv;
  const long long at = x(p.work);
  long long base = 0;  // pages before the sequences from b0 on
  for (int b0 = 0; b0 < a.c.B; b0 += NT) {
    const int n = b0 == 0 ? first : b0 + tid < a.c.B ? seq_work<WEIGHTS>(a, b0 + tid) : 0;
    long long run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    __syncthreads();
    if (lane == 31) s.sum[warp] = run;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
      if (w < warp) run += s.sum[w];
      all += s.sum[w];
    }
    if ((base + run - n) * a.c.Hkv <= at && at < (base + run) * a.c.Hkv) {
      s.b = b0 + tid;
      s.before = base + run - n;
    }
    base += all;
    if (base * a.c.Hkv > at) break;
  }
  __syncthreads();
  p.b = s.b;
  p.before = s.before;
  return p;
}

}  // namespace sage
