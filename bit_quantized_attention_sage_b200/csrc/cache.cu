// cache.cu -- what goes into, comes out of and is dropped from the paged
// 8-bit key/value cache: append, read back, evict.
//
// The codes of a page are its tokens divided by the page's scale, rounded to
// nearest even exactly: keys to int8 by an fp32 scale s = fp32(absmax / 127),
// values to e4m3 by a power of two.  A page that already holds tokens keeps
// its scale unless the new tokens need a larger one, in which case its codes
// are rescaled by the ratio.  All of it is one pass over the data: what bounds
// it is HBM (a prompt, a prune) or the launch (one token).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = [&] {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(code));
    __half_raw o;
    o.x = static_cast<unsigned short>(r & 0xFFFFu);
    return o;
  }();
  return __half2float(__half(h));
}

// round-half-even(x / s) for |x / s| <= 127.01, exactly.  x * inv (inv =
// fp32(1 / s)) is off by at most 2^-23 of 127; where that leaves the side of
// a tie open, the remainder x - (k + 1/2) s decides, which one fma gives
// without rounding (it is a small multiple of the last place of s or x).
__device__ __forceinline__ int key_code(float x, float s, float inv) {
  const float q = x * inv;
  float c = rintf(q);
  if (fabsf(fabsf(q - c) - 0.5f) < 6.1035156e-5f) {
    const float lo = floorf(q), r = fmaf(-(lo + 0.5f), s, x);
    c = r > 0.0f ? lo + 1.0f : r < 0.0f ? lo : 2.0f * rintf(0.5f * lo + 0.25f);
    // tie: the even one of lo and lo + 1 (0.5 lo + 0.25 is lo/2 + 1/4, whose
    // nearest integer is lo/2 for even lo and (lo + 1)/2 for odd lo)
  }
  return max(-127, min(127, static_cast<int>(c)));
}
// The same where 1 / s is no normal fp32 number (keys below 1e-36).
__device__ __forceinline__ int key_code_tiny(float x, float s) {
  const double q = s > 0.0f ? rint(static_cast<double>(x) / static_cast<double>(s)) : 0.0;
  return max(-127, min(127, static_cast<int>(q)));
}
// round-half-even(code * s_old / s_new): the product is exact in fp64, and a
// quotient of 24-bit numbers that is not a tie is farther from one than fp64
// rounds.
__device__ __forceinline__ int rescale_key(int code, float s_old, float s_new) {
  if (!(s_new > 0.0f)) return 0;
  const double q = rint(static_cast<double>(code) * s_old / static_cast<double>(s_new));
  return max(-127, min(127, static_cast<int>(q)));
}
// e4m3 code times 2^diff (diff <= 0), rounded to nearest even.
__device__ __forceinline__ uint32_t rescale_value(uint32_t code, int diff) {
  const float v = diff < -60 ? 0.0f * e4m3_value(code) : e4m3_value(code) * pow2i(diff);
  return cvt_e4m3x2(v, 0.0f) & 0xFFu;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

// Eight consecutive channels as fp32; VEC: one 16-byte load.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (VEC) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (sizeof(T) == 2) {
        T pr[2];
        *reinterpret_cast<uint32_t*>(pr) = w[i];
        f[2 * i] = to_f32(pr[0]);
        f[2 * i + 1] = to_f32(pr[1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = to_f32(p[i]);
  }
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  __syncthreads();  // red may still be read from an earlier call
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; i++) m = fmaxf(m, red[i]);
  return m;
}

// ---------------------------------------------------------------- append

// Block (touched page, head, batch): the new tokens of one page, held in
// registers between their maximum and their codes (one read).
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kThreads) k_append(const AppendArgs a) {
  __shared__ float red[kThreads / 32];
  constexpr int CH = D / 8;                      // 8-channel chunks of a token
  constexpr int PER = kPage * CH / kThreads;     // chunks per thread
  const int b = blockIdx.z, h = blockIdx.y;
  const CacheView& c = a.c;
  const int before = seq_length(c, b);
  int n = a.n;
  if (a.n_new) n = max(0, min(n, __ldg(a.n_new + b)));
  const int blk = before / kPage + static_cast<int>(blockIdx.x);
  const long long t0 = static_cast<long long>(blk) * kPage;
  const long long end = static_cast<long long>(before) + n;
  const int lo = static_cast<int>(max(t0, static_cast<long long>(before)) - t0);
  const int hi = static_cast<int>(min(static_cast<long long>(kPage), end - t0));
  if (n == 0 || hi <= lo) return;
  if (blk >= c.max_pages) {  // past the page table: recorded, not written
    if (threadIdx.x == 0 && atomicCAS(c.status, 0, 1) == 0) atomicExch(c.status + 1, 0x20003);
    return;
  }
  const int pg = page_id(c, b, blk);
  if (pg < 0) return;
  const size_t unit = static_cast<size_t>(pg) * c.Hkv + h;
  int8_t* kd = c.k_i8 + unit * (kPage * D);
  uint8_t* vd = c.v_f8 + unit * (kPage * D);
  const T* ks = static_cast<const T*>(a.k) + a.kb * b + a.kh * h;
  const T* vs = static_cast<const T*>(a.v) + a.vb * b + a.vh * h;

  float kx[PER][8], vx[PER][8];
  float ka = 0.0f, va = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int it = threadIdx.x + i * kThreads, r = it / CH, d = it % CH * 8;
    if (r >= lo && r < hi) {
      const long long t = t0 + r - before;
      load8<T, VEC>(ks + a.kn * t + d, kx[i]);
      load8<T, VEC>(vs + a.vn * t + d, vx[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int it = threadIdx.x + i * kThreads, r = it / CH, d = it % CH * 8;
    if (r >= lo && r < hi) {
      if (a.k_shift) {
#pragma unroll
        for (int e = 0; e < 8; e++)
          kx[i][e] = __fsub_rn(kx[i][e], __ldg(a.k_shift + static_cast<size_t>(h) * D + d + e));
      }
#pragma unroll
      for (int e = 0; e < 8; e++) {
        ka = fmaxf(ka, fabsf(kx[i][e]));
        va = fmaxf(va, fabsf(vx[i][e]));
      }
    }
  }
  const float s_old = lo > 0 ? c.k_scale[unit] : 0.0f;
  const int e_old = lo > 0 ? c.v_exp[unit] : kMinVExp;
  ka = block_max(ka, red);
  va = block_max(va, red);
  const float s = fmaxf(s_old, __fdiv_rn(ka, 127.0f));
  const int ve = max(e_old, value_exp(va));
  // every thread has read the old scales (block_max's barriers)
  if (threadIdx.x == 0) {
    c.k_scale[unit] = s;
    c.v_exp[unit] = static_cast<int8_t>(ve);
  }
  const bool tiny = !(s >= 1e-36f);
  const float inv = tiny ? 0.0f : __frcp_rn(s), pv = pow2i(-ve);
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int it = threadIdx.x + i * kThreads, r = it / CH, d = it % CH * 8;
    if (r >= lo && r < hi) {
      uint32_t kw[2], vw[2];
#pragma unroll
      for (int w = 0; w < 2; w++) {
        uint32_t u = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float x = kx[i][w * 4 + e];
          const int q = tiny ? key_code_tiny(x, s) : key_code(x, s, inv);
          u |= static_cast<uint32_t>(q & 0xFF) << (8 * e);
        }
        kw[w] = u;
        vw[w] = cvt_e4m3x4(vx[i][w * 4] * pv, vx[i][w * 4 + 1] * pv, vx[i][w * 4 + 2] * pv,
                           vx[i][w * 4 + 3] * pv);
      }
      *reinterpret_cast<uint2*>(kd + r * D + d) = make_uint2(kw[0], kw[1]);
      *reinterpret_cast<uint2*>(vd + r * D + d) = make_uint2(vw[0], vw[1]);
    } else if (r < lo) {  // tokens the page held: only a grown scale moves them
      if (s > s_old) {
        uint2 u = *reinterpret_cast<const uint2*>(kd + r * D + d);
        uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int j = 0; j < 2; j++) {
          uint32_t o = 0;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int code = static_cast<int8_t>(w[j] >> (8 * e));
            o |= static_cast<uint32_t>(rescale_key(code, s_old, s) & 0xFF) << (8 * e);
          }
          w[j] = o;
        }
        *reinterpret_cast<uint2*>(kd + r * D + d) = make_uint2(w[0], w[1]);
      }
      if (ve > e_old) {
        uint2 u = *reinterpret_cast<const uint2*>(vd + r * D + d);
        uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int j = 0; j < 2; j++) {
          uint32_t o = 0;
#pragma unroll
          for (int e = 0; e < 4; e++) o |= rescale_value((w[j] >> (8 * e)) & 0xFF, e_old - ve) << (8 * e);
          w[j] = o;
        }
        *reinterpret_cast<uint2*>(vd + r * D + d) = make_uint2(w[0], w[1]);
      }
    } else if (lo == 0) {  // a fresh page: the tokens to come read as zero
      *reinterpret_cast<uint2*>(kd + r * D + d) = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(vd + r * D + d) = make_uint2(0u, 0u);
    }
  }
  if (c.weight && threadIdx.x < kPage) {
    const int r = threadIdx.x;
    if (r >= lo && (r < hi || lo == 0)) c.weight[unit * kPage + r] = 0.0f;
  }
}

// ---------------------------------------------------------------- read back

// Block (64 tokens of the result, head, batch); thread: 4 channels, so a warp
// reads 128 bytes of codes and writes 512 of values.
template <int D>
__global__ void __launch_bounds__(kThreads) k_read(const ReadArgs a) {
  constexpr int CH = D / 4;
  const CacheView& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * kPage;
  const int len = seq_length(c, b);
  const int start = a.starts ? __ldg(a.starts + b) : 0;
  const size_t obase = (static_cast<size_t>(b) * c.Hkv + h) * a.n;
#pragma unroll
  for (int i = 0; i < kPage * CH / kThreads; i++) {
    const int it = threadIdx.x + i * kThreads, t = t0 + it / CH, d = it % CH * 4;
    if (t >= a.n) break;
    const long long p = static_cast<long long>(start) + t;
    float4 k = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = k;
    float w = 0.0f;
    if (p >= 0 && p < len) {
      const int pg = page_id(c, b, static_cast<int>(p / kPage));
      if (pg >= 0) {
        const size_t unit = static_cast<size_t>(pg) * c.Hkv + h;
        const size_t at = (unit * kPage + p % kPage) * D + d;
        const char4 kc = *reinterpret_cast<const char4*>(c.k_i8 + at);
        const uint32_t vc = *reinterpret_cast<const uint32_t*>(c.v_f8 + at);
        const float s = c.k_scale[unit], e = pow2i(c.v_exp[unit]);
        k = make_float4(kc.x * s, kc.y * s, kc.z * s, kc.w * s);
        if (a.k_shift) {
          const float4 f = *reinterpret_cast<const float4*>(a.k_shift + static_cast<size_t>(h) * D + d);
          k = make_float4(__fadd_rn(k.x, f.x), __fadd_rn(k.y, f.y), __fadd_rn(k.z, f.z),
                          __fadd_rn(k.w, f.w));
        }
        v = make_float4(e4m3_value(vc & 0xFF) * e, e4m3_value((vc >> 8) & 0xFF) * e,
                        e4m3_value((vc >> 16) & 0xFF) * e, e4m3_value(vc >> 24) * e);
        if (a.w && c.weight) w = c.weight[unit * kPage + p % kPage];
      }
    }
    const size_t o = (obase + t) * D + d;
    *reinterpret_cast<float4*>(a.k + o) = k;
    *reinterpret_cast<float4*>(a.v + o) = v;
    if (a.w && d == 0) a.w[obase + t] = w;
  }
}

// ---------------------------------------------------------------- evict

constexpr int kSelThreads = 1024;

// A weight as an unsigned key that sorts the same way (-0 as +0, NaN above
// every number).
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One block per (batch, head): which tokens stay.  The first `sink` and the
// last `recent` do; of the others the ones of largest weight, the lowest
// index among equal ones.  The smallest weight that stays is found by radix
// selection (four passes over 8 bits, a 256-bin histogram each), then one
// sweep in index order writes the survivors, every warp its own run of
// tokens.
__global__ void __launch_bounds__(kSelThreads) k_select(const EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int n_above[32], n_tie[32];
  const int bh = blockIdx.x, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CacheView& c = a.c;
  const int len = seq_length(c, b);
  const int n = min(len, a.keep);
  int* kept = a.kept + static_cast<size_t>(bh) * a.keep;
  if (h == 0 && tid == 0) a.lengths_out[b] = n;
  for (int i = n + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (n == len) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  // len > keep >= sink + recent: the contested tokens [lo, hi), of which
  // `need` stay
  const int lo = a.sink, hi = len - a.recent;
  const int need = n - a.sink - a.recent;
  auto key = [&](int i) -> uint32_t {
    const int pg = page_id(c, b, i / kPage);
    if (pg < 0) return 0u;
    return weight_key(c.weight[(static_cast<size_t>(pg) * c.Hkv + h) * kPage + i % kPage]);
  };
  uint32_t prefix = 0, left = static_cast<uint32_t>(need);
  if (need > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSelThreads) {
        const uint32_t k = key(i);
        if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 0xFF], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // the bin in which the count from the top reaches `left`
        uint32_t s = 0;
        for (int e = 0; e < 8; e++) s += hist[255 - (lane * 8 + e)];
        uint32_t run = s;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(kFull, run, o);
          if (lane >= o) run += v;
        }
        uint32_t at = run - s;  // keys in higher bins than this lane's
        if (at < left && run >= left) {
          for (int e = 0; e < 8; e++) {
            const int bin = 255 - (lane * 8 + e);
            if (at + hist[bin] >= left) {
              sh_prefix = (prefix << 8) | static_cast<uint32_t>(bin);
              sh_need = left - at;
              break;
            }
            at += hist[bin];
          }
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      left = sh_need;
    }
  }
  // tokens above the threshold `prefix` stay, and the first `left` equal to it
  const int seg = ((len + 31) / 32 + 31) / 32 * 32;
  const int s0 = min(len, warp * seg), s1 = min(len, s0 + seg);
  // 2: stays, 1: equal to the threshold, 0: goes
  auto judge = [&](int i) -> int {
    if (i < lo || i >= hi) return 2;
    if (need <= 0) return 0;
    const uint32_t k = key(i);
    return k > prefix ? 2 : k == prefix ? 1 : 0;
  };
  int above = 0, tie = 0;
  for (int i = s0 + lane; i - lane < s1; i += 32) {
    const int j = i < s1 ? judge(i) : 0;
    above += __popc(__ballot_sync(kFull, j == 2));
    tie += __popc(__ballot_sync(kFull, j == 1));
  }
  if (lane == 0) {
    n_above[warp] = above;
    n_tie[warp] = tie;
  }
  __syncthreads();
  int at = 0, ties = 0;
  for (int w = 0; w < warp; w++) {
    at += n_above[w];
    ties += n_tie[w];
  }
  at += min(ties, static_cast<int>(left));  // of the ties before, the first `left` stay
  for (int i = s0 + lane; i - lane < s1; i += 32) {
    const int j = i < s1 ? judge(i) : 0;
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t mt = __ballot_sync(kFull, j == 1);
    const bool stay = j == 2 || (j == 1 && ties + __popc(mt & lower) < static_cast<int>(left));
    const uint32_t ms = __ballot_sync(kFull, stay);
    if (stay) kept[at + __popc(ms & lower)] = i;
    at += __popc(ms);
    ties += __popc(mt);
  }
}

// Staging of an in-place prune, per (batch, head, block of the result).
struct Stage {
  int8_t* k;
  uint8_t* v;
  float *scale, *weight;
  int8_t* exp;
};
__host__ __device__ inline Stage stage_of(void* ws, size_t units, int D) {
  Stage s;
  char* p = static_cast<char*>(ws);
  s.k = reinterpret_cast<int8_t*>(p);
  p += units * kPage * D;
  s.v = reinterpret_cast<uint8_t*>(p);
  p += units * kPage * D;
  s.weight = reinterpret_cast<float*>(p);
  p += units * kPage * 4;
  s.scale = reinterpret_cast<float*>(p);
  p += units * 4;
  s.exp = reinterpret_cast<int8_t*>(p);
  return s;
}

__device__ __forceinline__ uint32_t abs_max4(uint32_t m, uint32_t w) {
  return __vmaxu4(m, __vabsss4(w));  // per byte; -128 (never written) reads as 127
}

// Block (64 survivors, head, batch): gather their codes, take the page's new
// scales from them and write the requantized codes to the result's page, or
// to the staging buffer of an in-place prune.
template <int D>
__global__ void __launch_bounds__(kThreads) k_gather(const EvictArgs a) {
  __shared__ float red[kThreads / 32];
  __shared__ int src[kPage];      // token, or -1
  __shared__ float s_src[kPage];
  __shared__ int e_src[kPage];
  __shared__ long long at_src[kPage];
  constexpr int CH = D / 16, PER = kPage * CH / kThreads;
  const CacheView& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x;
  const int len = seq_length(c, b), n = min(len, a.keep);
  const int m = min(kPage, n - blk * kPage);
  if (m <= 0 || (!a.pages_out && n == len)) return;
  const size_t ou = (static_cast<size_t>(b) * c.Hkv + h) * gridDim.x + blk;
  if (tid < kPage) {
    int t = -1;
    float s = 0.0f, w = 0.0f;
    int e = 0;
    long long at = 0;
    if (tid < m) {
      t = a.kept[(static_cast<size_t>(b) * c.Hkv + h) * a.keep + blk * kPage + tid];
      const int pg = page_id(c, b, t / kPage);
      if (pg < 0) {
        t = -1;
      } else {
        const size_t unit = static_cast<size_t>(pg) * c.Hkv + h;
        s = c.k_scale[unit];
        e = c.v_exp[unit];
        at = static_cast<long long>(unit * kPage + t % kPage);
        w = c.weight[at];
      }
    }
    src[tid] = t;
    s_src[tid] = s;
    e_src[tid] = e;
    at_src[tid] = at;
    if (a.pages_out) {
      const int po = page_id(c, a.pages_out, a.out_pages, b, blk);
      if (po >= 0) c.weight[(static_cast<size_t>(po) * c.Hkv + h) * kPage + tid] = w;
    } else {
      stage_of(a.ws, static_cast<size_t>(gridDim.x) * c.Hkv * c.B, D).weight[ou * kPage + tid] = w;
    }
  }
  __syncthreads();
  uint4 kc[PER], vc[PER];
  float ks = 0.0f;
  int ve = kMinVExp;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int it = tid + i * kThreads, r = it / CH, d = it % CH * 16;
    kc[i] = vc[i] = make_uint4(0u, 0u, 0u, 0u);
    if (src[r] >= 0) {
      kc[i] = *reinterpret_cast<const uint4*>(c.k_i8 + at_src[r] * D + d);
      vc[i] = *reinterpret_cast<const uint4*>(c.v_f8 + at_src[r] * D + d);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int it = tid + i * kThreads, r = it / CH;
    // largest |code| of the token: of the thread's 16 channels, then of its
    // CH lanes.  e4m3 codes without their sign order like their values.
    uint32_t mk = 0;
    mk = abs_max4(abs_max4(abs_max4(abs_max4(mk, kc[i].x), kc[i].y), kc[i].z), kc[i].w);
    uint32_t mv = __vmaxu4(__vmaxu4(vc[i].x & 0x7F7F7F7Fu, vc[i].y & 0x7F7F7F7Fu),
                           __vmaxu4(vc[i].z & 0x7F7F7F7Fu, vc[i].w & 0x7F7F7F7Fu));
    mk = __vmaxu4(mk, mk >> 16);
    mk = max(mk & 0xFF, (mk >> 8) & 0xFF);
    mv = __vmaxu4(mv, mv >> 16);
    mv = max(mv & 0xFF, (mv >> 8) & 0xFF);
#pragma unroll
    for (int o = CH / 2; o; o >>= 1) {
      mk = max(mk, __shfl_xor_sync(kFull, mk, o));
      mv = max(mv, __shfl_xor_sync(kFull, mv, o));
    }
    if (src[r] >= 0) {
      ks = fmaxf(ks, __fmul_rn(s_src[r], __fdiv_rn(static_cast<float>(mk), 127.0f)));
      // |value| = code * 2^e: its exponent is the code's, shifted
      if (mv) ve = max(ve, value_exp(e4m3_value(mv)) + e_src[r]);
    }
  }
  ks = block_max(ks, red);
  ve = static_cast<int>(block_max(static_cast<float>(ve), red));

  int8_t* kd;
  uint8_t* vd;
  if (a.pages_out) {
    const int po = page_id(c, a.pages_out, a.out_pages, b, blk);
    if (po < 0) return;
    const size_t unit = static_cast<size_t>(po) * c.Hkv + h;
    kd = c.k_i8 + unit * (kPage * D);
    vd = c.v_f8 + unit * (kPage * D);
    if (tid == 0) {
      c.k_scale[unit] = ks;
      c.v_exp[unit] = static_cast<int8_t>(ve);
    }
  } else {
    const Stage st = stage_of(a.ws, static_cast<size_t>(gridDim.x) * c.Hkv * c.B, D);
    kd = st.k + ou * (kPage * D);
    vd = st.v + ou * (kPage * D);
    if (tid == 0) {
      st.scale[ou] = ks;
      st.exp[ou] = static_cast<int8_t>(ve);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int it = tid + i * kThreads, r = it / CH, d = it % CH * 16;
    uint32_t kw[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w};
    uint32_t vw[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
    if (s_src[r] != ks) {
      const float s = s_src[r], ratio = ks > 0.0f ? s / ks : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint32_t o = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int code = static_cast<int8_t>(kw[j] >> (8 * e));
          // as key_code: the quotient in fp32, in fp64 next to a tie
          const float q = static_cast<float>(code) * ratio, f = rintf(q);
          const int r8 = fabsf(fabsf(q - f) - 0.5f) < 6.1035156e-5f
                             ? rescale_key(code, s, ks)
                             : max(-127, min(127, static_cast<int>(f)));
          o |= static_cast<uint32_t>(r8 & 0xFF) << (8 * e);
        }
        kw[j] = o;
      }
    }
    const int diff = e_src[r] - ve;
    if (diff != 0 && src[r] >= 0) {
      // diff > 0 happens where a page's largest tokens went: exact, as the
      // new exponent covers every survivor
      const float up = diff < -60 ? 0.0f : pow2i(min(diff, 126));
#pragma unroll
      for (int j = 0; j < 4; j++)
        vw[j] = cvt_e4m3x4(e4m3_value(vw[j] & 0xFF) * up, e4m3_value((vw[j] >> 8) & 0xFF) * up,
                           e4m3_value((vw[j] >> 16) & 0xFF) * up, e4m3_value(vw[j] >> 24) * up);
    }
    *reinterpret_cast<uint4*>(kd + r * D + d) = make_uint4(kw[0], kw[1], kw[2], kw[3]);
    *reinterpret_cast<uint4*>(vd + r * D + d) = make_uint4(vw[0], vw[1], vw[2], vw[3]);
  }
}

// In place: the staged blocks into the sequence's own first pages.
template <int D>
__global__ void __launch_bounds__(kThreads) k_commit(const EvictArgs a) {
  const CacheView& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, blk = blockIdx.x, tid = threadIdx.x;
  const int len = seq_length(c, b), n = min(len, a.keep);
  if (blk * kPage >= n || n == len) return;
  const int pg = page_id(c, b, blk);
  if (pg < 0) return;
  const size_t ou = (static_cast<size_t>(b) * c.Hkv + h) * gridDim.x + blk;
  const size_t unit = static_cast<size_t>(pg) * c.Hkv + h;
  const Stage st = stage_of(a.ws, static_cast<size_t>(gridDim.x) * c.Hkv * c.B, D);
#pragma unroll
  for (int i = tid; i < kPage * D / 16; i += kThreads) {
    reinterpret_cast<uint4*>(c.k_i8 + unit * (kPage * D))[i] =
        reinterpret_cast<const uint4*>(st.k + ou * (kPage * D))[i];
    reinterpret_cast<uint4*>(c.v_f8 + unit * (kPage * D))[i] =
        reinterpret_cast<const uint4*>(st.v + ou * (kPage * D))[i];
  }
  if (tid < kPage) c.weight[unit * kPage + tid] = st.weight[ou * kPage + tid];
  if (tid == 0) {
    c.k_scale[unit] = st.scale[ou];
    c.v_exp[unit] = st.exp[ou];
  }
}

template <typename T, int D>
void append_d(const AppendArgs& a, bool vec, dim3 grid, cudaStream_t s) {
  if (vec) k_append<T, D, true><<<grid, kThreads, 0, s>>>(a);
  else k_append<T, D, false><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
  // n tokens touch at most this many pages, wherever the first one starts
  const dim3 grid((a.n + kPage - 2) / kPage + 1, a.c.Hkv, a.c.B);
  const long long st = a.kb | a.kh | a.kn | a.vb | a.vh | a.vn;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15u) == 0 &&
                   st % 8 == 0;
  if (a.type == kTypeBf16) {
    if (a.c.D == 128) append_d<__nv_bfloat16, 128>(a, vec, grid, s);
    else append_d<__nv_bfloat16, 64>(a, vec, grid, s);
  } else {
    if (a.c.D == 128) append_d<__half, 128>(a, vec, grid, s);
    else append_d<__half, 64>(a, vec, grid, s);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s) {
  const dim3 grid((a.n + kPage - 1) / kPage, a.c.Hkv, a.c.B);
  if (a.c.D == 128) k_read<128><<<grid, kThreads, 0, s>>>(a);
  else k_read<64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

size_t cache_evict_ws_bytes(int B, int Hkv, int D, int keep) {
  const size_t units = static_cast<size_t>(B) * Hkv * ((keep + kPage - 1) / kPage);
  return (units * (2ull * kPage * D + kPage * 4 + 4 + 1) + 15) / 16 * 16;
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  k_select<<<a.c.B * a.c.Hkv, kSelThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((a.keep + kPage - 1) / kPage, a.c.Hkv, a.c.B);
  if (a.c.D == 128) k_gather<128><<<grid, kThreads, 0, s>>>(a);
  else k_gather<64><<<grid, kThreads, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.pages_out) return e;
  if (a.c.D == 128) k_commit<128><<<grid, kThreads, 0, s>>>(a);
  else k_commit<64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace sage
