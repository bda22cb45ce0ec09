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
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;

constexpr float kRound = 12582912.0f;       // 1.5 * 2^23
constexpr float kNearTie = 3.0517578e-5f;   // 2^-15: twice the error of x * fp32(1 / s) at 127
constexpr float kTinyScale = 1e-36f;        // below, neither s nor 1 / s need be a normal number
constexpr float kNearTieScaled = 1.5258789e-5f;  // 2^-16: twice that of code * fp32(s / s')

// The low bytes of four words as one.
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

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

// round-half-even(x / s) for |x / s| <= 127.01, exactly, by the slow way:
// x * inv (inv = fp32(1 / s)) is off by at most 2^-23 of 127; where that leaves
// the side of a tie open, the remainder x - (k + 1/2) s decides, which one fma
// gives without rounding (it is a small multiple of the last place of s or
// x).  `tiny`: 1 / s is no normal fp32 number (keys below 1e-36), fp64 decides.
__device__ __noinline__ int key_code_slow(float x, float s, float inv, bool tiny) {
  float c;
  if (tiny) {
    c = s > 0.0f ? static_cast<float>(rint(static_cast<double>(x) / static_cast<double>(s))) : 0.0f;
  } else {
    const float q = x * inv;
    c = rintf(q);
    if (fabsf(fabsf(q - c) - 0.5f) < kNearTie) {
      const float lo = floorf(q), r = fmaf(-(lo + 0.5f), s, x);
      c = r > 0.0f ? lo + 1.0f : r < 0.0f ? lo : 2.0f * rintf(0.5f * lo + 0.25f);
      // tie: the even one of lo and lo + 1 (0.5 lo + 0.25 is lo/2 + 1/4, whose
      // nearest integer is lo/2 for even lo and (lo + 1)/2 for odd lo)
    }
  }
  return max(-127, min(127, static_cast<int>(c)));
}
// Eight codes as two words, of finite |x| <= 127.01 s.  Adding 1.5 * 2^23 to
// the quotient (one rounding) leaves it, rounded, in the sum's low byte; only
// where one of the eight is next to a tie, or 1 / s is no normal number, does
// the slow way run.
__device__ __forceinline__ void key_codes(const float (&x)[8], float s, float inv, bool tiny, uint32_t (&w)[2]) {
  const float2 ii = make_float2(inv, inv), kk = make_float2(kRound, kRound), neg = make_float2(-1.0f, -1.0f);
  float worst = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const float2 a = make_float2(x[4 * i], x[4 * i + 1]), b = make_float2(x[4 * i + 2], x[4 * i + 3]);
    const float2 ya = __ffma2_rn(a, ii, kk), yb = __ffma2_rn(b, ii, kk);
    const float2 ra = __ffma2_rn(a, ii, __ffma2_rn(ya, neg, kk)), rb = __ffma2_rn(b, ii, __ffma2_rn(yb, neg, kk));
    worst = fmax3(worst, fmax3(fabsf(ra.x), fabsf(ra.y), fabsf(rb.x)), fabsf(rb.y));
    w[i] = low_bytes(ya.x, ya.y, yb.x, yb.y);
  }
  if (tiny || worst > 0.5f - kNearTie) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      uint32_t u = 0;
      for (int e = 0; e < 4; e++) {
        const float v = e == 0 ? x[4 * i] : e == 1 ? x[4 * i + 1] : e == 2 ? x[4 * i + 2] : x[4 * i + 3];
        u |= static_cast<uint32_t>(key_code_slow(v, s, inv, tiny) & 0xFF) << (8 * e);
      }
      w[i] = u;
    }
  }
}
// round-half-even(code * s_old / s_new): the product is exact in fp64, and a
// quotient of 24-bit numbers that is not a tie is farther from one than fp64
// rounds.
__device__ __forceinline__ int rescale_key(int code, float s_old, float s_new) {
  if (!(s_new > 0.0f)) return 0;
  const double q = rint(static_cast<double>(code) * s_old / static_cast<double>(s_new));
  return max(-127, min(127, static_cast<int>(q)));
}
__device__ __noinline__ uint32_t rescale_keys(uint32_t w, float s_old, float s_new) {
  uint32_t o = 0;
  for (int e = 0; e < 4; e++)
    o |= static_cast<uint32_t>(rescale_key(static_cast<int8_t>(w >> (8 * e)), s_old, s_new) & 0xFF) << (8 * e);
  return o;
}
// e4m3 code times 2^diff, rounded to nearest even.
__device__ __forceinline__ uint32_t rescale_value(uint32_t code, int diff) {
  const float v = diff < -60 ? 0.0f * e4m3_value(code) : e4m3_value(code) * pow2i(min(diff, 126));
  return cvt_e4m3x2(v, 0.0f) & 0xFFu;
}
__device__ __noinline__ uint32_t rescale_values(uint32_t w, int diff) {
  uint32_t o = 0;
  for (int e = 0; e < 4; e++) o |= rescale_value((w >> (8 * e)) & 0xFF, diff) << (8 * e);
  return o;
}
// Four e4m3 codes times a power of two that is exact in fp16.
__device__ __forceinline__ uint32_t scale_values(uint32_t w, __half2 f) {
  uint32_t a, b, r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b) : "r"(w));
  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), f);
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&b), f);
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)), "r"(*reinterpret_cast<const uint32_t*>(&y)));
  return r;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

// Eight consecutive 16-bit channels; VEC: one 16-byte load.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load8(const T* p) {
  if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + 2 * i;
    w[i] = q[0] | static_cast<uint32_t>(q[1]) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    T pr[2];
    *reinterpret_cast<uint32_t*>(pr) = w[i];
    f[2 * i] = to_f32(pr[0]);
    f[2 * i + 1] = to_f32(pr[1]);
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

// Measured, with the launch: 2040 tokens of 24 heads 14 us (2.6 TB/s: 1584
// blocks at three an SM, by 78 registers, are 3.6 rounds, each three dependent
// loads long), one token of 32 x 8 heads 7 us.  With keys and values in one block 24 us.
//
// Block (touched page and keys or values, head, batch): the new tokens of one
// page, held in registers as they came between their maximum and their codes,
// so they are read once.  Keys and values in blocks of their own: twice the
// blocks at half the registers, and a block is mostly latency (the sequence's
// length, the tokens, the page).
template <typename T, int D, bool VEC, bool KEYS>
__device__ __forceinline__ void append_page(const AppendArgs& a, int b, int h, int blk, int before, int lo,
                                            int hi, float* red) {
  constexpr int CH = D / 8;                   // 8-channel chunks of a token
  constexpr int PER = kPage * CH / kThreads;  // chunks per thread
  constexpr int RS = kThreads / CH;           // rows between a thread's chunks
  static_assert(kThreads % CH == 0, "a thread's chunks are of the same channels");
  const CacheView& c = a.c;
  const int r0 = threadIdx.x / CH, d = threadIdx.x % CH * 8;
  const T* src = static_cast<const T*>(KEYS ? a.k : a.v) + (KEYS ? a.kb : a.vb) * b + (KEYS ? a.kh : a.vh) * h + d;
  const long long sn = KEYS ? a.kn : a.vn, first = static_cast<long long>(blk) * kPage - before;
  uint4 x[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int r = r0 + i * RS;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= lo && r < hi) x[i] = load8<T, VEC>(src + sn * (first + r));
  }
  float sh[8];
#pragma unroll
  for (int e = 0; e < 8; e++)
    sh[e] = KEYS && a.k_shift ? __ldg(a.k_shift + static_cast<size_t>(h) * D + d + e) : 0.0f;
  const int pg = page_id(c, b, blk);
  if (pg < 0) return;
  const size_t unit = static_cast<size_t>(pg) * c.Hkv + h;
  uint8_t* dst = (KEYS ? reinterpret_cast<uint8_t*>(c.k_i8) : c.v_f8) + unit * (kPage * D) + d;
  const float s_old = KEYS && lo > 0 ? c.k_scale[unit] : 0.0f;
  const int e_old = !KEYS && lo > 0 ? c.v_exp[unit] : kMinVExp;
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int r = r0 + i * RS;
    if (r >= lo && r < hi) {
      float f[8];
      unpack8<T>(x[i], f);
#pragma unroll
      for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(__fsub_rn(f[e], sh[e])));
    }
  }
  m = block_max(m, red);
  const float s = fmaxf(s_old, __fdiv_rn(m, 127.0f));
  const int ve = max(e_old, value_exp(m));
  // every thread has read the old scale (block_max's barriers)
  if (threadIdx.x == 0) {
    if (KEYS) c.k_scale[unit] = s;
    else c.v_exp[unit] = static_cast<int8_t>(ve);
  }
  const bool tiny = !(s >= kTinyScale);
  const float inv = tiny ? 0.0f : __frcp_rn(s), pv = pow2i(-ve);
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int r = r0 + i * RS;
    uint2* p = reinterpret_cast<uint2*>(dst + r * D);
    if (r >= lo && r < hi) {
      uint32_t w[2];
      float f[8];
      unpack8<T>(x[i], f);
      if constexpr (KEYS) {
#pragma unroll
        for (int e = 0; e < 8; e++) f[e] = __fsub_rn(f[e], sh[e]);
        key_codes(f, s, inv, tiny, w);
      } else {
#pragma unroll
        for (int k = 0; k < 2; k++)
          w[k] = cvt_e4m3x4(f[k * 4] * pv, f[k * 4 + 1] * pv, f[k * 4 + 2] * pv, f[k * 4 + 3] * pv);
      }
      *p = make_uint2(w[0], w[1]);
    } else if (r < lo) {  // tokens the page held: only a grown scale moves them
      if (KEYS ? s > s_old : ve > e_old) {
        const uint2 u = *p;
        *p = KEYS ? make_uint2(rescale_keys(u.x, s_old, s), rescale_keys(u.y, s_old, s))
                  : make_uint2(rescale_values(u.x, e_old - ve), rescale_values(u.y, e_old - ve));
      }
    } else if (lo == 0) {  // a fresh page: the tokens to come read as zero
      *p = make_uint2(0u, 0u);
    }
  }
  if (KEYS && c.weight && threadIdx.x < kPage) {
    const int r = threadIdx.x;
    if (r >= lo && (r < hi || lo == 0)) c.weight[unit * kPage + r] = 0.0f;
  }
}

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kThreads) k_append(const AppendArgs a) {
  __shared__ float red[kThreads / 32];
  const int b = blockIdx.z, h = blockIdx.y;
  const int before = seq_length(a.c, b);
  int n = a.n;
  if (a.n_new) n = max(0, min(n, __ldg(a.n_new + b)));
  const int blk = before / kPage + static_cast<int>(blockIdx.x >> 1);
  const long long t0 = static_cast<long long>(blk) * kPage;
  const long long end = static_cast<long long>(before) + n;
  const int lo = static_cast<int>(max(t0, static_cast<long long>(before)) - t0);
  const int hi = static_cast<int>(min(static_cast<long long>(kPage), end - t0));
  if (n == 0 || hi <= lo) return;
  if (blk >= a.c.max_pages) {  // past the page table: recorded, not written
    if (threadIdx.x == 0 && atomicCAS(a.c.status, 0, 1) == 0) atomicExch(a.c.status + 1, 0x20003);
    return;
  }
  if (blockIdx.x & 1) append_page<T, D, VEC, false>(a, b, h, blk, before, lo, hi, red);
  else append_page<T, D, VEC, true>(a, b, h, blk, before, lo, hi, red);
}

// ---------------------------------------------------------------- read back

// Block (64 tokens of the result, head, batch); thread: 4 channels, so a warp
// reads 128 bytes of codes and writes 512 of values.  HBM bounds it: 4096
// tokens of 8 x 8 heads x 128 channels 56 us, 6.0 TB/s.
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

constexpr int kSelCluster = 4;   // blocks that share a (batch, head)
constexpr int kSelThreads = 512;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 16384;  // weights a block keeps in shared memory

// A weight as an unsigned key that sorts the same way (-0 as +0, NaN above
// every number).
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One cluster per (batch, head): which tokens stay.  The first `sink` and the
// last `recent` do; of the others the ones of largest weight, the lowest
// index among equal ones.  The smallest weight that stays is found by radix
// selection: three passes over 11, 11 and 10 bits (the first digit then splits
// an octave in four, so a heavy tail spreads over many bins).  Each of the four
// blocks takes a quarter of the sequence, then all of the bins, summed over the
// blocks' shared memories; a lone block took 45 us for 26520 tokens and left
// most SMs idle.  One sweep in index order then writes the survivors, every warp
// its own run of tokens.  The weights are read from memory once and kept in
// shared memory where they fit (65536 tokens); longer sequences read them
// again (L2) in every pass.  Measured: 8 x 8 heads of 16000 tokens 20 us, 24
// heads of 26520 21 us: the latency of the three passes and of the two sweeps,
// not the 4 MB of weights.  (With each block taking a quarter of the bins, three
// exchanges a pass instead of one, 21 and 22.)
__global__ void __cluster_dims__(kSelCluster, 1, 1) __launch_bounds__(kSelThreads) k_select(const EvictArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t sel[];  // read as uint4: bins, keys
  constexpr int W = kSelThreads / 32;
  static_assert(kSelThreads * 4 == kSelBins, "four bins of the histogram for every thread");
  static_assert(kSelBins % 4 == 0 && kPage % 4 == 0, "bins and keys start on 16 bytes");
  uint32_t* hist = sel;                 // [3][kSelBins], one for each pass
  uint32_t* keys = sel + 3 * kSelBins;  // [a.sel_keys], of this block's tokens
  int* unit = reinterpret_cast<int*>(keys + a.sel_keys);  // [a.sel_keys / 64]: (page, head) of its pages, or -1
  __shared__ uint32_t sh_prefix, sh_need, sh_sum[W];
  __shared__ int n_above[W], n_tie[W], total[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int bh = blockIdx.x / kSelCluster, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CacheView& c = a.c;
  const int len = seq_length(c, b);
  const int n = min(len, a.keep);
  int* kept = a.kept + static_cast<size_t>(bh) * a.keep;
  int* from = a.from + static_cast<size_t>(bh) * a.keep;
  auto unit_of = [&](int i) {
    const int pg = page_id(c, b, i / kPage);
    return pg < 0 ? -1 : pg * c.Hkv + h;
  };
  const int all_tid = rank * kSelThreads + tid, all = kSelCluster * kSelThreads;
  if (h == 0 && all_tid == 0) a.lengths_out[b] = n;
  for (int i = n + all_tid; i < a.keep; i += all) kept[i] = from[i] = -1;
  if (n == len) {  // (the whole cluster leaves)
    for (int i = all_tid; i < n; i += all) {
      kept[i] = i;
      from[i] = unit_of(i);
    }
    return;
  }
  // len > keep >= sink + recent: the contested tokens [lo, hi), of which
  // `need` stay; this block's tokens are [t0, t1), whole pages
  const int lo = a.sink, hi = len - a.recent;
  const int need = n - a.sink - a.recent;
  const int share = ((len + kSelCluster - 1) / kSelCluster + kPage - 1) / kPage * kPage;
  const int t0 = min(len, rank * share), t1 = min(len, t0 + share);
  auto fetch = [&](int i) -> uint32_t {
    const int u = unit_of(i);
    return u < 0 ? 0u : weight_key(c.weight[static_cast<size_t>(u) * kPage + i % kPage]);
  };
  const bool local = share <= a.sel_keys;
  if (local) {
    // a half warp a page, 16 bytes a lane
#pragma unroll 4
    for (int i = t0 + tid * 4; i < t1; i += kSelThreads * 4) {
      const int u = unit_of(i);
      float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (u >= 0) w = *reinterpret_cast<const float4*>(c.weight + static_cast<size_t>(u) * kPage + i % kPage);
      const bool ok = u >= 0;
      if (i % kPage == 0) unit[(i - t0) / kPage] = u;
      *reinterpret_cast<uint4*>(keys + i - t0) = make_uint4(ok ? weight_key(w.x) : 0u, ok ? weight_key(w.y) : 0u,
                                                            ok ? weight_key(w.z) : 0u, ok ? weight_key(w.w) : 0u);
    }
    __syncthreads();
  }
  auto key = [&](int i) -> uint32_t { return local ? keys[i - t0] : fetch(i); };
  uint32_t prefix = 0, left = static_cast<uint32_t>(need);
  if (need > 0) {
    const int c0 = max(t0, lo), c1 = min(t1, hi);
    for (int i = tid; i < 3 * kSelBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3; pass++) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t mask = (1u << bits) - 1u;
      uint32_t* bins = hist + pass * kSelBins;
      for (int i = c0 + tid; i < c1; i += kSelThreads) {
        const uint32_t k = key(i);
        if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&bins[(k >> shift) & mask], 1u);
      }
      cluster.sync();
      // this thread's four bins, from the top, of the whole cluster: every
      // block finds the threshold by itself, so this is the pass's only
      // exchange
      const int quad = kSelBins / 4 - 1 - tid;
      uint4 c4 = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int r = 0; r < kSelCluster; r++) {
        const uint4 o = reinterpret_cast<const uint4*>(cluster.map_shared_rank(bins, r))[quad];
        c4 = make_uint4(c4.x + o.x, c4.y + o.y, c4.z + o.z, c4.w + o.w);
      }
      const uint32_t cnt = c4.x + c4.y + c4.z + c4.w;
      uint32_t run = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, run, o);
        if (lane >= o) run += v;
      }
      if (lane == 31) sh_sum[warp] = run;
      __syncthreads();
      uint32_t mine = lane < warp ? sh_sum[lane & (W - 1)] : 0u;
#pragma unroll
      for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(kFull, mine, o);
      uint32_t before = run - cnt + mine;
      // the bin in which the count from the top reaches `left`
      if (before < left && before + cnt >= left) {
        const uint32_t down[4] = {c4.w, c4.z, c4.y, c4.x};
        int e = 0;
        while (before + down[e] < left) before += down[e++];
        sh_prefix = (prefix << bits) | static_cast<uint32_t>(4 * quad + 3 - e);
        sh_need = left - before;
      }
      __syncthreads();
      prefix = sh_prefix;
      left = sh_need;
    }
  }
  // tokens above the threshold `prefix` stay, and the first `left` equal to it
  const int seg = ((t1 - t0 + W - 1) / W + 31) / 32 * 32;
  const int s0 = min(t1, t0 + warp * seg), s1 = min(t1, s0 + seg);
  // 2: stays, 1: equal to the threshold, 0: goes
  auto fate = [&](int i) -> int {
    if (i < lo || i >= hi) return 2;
    if (need <= 0) return 0;
    const uint32_t k = key(i);
    return k > prefix ? 2 : k == prefix ? 1 : 0;
  };
  int above = 0, tie = 0;
#pragma unroll 4
  for (int i = s0 + lane; i < s1; i += 32) {
    const int j = fate(i);
    above += j == 2;
    tie += j == 1;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    above += __shfl_xor_sync(kFull, above, o);
    tie += __shfl_xor_sync(kFull, tie, o);
  }
  if (lane == 0) {
    n_above[warp] = above;
    n_tie[warp] = tie;
  }
  __syncthreads();
  int a_in = lane < W ? n_above[lane] : 0, t_in = lane < W ? n_tie[lane] : 0;
  int at = lane < warp ? a_in : 0, ties = lane < warp ? t_in : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a_in += __shfl_xor_sync(kFull, a_in, o);
    t_in += __shfl_xor_sync(kFull, t_in, o);
    at += __shfl_xor_sync(kFull, at, o);
    ties += __shfl_xor_sync(kFull, ties, o);
  }
  if (tid == 0) {
    total[0] = a_in;
    total[1] = t_in;
  }
  cluster.sync();
#pragma unroll
  for (int r = 0; r < kSelCluster; r++) {
    const int* other = cluster.map_shared_rank(total, r);
    if (r < rank) {
      at += other[0];
      ties += other[1];
    }
  }
  cluster.sync();  // no block leaves while another reads its totals
  at += min(ties, static_cast<int>(left));  // of the ties before, the first `left` stay
  for (int i = s0 + lane; i - lane < s1; i += 32) {
    const int j = i < s1 ? fate(i) : 0;
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t mt = __ballot_sync(kFull, j == 1);
    const bool stay = j == 2 || (j == 1 && ties + __popc(mt & lower) < static_cast<int>(left));
    const uint32_t ms = __ballot_sync(kFull, stay);
    if (stay) {
      kept[at + __popc(ms & lower)] = i;
      from[at + __popc(ms & lower)] = local ? unit[(i - t0) / kPage] : unit_of(i);
    }
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

// The page's new scale from its survivors, and their requantized codes to the
// result's page, or to the staging buffer of an in-place prune.
template <int D, bool KEYS, int PER>
__device__ __forceinline__ void requantize(const EvictArgs& a, int h, int po, size_t units, size_t ou,
                                           const uint4 (&x)[PER], const float (&s_src)[PER],
                                           const int (&e_src)[PER], const float (&w)[PER],
                                           const bool (&there)[PER], float* red) {
  constexpr int CH = D / 16;
  const CacheView& c = a.c;
  const int tid = threadIdx.x, d = tid % CH * 16;
  float top = KEYS ? 0.0f : static_cast<float>(kMinVExp);  // scale, or exponent
#pragma unroll
  for (int i = 0; i < PER; i++) {
    // largest |code| or |value| of the token, in fp16 (exact): of the
    // thread's 16 channels, then of its CH lanes
    const uint32_t q[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    __half2 m2 = __half2half2(__ushort_as_half(0));
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t p0, p1;
      if (KEYS)
        i8x4_to_f16(q[j], p0, p1);
      else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(p0), "=r"(p1) : "r"(q[j]));
      m2 = __hmax2(m2, __hmax2(__habs2(*reinterpret_cast<const __half2*>(&p0)), __habs2(*reinterpret_cast<const __half2*>(&p1))));
    }
#pragma unroll
    for (int o = CH / 2; o; o >>= 1) m2 = __hmax2(m2, __shfl_xor_sync(kFull, m2, o));
    const float big = fmaxf(__low2float(m2), __high2float(m2));
    if (there[i]) {
      if (KEYS)
        top = fmaxf(top, __fmul_rn(s_src[i], __fdiv_rn(fminf(big, 127.0f), 127.0f)));  // -128 is never written
      else if (big > 0.0f)  // |value| = code * 2^e: its exponent is the code's, shifted
        top = fmaxf(top, static_cast<float>(value_exp(big) + e_src[i]));
    }
  }
  top = block_max(top, red);
  const int ve = static_cast<int>(top);

  uint8_t* dst;
  if (a.pages_out) {
    const size_t unit = static_cast<size_t>(po) * c.Hkv + h;
    dst = (KEYS ? reinterpret_cast<uint8_t*>(c.k_i8) : c.v_f8) + unit * (kPage * D);
    if (KEYS) {
      if (tid == 0) c.k_scale[unit] = top;
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (d == 0) c.weight[unit * kPage + tid / CH + i * (kThreads / CH)] = w[i];
    } else if (tid == 0) {
      c.v_exp[unit] = static_cast<int8_t>(ve);
    }
  } else {
    const Stage st = stage_of(a.ws, units, D);
    dst = (KEYS ? reinterpret_cast<uint8_t*>(st.k) : st.v) + ou * (kPage * D);
    if (KEYS) {
      if (tid == 0) st.scale[ou] = top;
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (d == 0) st.weight[ou * kPage + tid / CH + i * (kThreads / CH)] = w[i];
    } else if (tid == 0) {
      st.exp[ou] = static_cast<int8_t>(ve);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int r = tid / CH + i * (kThreads / CH);
    uint32_t q[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    if constexpr (KEYS) {
      if (s_src[i] != top) {
        // round-half-even(code * ratio) in the low byte of the sum with 1.5 *
        // 2^23 (one rounding); next to a tie of any of the 16 fp64 decides.
        // |code| * s_src <= 127 top for every survivor, so nothing clamps;
        // a scale near the subnormal numbers is rounded by more than that
        // allows for, and the slow way does clamp.
        const float s = s_src[i], ratio = top > 0.0f ? s / top : 0.0f;
        float worst = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint32_t p0, p1;
          i8x4_to_f16(q[j], p0, p1);
          const float2 a2 = __half22float2(*reinterpret_cast<const __half2*>(&p0));
          const float2 b2 = __half22float2(*reinterpret_cast<const __half2*>(&p1));
          const float f[4] = {a2.x, a2.y, b2.x, b2.y};
          float y[4], rem[4];
#pragma unroll
          for (int e = 0; e < 4; e++) {
            y[e] = fmaf(f[e], ratio, kRound);
            rem[e] = fabsf(fmaf(f[e], ratio, __fsub_rn(kRound, y[e])));
          }
          worst = fmax3(worst, fmax3(rem[0], rem[1], rem[2]), rem[3]);
          q[j] = low_bytes(y[0], y[1], y[2], y[3]);
        }
        if (worst > 0.5f - kNearTieScaled || !(top >= kTinyScale)) {
          q[0] = rescale_keys(x[i].x, s, top);
          q[1] = rescale_keys(x[i].y, s, top);
          q[2] = rescale_keys(x[i].z, s, top);
          q[3] = rescale_keys(x[i].w, s, top);
        }
      }
    } else {
      const int diff = e_src[i] - ve;
      if (diff != 0 && there[i]) {
        // e4m3 values times 2^diff: exact in fp16 for |diff| <= 15 (diff > 0
        // happens where a page's largest tokens went; the new exponent covers
        // every survivor), so only the step back to e4m3 rounds
        if (diff >= -15 && diff <= 15) {
          const __half2 f = __half2half2(__float2half_rn(pow2i(diff)));
#pragma unroll
          for (int j = 0; j < 4; j++) q[j] = scale_values(q[j], f);
        } else {
#pragma unroll
          for (int j = 0; j < 4; j++) q[j] = rescale_values(q[j], diff);
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + r * D + d) = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// Block (64 survivors, head, batch).  A block is mostly the latency of its
// dependent loads, so there are two steps of them: the places of the thread's
// tokens (which the selection left with their page already looked up), the
// result's page and the lengths; then keys, values, scales and weights.
// Measured: 4096 of 16000 tokens of 8 x 8 heads 36 us, 134 MB at 3.7 TB/s (the
// survivors are runs of 128 bytes).  Persistent blocks with the next unit's
// codes on their way by cp.async took 8 us more, packed fp32 arithmetic
// changed nothing.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) k_gather(const EvictArgs a) {
  __shared__ float red[kThreads / 32];
  constexpr int CH = D / 16, PER = kPage * CH / kThreads;
  const CacheView& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, blk = blockIdx.x, blocks = gridDim.x;
  const int tid = threadIdx.x, d = tid % CH * 16;
  const int n = __ldg(a.lengths_out + b), len = a.pages_out ? 0 : seq_length(c, b);
  const size_t list = (static_cast<size_t>(b) * c.Hkv + h) * a.keep + blk * kPage;
  int t[PER], unit[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int r = tid / CH + i * (kThreads / CH);
    t[i] = unit[i] = -1;
    if (blk * kPage + r < a.keep) {
      t[i] = a.kept[list + r];
      unit[i] = a.from[list + r];
    }
  }
  const int po = a.pages_out ? page_id(c, a.pages_out, a.out_pages, b, blk, n > blk * kPage) : 0;
  if (n <= blk * kPage || po < 0 || (!a.pages_out && n == len)) return;
  uint4 k[PER], v[PER];
  float s_src[PER], w[PER];
  int e_src[PER];
  bool there[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
    s_src[i] = w[i] = 0.0f;
    e_src[i] = 0;
    there[i] = unit[i] >= 0;
    if (there[i]) {
      const size_t at = static_cast<size_t>(unit[i]) * kPage + t[i] % kPage;
      k[i] = *reinterpret_cast<const uint4*>(c.k_i8 + at * D + d);
      v[i] = *reinterpret_cast<const uint4*>(c.v_f8 + at * D + d);
      s_src[i] = c.k_scale[unit[i]];
      e_src[i] = c.v_exp[unit[i]];
      if (d == 0) w[i] = c.weight[at];
    }
  }
  const size_t units = static_cast<size_t>(blocks) * c.Hkv * c.B;
  const size_t ou = (static_cast<size_t>(b) * c.Hkv + h) * blocks + blk;
  requantize<D, true>(a, h, po, units, ou, k, s_src, e_src, w, there, red);
  requantize<D, false>(a, h, po, units, ou, v, s_src, e_src, w, there, red);
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
  const dim3 grid(2 * ((a.n + kPage - 2) / kPage + 1), a.c.Hkv, a.c.B);
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

// The survivors' (page, head), then, in place, the staged blocks.
size_t cache_evict_list_bytes(int B, int Hkv, int keep) {
  return (static_cast<size_t>(B) * Hkv * keep * 4 + 15) / 16 * 16;
}
size_t cache_evict_ws_bytes(int B, int Hkv, int D, int keep, bool in_place) {
  const size_t units = static_cast<size_t>(B) * Hkv * ((keep + kPage - 1) / kPage);
  return cache_evict_list_bytes(B, Hkv, keep) +
         (in_place ? (units * (2ull * kPage * D + kPage * 4 + 4 + 1) + 15) / 16 * 16 : 0);
}

cudaError_t cache_evict_prepare() {
  return cudaFuncSetAttribute(k_select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (3 * kSelBins + kSelKeys + kSelKeys / kPage) * 4);
}

cudaError_t launch_cache_evict(const EvictArgs& args, cudaStream_t s) {
  EvictArgs a = args;
  // shared memory for a block's share of as many weights as the page table holds
  const long long share = (static_cast<long long>(a.c.max_pages) + kSelCluster - 1) / kSelCluster * kPage;
  a.sel_keys = static_cast<int>(share < kSelKeys ? share : kSelKeys);
  a.from = static_cast<int*>(args.ws);
  a.ws = static_cast<char*>(args.ws) + cache_evict_list_bytes(a.c.B, a.c.Hkv, a.keep);
  k_select<<<a.c.B * a.c.Hkv * kSelCluster, kSelThreads, (3 * kSelBins + a.sel_keys + a.sel_keys / kPage) * 4, s>>>(a);
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
