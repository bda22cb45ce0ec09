// cache.cuh -- the paged 8-bit key/value cache: parameters, launch interface
// and the small device helpers its kernels share.
//
// Layout.  A page holds 64 tokens of every key/value head:
//   k_i8    int8 [pages][heads][64][D]   key codes, k = code * k_scale
//   k_scale f32  [pages][heads]          absmax / 127 of the page's keys
//   v_f8    e4m3 [pages][heads][64][D]   value codes, v = code * 2^v_exp
//   v_exp   int8 [pages][heads]          smallest e with absmax <= 448 * 2^e
// The codes of one page and head are contiguous (64 * D bytes), so a page is
// one TMA box.  The value scale is a power of two: an e4m3 code loses nothing
// by it (its relative step does not depend on the scale), a page that grows
// rescales its codes without a second rounding of normal ones, and the
// attention kernel folds it into the exponent of the softmax.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sage {

constexpr int kPage = 64;         // tokens per page
constexpr int kMinVExp = -40;     // floor of v_exp (also that of an all-zero page)
constexpr int kMaxShares = 320;  // blocks that share a decode call's pages, at most

enum { kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2 };

struct CacheView {
  int8_t* k_i8;
  float* k_scale;
  uint8_t* v_f8;
  int8_t* v_exp;
  float* weight;       // f32 [pages][heads][64], or null
  int n_pages, Hkv, D;
  const int* pages;    // [B][max_pages]
  const int* lengths;  // [B]
  int B, max_pages;
  int* status;         // device status word pair
};

// Tokens of sequence b that the page table can hold; a length outside
// [0, max_pages * 64] is recorded as an invalid argument and clamped.
__device__ __forceinline__ int clamp_length(int len, const CacheView& c) {
  const int cap = c.max_pages * kPage;
  if (len < 0 || len > cap) {
    if (atomicCAS(c.status, 0, 1 /* SAGE_ERR_INVALID_ARG */) == 0) atomicExch(c.status + 1, 0x20001);
    return len < 0 ? 0 : cap;
  }
  return len;
}
__device__ __forceinline__ int seq_length(const CacheView& c, int b) {
  return clamp_length(__ldg(c.lengths + b), c);
}

// Page id of block blk of sequence b in a table of `width` columns, or -1
// (recorded, if `record`) if it is no page.
__device__ __forceinline__ int page_id(const CacheView& c, const int* table, int width, int b, int blk,
                                       bool record = true) {
  const int pg = __ldg(table + static_cast<size_t>(b) * width + blk);
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(c.n_pages)) {
    if (record && atomicCAS(c.status, 0, 1 /* SAGE_ERR_INVALID_ARG */) == 0) atomicExch(c.status + 1, 0x20002);
    return -1;
  }
  return pg;
}
__device__ __forceinline__ int page_id(const CacheView& c, int b, int blk) {
  return page_id(c, c.pages, c.max_pages, b, blk);
}

// ---------------------------------------------------------------- masks

struct CacheMask {
  int mode;   // 0 none, 1 causal, 2 block-causal, 3 sliding window
  int block;  // block-causal block / window frame, tokens
  int win;    // frames per window
  int sink;   // reference context, tokens
};

// The keys that the query token at position g of `len` cached tokens sees:
// [0, sink) and [lo, hi).  g < 0 (more query tokens than cached ones) sees
// nothing under any mask but `none`.
struct KeyRange {
  int sink, lo, hi;
};
__device__ __forceinline__ KeyRange key_range(const CacheMask& m, long long g, int len) {
  KeyRange r{0, 0, len};
  if (m.mode == 0) return r;
  if (g < 0) {
    r.hi = 0;
    return r;
  }
  long long lo = 0, hi = g + 1;
  if (m.mode == 2) {
    hi = (g / m.block + 1) * m.block;
  } else if (m.mode == 3) {
    r.sink = min(m.sink, len);
    if (g < m.sink) {
      lo = hi = r.sink;
    } else {
      const long long f = (g - m.sink) / m.block;
      lo = m.sink + max(f - m.win + 1, 0ll) * m.block;
      hi = m.sink + (f + 1) * m.block;
    }
  }
  r.lo = static_cast<int>(min(lo, static_cast<long long>(len)));
  r.hi = static_cast<int>(min(hi, static_cast<long long>(len)));
  return r;
}

// The pages that the tokens [i0, i1] of a tile see together: [0, ns) and
// [ns + gap, ns + gap + rest).  key_range's lo and hi never decrease with g,
// and hi(g) >= lo(g + 1), so the two runs hold every visible key.
struct PageRuns {
  int n, ns, gap;
  __device__ __forceinline__ int page(int i) const { return i < ns ? i : i + gap; }
};
__device__ __forceinline__ PageRuns page_runs(const CacheMask& m, long long g0, long long g1,
                                              int len) {
  const KeyRange a = key_range(m, g0, len), b = key_range(m, g1, len);
  PageRuns r;
  const int end = (max(b.hi, b.sink) + kPage - 1) / kPage;
  r.ns = end;
  r.gap = 0;
  const int s = (max(a.sink, b.sink) + kPage - 1) / kPage;
  const int lo = a.lo / kPage;
  if (m.mode == 3 && lo > s) {
    r.ns = min(s, end);
    r.gap = min(lo, end) - r.ns;
  }
  r.n = end - r.gap;
  return r;
}

// 2^e as fp32, -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The smallest e with a <= 448 * 2^e (448 = 1.75 * 2^8), at least kMinVExp.
__device__ __forceinline__ int value_exp(float a) {
  const uint32_t u = __float_as_uint(a);
  if (u < 0x00800000u) return kMinVExp;  // zero and subnormals
  const int x = static_cast<int>(u >> 23) - 127;
  const int e = x - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return max(e, kMinVExp);
}

// ---------------------------------------------------------------- launches

struct RopeArgs {
  const void* x;
  void* y;
  int type, B, H, N, D, R;
  long long xb, xh, xn, yb, yh, yn;  // strides, elements
  const long long* pos64;            // one of the two: positions
  const int* pos32;
  long long pb;                      // position stride of the batch (0: shared)
  const double* inv_freq;            // [R / 2]
  float amplitude;
  int half, inverse;
  int sms;                           // of the device
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_tables(const RopeArgs& a, float* cosv, float* sinv, cudaStream_t s);

struct AppendArgs {
  CacheView c;  // lengths: tokens before the call
  const void *k, *v;
  int type, n;
  long long kb, kh, kn, vb, vh, vn;
  const int* n_new;      // [B] or null
  const float* k_shift;  // [Hkv][D] or null
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s);

struct ReadArgs {
  CacheView c;
  const int* starts;  // [B] or null
  int n;
  const float* k_shift;
  float *k, *v, *w;   // f32 [B][Hkv][n][D], [B][Hkv][n]; w may be null
};
cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t s);

struct EvictArgs {
  CacheView c;
  int keep, sink, recent;
  int* kept;         // [B][Hkv][keep]
  int* lengths_out;  // [B]
  const int* pages_out;  // [B][out_pages], or null: in place through the workspace
  int out_pages;
  int sel_keys;  // weights that k_select keeps in shared memory
  int* from;     // [B][Hkv][keep]: the survivors' (page, head)
  void* ws;
};
cudaError_t cache_evict_prepare();
size_t cache_evict_ws_bytes(int B, int Hkv, int D, int keep, bool in_place);
cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s);

struct CacheAttnMaps {
  CUtensorMap k, v;  // uint8 [pages * heads][64][D], box D x 32
};
struct CacheAttnArgs {
  CacheView c;
  const void* q;
  void* o;
  int type, H, G, Nq;
  int q_vec;         // query rows are 16-byte aligned
  long long qb, qh, qn, ob, oh, on;  // strides, elements
  const int* q_lens;                 // [B] or null
  CacheMask mask;
  float scale;       // softmax scale, natural units
  float* lse;        // f32 [B][H][Nq] or null
  const float* lse_in;
  int accumulate;    // cache_weights: add to the weights, or overwrite them
  // how the keys are cut: `chunks` ranges of `chunk_pages` pages of each query
  // tile; for at most 16 rows `chunks` blocks with equal shares of all pages,
  // or (`whole`) a block for every head
  int chunk_pages, chunks, whole;
  float *part_o, *part_ml;
  long long budget;
};
cudaError_t cache_prepare();
// rows of a query tile of the two attention kernels (the first: at most; one
// of eight rows where they suffice)
constexpr int kDecRows = 16, kPreRows = 256;
inline int decode_tile_rows(long long Nq, int G) { return Nq * G <= 8 ? 8 : kDecRows; }
cudaError_t cache_prefill_prepare();
cudaError_t launch_cache_prefill(const CacheAttnArgs& a, cudaStream_t s);
cudaError_t launch_cache_decode(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s);
cudaError_t cache_weights_prepare();
cudaError_t launch_cache_weights_few(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s);
cudaError_t launch_cache_weights(const CacheAttnArgs& a, cudaStream_t s);

}  // namespace sage
