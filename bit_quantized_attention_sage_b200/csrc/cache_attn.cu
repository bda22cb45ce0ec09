// cache_attn.cu -- attention over the paged 8-bit cache for few query rows
// (single tokens, grouped heads), the merge of KV ranges, and, in the same
// stream of keys, the attention weight that each cached key received.
//
// The query heads that share a key head are rows of one tile: row r of
// (sequence b, key head h) is token r / G, head h G + r % G.
//
// Scores.  Q goes to fp16 with a power of two per row (its largest element
// lands in [2^14, 2^15)): exact for bf16 and fp16 inputs down to 2^-31 of the
// row's maximum.  int8 key codes are exact in fp16, so the products are exact
// and only the fp32 accumulation rounds; the page's key scale, the row's
// power and log2(e) * softmax scale multiply the sum.
// Probabilities.  y = 2^(t + e - M + 7), t the score in log2 units, e the
// page's value exponent, M a reference maximum of t + e that follows the
// running one in steps of at least 2^8: y <= 2^15, and fp16(y) is off by at
// most 2^-11 of each weight down to 2^-21 of the largest term, where fp16's
// subnormal range begins.  The sum L takes y 2^-e in fp32 before that
// rounding.  e4m3 value codes are exact in fp16.  O = (sum y code) / L; the
// value scales need no multiplication.
//
// What bounds it: the codes, read once (2 D bytes a key and head).  Every
// warp walks half pages of its own (32 keys) through a private ring of three
// TMA loads (24 KB in flight a warp at D = 128, 192 KB an SM with two blocks),
// so no barrier joins the warps until the end.  Page ids, key scales and
// value exponents of a warp's next 32 half pages are fetched at once, one a
// lane; taken one by one inside the loop, their three dependent loads cost
// more than the tile.  16-row tiles on mma.sync (a sixteenth used for one
// row) keep the issue slots at about a third of the load time; a 128-row
// tcgen05 tile would need its codes converted through shared memory first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kHalf = 32;      // keys a tile
constexpr float kBoost = 7.0f;  // y = 2^7 at the reference maximum
constexpr float kLazy = 8.0f;   // growth of the maximum that moves the reference
constexpr float kLn2 = 0.69314718055994531f;

enum : int { kSiteDecPage = 0x20101, kSiteDecDrain };

// ---------------------------------------------------------------- tile access

// Byte offset of 16-byte chunk `ch` of row `r` in a TMA-swizzled tile of
// D-byte rows (128-byte swizzle for D = 128, 64-byte for D = 64).
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// D (fp32 16x8) += A (fp16 16x16) B (fp16 16x8)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 codes to two fp16 pairs, (bytes 0, 2) and (bytes 1, 3).
__device__ __forceinline__ void f8x4_to_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t p = __byte_perm(w, 0, 0x3120);
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(even), "=r"(odd) : "r"(p));
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w, int site) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > w.budget) {
      record_timeout(w.status, site);
      return;
    }
  }
}

// ---------------------------------------------------------------- decode

// A tile of the ring: half a page.
struct TileMeta {
  float ks;  // key scale
  int ve;    // value exponent
  int j0;    // first key, or -1: no page
  int unit;  // (page, head)
};

template <int D>
struct alignas(1024) DecSmem {
  uint8_t kv[kWarps][kStages][2][kHalf * D];  // TMA tiles: K, V
  __half q[kDecRows][D + 16];                 // padded: 8-byte reads of 4 rows on different banks
  float rowf[kDecRows];                       // 2^e * scale * log2(e) of each row
  float ml[kWarps][kDecRows][2];
  TileMeta meta[kWarps][kStages];
  uint64_t full[kWarps][kStages];
  int abort;
};

struct TileId {
  int b, h, rt, chunk;
};
__device__ __forceinline__ TileId tile_id(const CacheAttnArgs& a, int row_tiles) {
  // row tiles fastest (they read the same pages), then KV ranges
  unsigned i = blockIdx.x;
  TileId t;
  t.rt = i % row_tiles;
  i /= row_tiles;
  t.chunk = i % a.chunks;
  i /= a.chunks;
  t.h = i % a.c.Hkv;
  t.b = i / a.c.Hkv;
  return t;
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

// WEIGHTS: instead of attending, w[key] (+)= sum over the tile's rows of
// exp(s - lse), with the rows' lse given (at most 16 rows: one tile).
template <int D, bool WEIGHTS>
__global__ void __launch_bounds__(kWarps * 32, 2)
    k_cache_decode(const __grid_constant__ CacheAttnMaps maps, const CacheAttnArgs a, int row_tiles) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  DecSmem<D>& s = *reinterpret_cast<DecSmem<D>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const TileId id = tile_id(a, row_tiles);
  const int len = seq_length(a.c, id.b), qn = query_len(a, id.b);
  const int rows = qn * a.G, r0 = id.rt * kDecRows;
  if (r0 >= rows && !WEIGHTS) return;
  const int r1 = min(rows, r0 + kDecRows);
  const long long off = static_cast<long long>(len) - qn;  // position of token 0
  PageRuns runs;
  if constexpr (WEIGHTS) {  // every page: those that no row sees get 0
    runs.n = runs.ns = (len + kPage - 1) / kPage;
    runs.gap = 0;
  } else {
    runs = page_runs(a.mask, off + r0 / a.G, off + (r1 - 1) / a.G, len);
  }
  // the last range takes whatever a sequence longer than announced adds
  const int p0 = id.chunk * a.chunk_pages;
  const int p1 = id.chunk == a.chunks - 1 ? runs.n : min(runs.n, p0 + a.chunk_pages);
  // range 0 also serves an empty sequence
  if (p0 >= runs.n && (WEIGHTS || id.chunk > 0)) return;

  if (lane == 0) {
    for (int i = 0; i < kStages; i++) mbar_init(&s.full[warp][i], 1);
    if (warp == 0) s.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtx wc{a.budget, a.c.status, &s.abort};
  // this warp's half pages: warp, warp + kWarps, ... of the range's
  const int halves = max(0, 2 * (p1 - p0));
  const int mine = warp < halves ? (halves - warp + kWarps - 1) / kWarps : 0;
  TileMeta next{0.0f, 0, -1, 0};  // lane's tile of the current 32
  int issued = 0;
  auto issue = [&]() {  // the whole warp: the load of tile `issued`
    if ((issued & 31) == 0) {
      const int q = warp + (issued + lane) * kWarps;
      next = TileMeta{0.0f, 0, -1, 0};
      if (q < halves) {
        const int blk = runs.page(p0 + q / 2);
        const int pg = page_id(a.c, id.b, blk);
        if (pg >= 0) {
          next.unit = pg * a.c.Hkv + id.h;
          next.j0 = blk * kPage + (q & 1) * kHalf;
          next.ks = __ldg(a.c.k_scale + next.unit);
          if (!WEIGHTS) next.ve = __ldg(a.c.v_exp + next.unit);
        }
      }
    }
    if (lane == (issued & 31)) {
      const int st = issued % kStages;
      uint64_t* bar = &s.full[warp][st];
      if (next.j0 >= len) next.j0 = -1;  // the half behind the end
      s.meta[warp][st] = next;
      if (next.j0 < 0) {
        mbar_arrive(bar);  // nothing to load
      } else {
        mbar_arrive_expect_tx(bar, (WEIGHTS ? 1 : 2) * kHalf * D);
        const int y = next.j0 & (kPage - 1);
        tma_load_3d(s.kv[warp][st][0], &maps.k, bar, 0, y, next.unit);
        if (!WEIGHTS) tma_load_3d(s.kv[warp][st][1], &maps.v, bar, 0, y, next.unit);
      }
    }
    issued++;
  };
  while (issued < min(mine, kStages)) issue();
  for (int r = warp; r < kDecRows; r += kWarps) {
    const float f = stage_row<D>(a, id.b, id.h, r0 + r, r1, s.q[r], lane);
    if (lane == 0) s.rowf[r] = f * (a.scale * kLog2e);
  }
  __syncthreads();
  // A fragments of Q: k slots 2t, 2t + 1, 2t + 8, 2t + 9 of step kk are
  // channels 16 kk + 4 t .. + 3, the order in which ldmatrix hands out the
  // key codes' bytes
  uint32_t qa[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; kk++) {
    const uint2 x = *reinterpret_cast<const uint2*>(&s.q[g][kk * 16 + t * 4]);
    const uint2 y = *reinterpret_cast<const uint2*>(&s.q[g + 8][kk * 16 + t * 4]);
    qa[kk][0] = x.x;
    qa[kk][2] = x.y;
    qa[kk][1] = y.x;
    qa[kk][3] = y.y;
  }
  const float f0 = s.rowf[g], f1 = s.rowf[g + 8];
  KeyRange kr[2];
  float nl[2] = {-INFINITY, -INFINITY};  // WEIGHTS: -lse log2(e); -inf: weight 0
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int r = r0 + g + 8 * i;
    kr[i] = KeyRange{0, 0, 0};
    if (r < r1) {
      kr[i] = key_range(a.mask, off + r / a.G, len);
      if (WEIGHTS) {
        const float v = __ldg(a.lse_in + (static_cast<size_t>(id.b) * a.H + id.h * a.G + r % a.G) * a.Nq + r / a.G);
        if (v != -INFINITY) nl[i] = -v * kLog2e;
      }
    }
  }
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; i++)
#pragma unroll
    for (int e = 0; e < 4; e++) o[i][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

  bool ok = true;
  for (int i = 0; i < mine; i++) {
    const int st = i % kStages;
    ok = __all_sync(kFull, mbar_wait(&s.full[warp][st], (i / kStages) & 1, wc, kSiteDecPage));
    if (!ok) break;
    const TileMeta md = s.meta[warp][st];
    const int j0 = md.j0;
    if (j0 >= 0) {
      const uint32_t kb = smem_u32(s.kv[warp][st][0]), vb = smem_u32(s.kv[warp][st][1]);
      if (!WEIGHTS && j0 + kHalf > len) {
        // the sequence ends inside this tile: values behind it may be any
        // bytes (NaN among them), and zero weight times NaN is NaN.  The last
        // tile that this warp loads, so no later TMA load meets these writes.
        for (int x = lane; x < kHalf * D / 16; x += 32) {
          const int r = x / (D / 16);
          if (j0 + r >= len)
            *reinterpret_cast<uint4*>(s.kv[warp][st][1] + swz<D>(r, x % (D / 16))) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // scores: 4 tiles of 8 keys
      float sc[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; nt++) {
#pragma unroll
        for (int e = 0; e < 4; e++) sc[nt][e] = 0.0f;
#pragma unroll
        for (int c4 = 0; c4 < D / 64; c4++) {
          uint32_t kr4[4];
          ldsm4(kb + swz<D>(nt * 8 + (lane & 7), c4 * 4 + (lane >> 3)), kr4);
#pragma unroll
          for (int c = 0; c < 4; c++) {
            uint32_t b0, b1;
            i8x4_to_f16(kr4[c], b0, b1);
            mma16816(sc[nt], qa[c4 * 4 + c], b0, b1);
          }
        }
      }
      // a zero scale must not meet -inf as 0 * inf
      const float c0 = fmaxf(f0 * md.ks, FLT_MIN), c1 = fmaxf(f1 * md.ks, FLT_MIN);
      bool all = true;
#pragma unroll
      for (int i2 = 0; i2 < 2; i2++)
        all = all && (kr[i2].sink >= j0 + kHalf || (kr[i2].lo <= j0 && kr[i2].hi >= j0 + kHalf));
      if (!__all_sync(kFull, all)) {
#pragma unroll
        for (int nt = 0; nt < 4; nt++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const KeyRange& k = kr[e >> 1];
            const int j = j0 + nt * 8 + t * 2 + (e & 1);
            if (!(j < k.sink || (j >= k.lo && j < k.hi))) sc[nt][e] = -INFINITY;
          }
      }
      if constexpr (WEIGHTS) {
#pragma unroll
        for (int nt = 0; nt < 4; nt++) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            w[e] = ex2_approx(fmaf(sc[nt][e], c0, nl[0])) + ex2_approx(fmaf(sc[nt][2 + e], c1, nl[1]));
            w[e] += __shfl_xor_sync(kFull, w[e], 4);
            w[e] += __shfl_xor_sync(kFull, w[e], 8);
            w[e] += __shfl_xor_sync(kFull, w[e], 16);
          }
          if (g == (nt & 7)) {
            float* dst = a.c.weight + static_cast<size_t>(md.unit) * kPage + (j0 & (kPage - 1)) + nt * 8 + t * 2;
#pragma unroll
            for (int e = 0; e < 2; e++) {
              if (j0 + nt * 8 + t * 2 + e < len) {
                if (a.accumulate) atomicAdd(dst + e, w[e]);  // a page may serve two sequences
                else dst[e] = w[e];
              }
            }
          }
        }
      } else {
        const float ve = static_cast<float>(md.ve);
        float pm[2];
        pm[0] = fmax3(fmax3(sc[0][0], sc[0][1], sc[1][0]), fmax3(sc[1][1], sc[2][0], sc[2][1]),
                      fmaxf(sc[3][0], sc[3][1]));
        pm[1] = fmax3(fmax3(sc[0][2], sc[0][3], sc[1][2]), fmax3(sc[1][3], sc[2][2], sc[2][3]),
                      fmaxf(sc[3][2], sc[3][3]));
        bool grow = false;
#pragma unroll
        for (int i2 = 0; i2 < 2; i2++) {
          pm[i2] = fmaxf(pm[i2], __shfl_xor_sync(kFull, pm[i2], 1));
          pm[i2] = fmaxf(pm[i2], __shfl_xor_sync(kFull, pm[i2], 2));
          pm[i2] = fmaf(pm[i2], i2 ? c1 : c0, ve);
          grow = grow || pm[i2] > m[i2] + kLazy;
        }
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int i2 = 0; i2 < 2; i2++) {
            const float mn = fmaxf(m[i2], pm[i2]);
            const float al = m[i2] == mn ? 1.0f : ex2_approx(m[i2] - mn);  // 0 from -inf
            m[i2] = mn;
            l[i2] *= al;
#pragma unroll
            for (int d = 0; d < D / 8; d++) {
              o[d][2 * i2] *= al;
              o[d][2 * i2 + 1] *= al;
            }
          }
        }
        const float nm0 = m[0] == -INFINITY ? 0.0f : kBoost + ve - m[0];
        const float nm1 = m[1] == -INFINITY ? 0.0f : kBoost + ve - m[1];
        float rs[2] = {0.0f, 0.0f};
        uint32_t pa[2][4];
#pragma unroll
        for (int nt = 0; nt < 4; nt++) {
          const float y0 = ex2_approx(fmaf(sc[nt][0], c0, nm0)), y1 = ex2_approx(fmaf(sc[nt][1], c0, nm0));
          const float y2 = ex2_approx(fmaf(sc[nt][2], c1, nm1)), y3 = ex2_approx(fmaf(sc[nt][3], c1, nm1));
          rs[0] += y0 + y1;
          rs[1] += y2 + y3;
          const __half2 h0 = __floats2half2_rn(y0, y1), h1 = __floats2half2_rn(y2, y3);
          pa[nt / 2][(nt & 1) * 2] = *reinterpret_cast<const uint32_t*>(&h0);
          pa[nt / 2][(nt & 1) * 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
        }
        const float un = pow2i(min(-md.ve, 127));
        l[0] = fmaf(rs[0], un, l[0]);
        l[1] = fmaf(rs[1], un, l[1]);
        // O += P V: per 32 channels, 16 keys at a time
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
#pragma unroll
          for (int d2 = 0; d2 < D / 32; d2++) {
            uint32_t vr[4];  // keys 0-7 / 8-15 of two 16-channel chunks
            ldsm4t(vb + swz<D>(kk * 16 + (lane & 15), d2 * 2 + (lane >> 4)), vr);
#pragma unroll
            for (int c = 0; c < 2; c++) {
              uint32_t e0, o0, e1, o1;
              f8x4_to_f16(vr[2 * c], e0, o0);
              f8x4_to_f16(vr[2 * c + 1], e1, o1);
              mma16816(o[(d2 * 2 + c) * 2], pa[kk], e0, e1);
              mma16816(o[(d2 * 2 + c) * 2 + 1], pa[kk], o0, o1);
            }
          }
        }
      }
    }
    __syncwarp();
    if (issued < mine) issue();
  }
  if (!ok) {  // a wait ran out (recorded): let the loads in flight land, then leave
    if (lane == 0)
      for (int i = max(0, issued - kStages); i < issued; i++)
        drain_wait(&s.full[warp][i % kStages], (i / kStages) & 1, wc, kSiteDecDrain);
    __syncwarp();
  }
  if constexpr (WEIGHTS) return;
  // row sums over the four lanes of a row
#pragma unroll
  for (int i = 0; i < 2; i++) {
    l[i] += __shfl_xor_sync(kFull, l[i], 1);
    l[i] += __shfl_xor_sync(kFull, l[i], 2);
  }
  // join the warps: every tile has landed and been read, so the ring holds
  // the partial rows, fp32 [16][D] a warp
  __syncthreads();
  if (s.abort) return;
  float* part = reinterpret_cast<float*>(s.kv[warp][0][0]);
  static_assert(kStages * 2 * kHalf * D >= kDecRows * D * 4, "a warp's ring holds its partial rows");
#pragma unroll
  for (int d = 0; d < D / 16; d++) {
    // tiles 2 d and 2 d + 1 hold channels 16 d + 4 t + {0, 2} and + {1, 3}
    *reinterpret_cast<float4*>(part + g * D + d * 16 + t * 4) =
        make_float4(o[2 * d][0], o[2 * d + 1][0], o[2 * d][1], o[2 * d + 1][1]);
    *reinterpret_cast<float4*>(part + (g + 8) * D + d * 16 + t * 4) =
        make_float4(o[2 * d][2], o[2 * d + 1][2], o[2 * d][3], o[2 * d + 1][3]);
  }
  if (t == 0) {
    s.ml[warp][g][0] = m[0];
    s.ml[warp][g][1] = l[0];
    s.ml[warp][g + 8][0] = m[1];
    s.ml[warp][g + 8][1] = l[1];
  }
  __syncthreads();
  const int nch = min(a.chunks, (runs.n + a.chunk_pages - 1) / a.chunk_pages);
  constexpr size_t kWarpFloats = kStages * 2 * kHalf * D / 4;
  for (int x = threadIdx.x; x < kDecRows * D / 2; x += kWarps * 32) {
    const int r = x / (D / 2), d = x % (D / 2) * 2;
    if (r0 + r >= r1) break;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; w++) mx = fmaxf(mx, s.ml[w][r][0]);
    float ox = 0.0f, oy = 0.0f, ls = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      const float mw = s.ml[w][r][0];
      const float al = mw == -INFINITY ? 0.0f : ex2_approx(mw - mx);
      const float2 v = *reinterpret_cast<const float2*>(
          reinterpret_cast<const float*>(s.kv[0][0][0]) + w * kWarpFloats + r * D + d);
      ox = fmaf(al, v.x, ox);
      oy = fmaf(al, v.y, oy);
      ls = fmaf(al, s.ml[w][r][1], ls);
    }
    const size_t urow = (static_cast<size_t>(id.b) * a.c.Hkv + id.h) * (static_cast<size_t>(row_tiles) * kDecRows) + r0 + r;
    if (nch > 1) {
      const size_t pr = urow * a.chunks + id.chunk;
      *reinterpret_cast<float2*>(a.part_o + pr * D + d) = make_float2(ox, oy);
      if (d == 0) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(mx - kBoost, ls);
    } else {
      const float inv = ls > 0.0f ? 1.0f / ls : 0.0f;
      const int rr = r0 + r, tok = rr / a.G, head = id.h * a.G + rr % a.G;
      store_o2(a, a.ob * id.b + a.oh * head + a.on * tok + d, ox * inv, oy * inv);
      if (d == 0 && a.lse)
        a.lse[(static_cast<size_t>(id.b) * a.H + head) * a.Nq + tok] =
            ls > 0.0f ? (mx - kBoost + log2f(ls)) * kLn2 : -INFINITY;
    }
  }
}

// Join of the KV ranges: one warp per row, in range order.
template <int D>
__global__ void __launch_bounds__(128) k_cache_merge(const CacheAttnArgs a, int row_tiles, int tile_rows) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const long long per = static_cast<long long>(row_tiles) * tile_rows;
  const long long bh = row / per;
  if (bh >= static_cast<long long>(a.c.B) * a.c.Hkv) return;
  const int r = static_cast<int>(row - bh * per), b = static_cast<int>(bh / a.c.Hkv),
            h = static_cast<int>(bh % a.c.Hkv);
  const int len = seq_length(a.c, b), qn = query_len(a, b), rows = qn * a.G;
  if (r >= rows) return;
  const int r0 = r / tile_rows * tile_rows, r1 = min(rows, r0 + tile_rows);
  const long long off = static_cast<long long>(len) - qn;
  const PageRuns runs = page_runs(a.mask, off + r0 / a.G, off + (r1 - 1) / a.G, len);
  const int nch = min(a.chunks, (runs.n + a.chunk_pages - 1) / a.chunk_pages);
  if (nch <= 1) return;  // the attention kernel wrote this tile itself
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.chunks;
  float mx = -INFINITY;
  for (int i = lane; i < nch; i += 32) mx = fmaxf(mx, ml[i].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  constexpr int PER = D / 32;
  float o[PER], ls = 0.0f;
#pragma unroll
  for (int e = 0; e < PER; e++) o[e] = 0.0f;
  const float* po = a.part_o + row * a.chunks * D + lane * PER;
#pragma unroll 4
  for (int i = 0; i < nch; i++) {
    const float2 x = ml[i];
    const float al = x.x == -INFINITY ? 0.0f : ex2_approx(x.x - mx);
    ls = fmaf(al, x.y, ls);
#pragma unroll
    for (int e = 0; e < PER; e++) o[e] = fmaf(al, po[static_cast<size_t>(i) * D + e], o[e]);
  }
  const float inv = ls > 0.0f ? 1.0f / ls : 0.0f;
  const int tok = r / a.G, head = h * a.G + r % a.G;
  const size_t ob = a.ob * b + a.oh * head + a.on * tok + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2) store_o2(a, ob + e, o[e] * inv, o[e + 1] * inv);
  if (lane == 0 && a.lse)
    a.lse[(static_cast<size_t>(b) * a.H + head) * a.Nq + tok] =
        ls > 0.0f ? (mx + log2f(ls)) * kLn2 : -INFINITY;
}

}  // namespace

namespace {
template <int D, bool WEIGHTS>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(k_cache_decode<D, WEIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(sizeof(DecSmem<D>)));
}
template <int D, bool WEIGHTS>
cudaError_t launch_one(const CacheAttnMaps& m, const CacheAttnArgs& a, int row_tiles, cudaStream_t s) {
  const long long units = static_cast<long long>(a.c.B) * a.c.Hkv * row_tiles;
  const unsigned grid = static_cast<unsigned>(units * a.chunks);
  k_cache_decode<D, WEIGHTS><<<grid, kWarps * 32, sizeof(DecSmem<D>), s>>>(m, a, row_tiles);
  return cudaGetLastError();
}
}  // namespace

cudaError_t cache_prepare() {
  cudaError_t e = prepare_one<128, false>();
  if (e == cudaSuccess) e = prepare_one<64, false>();
  if (e == cudaSuccess) e = prepare_one<128, true>();
  if (e == cudaSuccess) e = prepare_one<64, true>();
  if (e == cudaSuccess) e = cache_prefill_prepare();
  if (e == cudaSuccess) e = cache_weights_prepare();
  return e;
}

cudaError_t launch_cache_decode(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  const int row_tiles = (a.Nq * a.G + kDecRows - 1) / kDecRows;
  const cudaError_t e = a.c.D == 128 ? launch_one<128, false>(m, a, row_tiles, s)
                                     : launch_one<64, false>(m, a, row_tiles, s);
  if (e != cudaSuccess || a.chunks == 1) return e;
  return launch_cache_merge(a, row_tiles, kDecRows, s);
}

cudaError_t launch_cache_weights_few(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  return a.c.D == 128 ? launch_one<128, true>(m, a, 1, s) : launch_one<64, true>(m, a, 1, s);
}

cudaError_t launch_cache_merge(const CacheAttnArgs& a, int row_tiles, int tile_rows, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.c.B) * a.c.Hkv * row_tiles * tile_rows;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (a.c.D == 128) k_cache_merge<128><<<grid, 128, 0, s>>>(a, row_tiles, tile_rows);
  else k_cache_merge<64><<<grid, 128, 0, s>>>(a, row_tiles, tile_rows);
  return cudaGetLastError();
}

}  // namespace sage
