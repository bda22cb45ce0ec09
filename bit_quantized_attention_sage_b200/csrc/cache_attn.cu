// cache_attn.cu -- attention over the paged 8-bit cache for few query rows
// (single tokens, grouped heads), the merge of its KV ranges, and the
// attention weight that each cached key received.
//
// The query heads that share a key head are rows of one tile: row r of
// (sequence b, key head h) is token r / G, head h G + r % G.
//
// Scores.  Q goes to fp16 with a power of two per row (its largest element
// lands in [2^14, 2^15)): exact for bf16 and fp16 inputs down to 2^-31 of the
// row's maximum.  int8 key codes are exact in fp16, so the products are exact
// and only the fp32 accumulation rounds; the page's key scale, the row's
// power and log2(e) * softmax scale multiply the sum.
// Probabilities.  y = 2^(t + e - M + 12), t the score in log2 units, e the
// page's value exponent, M the running maximum of t + e: fp16(y) is off by at
// most 2^-11 of each weight down to 2^-26 of the largest term, where fp16's
// subnormal range begins.  The sum L
// takes y 2^-e in fp32 before that rounding.  e4m3 value codes are exact in
// fp16.  O = (sum y code) / L; the value scales need no multiplication.
//
// What bounds it: the codes, read once (2 D bytes a key and head).  Every
// warp walks pages of its own through a private two-stage ring of TMA loads
// (32 KB in flight a warp at D = 128), so no barrier joins the warps until
// the end; 16-row tiles on mma.sync keep the tensor work (a sixteenth used
// for one row) under the load time, where a 128-row tcgen05 tile would not
// fit the registers and shared memory of that many loads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr float kBoost = 12.0f;
constexpr float kLn2 = 0.69314718055994531f;

enum : int { kSiteDecPage = 0x20101, kSiteDecDrain, kSiteWgtPage, kSiteWgtDrain };

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

template <int D>
struct alignas(1024) DecSmem {
  uint8_t kv[kWarps][kStages][2][kPage * D];  // TMA tiles: K, V
  __half q[kDecRows][D + 16];                 // padded: 8-byte reads of 4 rows on different banks
  float rowf[kDecRows];                       // 2^e * scale * log2(e) of each row
  float ml[kWarps][kDecRows][2];
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

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    k_cache_decode(const __grid_constant__ CacheAttnMaps maps, const CacheAttnArgs a, int row_tiles) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  DecSmem<D>& s = *reinterpret_cast<DecSmem<D>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const TileId id = tile_id(a, row_tiles);
  const int len = seq_length(a.c, id.b), qn = query_len(a, id.b);
  const int rows = qn * a.G, r0 = id.rt * kDecRows;
  if (r0 >= rows) return;
  const int r1 = min(rows, r0 + kDecRows);
  const long long off = static_cast<long long>(len) - qn;  // position of token 0
  const PageRuns runs = page_runs(a.mask, off + r0 / a.G, off + (r1 - 1) / a.G, len);
  // the last range takes whatever a sequence longer than announced adds
  const int p0 = id.chunk * a.chunk_pages;
  const int p1 = id.chunk == a.chunks - 1 ? runs.n : min(runs.n, p0 + a.chunk_pages);
  if (id.chunk > 0 && p0 >= runs.n) return;  // range 0 also serves an empty sequence

  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; w++)
      for (int i = 0; i < kStages; i++) mbar_init(&s.full[w][i], 1);
    s.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtx wc{a.budget, a.c.status, &s.abort};
  // this warp's pages: p0 + warp, p0 + warp + kWarps, ...; loads that the
  // ring holds are issued before the query rows are read
  const int mine = p0 + warp < p1 ? (p1 - p0 - warp + kWarps - 1) / kWarps : 0;
  auto issue = [&](int i) {  // lane 0: K and V of the warp's i-th page
    const int blk = runs.page(p0 + warp + i * kWarps);
    const int pg = page_id(a.c, id.b, blk);
    uint64_t* bar = &s.full[warp][i % kStages];
    if (pg < 0) {  // no page: nothing to load, the keys are masked below
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, 2 * kPage * D);
    const int z = pg * a.c.Hkv + id.h;
    tma_load_3d(s.kv[warp][i % kStages][0], &maps.k, bar, 0, 0, z);
    tma_load_3d(s.kv[warp][i % kStages][1], &maps.v, bar, 0, 0, z);
  };
  int issued = 0;
  if (lane == 0)
    for (; issued < min(mine, kStages); issued++) issue(issued);
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
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int r = r0 + g + 8 * i;
    kr[i] = key_range(a.mask, off + r / a.G, len);
    if (r >= r1) kr[i] = KeyRange{0, 0, 0};
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
    const int blk = runs.page(p0 + warp + i * kWarps), j0 = blk * kPage;
    const int pg = __ldg(a.c.pages + static_cast<size_t>(id.b) * a.c.max_pages + blk);
    const bool there = static_cast<unsigned>(pg) < static_cast<unsigned>(a.c.n_pages);
    if (there) {
      const size_t unit = static_cast<size_t>(pg) * a.c.Hkv + id.h;
      const float ks = __ldg(a.c.k_scale + unit);
      const int vexp = __ldg(a.c.v_exp + unit);
      const float ve = static_cast<float>(vexp);
      const uint32_t kb = smem_u32(s.kv[warp][st][0]), vb = smem_u32(s.kv[warp][st][1]);
      if (j0 + kPage > len) {
        // the sequence ends inside this page: values behind it may be any
        // bytes (NaN among them), and zero weight times NaN is NaN.  The last
        // page of the warp, so no later TMA load meets these writes.
        for (int x = lane; x < kPage * D / 16; x += 32) {
          const int r = x / (D / 16);
          if (j0 + r >= len)
            *reinterpret_cast<uint4*>(s.kv[warp][st][1] + swz<D>(r, x % (D / 16))) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // scores: 8 tiles of 8 keys
      float sc[8][4];
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
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
      const float c0 = f0 * ks, c1 = f1 * ks;
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
        sc[nt][0] *= c0;
        sc[nt][1] *= c0;
        sc[nt][2] *= c1;
        sc[nt][3] *= c1;
      }
      // keys [na, nb) of the page are masked for a row unless in its ranges
      bool all = true;
#pragma unroll
      for (int i2 = 0; i2 < 2; i2++)
        all = all && (kr[i2].sink >= j0 + kPage || (kr[i2].lo <= j0 && kr[i2].hi >= j0 + kPage));
      if (!__all_sync(kFull, all)) {
#pragma unroll
        for (int nt = 0; nt < 8; nt++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const KeyRange& k = kr[e >> 1];
            const int j = j0 + nt * 8 + t * 2 + (e & 1);
            if (!(j < k.sink || (j >= k.lo && j < k.hi))) sc[nt][e] = -INFINITY;
          }
      }
      float pm[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
        pm[0] = fmax3(pm[0], sc[nt][0], sc[nt][1]);
        pm[1] = fmax3(pm[1], sc[nt][2], sc[nt][3]);
      }
      const float un = pow2i(min(-vexp, 127));
      float nm[2];
#pragma unroll
      for (int i2 = 0; i2 < 2; i2++) {
        pm[i2] = fmaxf(pm[i2], __shfl_xor_sync(kFull, pm[i2], 1));
        pm[i2] = fmaxf(pm[i2], __shfl_xor_sync(kFull, pm[i2], 2));
        const float mn = fmaxf(m[i2], pm[i2] + ve);
        const float al = m[i2] == mn ? 1.0f : ex2_approx(m[i2] - mn);  // 0 from -inf
        m[i2] = mn;
        nm[i2] = mn == -INFINITY ? 0.0f : kBoost + ve - mn;
        l[i2] *= al;
#pragma unroll
        for (int d = 0; d < D / 8; d++) {
          o[d][2 * i2] *= al;
          o[d][2 * i2 + 1] *= al;
        }
      }
      float rs[2] = {0.0f, 0.0f};
      uint32_t pa[4][4];
#pragma unroll
      for (int nt = 0; nt < 8; nt++) {
        const float y0 = ex2_approx(sc[nt][0] + nm[0]), y1 = ex2_approx(sc[nt][1] + nm[0]);
        const float y2 = ex2_approx(sc[nt][2] + nm[1]), y3 = ex2_approx(sc[nt][3] + nm[1]);
        rs[0] += y0 + y1;
        rs[1] += y2 + y3;
        const __half2 h0 = __floats2half2_rn(y0, y1), h1 = __floats2half2_rn(y2, y3);
        pa[nt / 2][(nt & 1) * 2] = *reinterpret_cast<const uint32_t*>(&h0);
        pa[nt / 2][(nt & 1) * 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
      }
      l[0] = fmaf(rs[0], un, l[0]);
      l[1] = fmaf(rs[1], un, l[1]);
      // O += P V: per 32 channels, 16 keys at a time
#pragma unroll
      for (int kk = 0; kk < 4; kk++) {
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
    __syncwarp();
    if (lane == 0 && issued < mine) issue(issued++);
  }
  if (!ok) {  // a wait ran out (recorded): let the loads in flight land, then leave
    if (lane == 0)
      for (int i = max(0, issued - kStages); i < issued; i++)
        drain_wait(&s.full[warp][i % kStages], (i / kStages) & 1, wc, kSiteDecDrain);
    __syncwarp();
  }
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
  static_assert(kStages * 2 * kPage * D >= kDecRows * D * 4, "a warp's ring holds its partial rows");
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
  constexpr size_t kWarpFloats = kStages * 2 * kPage * D / 4;
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

// ---------------------------------------------------------------- weights

// w[key] (+)= sum over the query rows of exp(s - lse): scores as in the
// attention kernel, with the row's statistics known.  A warp owns a page (its
// keys are the columns of the score tiles, so a key's sum stays in one warp:
// no order of atomics enters it), 16 keys of it at a time as fp16 fragments
// in registers, over which all query rows of the block pass; the rows lie in
// shared memory, 128 at a time.
constexpr int kWgtWarps = 4;
constexpr int kWgtRows = 128;

template <int D>
struct alignas(1024) WgtSmem {
  uint8_t k[kWgtWarps][kPage * D];
  __half q[kWgtRows][D + 16];
  float2 row[kWgtRows];  // 2^e * scale * log2(e); lse * log2(e)
  KeyRange kr[kWgtRows];
  uint64_t full[kWgtWarps];
  int abort;
};

template <int D>
__global__ void __launch_bounds__(kWgtWarps * 32)
    k_cache_weights(const __grid_constant__ CacheAttnMaps maps, const CacheAttnArgs a, int page_groups) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  WgtSmem<D>& s = *reinterpret_cast<WgtSmem<D>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.x / page_groups;
  const int b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int len = seq_length(a.c, b), qn = query_len(a, b), rows = qn * a.G;
  const int n_blk = (len + kPage - 1) / kPage;
  int blk0 = static_cast<int>(blockIdx.x % page_groups) * kWgtWarps;
  if (blk0 >= n_blk) return;
  const long long off = static_cast<long long>(len) - qn;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWgtWarps; w++) mbar_init(&s.full[w], 1);
    s.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtx wc{a.budget, a.c.status, &s.abort};
  int loads = 0;  // page loads of this warp so far: the barrier's phase
  // one group of pages a block, more only where the sequence is longer than
  // announced
  for (; blk0 < n_blk; blk0 += page_groups * kWgtWarps) {
    const int blk = blk0 + warp, j0 = blk * kPage;
    int pg = -1;
    if (blk < n_blk) pg = page_id(a.c, b, blk);
    const bool mine = pg >= 0;
    const size_t unit = static_cast<size_t>(mine ? pg : 0) * a.c.Hkv + h;
    if (mine && lane == 0) {
      mbar_arrive_expect_tx(&s.full[warp], kPage * D);
      tma_load_3d(s.k[warp], &maps.k, &s.full[warp], 0, 0, static_cast<int>(unit));
    }
    const float ks = mine ? __ldg(a.c.k_scale + unit) : 0.0f;
    const uint32_t kb = smem_u32(s.k[warp]);
    float acc[8][2];  // keys 8 nt + 2 t, + 1
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i][0] = acc[i][1] = 0.0f;
    bool ok = __all_sync(kFull, !s.abort);
    for (int rb = 0; rb < rows; rb += kWgtRows) {
      const int nr = min(kWgtRows, rows - rb), nr16 = (nr + 15) / 16 * 16;
      __syncthreads();
      for (int r = warp; r < nr16; r += kWgtWarps) {
        const float f = stage_row<D>(a, b, h, rb + r, rows, s.q[r], lane);
        if (lane == 0) {
          float l2 = INFINITY;  // a row that saw nothing, or is not there: weight 0
          KeyRange k{0, 0, 0};
          if (r < nr) {
            const int rr = rb + r, tok = rr / a.G, head = h * a.G + rr % a.G;
            const float v = a.lse_in[(static_cast<size_t>(b) * a.H + head) * a.Nq + tok];
            if (v != -INFINITY) l2 = v * kLog2e;
            k = key_range(a.mask, off + tok, len);
          }
          s.row[r] = make_float2(f * (a.scale * kLog2e), l2);
          s.kr[r] = k;
        }
      }
      __syncthreads();
      if (!mine || !ok) continue;
      if (rb == 0) {
        ok = __all_sync(kFull, mbar_wait(&s.full[warp], loads & 1, wc, kSiteWgtPage));
        if (!ok) continue;
      }
#pragma unroll 1
      for (int n2 = 0; n2 < 4; n2++) {  // 16 keys
        uint32_t kf[2][D / 16][2];
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
          for (int c4 = 0; c4 < D / 64; c4++) {
            uint32_t r4[4];
            ldsm4(kb + swz<D>((n2 * 2 + x) * 8 + (lane & 7), c4 * 4 + (lane >> 3)), r4);
#pragma unroll
            for (int c = 0; c < 4; c++) i8x4_to_f16(r4[c], kf[x][c4 * 4 + c][0], kf[x][c4 * 4 + c][1]);
          }
        float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        for (int rt = 0; rt < nr16; rt += 16) {
          float sc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
          for (int kk = 0; kk < D / 16; kk++) {
            const uint2 x = *reinterpret_cast<const uint2*>(&s.q[rt + g][kk * 16 + t * 4]);
            const uint2 y = *reinterpret_cast<const uint2*>(&s.q[rt + g + 8][kk * 16 + t * 4]);
            const uint32_t qa[4] = {x.x, y.x, x.y, y.y};
            mma16816(sc[0], qa, kf[0][kk][0], kf[0][kk][1]);
            mma16816(sc[1], qa, kf[1][kk][0], kf[1][kk][1]);
          }
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const float2 rw = s.row[rt + g + 8 * i];
            const KeyRange k = s.kr[rt + g + 8 * i];
            const float c = rw.x * ks;
#pragma unroll
            for (int x = 0; x < 2; x++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const int j = j0 + (n2 * 2 + x) * 8 + t * 2 + e;
                const float y = ex2_approx(fmaf(sc[x][2 * i + e], c, -rw.y));
                if (j < k.sink || (j >= k.lo && j < k.hi)) sum[x][e] += y;
              }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (i == n2) {
            acc[2 * i][0] += sum[0][0];
            acc[2 * i][1] += sum[0][1];
            acc[2 * i + 1][0] += sum[1][0];
            acc[2 * i + 1][1] += sum[1][1];
          }
      }
    }
    if (!mine) continue;
    if (lane == 0) drain_wait(&s.full[warp], loads & 1, wc, kSiteWgtDrain);
    __syncwarp();
    loads++;
    if (!ok) continue;
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float v = acc[i][e];
        v += __shfl_xor_sync(kFull, v, 4);
        v += __shfl_xor_sync(kFull, v, 8);
        v += __shfl_xor_sync(kFull, v, 16);
        const int j = i * 8 + t * 2 + e;
        if (g == 0 && j0 + j < len) {
          float* w = a.c.weight + unit * kPage + j;
          if (a.accumulate) atomicAdd(w, v);  // a page may serve two sequences
          else *w = v;
        }
      }
  }
}

}  // namespace

cudaError_t cache_prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_cache_decode<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(DecSmem<128>)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cache_decode<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(DecSmem<64>)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cache_weights<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(WgtSmem<128>)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cache_weights<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(WgtSmem<64>)));
  return e == cudaSuccess ? cache_prefill_prepare() : e;
}

cudaError_t launch_cache_decode(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  const int row_tiles = (a.Nq * a.G + kDecRows - 1) / kDecRows;
  const long long units = static_cast<long long>(a.c.B) * a.c.Hkv * row_tiles;
  const unsigned grid = static_cast<unsigned>(units * a.chunks);
  if (a.c.D == 128)
    k_cache_decode<128><<<grid, kWarps * 32, sizeof(DecSmem<128>), s>>>(m, a, row_tiles);
  else
    k_cache_decode<64><<<grid, kWarps * 32, sizeof(DecSmem<64>), s>>>(m, a, row_tiles);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.chunks == 1) return e;
  return launch_cache_merge(a, row_tiles, kDecRows, s);
}

cudaError_t launch_cache_merge(const CacheAttnArgs& a, int row_tiles, int tile_rows, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.c.B) * a.c.Hkv * row_tiles * tile_rows;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (a.c.D == 128) k_cache_merge<128><<<grid, 128, 0, s>>>(a, row_tiles, tile_rows);
  else k_cache_merge<64><<<grid, 128, 0, s>>>(a, row_tiles, tile_rows);
  return cudaGetLastError();
}

cudaError_t launch_cache_weights(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  const int groups = a.chunks;  // page groups of kWgtWarps pages, set by the caller
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.c.B) * a.c.Hkv * groups);
  if (a.c.D == 128)
    k_cache_weights<128><<<grid, kWgtWarps * 32, sizeof(WgtSmem<128>), s>>>(m, a, groups);
  else
    k_cache_weights<64><<<grid, kWgtWarps * 32, sizeof(WgtSmem<64>), s>>>(m, a, groups);
  return cudaGetLastError();
}

}  // namespace sage
