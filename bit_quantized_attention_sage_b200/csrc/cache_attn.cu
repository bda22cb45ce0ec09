// cache_attn.cu -- attention over the paged 8-bit cache for few query rows
// (single tokens, grouped heads), the join of heads that several blocks shared,
// and, in the same stream of keys, the attention weight that each cached key
// received.
//
// The query heads that share a key head are rows of one tile: row r of
// (sequence b, key head h) is token r / G, head h G + r % G.
//
// Scores.  A query row becomes 22-bit integers v (a power of two puts its
// largest element into [2^21, 2^22)), exact for bf16 down to 2^-14 and fp16
// down to 2^-11 of the row's maximum and off by at most 2^-22 of it below, and
// those three int8 limbs, so Q K^T is three int8 products on the key codes as
// they lie in the cache: exact int32, no conversion of the codes (five
// instructions per four of them to fp16, half of the loop's issue slots).
// The limbs join in fp32, rounded twice (the lower two's sum, then the whole; by
// 2^-24 of sum |q k| each at most); the page's key scale, the row's power and
// log2(e) * softmax scale multiply the sum.
// Probabilities.  y = 2^(t + e - M + 7), t the score in log2 units, e the
// page's value exponent, M a reference maximum of t + e that follows the
// running one in steps of at least 2^8: y <= 2^15, and fp16(y) is off by at
// most 2^-11 of each weight down to 2^-21 of the largest term, where fp16's
// subnormal range begins.  The sum L takes y 2^-e in fp32 before that
// rounding, or, on pages far below the largest e, a power that is still a
// number (cache_dev.cuh).  e4m3 value codes are exact in fp16.
// O = (sum y code) / L; the value scales need no multiplication.
//
// What bounds it: the codes, read once (2 D bytes a key and head).  Every
// warp walks half pages of its own (32 keys) through a private ring of two
// TMA loads (16 KB in flight a warp at D = 128, 192 KB an SM with two blocks),
// so no barrier joins the warps until the end.  Page ids, key scales and
// value exponents of a warp's next 32 half pages are fetched at once, one a
// lane; taken one by one inside the loop, their three dependent loads cost
// more than the tile.  Keys are the 16 rows of the mma.sync tiles and query
// rows their 8 columns (S^T = K Q^T, O^T = V^T P^T): one head group of up to
// eight wastes no column, and a product covers 256 bytes of codes.  A 128-row
// tcgen05 tile would need its codes converted through shared memory first.
//
// Measured, 8 key heads x 128 channels: 32 tokens of 32 query heads on caches
// of up to 16000 tokens (286000 in all) 110-116 us, 5.3 TB/s; four of 64 query
// heads on 131071 tokens each 182-192 us, 5.9 TB/s.  The same loads without the arithmetic took
// 126 and 196 us from a cold L2, the kernels then 134 and 200.  One token on
// 500 tokens 10 us: five dependent loads, the instructions' first fetch and
// three tiles a warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
// Warps of a block (two an SM) and half pages on their way to each: a warp that
// holds 16 rows needs some 200 registers.
template <int NT>
struct Shape {
  static constexpr int kWarps = NT == 1 ? 6 : 4, kStages = NT == 1 ? 2 : 3;
};
constexpr int kJoinWarps = 6;
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

// D (int32 16x8) += A (int8 16x32) B (int8 32x8)
__device__ __forceinline__ void mma16832(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit elements held by the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

template <int D, int NT>
struct alignas(1024) DecSmem {
  static constexpr int kWarps = Shape<NT>::kWarps, kStages = Shape<NT>::kStages;
  uint8_t kv[kWarps][kStages][2][kHalf * D];  // TMA tiles: K, V
  int8_t q[3][kDecRows][D];                   // limbs of the query rows, low to high
  float rowf[kDecRows];                       // power of two * scale * log2(e) of each row
  float ml[kWarps][kDecRows][2];
  TileMeta meta[kWarps][kStages];
  PlaceSmem<kWarps> place;
  uint64_t full[kWarps][kStages];
  int abort;
};

// The first n query rows (from `rows` on: zero) as limbs.
template <int D, int NT>
__device__ __forceinline__ void stage_limbs(DecSmem<D, NT>& s, const CacheAttnArgs& a, int b, int h, int rows) {
  constexpr int CH = D / 8, n = 8 * NT, kWarps = Shape<NT>::kWarps;
  for (int i = threadIdx.x; i < n * CH; i += kWarps * 32) {
    const int r = i / CH, c = i % CH;
    const long long at[1] = {r < rows ? q8_at(a, b, h, r, c) : -1};
    uint4 raw[1];
    load_q8(a, at, raw);
    float f[8];
    q8_floats(a, raw[0], f);
    const float m = row_max<CH>(f);
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 8; e++) finite = finite && fabsf(f[e]) <= FLT_MAX;
    const uint32_t bad = __ballot_sync(kFull, !finite) >> (threadIdx.x & 31 & ~(CH - 1)) & ((1u << CH) - 1u);
    const int p = max(row_power(m) - 7, -126);  // m 2^-p in [2^21, 2^22)
    const float inv = pow2i(-p);
    uint32_t w[3][2] = {{0u, 0u}, {0u, 0u}, {0u, 0u}};
#pragma unroll
    for (int e = 0; e < 8; e++) {
      int v = __float2int_rn(f[e] * inv);
#pragma unroll
      for (int x = 0; x < 3; x++) {
        const int lo = static_cast<int8_t>(v);
        w[x][e >> 2] |= static_cast<uint32_t>(lo & 0xFF) << (8 * (e & 3));
        v = (v - lo) >> 8;
      }
    }
#pragma unroll
    for (int x = 0; x < 3; x++)
      *reinterpret_cast<uint2*>(&s.q[x][r][c * 8]) = make_uint2(w[x][0], w[x][1]);
    // (a row with a NaN or an infinity: its scores become NaN)
    if (c == 0) s.rowf[r] = bad ? __int_as_float(0x7FFFFFFF) : pow2i(p) * (a.scale * kLog2e);
  }
}

// One head's pages [p0, p1) (of the runs its rows visit): attention, or the
// weights.  `seen` counts the warp's tiles so far (the ring's phase).
template <int D, int NT, bool WEIGHTS>
__device__ __forceinline__ void decode_head(DecSmem<D, NT>& s, const CacheAttnMaps& maps, const CacheAttnArgs& a,
                                            int b, int h, int len, int qn, const PageRuns& runs, int p0,
                                            int p1, int np, int& seen, const WaitCtx& wc) {
  constexpr int ROWS = 8 * NT, kWarps = Shape<NT>::kWarps, kStages = Shape<NT>::kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rows = qn * a.G;
  const long long off = static_cast<long long>(len) - qn;  // position of token 0
  // this warp's half pages: warp, warp + kWarps, ... of the stretch's
  const int halves = 2 * (min(p1, runs.n) - p0);
  const int mine = warp < halves ? (halves - warp + kWarps - 1) / kWarps : 0;
  TileMeta next{0.0f, 0, -1, 0};  // lane's tile of the current 32
  int issued = 0;
  auto issue = [&]() {  // the whole warp: the load of tile `issued`
    if ((issued & 31) == 0) {
      const int q = warp + (issued + lane) * kWarps;
      next = TileMeta{0.0f, 0, -1, 0};
      if (q < halves) {
        const int blk = runs.page(p0 + q / 2);
        const int pg = page_id(a.c, b, blk);
        const int j0 = blk * kPage + (q & 1) * kHalf;
        if (pg >= 0 && j0 < len) {  // else: no page, or the half behind the end
          next.unit = pg * a.c.Hkv + h;
          next.j0 = j0;
          next.ks = __ldg(a.c.k_scale + next.unit);
          if (!WEIGHTS) next.ve = __ldg(a.c.v_exp + next.unit);
        }
      }
    }
    if (lane == (issued & 31)) {
      const int st = (seen + issued) % kStages;
      uint64_t* bar = &s.full[warp][st];
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
  stage_limbs(s, a, b, h, rows);
  __syncthreads();
  // B fragments of Q^T: channels 32 kk + 4 t .. + 3 and 16 on, of row g.  For
  // 16 rows they stay in shared memory: 48 registers would spill.
  auto q_frag = [&](int n, int kk, int x, int e) {
    return *reinterpret_cast<const uint32_t*>(&s.q[x][n * 8 + g][kk * 32 + e * 16 + t * 4]);
  };
  uint32_t qb[D / 32][3][2];
  if constexpr (NT == 1) {
#pragma unroll
    for (int kk = 0; kk < D / 32; kk++)
#pragma unroll
      for (int x = 0; x < 3; x++)
#pragma unroll
        for (int e = 0; e < 2; e++) qb[kk][x][e] = q_frag(0, kk, x, e);
  }
  float f[NT][2];
  KeyRange kr[NT][2];
  float nl[NT][2];  // WEIGHTS: -lse log2(e); -inf: weight 0
  bool bad[NT][2], any_bad = false;  // what the row sees is NaN
#pragma unroll
  for (int n = 0; n < NT; n++) {
#pragma unroll
    for (int e = 0; e < 2; e++) {  // rows that this lane's columns are
      const int r = n * 8 + t * 2 + e;
      f[n][e] = s.rowf[n * 8 + t * 2 + e];
      bad[n][e] = f[n][e] != f[n][e];
      kr[n][e] = KeyRange{0, 0, 0};
      nl[n][e] = -INFINITY;
      if (r < rows) {
        kr[n][e] = key_range(a.mask, off + r / a.G, len);
        if (WEIGHTS) {
          const float v = __ldg(a.lse_in + (static_cast<size_t>(b) * a.H + h * a.G + r % a.G) * a.Nq + r / a.G);
          if (v != v) bad[n][e] = true;
          else if (v != -INFINITY) nl[n][e] = -v * kLog2e;
        }
      }
      if (bad[n][e]) f[n][e] = 0.0f;
      any_bad = any_bad || bad[n][e];
    }
  }
  any_bad = __any_sync(kFull, any_bad);
  // keys [full_lo, full_hi) and those below full_sink are seen by every row
  // that is there: tiles inside need no mask.  Rows that are not there see
  // whatever those do and are never stored.
  const KeyRange ra = key_range(a.mask, off, len);
  const KeyRange rz = key_range(a.mask, off + max(qn - 1, 0), len);
  const int full_sink = min(ra.sink, rz.sink), full_lo = rz.lo, full_hi = min(ra.hi, rz.hi);

  float o[D / 16][NT][4];
#pragma unroll
  for (int i = 0; i < D / 16; i++)
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[i][n][e] = 0.0f;
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      m[n][e] = -INFINITY;
      l[n][e] = 0.0f;
    }

  bool ok = true;
  int top_exp = kMinVExp;  // the largest value exponent so far
  for (int i = 0; i < mine; i++) {
    const int st = (seen + i) % kStages;
    ok = __all_sync(kFull, mbar_wait(&s.full[warp][st], ((seen + i) / kStages) & 1, wc, kSiteDecPage));
    if (!ok) break;
    const TileMeta md = s.meta[warp][st];
    const int j0 = md.j0;
    if (j0 >= 0) {
      const uint32_t kb = smem_u32(s.kv[warp][st][0]), vb = smem_u32(s.kv[warp][st][1]);
      if (!WEIGHTS && j0 + kHalf > len) {
        // the sequence ends inside this tile: values behind it may be any
        // bytes (NaN among them), and zero weight times NaN is NaN.  The last
        // tile of this head that the warp loads: the next head's loads come
        // after the block's fence.
        for (int x = lane; x < kHalf * D / 16; x += 32) {
          const int r = x / (D / 16);
          if (j0 + r >= len)
            *reinterpret_cast<uint4*>(s.kv[warp][st][1] + swz<D>(r, x % (D / 16))) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // scores of two tiles of 16 keys: keys g and g + 8, rows 2 t and 2 t + 1
      float sc[2][NT][4];
      {
        uint32_t ka[2][D / 32][4];  // keys 0-7 / 8-15 of chunk 2 kk, then of 2 kk + 1
#pragma unroll
        for (int mt = 0; mt < 2; mt++)
#pragma unroll
          for (int kk = 0; kk < D / 32; kk++)
            ldsm4(kb + swz<D>(mt * 16 + (lane & 15), kk * 2 + (lane >> 4)), ka[mt][kk]);
        int low[2][NT][4];  // the two lower limbs joined
#pragma unroll
        for (int x = 0; x < 3; x++) {
          int acc[2][NT][4];
#pragma unroll
          for (int mt = 0; mt < 2; mt++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
              for (int e = 0; e < 4; e++) acc[mt][n][e] = 0;
#pragma unroll
          for (int kk = 0; kk < D / 32; kk++)
#pragma unroll
            for (int n = 0; n < NT; n++) {
              const uint32_t b0 = NT == 1 ? qb[kk][x][0] : q_frag(n, kk, x, 0);
              const uint32_t b1 = NT == 1 ? qb[kk][x][1] : q_frag(n, kk, x, 1);
#pragma unroll
              for (int mt = 0; mt < 2; mt++) mma16832(acc[mt][n], ka[mt][kk], b0, b1);
            }
#pragma unroll
          for (int mt = 0; mt < 2; mt++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
              for (int e = 0; e < 4; e++) {
                if (x == 0) low[mt][n][e] = acc[mt][n][e];
                else if (x == 1) low[mt][n][e] += acc[mt][n][e] * 256;
                else
                  sc[mt][n][e] = fmaf(static_cast<float>(acc[mt][n][e]), 65536.0f,
                                      static_cast<float>(low[mt][n][e]));
              }
        }
      }
      if (any_bad) {
#pragma unroll
        for (int mt = 0; mt < 2; mt++)
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (bad[n][e & 1]) sc[mt][n][e] = __int_as_float(0x7FFFFFFF);
      }
      if (!(j0 + kHalf <= full_sink || (j0 >= full_lo && j0 + kHalf <= full_hi))) {
#pragma unroll
        for (int mt = 0; mt < 2; mt++)
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const KeyRange& k = kr[n][e & 1];
              const int j = j0 + mt * 16 + g + (e >> 1) * 8;
              if (!(j < k.sink || (j >= k.lo && j < k.hi))) sc[mt][n][e] = -INFINITY;
            }
      }
      // a zero scale must not meet -inf as 0 * inf
      float c[NT][2];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) c[n][e] = fmaxf(f[n][e] * md.ks, FLT_MIN);
      if constexpr (WEIGHTS) {
        float w[4];  // keys g, g + 8, g + 16, g + 24
#pragma unroll
        for (int k = 0; k < 4; k++) {
          w[k] = 0.0f;
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++)
              w[k] += ex2_approx(fmaf(sc[k >> 1][n][(k & 1) * 2 + e], c[n][e], nl[n][e]));
          w[k] += __shfl_xor_sync(kFull, w[k], 1);
          w[k] += __shfl_xor_sync(kFull, w[k], 2);
        }
        // lane (g, t) writes key 8 t + g
        const float v = t == 0 ? w[0] : t == 1 ? w[1] : t == 2 ? w[2] : w[3];
        const int j = j0 + t * 8 + g;
        if (j < len) {
          float* dst = a.c.weight + static_cast<size_t>(md.unit) * kPage + (j & (kPage - 1));
          if (a.accumulate) atomicAdd(dst, v);  // a page may serve two sequences
          else *dst = v;
        }
      } else {
        const float ve = static_cast<float>(md.ve);
        float pm[NT][2];
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float x = fmax3(fmaxf(sc[0][n][e], sc[0][n][e + 2]), sc[1][n][e], sc[1][n][e + 2]);
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
            pm[n][e] = fmaf(x, c[n][e], ve);
            grow = grow || pm[n][e] > m[n][e] + kLazy;
          }
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const float mn = fmaxf(m[n][e], pm[n][e]);
              const float down = m[n][e] == mn ? 0.0f : m[n][e] - mn, al = ex2_approx(down);  // 0 from -inf
              m[n][e] = mn;
              l[n][e] = add_scaled(0.0f, l[n][e], down, al);
#pragma unroll
              for (int d = 0; d < D / 16; d++) {
                o[d][n][e] *= al;
                o[d][n][e + 2] *= al;
              }
            }
        }
        top_exp = max(top_exp, md.ve);
        const int fe = sum_exp(md.ve, top_exp);
        const float un = sum_unit(fe);
        uint32_t pb[2][NT][2];  // B fragments of P^T, 16 keys each
#pragma unroll
        for (int n = 0; n < NT; n++) {
          float nm[2], rs[2] = {0.0f, 0.0f};
#pragma unroll
          for (int e = 0; e < 2; e++) nm[e] = m[n][e] == -INFINITY ? 0.0f : kBoost + ve - m[n][e];
#pragma unroll
          for (int mt = 0; mt < 2; mt++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
              const float y0 = ex2_approx(fmaf(sc[mt][n][k * 2], c[n][0], nm[0]));
              const float y1 = ex2_approx(fmaf(sc[mt][n][k * 2 + 1], c[n][1], nm[1]));
              rs[0] += y0;
              rs[1] += y1;
              const __half2 y = __floats2half2_rn(y0, y1);
              pb[mt][n][k] = transpose8(*reinterpret_cast<const uint32_t*>(&y));
            }
          if (fe != md.ve) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const float nf = m[n][e] == -INFINITY ? 0.0f : kBoost + static_cast<float>(fe) - m[n][e];
              rs[e] = 0.0f;
#pragma unroll
              for (int k = 0; k < 4; k++)
                rs[e] += ex2_approx(fmaf(sc[k >> 1][n][(k & 1) * 2 + e], c[n][e], nf));
            }
          }
          l[n][0] = fmaf(rs[0], un, l[n][0]);
          l[n][1] = fmaf(rs[1], un, l[n][1]);
        }
        // O^T += V^T P^T: tiles of 16 channels, 16 keys at a time.  Row g of
        // the tile is channel 2 g, row g + 8 channel 2 g + 1.
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
#pragma unroll
          for (int d2 = 0; d2 < D / 32; d2++) {
            uint32_t vr[4];  // keys 0-7 / 8-15 of two 16-channel chunks
            ldsm4t(vb + swz<D>(kk * 16 + (lane & 15), d2 * 2 + (lane >> 4)), vr);
#pragma unroll
            for (int x = 0; x < 2; x++) {
              uint32_t va[4];
              f8x4_to_f16(vr[2 * x], va[0], va[1]);
              f8x4_to_f16(vr[2 * x + 1], va[2], va[3]);
#pragma unroll
              for (int n = 0; n < NT; n++) mma16816(o[d2 * 2 + x][n], va, pb[kk][n][0], pb[kk][n][1]);
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
        drain_wait(&s.full[warp][(seen + i) % kStages], ((seen + i) / kStages) & 1, wc, kSiteDecDrain);
    __syncwarp();
  }
  seen += mine;
  if constexpr (WEIGHTS) {
    __syncthreads();  // the query rows in shared memory are free again
    return;
  }
  // row sums over the eight lanes of a column
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      l[n][e] += __shfl_xor_sync(kFull, l[n][e], 4);
      l[n][e] += __shfl_xor_sync(kFull, l[n][e], 8);
      l[n][e] += __shfl_xor_sync(kFull, l[n][e], 16);
    }
  // join the warps: every tile has landed and been read, so the ring holds
  // the partial rows, fp32 [ROWS][D] a warp
  __syncthreads();
  if (s.abort) return;
  float* part = reinterpret_cast<float*>(s.kv[warp][0][0]);
  static_assert(kStages * 2 * kHalf * D >= ROWS * D * 4, "a warp's ring holds its partial rows");
#pragma unroll
  for (int n = 0; n < NT; n++) {
#pragma unroll
    for (int d = 0; d < D / 16; d++)
#pragma unroll
      for (int e = 0; e < 2; e++)
        *reinterpret_cast<float2*>(part + (n * 8 + t * 2 + e) * D + d * 16 + g * 2) =
            make_float2(o[d][n][e], o[d][n][e + 2]);
    if (g == 0) {
#pragma unroll
      for (int e = 0; e < 2; e++) {
        s.ml[warp][n * 8 + t * 2 + e][0] = m[n][e];
        s.ml[warp][n * 8 + t * 2 + e][1] = l[n][e];
      }
    }
  }
  __syncthreads();
  constexpr size_t kWarpFloats = kStages * 2 * kHalf * D / 4;
  const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (p0 == 0)) * ROWS;
  for (int x = threadIdx.x; x < ROWS * D / 2; x += kWarps * 32) {
    const int r = x / (D / 2), d = x % (D / 2) * 2;
    if (r >= rows) break;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; w++) mx = fmaxf(mx, s.ml[w][r][0]);
    float ox = 0.0f, oy = 0.0f, ls = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      const float mw = s.ml[w][r][0];
      // (no maximum: nothing seen, sum 0, or NaN alone, sum NaN)
      const bool none = mw == -INFINITY;
      const float al = none ? 0.0f * s.ml[w][r][1] : ex2_approx(mw - mx);
      const float2 v = *reinterpret_cast<const float2*>(
          reinterpret_cast<const float*>(s.kv[0][0][0]) + w * kWarpFloats + r * D + d);
      ox = fmaf(al, v.x, ox);
      oy = fmaf(al, v.y, oy);
      ls = add_scaled(ls, s.ml[w][r][1], none ? 0.0f : mw - mx, al);
    }
    if (p1 - p0 < np) {
      *reinterpret_cast<float2*>(a.part_o + (slot + r) * D + d) = make_float2(ox, oy);
      if (d == 0) *reinterpret_cast<float2*>(a.part_ml + (slot + r) * 2) = make_float2(mx - kBoost, ls);
    } else {
      const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
      const int tok = r / a.G, head = h * a.G + r % a.G;
      store_o2(a, a.ob * b + a.oh * head + a.on * tok + d, ox * inv, oy * inv);
      if (d == 0 && a.lse)
        a.lse[(static_cast<size_t>(b) * a.H + head) * a.Nq + tok] =
            ls == 0.0f ? -INFINITY : ls > 0.0f ? (mx - kBoost + log2f(ls)) * kLn2 : ls;
    }
  }
  // the ring held the partial rows: order them before the next head's loads
  fence_proxy_async_smem();
  __syncthreads();
}

// NT: query rows in eighths (8 NT rows).  WEIGHTS: instead of attending,
// w[key] (+)= sum over the rows of exp(s - lse), the rows' lse given.
template <int D, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(Shape<NT>::kWarps * 32, 2)
    k_cache_decode(const __grid_constant__ CacheAttnMaps maps, const CacheAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  constexpr int kWarps = Shape<NT>::kWarps, kStages = Shape<NT>::kStages;
  DecSmem<D, NT>& s = *reinterpret_cast<DecSmem<D, NT>*>(raw);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&maps.k);
    if (!WEIGHTS) tma_prefetch_desc(&maps.v);
    for (int w = 0; w < kWarps; w++)
      for (int i = 0; i < kStages; i++) mbar_init(&s.full[w][i], 1);
    s.abort = 0;
    fence_mbar_init();
  }
  const int c = blockIdx.x, n = gridDim.x;
  const WaitCtx wc{a.budget, a.c.status, &s.abort};
  // One loop for both ways of cutting, so that there is one copy of what it
  // does: a call's first microseconds are instructions that come from L2.
  int seen = 0, b, h = -1;  // h < 0: from the position x
  long long x, end, before = 0;
  if (a.whole) {
    __syncthreads();
    b = c / a.c.Hkv;
    h = c - b * a.c.Hkv;
    x = 0;
    end = seq_work<WEIGHTS>(a, b);
  } else {
    // (locate's barriers also publish the ring's)
    const Place pl = locate<kWarps, WEIGHTS>(s.place, a, [&](long long w) { return share_start(w, c, n); });
    if (!WEIGHTS) cudaTriggerProgrammaticLaunchCompletion();
    x = share_start(pl.work, c, n);
    end = share_start(pl.work, c + 1, n);
    before = pl.before;
    b = pl.b;
  }
  int np = 0, len = 0, qn = 0, p0 = 0;
  PageRuns runs{0, 0, 0};
  bool fresh = true;
  while (x < end && b < a.c.B) {
    if (fresh) {  // the first head of this block in sequence b
      fresh = false;
      np = seq_work<WEIGHTS>(a, b);
      len = seq_length(a.c, b);
      qn = query_len(a, b);
      runs = seq_runs<WEIGHTS>(a, b, len, qn);
      if (h < 0 && np > 0) {
        const long long rel = x - before * a.c.Hkv;
        h = static_cast<int>(rel / np);
        p0 = static_cast<int>(rel - static_cast<long long>(h) * np);
      }
    }
    if (np == 0 || h == a.c.Hkv) {
      before += np;
      b++;
      h = -1;
      fresh = true;
      continue;
    }
    const int p1 = static_cast<int>(min(static_cast<long long>(np), p0 + (end - x)));
    decode_head<D, NT, WEIGHTS>(s, maps, a, b, h, len, qn, runs, p0, p1, np, seen, wc);
    if (s.abort) return;
    x += p1 - p0;
    p0 = 0;
    h++;
  }
}

// Join of the heads that stretches cut, a block a head and slice of its
// channels (gridDim.y slices): first the factor of every partial result (2^(its
// maximum - the largest)), a warp a row; then threads (group, row, 4 channels),
// each group every so many-th partial, the groups summed in order.
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) k_cache_join(const CacheAttnArgs a, int n) {
  constexpr int NT = kJoinWarps * 32;
  const int Q = D / 4 / gridDim.y, d0 = blockIdx.y * (D / gridDim.y);
  __shared__ long long sum[2][kJoinWarps];
  __shared__ float fac[kMaxShares][ROWS];  // maximum, then factor
  __shared__ float lsum[kMaxShares][ROWS];
  __shared__ float tot[2][ROWS];           // largest maximum, joined sum
  __shared__ float4 sh_o[NT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv;
  // Launched under the attention kernel's tail.  Every block waits for that,
  // also one with nothing to join: what comes next in the stream waits for
  // this kernel only, so it must not end before the attention has.
  const int np = seq_work<false>(a, b);
  if (np == 0) {
    cudaGridDependencySynchronize();
    return;
  }
  long long sb = 0, sw = 0;  // pages of one head before b, and in all
  for (int i = tid; i < a.c.B; i += NT) {
    const int v = seq_work<false>(a, i);
    sw += v;
    if (i < b) sb += v;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sb += __shfl_xor_sync(kFull, sb, o);
    sw += __shfl_xor_sync(kFull, sw, o);
  }
  if (lane == 0) {
    sum[0][warp] = sb;
    sum[1][warp] = sw;
  }
  __syncthreads();
  long long before = 0, work = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; w++) {
    before += sum[0][w];
    work += sum[1][w];
  }
  work *= a.c.Hkv;
  const long long x0 = before * a.c.Hkv + static_cast<long long>(h) * np;
  const int c0 = share_of(work, x0, n), c1 = share_of(work, x0 + np - 1, n);
  cudaGridDependencySynchronize();
  if (c0 == c1) return;  // one block had the whole head and wrote it
  const int qn = query_len(a, b), rows = qn * a.G, k = c1 - c0 + 1;
  // the first partial of the head lies in slot 2 c + 1, the others in 2 c
  auto slot = [&](int i) { return (2 * static_cast<size_t>(c0 + i) + (i == 0)) * ROWS; };
  for (int i = tid; i < k * ROWS; i += NT) {
    const int p = i / ROWS, r = i % ROWS;
    float2 ml = make_float2(-INFINITY, 0.0f);
    // (a block without a page of its own wrote nothing)
    if (r < rows && share_start(work, c0 + p, n) < share_start(work, c0 + p + 1, n))
      ml = *reinterpret_cast<const float2*>(a.part_ml + (slot(p) + r) * 2);
    fac[p][r] = ml.x;
    lsum[p][r] = ml.y;
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kJoinWarps) {
    float mx = -INFINITY, ls = 0.0f;
    for (int p = lane; p < k; p += 32) mx = fmaxf(mx, fac[p][r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    for (int p = lane; p < k; p += 32) {
      const float down = fac[p][r] == -INFINITY ? 0.0f : fac[p][r] - mx;
      const float al = fac[p][r] == -INFINITY ? 0.0f * lsum[p][r] : ex2_approx(down);
      fac[p][r] = al;
      ls = add_scaled(ls, lsum[p][r], down, al);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(kFull, ls, o);
    if (lane == 0) {
      tot[0][r] = mx;
      tot[1][r] = ls;
    }
  }
  __syncthreads();
  const int items = rows * Q;
  const int groups = max(1, NT / items);
  for (int it0 = 0; it0 < items; it0 += NT) {
    const int grp = groups > 1 ? tid / items : 0, it = groups > 1 ? tid % items : it0 + tid;
    const bool live = grp < groups && it < items;
    const int r = live ? it / Q : 0, d = d0 + it % Q * 4;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live) {
#pragma unroll 8
      for (int p = grp; p < k; p += groups) {
        const float al = fac[p][r];
        const float4 v = *reinterpret_cast<const float4*>(a.part_o + (slot(p) + r) * D + d);
        if (al != 0.0f)  // (memory that no block wrote is not used)
          o = make_float4(fmaf(al, v.x, o.x), fmaf(al, v.y, o.y), fmaf(al, v.z, o.z), fmaf(al, v.w, o.w));
      }
    }
    if (groups > 1) {
      sh_o[tid] = o;
      __syncthreads();
      if (live && grp == 0) {
        for (int x = 1; x < groups; x++) {
          const float4 v = sh_o[x * items + it];
          o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
      }
    }
    if (!live || grp != 0) continue;
    const float ls = tot[1][r], inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    const int tok = r / a.G, head = h * a.G + r % a.G;
    const size_t ob = a.ob * b + a.oh * head + a.on * tok + d;
    store_o2(a, ob, o.x * inv, o.y * inv);
    store_o2(a, ob + 2, o.z * inv, o.w * inv);
    if (d == 0 && a.lse)
      a.lse[(static_cast<size_t>(b) * a.H + head) * a.Nq + tok] =
          ls == 0.0f ? -INFINITY : ls > 0.0f ? (tot[0][r] + log2f(ls)) * kLn2 : ls;
  }
}

}  // namespace

namespace {
template <int D, int NT, bool WEIGHTS>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(k_cache_decode<D, NT, WEIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(sizeof(DecSmem<D, NT>)));
}
template <int D>
cudaError_t prepare_d() {
  cudaError_t e = prepare_one<D, 1, false>();
  if (e == cudaSuccess) e = prepare_one<D, 2, false>();
  if (e == cudaSuccess) e = prepare_one<D, 1, true>();
  if constexpr (D == 64) {  // (weights of more than 8 rows at D = 128: cache_weights.cu)
    if (e == cudaSuccess) e = prepare_one<D, 2, true>();
  }
  return e;
}
template <int D, bool WEIGHTS>
cudaError_t launch_d(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  const bool one = decode_tile_rows(a.Nq, a.G) == 8;
  if constexpr (WEIGHTS && D == 128) {
    k_cache_decode<D, 1, true><<<a.chunks, Shape<1>::kWarps * 32, sizeof(DecSmem<D, 1>), s>>>(m, a);
  } else {
    if (one) k_cache_decode<D, 1, WEIGHTS><<<a.chunks, Shape<1>::kWarps * 32, sizeof(DecSmem<D, 1>), s>>>(m, a);
    else k_cache_decode<D, 2, WEIGHTS><<<a.chunks, Shape<2>::kWarps * 32, sizeof(DecSmem<D, 2>), s>>>(m, a);
  }
  cudaError_t e = cudaGetLastError();
  if (WEIGHTS || e != cudaSuccess || a.whole) return e;
  // the join starts while the last attention blocks still run and waits for
  // them on the device (programmatic dependent launch)
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const unsigned heads = static_cast<unsigned>(a.c.B) * a.c.Hkv;
  // few heads, each cut into many stretches: slices of their channels
  unsigned slices = 1;
  while (slices < 8 && 2 * slices * heads <= static_cast<unsigned>(a.chunks)) slices *= 2;
  cfg.gridDim = dim3(heads, slices);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return one ? cudaLaunchKernelEx(&cfg, k_cache_join<D, 8>, a, a.chunks)
             : cudaLaunchKernelEx(&cfg, k_cache_join<D, 16>, a, a.chunks);
}
}  // namespace

cudaError_t cache_prepare() {
  cudaError_t e = prepare_d<128>();
  if (e == cudaSuccess) e = prepare_d<64>();
  if (e == cudaSuccess) e = cache_prefill_prepare();
  if (e == cudaSuccess) e = cache_weights_prepare();
  if (e == cudaSuccess) e = cache_evict_prepare();
  return e;
}

cudaError_t launch_cache_decode(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  return a.c.D == 128 ? launch_d<128, false>(m, a, s) : launch_d<64, false>(m, a, s);
}
cudaError_t launch_cache_weights_few(const CacheAttnMaps& m, const CacheAttnArgs& a, cudaStream_t s) {
  return a.c.D == 128 ? launch_d<128, true>(m, a, s) : launch_d<64, true>(m, a, s);
}

}  // namespace sage
