// cache_weights.cu -- the attention weight that every cached key received:
//   w[key] (+)= sum over query rows of exp(s - lse),
// s the score, lse the row's log-sum-exp from the attention call.
//
// The score tile is taken transposed, S^T = K Q^T: a thread owns a key (TMEM
// lane) and adds up over the query rows (TMEM columns), so a key's sum stays
// in one register, in row order, with no atomics or exchanges between
// threads; the rows' constants (lse * log2(e), see stage_rows_common) are the
// same for all threads and come as broadcasts from shared memory.
// Operands as in cache_prefill.cu: int8 key codes exactly as fp16, query rows
// as fp16 with a power of two; the key scale multiplies the fp32 sum.
//
// A block, one an SM, takes an equal stretch of the line of all pages (see
// cache_dev.cuh) and walks it head by head in tiles of 128 keys (two pages),
// 128 query rows at a time, 22 warps:
//   0-11    sums, four warps a tile, a thread a key; they stage the rows
//   12-19   key codes to fp16 operands, four warps a tile
//   20      issues the products into four TMEM buffers of 128 columns
//   21      copies pages, whole, into a ring of raw tiles
// so copies, conversions and products run under the sums.
//
// 40 us for two sequences of 32000 and 20988 keys, 8 heads, 32 tokens of 4
// query heads each: 350 TFLOP/s, 1.4 TB/s.  A tile takes some 1650 clocks; exp2
// (16 a clock and SM) is 1024 of them, and the sums' broadcasts, the codes'
// conversion and the products' operands share the rest of the shared memory's
// time.  A block's start and the first rows take 9 us.  704 threads leave 80
// registers each, of which the roles spill 114 bytes (96 at D = 64).  Every warp doing copies,
// products and sums in turn (two blocks an SM): 58 us, the blocks fell into
// phase and exp2 idled half the time.  Groups of summing warps: two 47 us,
// three 41, four 41; one group that converts: 47; products of 64 rows into
// eight buffers: 52.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGroups = 3;     // groups of 128 threads that sum
constexpr int kSum = kGroups * 128;
constexpr int kConvert = 128;  // threads that convert a tile, in two groups
constexpr int kMma = (kSum + 2 * kConvert) / 32;  // the warp that issues products
constexpr int kThreads = kMma * 32 + 64;
constexpr int kRows = 128;     // query rows a pass
constexpr int kKeys = 128;     // keys a tile
constexpr int NR = 5;          // raw tiles: 80 KB of a GPU's pages on their way
constexpr int NS = 3;          // operand stages
constexpr int NT = 4;          // TMEM buffers
// Tiles whose page data is kept.  Page data t is written when raw tile t - NR
// is converted, so the products of t - NR - NS are done, and the sums of
// t - NR - NS - NT.
constexpr int kMeta = 16;
static_assert(NR + NS + NT <= kMeta, "page data in use would be overwritten");

enum : int { kSiteWgtRaw = 0x20301, kSiteWgtCode, kSiteWgtEmpty, kSiteWgtK, kSiteWgtT, kSiteWgtFull, kSiteWgtDrain };

struct TileMeta {
  int unit[2];  // (page, head), or -1: no page
  float ks[2];
};

template <int D>
struct alignas(1024) WgtSmem {
  uint8_t k[NS][kKeys * D * 2];  // fp16 operand tiles
  int8_t raw[NR][kKeys * D];     // codes as they lie in the pages
  uint8_t q[kRows * D * 2];
  float c[kRows], nl[kRows];     // the row's power of two (where each has its own); -lse * log2(e)
  int power[2];                  // least and greatest
  KeyRange kr[kRows];
  TileMeta meta[kMeta];
  PlaceSmem<kThreads / 32> place;
  uint64_t r_full[NR], r_empty[NR], k_full[NS], k_empty[NS], t_full[NT], t_empty[NT], drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// acc += exp2(S k2 - lse) over N query rows (columns n0 on), k2 the key scale,
// the softmax's and the rows' power of two (OWN: each row has its own); rows
// that do not see key j add nothing.
template <int D, int N, bool OWN, bool ALL>
__device__ __forceinline__ void add_columns(const WgtSmem<D>& s, const uint32_t (&r)[N], int n0, float2 k2,
                                            int j, float2 (&acc)[2]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const float4 nl = *reinterpret_cast<const float4*>(s.nl + n0 + e);
    float2 x = make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
    float2 y = make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
    if constexpr (OWN) {
      const float4 c = *reinterpret_cast<const float4*>(s.c + n0 + e);
      x = __fmul2_rn(x, make_float2(c.x, c.y));
      y = __fmul2_rn(y, make_float2(c.z, c.w));
    }
    x = __ffma2_rn(x, k2, make_float2(nl.x, nl.y));
    y = __ffma2_rn(y, k2, make_float2(nl.z, nl.w));
    x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    if constexpr (!ALL) {
      float* f[4] = {&x.x, &x.y, &y.x, &y.y};
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const KeyRange k = s.kr[n0 + e + q];
        if (!(j < k.sink || (j >= k.lo && j < k.hi))) *f[q] = 0.0f;
      }
    }
    acc[0] = __fadd2_rn(acc[0], x);
    acc[1] = __fadd2_rn(acc[1], y);
  }
}
template <int D, bool OWN, bool ALL>
__device__ __forceinline__ float sum_rows(const WgtSmem<D>& s, uint32_t tS, int n, float k2, int j) {
  const float2 k = make_float2(k2, k2);
  float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  int n0 = 0;
#pragma unroll 1
  for (; n0 + 32 <= n; n0 += 32) {
    uint32_t r[32];
    tmem_ld32(tS + n0, r);
    add_columns<D, 32, OWN, ALL>(s, r, n0, k, j, acc);
  }
  if (n0 < n) {  // 16 more
    uint32_t r[16];
    tmem_ld16(tS + n0, r);
    add_columns<D, 16, OWN, ALL>(s, r, n0, k, j, acc);
  }
  const float2 x = __fadd2_rn(acc[0], acc[1]);
  return x.x + x.y;
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void copy_page(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Query rows as stage_rows lays them out, but with one power of two for all of
// them where their own differ by 2^12 at most: the sums then read one constant
// a row and not two (shared memory is what bounds them).  The least row's
// largest channel still lies 2^16 above the normal fp16 numbers' end, so what
// its channels lose is 2^-27 of that, below the fp32 rounding of the sum.
// Returns the power, or kOwnPowers; power[] holds {kOwnPowers, -kOwnPowers}; sync: a
// barrier of the NT threads.
constexpr int kOwnPowers = 1000, kSpread = 12;
template <int D, int NT, typename S>
__device__ __forceinline__ int stage_rows_common(const CacheAttnArgs& a, int b, int h, int r0, int rows, int n,
                                                 uint8_t* tile, float* factor, int* power, int tid, S sync) {
  constexpr int CH = D / 8, UN = (kRows * CH + NT - 1) / NT;
  long long at[UN];
  uint4 raw[UN];
#pragma unroll
  for (int u = 0; u < UN; u++) {
    const int i = tid + u * NT, r = r0 + i / CH;
    at[u] = i < n * CH && r < rows ? q8_at(a, b, h, r, i % CH) : -1;
  }
  load_q8(a, at, raw);
  int own[UN], lo = kOwnPowers, hi = -kOwnPowers;
#pragma unroll
  for (int u = 0; u < UN; u++) {
    float f[8];
    q8_floats(a, raw[u], f);
    const float m = row_max<CH>(f);
    own[u] = row_power(m);
    if (m != 0.0f) {
      lo = min(lo, own[u]);
      hi = max(hi, own[u]);
    }
  }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
  if ((tid & 31) == 0) {
    atomicMin(&power[0], lo);
    atomicMax(&power[1], hi);
  }
  sync();
  lo = power[0];
  hi = power[1];
  const int all = hi < lo ? 0 : hi - lo <= kSpread ? hi : kOwnPowers;
#pragma unroll
  for (int u = 0; u < UN; u++) {
    const int i = tid + u * NT;
    if (i >= n * CH) break;
    float f[8];
    q8_floats(a, raw[u], f);
    store_q8(tile, i / CH, i % CH, f, all == kOwnPowers ? own[u] : all);
    if (i % CH == 0) factor[i / CH] = pow2i(own[u]);
  }
  return all;
}

// What a pass (a head's pages, 128 query rows) is about.
struct Pass {
  int b, h, len, p0, p1;
  long long off;  // position of token 0
  int rb, nr, n;  // first row, rows, rows rounded up to 16
  KeyRange ra, rz;  // of the first and the last row
  __device__ __forceinline__ int tiles() const { return (p1 - p0 + 1) / 2; }
  __device__ __forceinline__ int first(int i) const { return (p0 + 2 * i) * kPage; }
  __device__ __forceinline__ int last(int i) const { return min(len, min(p1, p0 + 2 * i + 2) * kPage); }
  // no row sees a key of tile i / all see all
  __device__ __forceinline__ bool none(int i) const {
    return n == 0 || (first(i) >= max(ra.sink, rz.sink) && (first(i) >= rz.hi || last(i) <= ra.lo));
  }
  __device__ __forceinline__ bool all(int i) const {
    return min(ra.sink, rz.sink) >= last(i) || (rz.lo <= first(i) && ra.hi >= last(i));
  }
  // the next tile from i on that some row sees
  __device__ __forceinline__ int next(int i) const {
    while (i < tiles() && none(i)) i++;
    return i;
  }
};

// The passes of this block's stretch, in the order that every role walks them.
template <typename F>
__device__ __forceinline__ void each_pass(const CacheAttnArgs& a, const Place& pl, F f) {
  long long x = share_start(pl.work, blockIdx.x, gridDim.x);
  const long long end = share_start(pl.work, blockIdx.x + 1, gridDim.x);
  long long before = pl.before;
  Pass p;
  for (int b = pl.b; x < end && b < a.c.B; b++) {
    const int len = seq_length(a.c, b), np = (len + kPage - 1) / kPage;
    if (np == 0) continue;
    const int qn = query_len(a, b), rows = qn * a.G;
    p.b = b;
    p.len = len;
    p.off = static_cast<long long>(len) - qn;
    for (long long rel = x - before * a.c.Hkv; x < end && rel < static_cast<long long>(np) * a.c.Hkv;) {
      p.h = static_cast<int>(rel / np);
      p.p0 = static_cast<int>(rel - static_cast<long long>(p.h) * np);
      p.p1 = static_cast<int>(min(static_cast<long long>(np), p.p0 + (end - x)));
      p.rb = 0;
      do {  // (no query rows: one pass, which writes zeros)
        p.nr = min(kRows, rows - p.rb);
        p.n = (p.nr + 15) / 16 * 16;
        p.ra = key_range(a.mask, p.off + p.rb / a.G, len);
        p.rz = key_range(a.mask, p.off + max(p.rb + p.nr - 1, 0) / a.G, len);
        f(p);
        p.rb += kRows;
      } while (p.rb < rows);
      x += p.p1 - p.p0;
      rel += p.p1 - p.p0;
    }
    before += np;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_cache_weights(const CacheAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  WgtSmem<D>& s = *reinterpret_cast<WgtSmem<D>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NR; i++) {
      mbar_init(&s.r_full[i], 1);
      mbar_init(&s.r_empty[i], kConvert / 32);
    }
    for (int i = 0; i < NS; i++) {
      mbar_init(&s.k_full[i], kConvert / 32);
      mbar_init(&s.k_empty[i], 1);
    }
    for (int i = 0; i < NT; i++) {
      mbar_init(&s.t_full[i], 1);
      mbar_init(&s.t_empty[i], 4);
    }
    mbar_init(&s.drain, 1);
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&s.tmem_base, NT * kRows);
    tmem_relinquish();
  }
  tc_fence_before();
  // (locate's barriers also publish these)
  const Place pl = locate<kThreads / 32, true>(
      s.place, a, [&](long long w) { return share_start(w, blockIdx.x, gridDim.x); });
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const WaitCtx wc{a.budget, a.c.status, &s.abort};
  auto wait = [&](uint64_t* bar, int phase, int site) {
    return static_cast<bool>(__all_sync(kFull, mbar_wait(bar, phase & 1, wc, site)));
  };
  // The budget of what is waited for at the end, whatever the waits before
  // came to: nothing may be on its way when shared memory and TMEM go.
  auto drain = [&](uint64_t* bar, int phase) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, phase & 1)) {
      if (clock64() - t0 > wc.budget) {
        record_timeout(wc.status, kSiteWgtDrain);
        break;
      }
    }
  };
  int t = 0;       // tile: its ring slots and phases follow
  bool ok = true;  // of the warp; after a wait that ran out it still meets the barriers

  if (warp >= kMma) {
    if (warp == kMma) {
      const uint32_t q0 = kDescLoK | (smem_u32(s.q) >> 4), k0 = kDescLoK | (smem_u32(s.k[0]) >> 4);
      each_pass(a, pl, [&](const Pass& p) {
        const int n_tiles = p.tiles();
        bar_sync(1, kSum + 32);  // the rows are staged
        for (int i = p.next(0); ok && i < n_tiles; i = p.next(i + 1), t++) {
          const int st = t % NS, buf = t % NT;
          if (!wait(&s.k_full[st], t / NS, kSiteWgtK) || (t >= NT && !wait(&s.t_empty[buf], t / NT - 1, kSiteWgtT))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            mma_rows<D>(tmem + buf * kRows, k0 + st * ((kKeys * D * 2) >> 4), q0, idesc_f16(128, p.n));
            mma_commit(&s.k_empty[st]);
            mma_commit(&s.t_full[buf]);
          }
          __syncwarp();
        }
      });
      if (elect_one()) {
        mma_commit(&s.drain);
        drain(&s.drain, 0);
      }
      __syncwarp();
    } else if (warp == kMma + 1) {
      each_pass(a, pl, [&](const Pass& p) {
        int base = 0, unit = -1;
        float ks = 0.0f;
        const int n_tiles = p.tiles();
        bool fresh = true;
        for (int i = p.next(0); ok && i < n_tiles; i = p.next(i + 1), t++) {
          const int pg = p.p0 + 2 * i;
          if (fresh || pg - base >= 32) {  // lane l holds page base + l
            base = pg;
            fresh = false;
            unit = -1;
            ks = 0.0f;
            const int id = base + lane < p.p1 ? page_id(a.c, p.b, base + lane) : -1;
            if (id >= 0) {
              unit = id * a.c.Hkv + p.h;
              ks = __ldg(a.c.k_scale + unit);
            }
          }
          const int st = t % NR, at = pg - base;
          if (t >= NR && !wait(&s.r_empty[st], t / NR - 1, kSiteWgtRaw)) {
            ok = false;
            break;
          }
          const bool mine = lane == at || lane == at + 1;
          if (mine) {
            s.meta[t % kMeta].unit[lane - at] = unit;
            s.meta[t % kMeta].ks[lane - at] = ks;
          }
          const uint32_t has = __ballot_sync(kFull, mine && unit >= 0);
          __syncwarp();  // both pages' data before the arrival that publishes it
          if (lane == at) mbar_arrive_expect_tx(&s.r_full[st], __popc(has) * (kPage * D));
          __syncwarp();  // the copies' bytes are expected before the copies
          if (mine && unit >= 0)
            copy_page(s.raw[st] + (lane - at) * (kPage * D), a.c.k_i8 + static_cast<size_t>(unit) * (kPage * D),
                      kPage * D, &s.r_full[st]);
        }
      });
      for (int u = max(0, t - NR); u < t; u++) drain(&s.r_full[u % NR], u / NR);
    }
  } else if (warp >= kSum / 32) {
    // Chunks of 8 codes, in the pages' order: loads and stores meet no bank
    // twice.  A step of 128 chunks is 8 or 16 keys, so the swizzle is the same.
    constexpr int CH = D / 8, STEP = kConvert / CH, N = kKeys / STEP;
    const int e = tid & (kConvert - 1), wg = (tid - kSum) / kConvert;
    const uint32_t dst = op_off(e / CH, e % CH);
    each_pass(a, pl, [&](const Pass& p) {
      const int n_tiles = p.tiles();
      for (int i = p.next(0); ok && i < n_tiles; i = p.next(i + 1), t++) {
        if ((t & 1) != wg) continue;
        const int sr = t % NR, st = t % NS;
        if (!wait(&s.r_full[sr], t / NR, kSiteWgtCode) ||
            (t >= NS && !wait(&s.k_empty[st], t / NS - 1, kSiteWgtEmpty))) {
          ok = false;
          break;
        }
        const TileMeta& m = s.meta[t % kMeta];
        const bool have[2] = {m.unit[0] >= 0, m.unit[1] >= 0};
        const uint8_t* src = reinterpret_cast<const uint8_t*>(s.raw[sr]) + e * 8;
#pragma unroll
        for (int k = 0; k < N; k++) {
          uint2 v = *reinterpret_cast<const uint2*>(src + k * (kConvert * 8));
          if (!have[k / (N / 2)]) v = make_uint2(0u, 0u);
          uint4 o;
          i8x4_to_f16(v.x, o.x, o.y);
          i8x4_to_f16(v.y, o.z, o.w);
          *reinterpret_cast<uint4*>(s.k[st] + dst + k * STEP * 128) = o;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.r_empty[sr]);
          mbar_arrive(&s.k_full[st]);
        }
      }
    });
  } else {
    const int wg = warp >> 2, quad = warp & 3, key = quad * 32 + lane, g = quad >> 1;
    each_pass(a, pl, [&](const Pass& p) {
      const int n_tiles = p.tiles();
      if (tid < 2) s.power[tid] = tid ? -kOwnPowers : kOwnPowers;
      bar_sync(2, kSum);  // all products and sums with the last rows are done
      float lse = -INFINITY;  // of a row that saw nothing, or is not there: weight 0
      KeyRange k{0, 0, 0};
      if (tid < p.nr) {
        const int rr = p.rb + tid, tok = rr / a.G, head = p.h * a.G + (rr - tok * a.G);
        lse = __ldg(a.lse_in + (static_cast<size_t>(p.b) * a.H + head) * a.Nq + tok);
        k = key_range(a.mask, p.off + tok, p.len);
      }
      const int power = stage_rows_common<D, kSum>(a, p.b, p.h, p.rb, p.rb + p.nr, p.n, s.q, s.c, s.power, tid,
                                                   [] { bar_sync(2, kSum); });
      const bool own = power == kOwnPowers;
      const float common = own ? 1.0f : pow2i(power);
      if (tid < p.n) {
        s.nl[tid] = lse == -INFINITY ? lse : -lse * kLog2e;
        s.kr[tid] = k;
      }
      fence_proxy_async_smem();
      bar_sync(1, kSum + 32);
      for (int j = 0; ok && j < n_tiles; j++) {
        const bool none = p.none(j);
        const int mine = t;
        if (!none) t++;
        // tiles that no row sees go to the groups in turn, too
        if (none ? j % kGroups != wg || p.rb > 0 || a.accumulate : mine % kGroups != wg) continue;
        const int at = p.first(j) + key;  // key index
        float sum = 0.0f;
        int unit = -1;
        if (none) {
          const int blk = p.p0 + 2 * j + g;
          const int pg = blk < p.p1 ? page_id(a.c, p.b, blk) : -1;
          unit = pg < 0 ? -1 : pg * a.c.Hkv + p.h;
        } else {
          const int buf = mine % NT;
          const uint32_t tS = tmem + buf * kRows + (static_cast<uint32_t>(quad * 32) << 16);
          const bool all = p.all(j);
          if (!wait(&s.t_full[buf], mine / NT, kSiteWgtFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const TileMeta& m = s.meta[mine % kMeta];
          unit = m.unit[g];
          const float k2 = m.ks[g] * (a.scale * kLog2e) * common;
          // (the masked forms are rare: a tile or two of a causal call)
          if (own) sum = all ? sum_rows<D, true, true>(s, tS, p.n, k2, at) : sum_rows<D, true, false>(s, tS, p.n, k2, at);
          else sum = all ? sum_rows<D, false, true>(s, tS, p.n, k2, at) : sum_rows<D, false, false>(s, tS, p.n, k2, at);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.t_empty[buf]);
        }
        if (unit >= 0 && at < p.len) {
          float* w = a.c.weight + static_cast<size_t>(unit) * kPage + (key & (kPage - 1));
          if (a.accumulate || p.rb > 0) atomicAdd(w, sum);  // a page may serve two sequences
          else *w = sum;
        }
      }
    });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, NT * kRows);
  }
}

}  // namespace

cudaError_t cache_weights_prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_cache_weights<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(WgtSmem<128>)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cache_weights<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(WgtSmem<64>)));
  return e;
}

cudaError_t launch_cache_weights(const CacheAttnArgs& a, cudaStream_t s) {
  if (a.c.D == 128) k_cache_weights<128><<<a.chunks, kThreads, sizeof(WgtSmem<128>), s>>>(a);
  else k_cache_weights<64><<<a.chunks, kThreads, sizeof(WgtSmem<64>), s>>>(a);
  return cudaGetLastError();
}

}  // namespace sage
