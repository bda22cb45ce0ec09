// cache_prefill.cu -- attention over the paged 8-bit cache for many query
// rows (prompts, latent frames): the arithmetic of cache_attn.cu on tcgen05.
//
// A block owns 256 query rows of one (sequence, key head), two tiles of 128,
// and walks KV tiles of 128 keys (two pages).  16 warps:
//   0-3, 4-7   softmax of tile 0 and 1, a thread a row: S from TMEM, running
//              maximum, y = 2^(t + e - M + 7), fp16(y) back into the TMEM
//              columns of S, where the second product reads it as operand A,
//              64 keys at a time.  M moves, and O is rescaled, only when a
//              row's maximum grew by more than 2^8 (y <= 2^15 then still fits
//              fp16), so a tile's maximum is off the path to its exponentials.
//   8-11       codes from global memory to fp16 operands in shared memory, in
//              the 128-byte swizzle the tensor core reads; K exactly, V
//              exactly, the next tile's codes already in flight in registers.
//   12         issues every tcgen05.mma: for each tile in turn O += P V of
//              one KV tile and S = Q K^T of the next, so one tile's products
//              run under the other's softmax.
// What bounds it: 4 D flops a (row, key) on the fp16 tensor pipe and one exp2
// on the MUFU take the same 2048 clocks a KV tile at D = 128.  fp16 operands
// rather than the codes' own 8-bit kinds: Q is not quantized, and an int8 or
// e4m3 product would need it (and P) in two limbs or more, the same tensor
// time without the exactness.  256 rows a block halve the conversions per
// row, which then fit the issue slots that the softmax leaves.
//
// Measured: 24 heads, 2040 rows on 26520 tokens, 128 channels, 830-857 us, 780
// to 810 TFLOP/s.  A KV tile takes some 4200 clocks: of each row tile's chain,
// softmax 2550 (the two tiles' overlap for a third of it), the slowest of its
// four warps 390 more, O += P V and the next S 820, and 250 until the S is
// seen; the products alone, issued back to back, take 2048.  Tried and slower
// or no faster: two S buffers of 64 keys a row tile (905 us: another exchange
// for every 64 keys), the two row tiles' softmax in turns (925), a share of
// the exponentials on the fma pipes (equal), single-lane issue (851).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int kThreads = 512;
constexpr int kConvert = 128;  // of these
constexpr int NS = 2;
constexpr float kBoost = 7.0f;   // y = 2^7 at the reference maximum
constexpr float kLazy = 8.0f;    // growth of the maximum that forces a rescale
constexpr int kRegsSoftmax = 184, kRegsConvert = 104, kRegsIssue = 40;
static_assert(kRegsSoftmax * 256 + kRegsConvert * 128 + kRegsIssue * 128 <= 65536,
              "register split within the launch's share");

enum : int { kSitePreKEmpty = 0x20201, kSitePreVEmpty, kSitePreK, kSitePreV, kSitePreP, kSitePreS,
             kSitePreDrain };

// A KV tile's two pages: first key (-1: no page), key scale, value exponent.
struct TileMeta {
  int j0[2];
  float ks[2];
  int ve[2];
};

template <int D>
struct alignas(1024) PreSmem {
  uint8_t q[2][BM * D * 2];   // fp16 [D / 64][128 rows][128 bytes], 128-byte swizzle
  uint8_t k[NS][BN * D * 2];  // the same over keys (K-major B operand)
  uint8_t v[NS][BN * D * 2];  // the same (MN-major B operand)
  float rowf[2 * BM];
  TileMeta meta[4];  // of KV tile it in slot it % 4
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  uint64_t s_full[2], p_full[2][2], drain;  // p_full[tile][half]: P of 64 keys
  uint32_t tmem_base;
  int abort;
};

// D[tmem] (+)= A[tmem] B[smem], f16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------- converters

// Lane l of a converter warp holds page l of the next 32 (16 KV tiles).
struct PageOf {
  int j0, unit, ve;
  float ks;
};
__device__ __forceinline__ PageOf page_of(const CacheAttnArgs& a, const PageRuns& runs, int b, int h, int i,
                                          int end) {
  PageOf p{-1, 0, 0, 0.0f};
  if (i < end) {
    const int blk = runs.page(i);
    const int pg = __ldg(a.c.pages + static_cast<size_t>(b) * a.c.max_pages + blk);
    if (static_cast<unsigned>(pg) < static_cast<unsigned>(a.c.n_pages)) {
      p.j0 = blk * kPage;
      p.unit = pg * a.c.Hkv + h;
      p.ks = __ldg(a.c.k_scale + p.unit);
      p.ve = __ldg(a.c.v_exp + p.unit);
    }
  }
  return p;
}

// A converter thread's chunks (16 codes) of a KV tile: chunk column c and rows
// row0 + i * STEP.  Eight neighbouring lanes take four chunks of two rows, so
// that their 16-byte stores hit eight different banks (rows r and r + 1 swizzle
// to the other half of the banks); a warp still reads whole rows.
template <int D>
struct Chunks {
  static constexpr int CH = D / 16, N = D / 16, STEP = BN / N;
  static_assert(N * STEP == BN && kConvert * N == BN * CH, "every chunk has its thread");
  int c, row0;
  uint32_t off0, off1;  // of chunks 2 c and 2 c + 1 of row0 in an operand tile
  __device__ __forceinline__ explicit Chunks(int tid) {
    const int lane = tid & 31, w = tid >> 5;
    if (D == 128) {
      c = (lane & 3) | ((lane >> 1) & 4);
      row0 = w * 4 + ((lane >> 2) & 1) + ((lane >> 3) & 2);
    } else {
      c = lane & 3;
      row0 = w * 8 + (lane >> 2);
    }
    off0 = op_off(row0, 2 * c);
    off1 = op_off(row0, 2 * c + 1);
  }
};
template <int D>
__device__ __forceinline__ void load_codes(uint4 (&r)[D / 16], const uint8_t* codes, const Chunks<D>& ch,
                                           const int (&unit)[2], const int (&j0)[2]) {
  constexpr int N = Chunks<D>::N, STEP = Chunks<D>::STEP;
#pragma unroll
  for (int g = 0; g < 2; g++) {
    const uint8_t* p = codes + static_cast<size_t>(unit[g]) * (kPage * D) + ch.row0 * D + ch.c * 16;
#pragma unroll
    for (int i = 0; i < N / 2; i++)
      r[g * (N / 2) + i] = j0[g] < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                     : __ldg(reinterpret_cast<const uint4*>(p + i * STEP * D));
  }
}
// 16 codes to 16 fp16 values, two chunks of a row.
template <int D, bool VALUES>
__device__ __forceinline__ void store_codes(uint8_t* tile, const uint4 (&r)[D / 16], const Chunks<D>& ch,
                                            const int (&j0)[2], int len) {
  constexpr int N = Chunks<D>::N, STEP = Chunks<D>::STEP;
#pragma unroll
  for (int i = 0; i < N; i++) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
    uint32_t o[8];
    if constexpr (VALUES) {
#pragma unroll
      for (int j = 0; j < 4; j++)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(o[2 * j]), "=r"(o[2 * j + 1]) : "r"(w[j]));
      // values behind the sequence's end may be any bytes, NaN among them
      const int g = i / (N / 2);
      if (j0[g] + kPage > len && j0[g] + ch.row0 + (i % (N / 2)) * STEP >= len) {
#pragma unroll
        for (int j = 0; j < 8; j++) o[j] = 0u;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) i8x4_to_f16(w[j], o[2 * j], o[2 * j + 1]);
    }
    *reinterpret_cast<uint4*>(tile + ch.off0 + i * STEP * 128) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(tile + ch.off1 + i * STEP * 128) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int D>
__device__ __forceinline__ void convert(PreSmem<D>& s, const CacheAttnArgs& a, const PageRuns& runs, int b,
                                        int h, int p0, int p1, int nk, int len, const WaitCtx& w) {
  constexpr uint32_t kFull = 0xffffffffu;
  const int tid = threadIdx.x & (kConvert - 1), lane = tid & 31;
  const Chunks<D> ch(tid);
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.c.k_i8);
  PageOf cur = page_of(a, runs, b, h, p0 + lane, p1);
  uint4 kr[D / 16], vr[D / 16];
  int unit[2], j0[2];
#pragma unroll
  for (int g = 0; g < 2; g++) {
    unit[g] = __shfl_sync(kFull, cur.unit, g);
    j0[g] = __shfl_sync(kFull, cur.j0, g);
  }
  load_codes<D>(kr, kc, ch, unit, j0);
  load_codes<D>(vr, a.c.v_f8, ch, unit, j0);
  for (int it = 0; it < nk; it++) {
    const int st = it % NS, at = (2 * it) & 31;
    const uint32_t ph = ((it / NS) & 1) ^ 1;
    if (it >= NS && !__all_sync(kFull, mbar_wait(&s.k_empty[st], ph, w, kSitePreKEmpty))) return;
    store_codes<D, false>(s.k[st], kr, ch, j0, len);
    // the tile's page data for the softmax.  Slot it % 4 was last read by the
    // softmax of tile it - 4, whose P went into a product issued before the
    // S of tile it - 2 that k_empty has just reported.
    if (tid < 32 && (lane & ~1) == at) {
      TileMeta& m = s.meta[it & 3];
      m.j0[lane & 1] = cur.j0;
      m.ks[lane & 1] = cur.ks;
      m.ve[lane & 1] = cur.ve;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.k_full[st]);
    int un[2], jn[2];
    if (at == 30) cur = page_of(a, runs, b, h, p0 + 2 * it + 2 + lane, p1);
#pragma unroll
    for (int g = 0; g < 2; g++) {
      un[g] = __shfl_sync(kFull, cur.unit, (at + 2 + g) & 31);
      jn[g] = __shfl_sync(kFull, cur.j0, (at + 2 + g) & 31);
    }
    load_codes<D>(kr, kc, ch, un, jn);
    if (it >= NS && !__all_sync(kFull, mbar_wait(&s.v_empty[st], ph, w, kSitePreVEmpty))) return;
    store_codes<D, true>(s.v[st], vr, ch, j0, len);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.v_full[st]);
    load_codes<D>(vr, a.c.v_f8, ch, un, jn);
#pragma unroll
    for (int g = 0; g < 2; g++) {
      unit[g] = un[g];
      j0[g] = jn[g];
    }
  }
}

// ---------------------------------------------------------------- tensor core

// O (+)= P V of 64 keys.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t tP, uint32_t tO, uint32_t v, bool first) {
  constexpr uint32_t id = idesc_f16(BM, D) | kIdescBMajorMN;
#pragma unroll
  for (int kk = 0; kk < kPage / 16; kk++)
    mma_f16_ts(tO, tP + kk * 8, desc_of(v + kk * (2048 >> 4)), id, kk > 0 ? 1u : (first ? 0u : 1u));
}

// By a whole warp, one elected lane of which issues: the waits and the
// operands' addresses then stay uniform (a single-lane branch around all of it
// took 90 clocks a product, most of them moves to uniform registers).
template <int D>
__device__ __forceinline__ void issue(PreSmem<D>& s, uint32_t tmem, int nk, int tiles, const WaitCtx& w) {
  constexpr uint32_t kFull = 0xffffffffu;
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    return __all_sync(kFull, mbar_wait(bar, parity, w, site));
  };
  const uint32_t q0 = kDescLoK | (smem_u32(s.q[0]) >> 4), k0 = kDescLoK | (smem_u32(s.k[0]) >> 4);
  const uint32_t v0 = kDescLoV | (smem_u32(s.v[0]) >> 4);
  constexpr uint32_t kTile = (BN * D * 2) >> 4, kHalf = (kPage * 128) >> 4;
  bool ok = wait(&s.k_full[0], 0, kSitePreK);
  if (ok) {
    tc_fence_after();
    if (elect_one()) {
      for (int t = 0; t < tiles; t++) {
        mma_rows<D>(tmem + t * BN, q0 + t * kTile, k0, idesc_f16(BM, BN));
        mma_commit(&s.s_full[t]);
      }
      mma_commit(&s.k_empty[0]);
    }
    __syncwarp();
  }
  for (int it = 0; ok && it < nk; it++) {
    const int st = it % NS, sn = (it + 1) % NS;
    const bool more = it + 1 < nk;
    ok = wait(&s.v_full[st], (it / NS) & 1, kSitePreV);
    for (int t = 0; ok && t < tiles; t++) {
      const uint32_t tS = tmem + t * BN, tO = tmem + 2 * BN + t * D;
      ok = wait(&s.p_full[t][0], it & 1, kSitePreP);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) issue_pv<D>(tS, tO, v0 + st * kTile, it == 0);
      __syncwarp();
      ok = wait(&s.p_full[t][1], it & 1, kSitePreP);
      if (ok && more && t == 0) ok = wait(&s.k_full[sn], ((it + 1) / NS) & 1, kSitePreK);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        issue_pv<D>(tS + 32, tO, v0 + st * kTile + kHalf, false);
        if (t == tiles - 1) mma_commit(&s.v_empty[st]);
        if (more) {
          mma_rows<D>(tS, q0 + t * kTile, k0 + sn * kTile, idesc_f16(BM, BN));
          if (t == tiles - 1) mma_commit(&s.k_empty[sn]);
        }
        mma_commit(&s.s_full[t]);  // the next S, or the finished O
      }
      __syncwarp();
    }
  }
  // everything issued completes before TMEM is freed
  if (elect_one()) {
    mma_commit(&s.drain);
    const long long t0 = clock64();
    while (!mbar_try_wait(&s.drain, 0)) {
      if (clock64() - t0 > w.budget) {
        record_timeout(w.status, kSitePreDrain);
        break;
      }
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- softmax

template <int D>
__device__ __forceinline__ void softmax(PreSmem<D>& s, const CacheAttnArgs& a, uint32_t tmem, int b, int h,
                                        int t, int r0, int r1, const PageRuns& runs, int p0, int p1, int nk,
                                        int len, long long off, int chunk, int nch, int row_tiles,
                                        const WaitCtx& w) {
  constexpr uint32_t kFull = 0xffffffffu, kNegInf = 0xFF800000u;
  const int quad = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int r = t * BM + quad * 32 + lane, row = r0 + r;
  const bool valid = row < r1;
  const uint32_t lo = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + t * BN + lo, tO = tmem + 2 * BN + t * D + lo;
  const float f = s.rowf[r] * (a.scale * kLog2e);
  // a row that is not there sees every key (its scores are 0) and is never
  // stored: masked, it would send its whole warp through the masking code
  KeyRange kr{0, 0, 0x7FFFFFFF};
  if (valid) kr = key_range(a.mask, off + row / a.G, len);
  float m = -INFINITY, l = 0.0f;
  int top_exp = kMinVExp;  // the largest value exponent so far
  bool ok = true;
  for (int it = 0; it < nk; it++) {
    ok = __all_sync(kFull, mbar_wait(&s.s_full[t], it & 1, w, kSitePreS));
    if (!ok) break;
    tc_fence_after();
    const TileMeta md = s.meta[it & 3];
    // a zero scale must not meet -inf as 0 * inf
    const float c[2] = {fmaxf(f * md.ks[0], FLT_MIN), fmaxf(f * md.ks[1], FLT_MIN)};
    const float ve[2] = {static_cast<float>(md.ve[0]), static_cast<float>(md.ve[1])};
    top_exp = max(top_exp, max(md.ve[0], md.ve[1]));
    const int fe[2] = {sum_exp(md.ve[0], top_exp), sum_exp(md.ve[1], top_exp)};
    uint32_t sv[128];
    tmem_ld128(tS, sv);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int j0 = md.j0[i];
      const bool all = j0 >= 0 && (kr.sink >= j0 + kPage || (kr.lo <= j0 && kr.hi >= j0 + kPage));
      if (!__all_sync(kFull, all)) {
        const int na = j0 < 0 ? 0 : min(max(kr.sink - j0, 0), kPage);
        const int nb = min(max(kr.lo - j0, 0), kPage);
        const int nc = j0 < 0 ? nb : min(max(kr.hi - j0, nb), kPage);
        const uint32_t nbc = static_cast<uint32_t>(nc - nb);
#pragma unroll
        for (int j = 0; j < kPage; j++)
          sv[i * 64 + j] = (j < na || static_cast<uint32_t>(j - nb) < nbc) ? sv[i * 64 + j] : kNegInf;
      }
    }
    // The exponentials of the first half start at once, against the reference
    // maximum in hand, and the tile's maximum is taken beside them (its
    // instructions fit between those of the MUFU).  Only if that has grown by
    // more than 2^8, or is the row's first, is the half done again.
    float mx[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
    float sum;
    {
      const float nm = (m == -INFINITY ? 0.0f : kBoost - m) + ve[0];
      float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      const float2 cc = make_float2(c[0], c[0]), nn = make_float2(nm, nm);
#pragma unroll
      for (int j = 0; j < 32; j++) {
        const float s0 = __uint_as_float(sv[2 * j]), s1 = __uint_as_float(sv[2 * j + 1]);
        float2 x = __ffma2_rn(make_float2(s0, s1), cc, nn);
        x.x = ex2_approx(x.x);
        x.y = ex2_approx(x.y);
        mx[0][j & 1] = fmax3(mx[0][j & 1], s0, s1);
        mx[1][j & 1] = fmax3(mx[1][j & 1], __uint_as_float(sv[64 + 2 * j]), __uint_as_float(sv[65 + 2 * j]));
        acc[j & 1] = __fadd2_rn(acc[j & 1], x);
        const __half2 y = __floats2half2_rn(x.x, x.y);
        sv[j] = *reinterpret_cast<const uint32_t*>(&y);
      }
      const float2 a2 = __fadd2_rn(acc[0], acc[1]);
      sum = a2.x + a2.y;
    }
    const float top = fmaxf(fmaf(fmaxf(mx[0][0], mx[0][1]), c[0], ve[0]),
                            fmaf(fmaxf(mx[1][0], mx[1][1]), c[1], ve[1]));
    // (a page far below the largest exponent takes its sum there, too)
    if (__any_sync(kFull, top > m + kLazy) || fe[0] != md.ve[0]) {
      const float mn = fmaxf(m, top);
      const float down = mn == m ? 0.0f : m - mn, al = ex2_approx(down);  // 0 from -inf
      // O holds the sum of the tiles before: its last product completed
      // before s_full did
      if (it > 0) {
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          tmem_ld32(tO + d, o);
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
          tmem_st32(tO + d, o);
        }
      }
      l = add_scaled(0.0f, l, down, al);
      m = mn;
      const float nm = (m == -INFINITY ? 0.0f : kBoost - m) + ve[0];
      const float nf = (m == -INFINITY ? 0.0f : kBoost - m) + static_cast<float>(fe[0]);
      sum = 0.0f;
      // S is still in TMEM; P of 32 keys takes the columns of the 16 before
#pragma unroll 1
      for (int k = 0; k < kPage; k += 32) {
        uint32_t x[32], y[16];
        tmem_ld32(tS + k, x);
#pragma unroll
        for (int e = 0; e < 32; e++) {
          const int j = md.j0[0] + k + e;
          const bool see = md.j0[0] >= 0 && (j < kr.sink || (j >= kr.lo && j < kr.hi));
          const float v = see ? ex2_approx(fmaf(__uint_as_float(x[e]), c[0], nm)) : 0.0f;
          if (fe[0] == md.ve[0]) sum += v;
          else sum += see ? ex2_approx(fmaf(__uint_as_float(x[e]), c[0], nf)) : 0.0f;
          x[e] = __float_as_uint(v);
        }
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const __half2 h2 = __floats2half2_rn(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
          y[e] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        tmem_st16(tS + k / 2, y);
      }
    } else {
      uint32_t pk[32];
#pragma unroll
      for (int j = 0; j < 32; j++) pk[j] = sv[j];
      tmem_st32(tS, pk);
    }
    l = fmaf(sum, sum_unit(fe[0]), l);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.p_full[t][0]);
    {
      const float base = m == -INFINITY ? 0.0f : kBoost - m;
      float far_sum = 0.0f;
      if (fe[1] != md.ve[1]) {
        const float nf = base + static_cast<float>(fe[1]);
#pragma unroll
        for (int j = 0; j < kPage; j++) far_sum += ex2_approx(fmaf(__uint_as_float(sv[64 + j]), c[1], nf));
      }
      float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      const float2 cc = make_float2(c[1], c[1]), nn = make_float2(base + ve[1], base + ve[1]);
      uint32_t pk[32];
#pragma unroll
      for (int j = 0; j < 32; j++) {
        float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[64 + 2 * j]), __uint_as_float(sv[65 + 2 * j])), cc, nn);
        x.x = ex2_approx(x.x);
        x.y = ex2_approx(x.y);
        acc[j & 1] = __fadd2_rn(acc[j & 1], x);
        const __half2 y = __floats2half2_rn(x.x, x.y);
        pk[j] = *reinterpret_cast<const uint32_t*>(&y);
      }
      tmem_st32(tS + 32, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.p_full[t][1]);
      const float2 a2 = __fadd2_rn(acc[0], acc[1]);
      l = fmaf(fe[1] == md.ve[1] ? a2.x + a2.y : far_sum, sum_unit(fe[1]), l);
    }
  }
  if (!ok) return;
  if (nk > 0) {
    if (!__all_sync(kFull, mbar_wait(&s.s_full[t], nk & 1, w, kSitePreS))) return;
    tc_fence_after();
  }
  if (__all_sync(kFull, !valid)) return;
  const bool part = nch > 1;
  const size_t urow = (static_cast<size_t>(b) * a.c.Hkv + h) * (static_cast<size_t>(row_tiles) * (2 * BM)) + row;
  const size_t pr = urow * a.chunks + chunk;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = row / a.G, head = h * a.G + row % a.G;
  const size_t ob = a.ob * b + a.oh * static_cast<size_t>(head) + a.on * static_cast<size_t>(tok);
  const bool vec = ((reinterpret_cast<uintptr_t>(a.o) | (a.ob * 2) | (a.oh * 2) | (a.on * 2)) & 15) == 0;
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    uint32_t o[32];
    if (nk > 0) {
      tmem_ld32(tO + d, o);
    } else {
#pragma unroll
      for (int e = 0; e < 32; e++) o[e] = 0u;
    }
    if (!valid) continue;
    if (part) {
      float4* dst = reinterpret_cast<float4*>(a.part_o + pr * D + d);
#pragma unroll
      for (int e = 0; e < 8; e++)
        dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                             __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
      continue;
    }
    uint32_t y[16];
#pragma unroll
    for (int e = 0; e < 16; e++) {
      const float x0 = __uint_as_float(o[2 * e]) * inv, x1 = __uint_as_float(o[2 * e + 1]) * inv;
      if (a.type == kTypeBf16) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(x0, x1);
        y[e] = *reinterpret_cast<const uint32_t*>(&z);
      } else {
        const __half2 z = __floats2half2_rn(x0, x1);
        y[e] = *reinterpret_cast<const uint32_t*>(&z);
      }
    }
    uint16_t* dst = static_cast<uint16_t*>(a.o) + ob + d;
    if (vec) {
#pragma unroll
      for (int e = 0; e < 4; e++)
        reinterpret_cast<uint4*>(dst)[e] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; e++) {
        dst[2 * e] = static_cast<uint16_t>(y[e]);
        dst[2 * e + 1] = static_cast<uint16_t>(y[e] >> 16);
      }
    }
  }
  if (!valid) return;
  if (part) {
    *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m - kBoost, l);
  } else if (a.lse) {
    a.lse[(static_cast<size_t>(b) * a.H + head) * a.Nq + tok] =
        l == 0.0f ? -INFINITY : l > 0.0f ? (m - kBoost + log2f(l)) * 0.69314718055994531f : l;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_cache_prefill(const CacheAttnArgs a, int row_tiles) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  PreSmem<D>& s = *reinterpret_cast<PreSmem<D>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // KV ranges fastest; row tiles from the last to the first (under a causal
  // mask the last see most)
  unsigned i = blockIdx.x;
  const int chunk = static_cast<int>(i % a.chunks);
  i /= a.chunks;
  const int h = static_cast<int>(i % a.c.Hkv);
  i /= a.c.Hkv;
  const int b = static_cast<int>(i % a.c.B);
  const int rt = row_tiles - 1 - static_cast<int>(i / a.c.B);
  const int len = seq_length(a.c, b), qn = query_len(a, b), rows = qn * a.G;
  const int r0 = rt * (2 * BM);
  if (r0 >= rows) return;
  const int r1 = min(rows, r0 + 2 * BM);
  const long long off = static_cast<long long>(len) - qn;
  const PageRuns runs = page_runs(a.mask, off + r0 / a.G, off + (r1 - 1) / a.G, len);
  const int nch = min(a.chunks, (runs.n + a.chunk_pages - 1) / a.chunk_pages);
  const int p0 = chunk * a.chunk_pages;
  const int p1 = chunk == a.chunks - 1 ? runs.n : min(runs.n, p0 + a.chunk_pages);
  if (chunk > 0 && p0 >= runs.n) return;
  const int nk = p1 > p0 ? (p1 - p0 + 1) / 2 : 0;
  const int tiles = r1 - r0 > BM ? 2 : 1;

  if (threadIdx.x == 0) {
    for (int j = 0; j < NS; j++) {
      mbar_init(&s.k_full[j], kConvert / 32);
      mbar_init(&s.k_empty[j], 1);
      mbar_init(&s.v_full[j], kConvert / 32);
      mbar_init(&s.v_empty[j], 1);
    }
    for (int j = 0; j < 2; j++) {
      mbar_init(&s.s_full[j], 1);
      mbar_init(&s.p_full[j][0], 4);
      mbar_init(&s.p_full[j][1], 4);
    }
    mbar_init(&s.drain, 1);
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  for (int t = 0; t < tiles; t++)
    stage_rows<D, kThreads>(a, b, h, r0 + t * BM, r1, BM, s.q[t], s.rowf + t * BM, threadIdx.x);
  // a page id that is none is recorded once, by the first range
  if (chunk == 0)
    for (int j = threadIdx.x; j < runs.n; j += kThreads) (void)page_id(a.c, b, runs.page(j));
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const WaitCtx w{a.budget, a.c.status, &s.abort};
  if (warp < 8) {
    set_regs_up<kRegsSoftmax>();
    const int t = warp >> 2;
    if (t < tiles)
      softmax<D>(s, a, tmem, b, h, t, r0, r1, runs, p0, p1, nk, len, off, chunk, nch, row_tiles, w);
  } else if (warp < 12) {
    set_regs_down<kRegsConvert>();
    convert<D>(s, a, runs, b, h, p0, p1, nk, len, w);
  } else {
    set_regs_down<kRegsIssue>();
    if (warp == 12 && nk > 0) issue<D>(s, tmem, nk, tiles, w);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Join of the KV ranges, the ranges in order; a block joins 16 rows of one
// tile (what they share, the tile's pages and ranges, is worked out once), a
// warp a row at a time.  A lane holds the factor of one range; the partial
// rows come four at a time, on their way before the factors are known.
// Measured: 24 heads x 2040 rows of three ranges 27 us, 76 MB, behind the
// attention and not under it (a warp a row that worked out everything for
// itself 45).
constexpr int kMergeRows = 16;
template <int D>
__global__ void __launch_bounds__(128) k_cache_merge(const CacheAttnArgs a, int row_tiles) {
  constexpr uint32_t kFull = 0xffffffffu;
  constexpr int PER = D / 32;
  static_assert(kPreRows % kMergeRows == 0, "rows of one tile");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = row_tiles * (kPreRows / kMergeRows);  // of a (sequence, key head)
  const int bh = static_cast<int>(blockIdx.x) / blocks, first = (static_cast<int>(blockIdx.x) - bh * blocks) * kMergeRows;
  const int b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
  const int len = seq_length(a.c, b), qn = query_len(a, b), rows = qn * a.G;
  const int r0 = first / kPreRows * kPreRows, r1 = min(rows, r0 + kPreRows);
  int nch = 0;
  if (first < rows) {
    const long long off = static_cast<long long>(len) - qn;
    const PageRuns runs = page_runs(a.mask, off + r0 / a.G, off + (r1 - 1) / a.G, len);
    nch = min(a.chunks, (runs.n + a.chunk_pages - 1) / a.chunk_pages);
  }
  // The attention kernel gives no signal of its own, so this kernel's blocks
  // come as its last blocks leave.  Every block waits, also one with nothing to
  // join: what comes next in the stream waits for this kernel only, so it must
  // not end before the attention has.
  cudaGridDependencySynchronize();
  if (nch <= 1) return;  // the attention kernel wrote this tile itself
  auto load = [&](const float* p, float (&v)[PER]) {
    if constexpr (PER == 4) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(p);
      v[0] = x.x, v[1] = x.y;
    }
  };
  for (int r = first + warp; r < min(r1, first + kMergeRows); r += 4) {
    const size_t row = static_cast<size_t>(bh) * row_tiles * kPreRows + r;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * a.chunks;
    const float* po = a.part_o + row * a.chunks * D + lane * PER;
    float v[4][PER];
#pragma unroll
    for (int k = 0; k < 4; k++) load(po + static_cast<size_t>(min(k, nch - 1)) * D, v[k]);
    float o[PER], ls = 0.0f, mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < PER; e++) o[e] = 0.0f;
    for (int i = lane; i < nch; i += 32) mx = fmaxf(mx, ml[i].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, x));
    for (int i0 = 0; i0 < nch; i0 += 32) {
      float al = 0.0f;
      const int mine = i0 + lane;
      if (mine < nch) {
        const float2 x = ml[mine];
        // (no maximum: nothing seen, sum 0, or NaN alone, sum NaN)
        const float down = x.x == -INFINITY ? 0.0f : x.x - mx;
        al = x.x == -INFINITY ? 0.0f * x.y : ex2_approx(down);
        ls = add_scaled(ls, x.y, down, al);
      }
      const int n = min(32, nch - i0);
#pragma unroll 1
      for (int k0 = 0; k0 < n; k0 += 4) {
        if (i0 + k0 > 0) {
#pragma unroll
          for (int k = 0; k < 4; k++) load(po + static_cast<size_t>(min(i0 + k0 + k, nch - 1)) * D, v[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float x = __shfl_sync(kFull, al, (k0 + k) & 31);
          // ranges past the end: their factor is 0, the row read in their
          // place finite
#pragma unroll
          for (int e = 0; e < PER; e++) o[e] = fmaf(k0 + k < n ? x : 0.0f, v[k][e], o[e]);
        }
      }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) ls += __shfl_xor_sync(kFull, ls, x);
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    const int tok = r / a.G, head = h * a.G + (r - tok * a.G);
    const size_t ob = a.ob * b + a.oh * head + a.on * tok + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e += 2) store_o2(a, ob + e, o[e] * inv, o[e + 1] * inv);
    if (lane == 0 && a.lse)
      a.lse[(static_cast<size_t>(b) * a.H + head) * a.Nq + tok] =
          ls == 0.0f ? -INFINITY : ls > 0.0f ? (mx + log2f(ls)) * 0.69314718055994531f : ls;
  }
}

}  // namespace

cudaError_t cache_prefill_prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_cache_prefill<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(PreSmem<128>)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cache_prefill<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(PreSmem<64>)));
  return e;
}

cudaError_t launch_cache_prefill(const CacheAttnArgs& a, cudaStream_t s) {
  const int row_tiles = (a.Nq * a.G + kPreRows - 1) / kPreRows;
  const long long units = static_cast<long long>(a.c.B) * a.c.Hkv * row_tiles;
  const unsigned grid = static_cast<unsigned>(units * a.chunks);
  if (a.c.D == 128) k_cache_prefill<128><<<grid, kThreads, sizeof(PreSmem<128>), s>>>(a, row_tiles);
  else k_cache_prefill<64><<<grid, kThreads, sizeof(PreSmem<64>), s>>>(a, row_tiles);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.chunks == 1) return e;
  // programmatic dependent launch: the merge's launch is under the attention,
  // its blocks come when every attention block has ended
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * (kPreRows / kMergeRows)));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.c.D == 128 ? cudaLaunchKernelEx(&cfg, k_cache_merge<128>, a, row_tiles)
                      : cudaLaunchKernelEx(&cfg, k_cache_merge<64>, a, row_tiles);
}

}  // namespace sage
