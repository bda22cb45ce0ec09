// cache_weights.cu -- the attention weight that every cached key received:
//   w[key] (+)= sum over query rows of exp(s - lse),
// s the score, lse the row's log-sum-exp from the attention call.
//
// The score tile is taken transposed, S^T = K Q^T: a thread owns a key (TMEM
// lane) and adds up over the query rows (TMEM columns), so a key's sum stays
// in one register, in row order, with no atomics or exchanges between
// threads; the row's constants (power of two * scale * log2(e), lse * log2(e))
// are the same for all threads and come as broadcasts from shared memory.
// Operands as in cache_prefill.cu: int8 key codes exactly as fp16, query rows
// as fp16 with a power of two; the key scale multiplies the fp32 sum.
//
// A block of 256 threads holds 256 keys (four pages, two M = 128 tiles) and
// passes the query rows in blocks of 128; the next keys' codes are loaded
// into registers under the current ones' work, and two blocks an SM fill each
// other's waits.  What bounds it: the key codes (D bytes a key and head) for
// few rows, exp2 (16 a clock and SM) from about 64 rows on.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_dev.cuh"
#include "sm100.cuh"

namespace sage {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kRows = 128;  // query rows a pass
constexpr int kKeys = 256;  // keys a pass

enum : int { kSiteWgtMma = 0x20301 };

template <int D>
struct alignas(1024) WgtSmem {
  uint8_t k[2][128 * D * 2];  // fp16 operand tiles of 128 keys
  uint8_t q[kRows * D * 2];   // and of the query rows
  float factor[kRows];
  float c[kRows], nl[kRows];  // factor * scale * log2(e); -lse * log2(e)
  KeyRange kr[kRows];
  uint64_t done;
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

// Codes of 256 keys, 16 bytes a chunk: page p of the pass holds chunks
// [p * 64 * CH, ...), so a chunk's page is known from its index.
template <int D>
__device__ __forceinline__ void load_keys(uint4 (&r)[D / 16], const CacheAttnArgs& a, const int (&unit)[4],
                                          int tid) {
  constexpr int CH = D / 16;
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int row = tid / CH + i * (kThreads / CH), c = tid % CH;
    // kThreads / CH rows a step: 32 (D = 128) or 64 (D = 64), within one page
    const int u = unit[i * (kThreads / CH) / kPage];
    r[i] = u < 0 ? make_uint4(0u, 0u, 0u, 0u)
                 : __ldg(reinterpret_cast<const uint4*>(
                       a.c.k_i8 + (static_cast<size_t>(u) * kPage + (row & (kPage - 1))) * D + c * 16));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) k_cache_weights(const CacheAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  WgtSmem<D>& s = *reinterpret_cast<WgtSmem<D>*>(raw);
  constexpr int CH = D / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks), bh = static_cast<int>(blockIdx.x / a.chunks);
  const int b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int len = seq_length(a.c, b), qn = query_len(a, b), rows = qn * a.G;
  const int n_blk = (len + kPage - 1) / kPage;
  const int p0 = chunk * a.chunk_pages;
  // the last range takes whatever a sequence longer than announced adds
  const int p1 = chunk == a.chunks - 1 ? n_blk : min(n_blk, p0 + a.chunk_pages);
  if (p0 >= p1) return;
  const long long off = static_cast<long long>(len) - qn;
  if (tid == 0) {
    mbar_init(&s.done, 1);
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&s.tmem_base, 256);
    tmem_relinquish();
  }
  const WaitCtx wc{a.budget, a.c.status, &s.abort};
  auto units = [&](int p, int (&u)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int pg = p + i < p1 ? page_id(a.c, b, p + i) : -1;
      u[i] = pg < 0 ? -1 : pg * a.c.Hkv + h;
    }
  };
  int unit[4];
  units(p0, unit);
  uint4 kr[CH];
  load_keys<D>(kr, a, unit, tid);

  const int tile = warp >> 2, quad = warp & 3;
  const int key = tile * 128 + quad * 32 + lane;  // of the pass
  int staged = -1;                                // row block in s.q
  uint32_t phase = 0;
  bool ok = true;
  for (int p = p0; p < p1 && ok; p += 4) {
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int row = tid / CH + i * (kThreads / CH), c = tid % CH;
      const uint32_t w[4] = {kr[i].x, kr[i].y, kr[i].z, kr[i].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; j++) i8x4_to_f16(w[j], o[2 * j], o[2 * j + 1]);
      store_pair<D>(s.k[row >> 7], row & 127, c, o);
    }
    // this thread's key
    const int mu = quad < 2 ? (tile ? unit[2] : unit[0]) : (tile ? unit[3] : unit[1]);
    const float ks = mu < 0 ? 0.0f : __ldg(a.c.k_scale + mu);
    const long long j = static_cast<long long>(p) * kPage + key;
    const int mine = mu;
    units(p + 4, unit);
    load_keys<D>(kr, a, unit, tid);
    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    const int first = p * kPage, last = min(len, first + kKeys);
    for (int rb = 0; rb < rows && ok; rb += kRows) {
      const int nr = min(kRows, rows - rb), n = (nr + 15) / 16 * 16;
      // does any row of the block see any of these keys, and all see all?
      const KeyRange ra = key_range(a.mask, off + rb / a.G, len);
      const KeyRange rz = key_range(a.mask, off + (rb + nr - 1) / a.G, len);
      const bool none = first >= max(ra.sink, rz.sink) && (first >= rz.hi || last <= ra.lo);
      if (none) continue;
      const bool all = min(ra.sink, rz.sink) >= last || (rz.lo <= first && ra.hi >= last);
      if (staged != rb) {
        staged = rb;
        stage_rows<D, kThreads>(a, b, h, rb, rows, n, s.q, s.factor, tid);
        __syncthreads();
        if (tid < n) {
          float nl = -INFINITY;  // a row that saw nothing, or is not there: weight 0
          KeyRange k{0, 0, 0};
          if (tid < nr) {
            const int rr = rb + tid, tok = rr / a.G, head = h * a.G + rr % a.G;
            const float v = __ldg(a.lse_in + (static_cast<size_t>(b) * a.H + head) * a.Nq + tok);
            if (v != -INFINITY) nl = -v * kLog2e;
            k = key_range(a.mask, off + tok, len);
          }
          s.c[tid] = s.factor[tid] * (a.scale * kLog2e);
          s.nl[tid] = nl;
          s.kr[tid] = k;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      const uint32_t tmem = s.tmem_base;
      if (tid == 0) {
        mma_rows<D>(tmem, smem_u32(s.k[0]), smem_u32(s.q), idesc_f16(128, n));
        if (last - first > 128) mma_rows<D>(tmem + 128, smem_u32(s.k[1]), smem_u32(s.q), idesc_f16(128, n));
        mma_commit(&s.done);
      }
      __syncwarp();
      ok = __syncthreads_and(mbar_wait(&s.done, phase, wc, kSiteWgtMma));
      phase ^= 1;
      if (!ok) break;
      tc_fence_after();
      if (tile * 128 < last - first) {
        const uint32_t tS = tmem + tile * 128 + (static_cast<uint32_t>(quad * 32) << 16);
        const float2 k2 = make_float2(ks, ks);
#pragma unroll 1
        for (int n0 = 0; n0 < n; n0 += 16) {
          uint32_t r[16];
          tmem_ld16(tS + n0, r);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 c = *reinterpret_cast<const float4*>(s.c + n0 + e);
            const float4 nl = *reinterpret_cast<const float4*>(s.nl + n0 + e);
            float2 x = __fmul2_rn(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), k2);
            float2 y = __fmul2_rn(make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), k2);
            x = __ffma2_rn(x, make_float2(c.x, c.y), make_float2(nl.x, nl.y));
            y = __ffma2_rn(y, make_float2(c.z, c.w), make_float2(nl.z, nl.w));
            x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            if (!all) {
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
      }
    }
    if (ok && mine >= 0 && j < len) {
      const float2 t = __fadd2_rn(acc[0], acc[1]);
      float* w = a.c.weight + static_cast<size_t>(mine) * kPage + (key & (kPage - 1));
      if (a.accumulate) atomicAdd(w, t.x + t.y);  // a page may serve two sequences
      else *w = t.x + t.y;
    }
    // the operand tiles and TMEM are free again
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (!ok) {
    // a wait ran out (recorded): give the products in flight their time
    if (tid == 0) {
      const long long t0 = clock64();
      while (!mbar_try_wait(&s.done, phase ^ 1) && clock64() - t0 < wc.budget) {
      }
    }
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(s.tmem_base, 256);
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
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.c.B) * a.c.Hkv * a.chunks);
  if (a.c.D == 128) k_cache_weights<128><<<grid, kThreads, sizeof(WgtSmem<128>), s>>>(a);
  else k_cache_weights<64><<<grid, kThreads, sizeof(WgtSmem<64>), s>>>(a);
  return cudaGetLastError();
}

}  // namespace sage
