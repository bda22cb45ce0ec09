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
  float c[kRows], nl[kRows];  // power of two * scale * log2(e); -lse * log2(e)
  KeyRange kr[kRows];
  uint64_t done[2];           // scores of the two key tiles
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

// A thread's chunks (16 codes) of 256 keys: chunk column c, rows row0 + i *
// STEP.  Eight neighbouring lanes take four chunks of two rows, so that their
// 16-byte stores hit eight different banks; a warp still reads whole rows.
template <int D>
struct KeyChunks {
  static constexpr int CH = D / 16, N = kKeys * CH / kThreads, STEP = kKeys / N;
  int c, row0;
  uint32_t off0, off1;
  __device__ __forceinline__ explicit KeyChunks(int tid) {
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
__device__ __forceinline__ void load_keys(uint4 (&r)[D / 16], const CacheAttnArgs& a, const int (&unit)[4],
                                          const KeyChunks<D>& ch) {
  using K = KeyChunks<D>;
#pragma unroll
  for (int p = 0; p < 4; p++) {
    const int8_t* src = a.c.k_i8 + static_cast<size_t>(max(unit[p], 0)) * (kPage * D) + ch.row0 * D + ch.c * 16;
#pragma unroll
    for (int i = 0; i < K::N / 4; i++)
      r[p * (K::N / 4) + i] = unit[p] < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                          : __ldg(reinterpret_cast<const uint4*>(src + i * K::STEP * D));
  }
}

// acc += exp2(S ks c - lse) over N query rows (columns n0 on); rows that do not
// see key j add nothing.
template <int D, int N>
__device__ __forceinline__ void add_columns(const WgtSmem<D>& s, const uint32_t (&r)[N], int n0, float2 k2,
                                            bool all, long long j, float2 (&acc)[2]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
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

template <int D>
__global__ void __launch_bounds__(kThreads, 2) k_cache_weights(const CacheAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_misaligned(raw, a.c.status)) return;
  WgtSmem<D>& s = *reinterpret_cast<WgtSmem<D>*>(raw);
  constexpr int CH = D / 16;  // chunks of a thread
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
    mbar_init(&s.done[0], 1);
    mbar_init(&s.done[1], 1);
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
  // the pass's pages, and the next one's: a pass ahead of their codes, which
  // are a pass ahead of their conversion
  int unit[4], next[4];
  units(p0, unit);
  uint4 kr[CH];
  const KeyChunks<D> ch(tid);
  load_keys<D>(kr, a, unit, ch);
  units(p0 + 4, next);

  const int tile = warp >> 2, quad = warp & 3;
  const int key = tile * 128 + quad * 32 + lane;  // of the pass
  int staged = -1;                                // row block in s.q
  uint32_t phase = 0;
  bool ok = true;    // of this warp: a wait that ran out makes it false for good
  bool live = true;  // of the block, as of its last barrier
  bool pending = false;
  for (int p = p0; p < p1 && live; p += 4) {
#pragma unroll
    for (int i = 0; i < KeyChunks<D>::N; i++) {
      const uint32_t w[4] = {kr[i].x, kr[i].y, kr[i].z, kr[i].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; j++) i8x4_to_f16(w[j], o[2 * j], o[2 * j + 1]);
      // rows 128 on are the second tile, which follows the first
      const uint32_t at = i * KeyChunks<D>::STEP < 128 ? i * KeyChunks<D>::STEP * 128
                                                      : 128 * D * 2 + (i * KeyChunks<D>::STEP - 128) * 128;
      *reinterpret_cast<uint4*>(s.k[0] + ch.off0 + at) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(s.k[0] + ch.off1 + at) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    // this thread's key
    const int mu = quad < 2 ? (tile ? unit[2] : unit[0]) : (tile ? unit[3] : unit[1]);
    const float ks = mu < 0 ? 0.0f : __ldg(a.c.k_scale + mu);
    const long long j = static_cast<long long>(p) * kPage + key;
    const int mine = mu;
    load_keys<D>(kr, a, next, ch);
#pragma unroll
    for (int i = 0; i < 4; i++) unit[i] = next[i];
    units(p + 8, next);
    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    const int first = p * kPage, last = min(len, first + kKeys);
    for (int rb = 0; rb < rows; rb += kRows) {
      const int nr = min(kRows, rows - rb), n = (nr + 15) / 16 * 16;
      // does any row of the block see any of these keys, and all see all?
      const KeyRange ra = key_range(a.mask, off + rb / a.G, len);
      const KeyRange rz = key_range(a.mask, off + (rb + nr - 1) / a.G, len);
      const bool none = first >= max(ra.sink, rz.sink) && (first >= rz.hi || last <= ra.lo);
      if (none) continue;
      const bool all = min(ra.sink, rz.sink) >= last || (rz.lo <= first && ra.hi >= last);
      if (staged != rb) {
        if (staged >= 0) __syncthreads();  // the last block's products and constants are done with
        staged = rb;
        if (tid < n) {
          float nl = -INFINITY;  // a row that saw nothing, or is not there: weight 0
          KeyRange k{0, 0, 0};
          if (tid < nr) {
            const int rr = rb + tid, tok = rr / a.G, head = h * a.G + rr % a.G;
            const float v = __ldg(a.lse_in + (static_cast<size_t>(b) * a.H + head) * a.Nq + tok);
            if (v != -INFINITY) nl = -v * kLog2e;
            k = key_range(a.mask, off + tok, len);
          }
          s.nl[tid] = nl;
          s.kr[tid] = k;
        }
        stage_rows<D, kThreads>(a, b, h, rb, rows, n, s.q, s.c, tid);
        __syncthreads();
        if (tid < n) s.c[tid] *= a.scale * kLog2e;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      live = !__syncthreads_or(!ok);
      if (!live) break;
      tc_fence_after();
      const uint32_t tmem = s.tmem_base;
      if (warp == 0) {
        const uint32_t q0 = kDescLoK | (smem_u32(s.q) >> 4), k0 = kDescLoK | (smem_u32(s.k[0]) >> 4);
        if (elect_one()) {
          mma_rows<D>(tmem, k0, q0, idesc_f16(128, n));
          mma_commit(&s.done[0]);
          if (last - first > 128) mma_rows<D>(tmem + 128, k0 + ((128 * D * 2) >> 4), q0, idesc_f16(128, n));
          mma_commit(&s.done[1]);
        }
        __syncwarp();
      }
      ok = ok && __all_sync(kFull, mbar_wait(&s.done[tile], phase, wc, kSiteWgtMma));
      phase ^= 1;
      pending = true;
      tc_fence_after();
      if (ok && tile * 128 < last - first) {
        const uint32_t tS = tmem + tile * 128 + (static_cast<uint32_t>(quad * 32) << 16);
        const float2 k2 = make_float2(ks, ks);
        // 64 columns at a time (the load's latency is paid once for them),
        // the rest in steps of 16
        int n0 = 0;
#pragma unroll 1
        for (; n0 + 64 <= n; n0 += 64) {
          uint32_t r[64];
          tmem_ld64(tS + n0, r);
          add_columns<D, 64>(s, r, n0, k2, all, j, acc);
        }
#pragma unroll 1
        for (; n0 < n; n0 += 16) {
          uint32_t r[16];
          tmem_ld16(tS + n0, r);
          add_columns<D, 16>(s, r, n0, k2, all, j, acc);
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
    live = !__syncthreads_or(!ok);
    tc_fence_after();
  }
  // Both tiles' last products are done before their shared memory and TMEM
  // go (after a wait that ran out, recorded, that takes its time once more).
  if (pending && tid == 0) {
    const long long t0 = clock64();
    while (!mbar_try_wait(&s.done[1], phase ^ 1) && clock64() - t0 < wc.budget) {
    }
  }
  __syncthreads();
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
