// rope.cu -- rotary positions of query and key heads.
//
// Pair p of a head (channels 2p, 2p + 1 interleaved, or p, p + R/2 in halves)
// at position n turns by the angle n * f_p and is scaled by an amplitude a:
//   y0 = a (x0 cos - x1 sin),  y1 = a (x0 sin + x1 cos);
// channels from R on pass through.  The inverse turns by the negative angle:
// the transposed map, i.e. the gradient of the forward one.
//
// What bounds it: x read and y written once (HBM for a clip, the launch for a
// token).  Angles need 64 bits (n * f in fp32 is off by whole radians at far
// positions), so a block computes each cos/sin once, in shared memory, and
// uses it for all its heads: the fp64 work is 1/heads of an element's.  Four
// heads' loads are on their way at once (one after another 55 us).
// Measured: a clip of 12 heads x 32760 tokens x 128 channels, half of them
// turned, 36 us, 5.6 TB/s (copy 6.5); a token of 16 x 32 heads 5.5 us, most of
// it the launch and the angles' latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"

namespace sage {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 1024;  // cos/sin pairs a block keeps (8 KB)

// cos and sin of n * f: the product and its whole turns in fp64, the
// remaining fraction of a turn (at most half) rounded to fp32 once.
__device__ __forceinline__ float2 turn(double n, double f, float amp, bool inverse) {
  double t = n * f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= rint(t);
  float s, c;
  sincospif(2.0f * static_cast<float>(t), &s, &c);
  return make_float2(c * amp, inverse ? -s * amp : s * amp);
}

__device__ __forceinline__ double position(const RopeArgs& a, int b, int n) {
  const long long i = a.pb * b + n;
  return a.pos64 ? static_cast<double>(a.pos64[i]) : static_cast<double>(a.pos32[i]);
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float2 f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ uint32_t pack(float2 f) {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};

// 16 bytes of channels as fp32 values and back.
template <typename T>
__device__ __forceinline__ void unpack16(uint4 u, float (&f)[Elem<T>::kVec]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (Elem<T>::kVec == 8) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 v = Elem<T>::unpack(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = __uint_as_float(w[i]);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&f)[Elem<T>::kVec]) {
  if constexpr (Elem<T>::kVec == 8)
    return make_uint4(Elem<T>::pack(make_float2(f[0], f[1])), Elem<T>::pack(make_float2(f[2], f[3])),
                      Elem<T>::pack(make_float2(f[4], f[5])), Elem<T>::pack(make_float2(f[6], f[7])));
  else
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}

__device__ __forceinline__ void rotate(float& x0, float& x1, float2 cs) {
  const float a = x0, b = x1;
  x0 = fmaf(a, cs.x, -(b * cs.y));
  x1 = fmaf(a, cs.y, b * cs.x);
}

// Block (token tile, head group, batch).  VEC: 16-byte accesses (every
// address and run of channels a multiple of 16 bytes), else one pair or one
// passed channel per item.
template <typename T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const RopeArgs a, int tile, int heads) {
  __shared__ float2 cs[kRopePairs];
  const int b = blockIdx.z, n0 = blockIdx.x * tile, h0 = blockIdx.y * heads;
  const int nt = min(tile, a.N - n0), nh = min(heads, a.H - h0), R2 = a.R / 2;
  for (int i = threadIdx.x; i < nt * R2; i += kRopeThreads)
    cs[i] = turn(position(a, b, n0 + i / R2), __ldg(a.inv_freq + i % R2), a.amplitude, a.inverse);
  __syncthreads();
  const T* x = static_cast<const T*>(a.x) + a.xb * b;
  T* y = static_cast<T*>(a.y) + a.yb * b;
  if constexpr (VEC) {
    constexpr int V = Elem<T>::kVec;
    // items of a token: rotated runs (half: a run of V pairs, two accesses),
    // then the passed channels
    const int nr = HALF ? R2 / V : a.R / V;
    const int per = nr + (a.D - a.R) / V;
    const int items = nt * per;
    // an item's channels are the same in every head, and so are its angles;
    // four heads' loads are in flight at once
    constexpr int U = 4;
    for (int i = threadIdx.x; i < items; i += kRopeThreads) {
      const int t = i / per, c = i - t * per;
      const bool pass = c >= nr;
      const int d = pass ? a.R + (c - nr) * V : c * V;
      constexpr int P = HALF ? V : V / 2;  // pairs of an item
      float2 w[P];
      if (!pass) {
#pragma unroll
        for (int e = 0; e < P; e++) w[e] = cs[t * R2 + (HALF ? d : d / 2) + e];
      }
      const T* xr = x + a.xh * h0 + a.xn * (n0 + t) + d;
      T* yr = y + a.yh * h0 + a.yn * (n0 + t) + d;
      for (int hi = 0; hi < nh; hi += U) {
        uint4 u[U], v[U];
#pragma unroll
        for (int k = 0; k < U; k++) {
          if (hi + k >= nh) break;
          const T* p = xr + a.xh * (hi + k);
          u[k] = *reinterpret_cast<const uint4*>(p);
          if (HALF && !pass) v[k] = *reinterpret_cast<const uint4*>(p + R2);
        }
#pragma unroll
        for (int k = 0; k < U; k++) {
          if (hi + k >= nh) break;
          T* p = yr + a.yh * (hi + k);
          if (pass) {
            *reinterpret_cast<uint4*>(p) = u[k];
            continue;
          }
          float f[V];
          unpack16<T>(u[k], f);
          if constexpr (HALF) {
            float g[V];
            unpack16<T>(v[k], g);
#pragma unroll
            for (int e = 0; e < V; e++) rotate(f[e], g[e], w[e]);
            *reinterpret_cast<uint4*>(p + R2) = pack16<T>(g);
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) rotate(f[e], f[e + 1], w[e / 2]);
          }
          *reinterpret_cast<uint4*>(p) = pack16<T>(f);
        }
      }
    }
  } else {
    const int per = R2 + a.D - a.R;
    const long long items = static_cast<long long>(nh) * nt * per;
    for (long long i = threadIdx.x; i < items; i += kRopeThreads) {
      const int hi = static_cast<int>(i / (nt * per)), j = static_cast<int>(i % (nt * per));
      const int t = j / per, c = j - t * per;
      const T* xr = x + a.xh * (h0 + hi) + a.xn * (n0 + t);
      T* yr = y + a.yh * (h0 + hi) + a.yn * (n0 + t);
      if (c >= R2) {
        yr[a.R + c - R2] = xr[a.R + c - R2];
        continue;
      }
      const int d0 = HALF ? c : 2 * c, d1 = HALF ? c + R2 : 2 * c + 1;
      float f = Elem<T>::get(xr[d0]), g = Elem<T>::get(xr[d1]);
      rotate(f, g, cs[t * R2 + c]);
      yr[d0] = Elem<T>::put(f);
      yr[d1] = Elem<T>::put(g);
    }
  }
}

__global__ void __launch_bounds__(kRopeThreads) k_rope_tables(const RopeArgs a, float* cosv, float* sinv) {
  const int R2 = a.R / 2;
  const long long total = static_cast<long long>(a.N) * R2;
  for (long long i = blockIdx.x * static_cast<long long>(kRopeThreads) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kRopeThreads) {
    const float2 t = turn(position(a, 0, static_cast<int>(i / R2)), __ldg(a.inv_freq + i % R2),
                          a.amplitude, false);
    cosv[i] = t.x;
    sinv[i] = t.y;
  }
}

template <typename T>
cudaError_t launch_type(const RopeArgs& a, bool vec, cudaStream_t s) {
  // tokens per block: as many as the cos/sin buffer holds, 16 at most; the
  // heads are cut into groups only until there is a block for every SM (every
  // group computes its angles again).  Cut until there are one, two, four
  // blocks an SM, us, R = D = 128: one token of 64 x 32 heads 8.2 : 8.2 : 10.2,
  // 4 x 100 tokens of 24 heads 8.2 : 10.2 : 12.3, 2040 tokens of 24 heads 12.3 :
  // 14.3 : 18.4, 9000 of 12 heads 20.5 : 20.5 : 24.6; fewer blocks were slower on
  // none of 13 shapes.
  const int tile = min(max(1, kRopePairs / max(1, a.R / 2)), min(a.N, 16));
  const int nb = (a.N + tile - 1) / tile;
  int groups = 1;
  while (groups < a.H && static_cast<long long>(nb) * a.B * groups < a.sms) groups *= 2;
  const int heads = (a.H + groups - 1) / groups;
  const dim3 grid(nb, (a.H + heads - 1) / heads, a.B);
  if (a.half) {
    if (vec) k_rope<T, true, true><<<grid, kRopeThreads, 0, s>>>(a, tile, heads);
    else k_rope<T, true, false><<<grid, kRopeThreads, 0, s>>>(a, tile, heads);
  } else {
    if (vec) k_rope<T, false, true><<<grid, kRopeThreads, 0, s>>>(a, tile, heads);
    else k_rope<T, false, false><<<grid, kRopeThreads, 0, s>>>(a, tile, heads);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const int size = a.type == kTypeF32 ? 4 : 2, V = 16 / size;
  const long long st = a.xb | a.xh | a.xn | a.yb | a.yh | a.yn;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) & 15u) == 0 &&
                   st % V == 0 && a.D % V == 0 && a.R % (a.half ? 2 * V : V) == 0;
  if (a.type == kTypeF32) return launch_type<float>(a, vec, s);
  if (a.type == kTypeF16) return launch_type<__half>(a, vec, s);
  return launch_type<__nv_bfloat16>(a, vec, s);
}

cudaError_t launch_rope_tables(const RopeArgs& a, float* cosv, float* sinv, cudaStream_t s) {
  const long long total = static_cast<long long>(a.N) * (a.R / 2);
  const long long blocks = (total + kRopeThreads - 1) / kRopeThreads;
  k_rope_tables<<<static_cast<int>(blocks < 2368 ? blocks : 2368), kRopeThreads, 0, s>>>(a, cosv, sinv);
  return cudaGetLastError();
}

}  // namespace sage
