// api_cache.cu -- C ABI of the rotary positions and the paged 8-bit cache
// (include/sage.h): argument checks and launches.  As in api.cu nothing
// allocates device memory, nothing throws, and every error that the host can
// see is returned before anything is enqueued.
#include <algorithm>
#include <cmath>

#include "api.cuh"
#include "cache.cuh"
#include "sage.h"

#define SAGE_EXPORT extern "C" __attribute__((visibility("default")))

using namespace sage;

namespace {

bool al(const void* p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sage_status status_of(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

bool cache_ok(const sage_kv_cache* c) {
  return c && al(c->k_i8, 16) && al(c->v_f8, 16) && al(c->k_scale, 4) && c->v_exp &&
         (!c->weight || al(c->weight, 16)) && c->n_pages >= 1 && c->heads >= 1 && c->heads <= 65535 &&
         (c->D == 64 || c->D == 128);
}
bool seqs_ok(const sage_kv_seqs* s) {
  return s && al(s->pages, 4) && al(s->lengths, 4) && s->B >= 1 && s->B <= 65535 && s->max_pages >= 1 &&
         s->max_pages <= (1 << 24);
}
// Tiles of the TMA maps and (page, head) units are counted in 32 bits.
bool cache_fits(const sage_kv_cache* c) {
  return static_cast<long long>(c->n_pages) * c->heads <= (1ll << 30);
}
CacheView view_of(const sage_kv_cache* c, const sage_kv_seqs* s, int* status) {
  CacheView v{};
  v.k_i8 = c->k_i8;
  v.k_scale = c->k_scale;
  v.v_f8 = c->v_f8;
  v.v_exp = c->v_exp;
  v.weight = c->weight;
  v.n_pages = c->n_pages;
  v.Hkv = c->heads;
  v.D = c->D;
  v.pages = s->pages;
  v.lengths = s->lengths;
  v.B = s->B;
  v.max_pages = s->max_pages;
  v.status = status;
  return v;
}

bool strides_ok(const long long st[3]) { return st && st[0] >= 0 && st[1] >= 0 && st[2] >= 0; }

sage_status mask_of(int mask, int block, int win, int sink, CacheMask* m) {
  if (mask < 0 || mask > 3) return SAGE_ERR_INVALID_ARG;
  if (mask >= 2 && block < 1) return SAGE_ERR_INVALID_ARG;
  if (mask == 3 && (win < 1 || sink < 0)) return SAGE_ERR_INVALID_ARG;
  *m = CacheMask{mask, mask >= 2 ? block : 1, mask == 3 ? win : 1, mask == 3 ? sink : 0};
  return SAGE_OK;
}

// How an attention call is cut, and the floats of its partial results.
struct Plan {
  bool prefill;  // tcgen05 kernel, else the mma.sync one
  int chunk_pages, chunks, whole;
  long long blocks;
  size_t rows;   // of partial results
  size_t ws;
};
// Pages that one query tile of `tile_tokens` tokens visits at most.
int visited_pages(const CacheMask& m, int max_len, int tile_tokens) {
  const long long pages = (static_cast<long long>(max_len) + kPage - 1) / kPage;
  if (m.mode != 3) return static_cast<int>(pages);
  const long long win = static_cast<long long>(m.win) * m.block + m.block + tile_tokens;
  return static_cast<int>(std::min(pages, (m.sink + kPage - 1ll) / kPage + win / kPage + 3));
}
// Blocks that share `pages` pages of every head: two an SM, with eight pages
// (four tiles a warp) each at least.  Or, `whole`, a block a head: no look-up
// of its place and no join, but the heads of the last round walk their pages
// alone, 0.32 us each.  Whole against shared, us, at 4 x 128 query heads:
//   8 heads     1000 tokens 18 : 20   2000 23 : 20   4000  33 :  26
//   128 heads   1000 tokens 21 : 28   4000 41 : 48
//   512 heads   1000 tokens 46 : 50   4000 106 : 118 (of uneven lengths 83 : 89)
// The bounds, whole against shared from a cold L2 (in brackets a warm one):
//   24 pages, 8 heads      18 : 18 (18 : 17), 28 pages 21 : 23 (21 : 22), 32
//                          pages 23 : 18 (23 : 17)
//   64 pages, heads of the last round (of 296), one round:
//     72   37 : 39 (35 : 31)    96   39 : 43 (37 : 34)   104   39 : 45 (36 : 36)
//   two rounds:
//     72  100 : 96 (90 : 82)    96  102 : 102 (90 : 85)  104  102 : 104 (90 : 87)
// and past 64 pages one long sequence among short ones would cost more than
// there is to gain.  (The weights have no join to save: 128 heads of 8000
// tokens 39 us whole, 34 shared; equal at 1000.)
void plan_decode(long long units, int pages, int sms, bool join, int* chunks, int* whole) {
  const long long slots = std::min<long long>(2ll * sms, kMaxShares);
  *whole = pages <= 8 || (join && (pages <= 24 || (pages <= 64 && (units - 1) % slots + 1 >= slots / 3)));
  *chunks = static_cast<int>(*whole ? units : std::min(slots, (units * pages + 7) / 8));
}

Plan plan_of(const CacheMask& m, int B, int Hkv, int G, int Nq, int D, int max_len, int sms) {
  Plan p{};
  const long long qrows = static_cast<long long>(Nq) * G;
  // (16 rows of 16 x 8 heads of 8000 tokens: 122 us against 156 on tcgen05's
  // 256-row tiles, 73 against 115 with 64 channels)
  p.prefill = qrows > kDecRows;
  if (!p.prefill) {
    const long long units = static_cast<long long>(B) * Hkv;
    plan_decode(units, visited_pages(m, max_len, Nq), sms, true, &p.chunks, &p.whole);
    p.blocks = p.chunks;
    p.rows = p.whole ? 0 : 2ull * p.chunks * decode_tile_rows(Nq, G);
  } else {
    const int row_tiles = static_cast<int>((qrows + kPreRows - 1) / kPreRows);
    const long long units = static_cast<long long>(B) * Hkv * row_tiles;
    const int pages = visited_pages(m, max_len, (kPreRows + G - 1) / G + 1);
    // one block an SM: the fewest ranges whose last round of blocks leaves at
    // most a tenth of the SMs' time unused, of 16 pages at least (24 heads, 2040
    // rows on 26520 tokens: three ranges 798 us, one 1032; 8 heads, 256 rows: 67
    // against 526)
    long long cp = std::max(4, pages);
    double best = 0.0;
    for (long long n = 1; n <= 64 && (n == 1 || pages / n >= 16); n++) {
      const double rounds = static_cast<double>(units * n) / sms;
      const double used = rounds / std::ceil(rounds);
      if (used > best + 1e-9) {
        best = used;
        cp = ((pages + n - 1) / n + 1) / 2 * 2;
      }
      if (used >= 0.9) break;
    }
    p.chunk_pages = static_cast<int>(std::max(4ll, cp));
    p.chunks = static_cast<int>(std::max(1ll, (pages + p.chunk_pages - 1ll) / p.chunk_pages));
    p.blocks = units * p.chunks;
    p.rows = p.chunks > 1 ? static_cast<size_t>(units) * kPreRows * p.chunks : 0;
  }
  p.ws = p.rows * (static_cast<size_t>(D) + 2) * 4;
  return p;
}
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

bool attn_shape_ok(const sage_kv_cache* c, const sage_kv_seqs* s, int H, int Nq, int max_len) {
  if (H < 0 || H % c->heads || Nq < 0 || Nq > (1 << 24)) return false;
  if (max_len < 0 || max_len > static_cast<long long>(s->max_pages) * kPage) return false;
  return static_cast<long long>(H / c->heads) * Nq <= (1 << 28);
}

bool maps_of(const sage_kv_cache* c, CacheAttnMaps* m) {
  const uint64_t tiles = static_cast<uint64_t>(c->n_pages) * c->heads;
  return api_tile_map(&m->k, c->k_i8, kPage, tiles, c->D, kPage / 2) &&
         api_tile_map(&m->v, c->v_f8, kPage, tiles, c->D, kPage / 2);
}

// A query without rows: the weights' sum over none of them is zero.
bool no_rows(const sage_kv_query* q) { return q->H == 0 || q->Nq == 0; }

sage_status attn_common(const sage_kv_cache* c, const sage_kv_seqs* s, const sage_kv_query* q, int mask,
                        int mask_block, int win, int sink, CacheAttnArgs* a) {
  if (!cache_ok(c) || !seqs_ok(s) || !q) return SAGE_ERR_INVALID_ARG;
  if (!attn_shape_ok(c, s, q->H, q->Nq, q->max_len)) return SAGE_ERR_INVALID_ARG;
  if (q->type != kTypeBf16 && q->type != kTypeF16) return SAGE_ERR_INVALID_ARG;
  if ((!no_rows(q) && !al(q->q, 2)) || !strides_ok(q->q_strides) || (q->q_lens && !al(q->q_lens, 4)))
    return SAGE_ERR_INVALID_ARG;
  if (!std::isfinite(q->scale) || q->scale < 0.0f) return SAGE_ERR_INVALID_ARG;
  const sage_status st = mask_of(mask, mask_block, win, sink, &a->mask);
  if (st != SAGE_OK) return st;
  // (the join of a decode call has a block for every head)
  if (!cache_fits(c) || static_cast<long long>(s->B) * c->heads > (1ll << 31) - 1) return SAGE_ERR_UNSUPPORTED;
  int* status = api_status_word();
  if (!status) return SAGE_ERR_CUDA;
  a->c = view_of(c, s, status);
  a->q = q->q;
  a->type = q->type;
  a->H = q->H;
  a->G = q->H / c->heads;
  a->Nq = q->Nq;
  a->qb = q->q_strides[0];
  a->qh = q->q_strides[1];
  a->qn = q->q_strides[2];
  a->q_vec = al(q->q, 16) && ((a->qb | a->qh | a->qn) & 7) == 0;
  a->q_lens = q->q_lens;
  a->scale = q->scale;
  a->budget = api_wait_budget();
  return SAGE_OK;
}

}  // namespace

// ---------------------------------------------------------------- rotary positions

SAGE_EXPORT sage_status sage_rope(const void* x, void* y, int type, int B, int H, int N, int D, int R,
                                  const long long x_strides[3], const long long y_strides[3],
                                  const void* positions, int positions_64, long long positions_stride,
                                  const double* inv_freq, float amplitude, int half, int inverse,
                                  void* stream) {
  if (type < kTypeBf16 || type > kTypeF32) return SAGE_ERR_INVALID_ARG;
  const uintptr_t es = type == kTypeF32 ? 4 : 2;
  if (B < 1 || H < 1 || N < 1 || D < 1 || R < 0 || R > D || (R & 1)) return SAGE_ERR_INVALID_ARG;
  if (B > 65535 || H > 65535 || N > (1 << 30)) return SAGE_ERR_INVALID_ARG;
  if (!al(x, es) || !al(y, es) || !strides_ok(x_strides) || !strides_ok(y_strides))
    return SAGE_ERR_INVALID_ARG;
  if (!al(positions, positions_64 ? 8 : 4) || positions_stride < 0 || (R > 0 && !al(inv_freq, 8)))
    return SAGE_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return SAGE_ERR_INVALID_ARG;
  if (R > 2048 || D > 65536) return SAGE_ERR_UNSUPPORTED;
  if (!api_status_word()) return SAGE_ERR_CUDA;
  RopeArgs a{};
  a.x = x;
  a.y = y;
  a.type = type;
  a.B = B;
  a.H = H;
  a.N = N;
  a.D = D;
  a.R = R;
  a.xb = x_strides[0];
  a.xh = x_strides[1];
  a.xn = x_strides[2];
  a.yb = y_strides[0];
  a.yh = y_strides[1];
  a.yn = y_strides[2];
  (positions_64 ? reinterpret_cast<const void*&>(a.pos64) : reinterpret_cast<const void*&>(a.pos32)) =
      positions;
  a.pb = positions_stride;
  a.inv_freq = inv_freq;
  a.amplitude = amplitude;
  a.half = half != 0;
  a.inverse = inverse != 0;
  a.sms = sm_count();
  if (!a.sms) return SAGE_ERR_CUDA;
  return status_of(launch_rope(a, static_cast<cudaStream_t>(stream)));
}

SAGE_EXPORT sage_status sage_rope_tables(int N, int R, const void* positions, int positions_64,
                                         const double* inv_freq, float amplitude, float* cosv,
                                         float* sinv, void* stream) {
  if (N < 1 || N > (1 << 30) || R < 2 || (R & 1) || R > 65536) return SAGE_ERR_INVALID_ARG;
  if (!al(positions, positions_64 ? 8 : 4) || !al(inv_freq, 8) || !al(cosv, 4) || !al(sinv, 4))
    return SAGE_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return SAGE_ERR_INVALID_ARG;
  if (!api_status_word()) return SAGE_ERR_CUDA;
  RopeArgs a{};
  a.N = N;
  a.R = R;
  if (positions_64) a.pos64 = static_cast<const long long*>(positions);
  else a.pos32 = static_cast<const int*>(positions);
  a.inv_freq = inv_freq;
  a.amplitude = amplitude;
  return status_of(launch_rope_tables(a, cosv, sinv, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- cache

SAGE_EXPORT sage_status sage_cache_append(const sage_kv_cache* cache, const sage_kv_seqs* seqs, const void* k,
                                          const void* v, int type, int n, const long long k_strides[3],
                                          const long long v_strides[3], const int32_t* n_new,
                                          const float* k_shift, void* stream) {
  if (!cache_ok(cache) || !seqs_ok(seqs)) return SAGE_ERR_INVALID_ARG;
  if (type != kTypeBf16 && type != kTypeF16) return SAGE_ERR_INVALID_ARG;
  if (n < 1 || n > (1 << 28) || !al(k, 2) || !al(v, 2) || !strides_ok(k_strides) || !strides_ok(v_strides))
    return SAGE_ERR_INVALID_ARG;
  if ((n_new && !al(n_new, 4)) || (k_shift && !al(k_shift, 4))) return SAGE_ERR_INVALID_ARG;
  if (!cache_fits(cache)) return SAGE_ERR_UNSUPPORTED;
  int* status = api_status_word();
  if (!status) return SAGE_ERR_CUDA;
  AppendArgs a{};
  a.c = view_of(cache, seqs, status);
  a.k = k;
  a.v = v;
  a.type = type;
  a.n = n;
  a.kb = k_strides[0];
  a.kh = k_strides[1];
  a.kn = k_strides[2];
  a.vb = v_strides[0];
  a.vh = v_strides[1];
  a.vn = v_strides[2];
  a.n_new = n_new;
  a.k_shift = k_shift;
  return status_of(launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

SAGE_EXPORT sage_status sage_cache_read(const sage_kv_cache* cache, const sage_kv_seqs* seqs, int n,
                                        const int32_t* starts, const float* k_shift, float* k, float* v,
                                        float* weight, void* stream) {
  if (!cache_ok(cache) || !seqs_ok(seqs) || n < 1 || n > (1 << 30)) return SAGE_ERR_INVALID_ARG;
  if (!al(k, 16) || !al(v, 16) || (starts && !al(starts, 4)) || (k_shift && !al(k_shift, 16)))
    return SAGE_ERR_INVALID_ARG;
  if (weight && (!al(weight, 4) || !cache->weight)) return SAGE_ERR_INVALID_ARG;
  if (!cache_fits(cache)) return SAGE_ERR_UNSUPPORTED;
  int* status = api_status_word();
  if (!status) return SAGE_ERR_CUDA;
  ReadArgs a{};
  a.c = view_of(cache, seqs, status);
  a.starts = starts;
  a.n = n;
  a.k_shift = k_shift;
  a.k = k;
  a.v = v;
  a.w = weight;
  return status_of(launch_cache_read(a, static_cast<cudaStream_t>(stream)));
}

SAGE_EXPORT size_t sage_cache_attn_workspace_bytes(int B, int heads, int H, int Nq, int D, int max_len,
                                                   int mask, int mask_block, int win, int sink) {
  CacheMask m;
  if (B < 1 || B > 65535 || heads < 1 || heads > 65535 || H < 1 || H % heads || Nq < 1 || Nq > (1 << 24) ||
      static_cast<long long>(H / heads) * Nq > (1 << 28) || (D != 64 && D != 128) || max_len < 0 ||
      max_len > (1 << 30) || mask_of(mask, mask_block, win, sink, &m) != SAGE_OK)
    return 0;
  const int sms = sm_count();
  if (!sms) return 0;
  return std::max<size_t>(16, plan_of(m, B, heads, H / heads, Nq, D, max_len, sms).ws);
}

SAGE_EXPORT sage_status sage_cache_attn(const sage_kv_cache* cache, const sage_kv_seqs* seqs,
                                        const sage_kv_query* query, int mask, int mask_block, int win,
                                        int sink, void* out, const long long o_strides[3], float* lse,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!al(out, 2) || !strides_ok(o_strides) || (lse && !al(lse, 4))) return SAGE_ERR_INVALID_ARG;
  if (!query || no_rows(query)) return SAGE_ERR_INVALID_ARG;
  CacheAttnArgs a{};
  const sage_status st = attn_common(cache, seqs, query, mask, mask_block, win, sink, &a);
  if (st != SAGE_OK) return st;
  const int sms = sm_count();
  if (!sms) return SAGE_ERR_CUDA;
  const Plan p = plan_of(a.mask, seqs->B, cache->heads, a.G, a.Nq, cache->D, query->max_len, sms);
  if (p.blocks > (1ll << 31) - 1) return SAGE_ERR_UNSUPPORTED;
  if (p.ws && (!al(workspace, 16) || workspace_bytes < p.ws)) return SAGE_ERR_INVALID_ARG;
  a.o = out;
  a.ob = o_strides[0];
  a.oh = o_strides[1];
  a.on = o_strides[2];
  a.lse = lse;
  a.chunk_pages = p.chunk_pages;
  a.chunks = p.chunks;
  a.part_o = static_cast<float*>(workspace);
  a.whole = p.whole;
  a.part_ml = a.part_o + p.rows * cache->D;
  if (p.prefill) return status_of(launch_cache_prefill(a, static_cast<cudaStream_t>(stream)));
  CacheAttnMaps maps;
  if (!maps_of(cache, &maps)) return SAGE_ERR_CUDA;
  return status_of(launch_cache_decode(maps, a, static_cast<cudaStream_t>(stream)));
}

SAGE_EXPORT sage_status sage_cache_weights(const sage_kv_cache* cache, const sage_kv_seqs* seqs,
                                           const sage_kv_query* query, int mask, int mask_block, int win,
                                           int sink, const float* lse, int accumulate, void* stream) {
  if (!query || (!no_rows(query) && !al(lse, 4)) || !cache_ok(cache) || !cache->weight)
    return SAGE_ERR_INVALID_ARG;
  CacheAttnArgs a{};
  const sage_status st = attn_common(cache, seqs, query, mask, mask_block, win, sink, &a);
  if (st != SAGE_OK) return st;
  if (no_rows(query)) {
    if (accumulate) return SAGE_OK;
    // one group of no tokens: the few-row kernel then reads no query row
    a.G = 1;
    a.H = cache->heads;
    a.Nq = 0;
    a.q_lens = nullptr;
  }
  a.lse_in = lse;
  a.accumulate = accumulate != 0;
  const int sms = sm_count();
  if (!sms) return SAGE_ERR_CUDA;
  const int pages = std::max(1, (query->max_len + kPage - 1) / kPage);
  const long long units = static_cast<long long>(seqs->B) * cache->heads;
  // Up to eight query rows the keys stream past one mma.sync tile, up to 16
  // with 64 channels (16 rows of 16 x 8 heads of 8000 tokens: 41 us against 47;
  // with 128 channels 76 against 59).
  if (static_cast<long long>(a.Nq) * a.G > (cache->D == 64 ? kDecRows : kDecRows / 2)) {
    // a block an SM, with eight pages each at least
    a.chunks = static_cast<int>(std::min<long long>(sms, (units * pages + 7) / 8));
    return status_of(launch_cache_weights(a, static_cast<cudaStream_t>(stream)));
  }
  plan_decode(units, pages, sms, false, &a.chunks, &a.whole);
  CacheAttnMaps maps;
  if (!maps_of(cache, &maps)) return SAGE_ERR_CUDA;
  return status_of(launch_cache_weights_few(maps, a, static_cast<cudaStream_t>(stream)));
}

SAGE_EXPORT size_t sage_cache_evict_workspace_bytes(int B, int heads, int D, int keep, int in_place) {
  if (B < 1 || B > 65535 || heads < 1 || heads > 65535 || (D != 64 && D != 128) || keep < 1 ||
      keep > (1 << 30))
    return 0;
  return cache_evict_ws_bytes(B, heads, D, keep, in_place != 0);
}

SAGE_EXPORT sage_status sage_cache_evict(const sage_kv_cache* cache, const sage_kv_seqs* seqs, int keep,
                                         int sink, int recent, const int32_t* pages_out, int out_pages,
                                         int32_t* kept, int32_t* lengths_out, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  if (!cache_ok(cache) || !cache->weight || !seqs_ok(seqs)) return SAGE_ERR_INVALID_ARG;
  if (keep < 1 || keep > (1 << 30) || sink < 0 || recent < 0 ||
      static_cast<long long>(sink) + recent > keep)
    return SAGE_ERR_INVALID_ARG;
  if (!al(kept, 4) || !al(lengths_out, 4)) return SAGE_ERR_INVALID_ARG;
  const int need = (keep + kPage - 1) / kPage;
  if (pages_out && (!al(pages_out, 4) || out_pages < need)) return SAGE_ERR_INVALID_ARG;
  if (!al(workspace, 16) ||
      workspace_bytes < cache_evict_ws_bytes(seqs->B, cache->heads, cache->D, keep, !pages_out))
    return SAGE_ERR_INVALID_ARG;
  if (!cache_fits(cache) || static_cast<long long>(seqs->B) * cache->heads > (1 << 28))
    return SAGE_ERR_UNSUPPORTED;
  if (lengths_out == seqs->lengths) return SAGE_ERR_INVALID_ARG;
  int* status = api_status_word();
  if (!status) return SAGE_ERR_CUDA;
  EvictArgs a{};
  a.c = view_of(cache, seqs, status);
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.kept = kept;
  a.lengths_out = lengths_out;
  a.pages_out = pages_out;
  a.out_pages = out_pages;
  a.ws = workspace;
  return status_of(launch_cache_evict(a, static_cast<cudaStream_t>(stream)));
}
