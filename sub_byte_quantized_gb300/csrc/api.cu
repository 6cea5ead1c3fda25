// C ABI of the library: host-side validation, workspace layout and kernel launches.
// Nothing here allocates, synchronises or prints; failures return a kvq_status and record a
// one-line reason readable through kvq_last_error().
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "kvq_internal.cuh"

namespace {

thread_local char g_last_error[256] = "";
thread_local cudaEvent_t g_ev_begin = nullptr, g_ev_end = nullptr;

kvq_status fail(kvq_status st, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Whether two runs of bytes share one (NULL: no run).
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && (x <= y ? y - x < na : x - y < nb);
}

size_t row_bytes_of(int layout, int D) {
  if (D != 128 && D != 256) return 0;
  const int nb = D / kvq::kBlock;
  switch (layout) {
    case KVQ_Q4_0: return 16 * (size_t)nb;
    case KVQ_Q6_0: return 24 * (size_t)nb;
    case KVQ_HAD_INT4: return (size_t)D / 2;
    case KVQ_HAD_INT2: return (size_t)D / 4;
    case KVQ_Q8_0: return 32 * (size_t)nb;
    case KVQ_ASYM4_G32: return 16 * (size_t)nb;
    case KVQ_INT8_B64:
    case KVQ_E4M3_B64: return (size_t)D;
    default: return 0;
  }
}

// The K and V layouts of a cache's layout field (plain, or KVQ_MIXED(k, v)); false when invalid.
bool split_layout(int32_t layout, int &k, int &v) {
  k = layout & 0xFF;
  v = (layout >> 8) ? (layout >> 8) - 1 : k;
  if ((layout >> 8) > kvq::kLastLayout + 1 || layout < 0) return false;
  if (k > kvq::kLastLayout || v > kvq::kLastLayout) return false;
  if (kvq::is_b64(k) || kvq::is_b64(v)) return k == v;   // their kernels take one layout in both planes
  return kvq::is_hadamard(k) == kvq::is_hadamard(v);
}

// Bytes of `rows` token rows' scales in a plain layout (the block layouts': whole blocks of 64 rows).
size_t scale_bytes_of(int layout, size_t rows, int D) {
  if (kvq::is_b64(layout)) return rows / 64 * sizeof(float);
  return kvq::is_hadamard(layout) ? rows * sizeof(float) : rows * (D / kvq::kBlock) * 2;
}

// Layout checks shared by the contiguous and paged caches: both planes' layouts, head_dim, the
// window option and the plane pointers each plane's layout needs.
kvq_status check_planes(int32_t layout, int32_t head_dim, int32_t n_recent, const void *k_zero, const void *v_zero,
                        const float *k_recent, const float *v_recent, kvq::CacheView &v) {
  int kl, vl;
  if (!split_layout(layout, kl, vl)) return fail(KVQ_EINVAL, "unknown layout %d (or a rotated/unrotated mix)", layout);
  if (head_dim != 128 && head_dim != 256) return fail(KVQ_ESHAPE, "head_dim %d not 128/256", head_dim);
  if (n_recent < 0) return fail(KVQ_EINVAL, "n_recent < 0");
  if (!kvq::is_hadamard(kl) && n_recent != 0) return fail(KVQ_EUNSUPPORTED, "n_recent is an option of the Hadamard layouts");
  if (kl == KVQ_ASYM4_G32 && !k_zero) return fail(KVQ_EINVAL, "zero-point planes are NULL");
  if (vl == KVQ_ASYM4_G32 && !v_zero) return fail(KVQ_EINVAL, "zero-point planes are NULL");
  if ((k_zero && !aligned(k_zero, 16)) || (v_zero && !aligned(v_zero, 16)))
    return fail(KVQ_EALIGN, "zero plane not 16-byte aligned");
  if (kvq::is_hadamard(kl) && n_recent > 0) {
    if (!k_recent || !v_recent) return fail(KVQ_EINVAL, "recent-window planes are NULL");
    if (!aligned(k_recent, 16) || !aligned(v_recent, 16)) return fail(KVQ_EALIGN, "window plane not 16-byte aligned");
  }
  v.layout = kl;
  v.v_layout = vl;
  v.row_bytes = (int)row_bytes_of(kl, head_dim);
  v.v_row_bytes = (int)row_bytes_of(vl, head_dim);
  v.n_recent = kvq::is_hadamard(kl) ? n_recent : 0;
  return KVQ_OK;
}

kvq_status check_cache(const kvq_cache *c, kvq::CacheView &v) {
  if (!c) return fail(KVQ_EINVAL, "cache is NULL");
  kvq_status st = check_planes(c->layout, c->head_dim, c->n_recent, c->k_zero, c->v_zero, c->k_recent, c->v_recent, v);
  if (st != KVQ_OK) return st;
  if (c->batch < 1 || c->n_kv_heads < 1 || c->capacity < 1)
    return fail(KVQ_EINVAL, "batch, n_kv_heads and capacity must be >= 1");
  if (kvq::is_b64(v.layout) && c->capacity % 64) return fail(KVQ_ESHAPE, "capacity %d not a multiple of 64 (block layouts)", c->capacity);
  const void *ptrs[] = {c->k_payload, c->v_payload, c->k_scale, c->v_scale};
  for (const void *p : ptrs) {
    if (!p) return fail(KVQ_EINVAL, "payload/scale pointer is NULL");
    if (!aligned(p, 16)) return fail(KVQ_EALIGN, "payload/scale pointer not 16-byte aligned");
  }
  v.B = c->batch; v.H = c->n_kv_heads; v.D = c->head_dim; v.cap = c->capacity;
  v.payload[0] = static_cast<uint8_t *>(c->k_payload);
  v.payload[1] = static_cast<uint8_t *>(c->v_payload);
  v.scale[0] = c->k_scale; v.scale[1] = c->v_scale;
  v.zero[0] = static_cast<__half *>(c->k_zero);
  v.zero[1] = static_cast<__half *>(c->v_zero);
  v.ring[0] = c->k_recent; v.ring[1] = c->v_recent;
  v.page_shift = -1; v.table_stride = 0; v.n_pages = 0; v.table = nullptr;
  return KVQ_OK;
}

// log2 of a paged cache's page size; -1 when it is none.
int page_shift_of(int page_size) {
  for (int k = kvq::kMinPageShift; k <= 20; ++k)
    if (page_size == (1 << k)) return k;
  return -1;
}

// Validation of a paged pool and its block table.
kvq_status check_paged_cache(const kvq_paged_cache *c, kvq::CacheView &v) {
  if (!c) return fail(KVQ_EINVAL, "cache is NULL");
  kvq_status st = check_planes(c->layout, c->head_dim, c->n_recent, c->k_zero, c->v_zero, c->k_recent, c->v_recent, v);
  if (st != KVQ_OK) return st;
  if (c->batch < 1 || c->n_kv_heads < 1 || c->n_pages < 1 || c->max_pages_per_seq < 1)
    return fail(KVQ_EINVAL, "batch, n_kv_heads, n_pages and max_pages_per_seq must be >= 1");
  const int shift = page_shift_of(c->page_size);
  if (shift < 0) return fail(KVQ_ESHAPE, "page_size %d is not a power of two in [64, 2^20]", c->page_size);
  if ((long long)c->max_pages_per_seq * c->page_size > INT_MAX)
    return fail(KVQ_ECAPACITY, "max_pages_per_seq * page_size exceeds INT_MAX tokens");
  const void *ptrs[] = {c->k_payload, c->v_payload, c->k_scale, c->v_scale, c->block_table};
  for (const void *p : ptrs) {
    if (!p) return fail(KVQ_EINVAL, "payload/scale/block_table pointer is NULL");
    if (!aligned(p, 16)) return fail(KVQ_EALIGN, "payload/scale/block_table pointer not 16-byte aligned");
  }
  v.B = c->batch; v.H = c->n_kv_heads; v.D = c->head_dim;
  v.cap = c->max_pages_per_seq * c->page_size;
  v.payload[0] = static_cast<uint8_t *>(c->k_payload);
  v.payload[1] = static_cast<uint8_t *>(c->v_payload);
  v.scale[0] = c->k_scale; v.scale[1] = c->v_scale;
  v.zero[0] = static_cast<__half *>(c->k_zero);
  v.zero[1] = static_cast<__half *>(c->v_zero);
  v.ring[0] = c->k_recent; v.ring[1] = c->v_recent;
  v.page_shift = shift; v.table_stride = c->max_pages_per_seq; v.n_pages = c->n_pages;
  v.table = c->block_table;
  return KVQ_OK;
}

// Validation of an append (no launch). want_layout < 0 accepts the cache's own layout.
kvq_status check_store(int want_layout, const kvq_cache *cache, const void *k_new, const void *v_new, int dtype,
                       int n_new, int pos0, kvq::CacheView &v) {
  kvq_status st = check_cache(cache, v);
  if (st != KVQ_OK) return st;
  if (want_layout >= 0 && (v.layout != want_layout || v.v_layout != want_layout))
    return fail(KVQ_EUNSUPPORTED, "cache layout %d does not match this store (kvq_store takes any layout)",
                cache->layout);
  if (dtype < KVQ_F32 || dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown dtype %d", dtype);
  if (n_new < 0 || pos0 < 0) return fail(KVQ_EINVAL, "n_new and pos0 must be >= 0");
  if ((long long)pos0 + n_new > v.cap) return fail(KVQ_ECAPACITY, "pos0 + n_new = %lld > capacity %d",
                                                  (long long)pos0 + n_new, v.cap);
  if (n_new == 0) return KVQ_OK;
  if (!k_new || !v_new) return fail(KVQ_EINVAL, "k_new/v_new is NULL");
  if (!aligned(k_new, 16) || !aligned(v_new, 16)) return fail(KVQ_EALIGN, "k_new/v_new not 16-byte aligned");
  return KVQ_OK;
}

kvq_status store_common(int want_layout, const kvq_cache *cache, const void *k_new, const void *v_new, int dtype,
                        int n_new, int pos0, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq_status st = check_store(want_layout, cache, k_new, v_new, dtype, n_new, pos0, v);
  if (st != KVQ_OK || n_new == 0) return st;
  cudaError_t e = kvq::launch_store(v, k_new, v_new, dtype, n_new, pos0, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "store launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// Automatic split-K chunk, sized for the tensor-core kernel that will run. Decode (up to eight
// query rows per kv head), one wave: for the per-warp kernel four times the smallest multiple of
// 32 tokens (a warp's stage) that gives one slice to every resident warp (four warps per chunk);
// for the warp-specialised kernels (Q6_0, asymmetric) the smallest multiple of 64 that gives one
// chunk to every resident CTA. Many rows: about four waves of 64-row CTAs on the row-side kernel,
// the fewest waves x stages of 256-row CTAs on the tcgen05 kernel.
// `work` = body tokens summed over every (batch, kv head) (0: n_body for each of them); a ragged
// batch passes its true total so the chunk fits the work that exists.
// n_wchunks: window chunks per (batch, kv head) that the row-side kernel scores in the same grid.
int auto_chunk(const kvq::CacheView &c, int rows, int n_body, int n_heads, long long work = 0, int n_wchunks = 0) {
  const int sms = kvq::sm_count();
  const bool total_given = work > 0;
  if (!total_given) work = (long long)(n_body > 0 ? n_body : 1) * n_heads;
  long long chunk;
  if (kvq::is_b64(c.layout)) {
    // every resident CTA takes as many tokens; each group of query rows counts
    const long long ctas = (long long)sms * kvq::b64_ctas(c.D, rows), per = kvq::b64_group(c.D, rows), groups = (rows + per - 1) / per;
    chunk = ((work * groups + ctas - 1) / ctas + 63) / 64 * 64;
  } else if (c.layout == KVQ_Q6_0 && kvq::mma_q6_shape(c.D, rows) && !kvq::prefill_shape(c.layout, c.v_layout, c.D, rows)) {
    // one chunk per resident CTA; each group of four query rows has its own CTAs
    const long long ctas = (long long)sms * kvq::kMmaQ6CtasPerSm(c.D);
    const long long groups = (rows + 3) / 4;
    chunk = ((work * groups + ctas - 1) / ctas + 63) / 64 * 64;
  } else if (kvq::prefill_shape(c.layout, c.v_layout, c.D, rows) && rows <= 16 &&
             !kvq::decode_kernel(c.layout, c.v_layout)) {
    // row-side kernel in its decode form (one row block, the warps split the tokens): one chunk per
    // resident CTA, as many chunks per (batch, kv head) as fit one wave
    const long long ctas = (long long)sms * (kvq::is_hadamard(c.layout) ? kvq::kPrefillCtasPerSm : 2);
    long long per_head = ctas / (n_heads > 0 ? n_heads : 1);   // (the window is scored in phase 2)
    if (per_head < 1) per_head = 1;
    const long long body = total_given ? (work + n_heads - 1) / n_heads : (n_body > 0 ? n_body : 1);
    chunk = ((body + per_head - 1) / per_head + 63) / 64 * 64;
  } else if (kvq::tc_prefill_shape(c.layout, c.v_layout, c.D, rows)) {
    // tcgen05 kernel, one CTA of 256 rows per SM: the number of body chunks per row block (1..8)
    // whose grid takes the fewest waves x (stages per chunk + about two stages of fixed cost per CTA)
    const long long units = (long long)((rows + kvq::kTcRows - 1) / kvq::kTcRows) * n_heads;
    const long long body = total_given ? (work + n_heads - 1) / n_heads : (n_body > 0 ? n_body : 1);
    const long long stages = (body + 63) / 64;
    long long best = 1, best_cost = -1;
    for (long long n = 1; n <= 8; ++n) {
      const long long per = (stages + n - 1) / n;
      if (per * 64 > 8192) continue;
      const long long waves = (units * n + sms - 1) / sms;
      const long long cost = waves * (per + 2);
      if (best_cost < 0 || cost < best_cost) { best = n; best_cost = cost; }
    }
    chunk = ((stages + best - 1) / best) * 64;
  } else if (kvq::prefill_shape(c.layout, c.v_layout, c.D, rows)) {
    // row-side kernel: CTAs of 64 query rows; split the body into enough chunks for about four
    // waves of resident CTAs
    const long long row_ctas = (long long)((rows + kvq::kPrefillRows - 1) / kvq::kPrefillRows) * n_heads;
    const long long want = 4LL * sms * kvq::kPrefillCtasPerSm;
    long long n_chunks = (want + row_ctas - 1) / row_ctas;
    if (n_chunks < 1) n_chunks = 1;
    const long long body = total_given ? (work + n_heads - 1) / n_heads : (n_body > 0 ? n_body : 1);
    chunk = ((body + n_chunks - 1) / n_chunks + 63) / 64 * 64;
  } else if (kvq::uses_mma4(c.layout)) {
    // warp-specialised 4-bit kernel: one chunk per resident CTA, as many chunks per (batch, kv
    // head) as fit one wave
    const long long ctas = (long long)sms * kvq::kMma4CtasPerSm;
    long long per_head = ctas / (n_heads > 0 ? n_heads : 1);
    if (per_head < 1) per_head = 1;
    const long long body = total_given ? (work + n_heads - 1) / n_heads : (n_body > 0 ? n_body : 1);
    chunk = ((body + per_head - 1) / per_head + 63) / 64 * 64;
  } else {
    const long long warps = (long long)sms * kvq::kMmaWarpsPerSm;
    chunk = 4 * (((work + warps - 1) / warps + 31) / 32 * 32);   // a warp's slice: whole 32-token stages
  }
  if (chunk > 8192) chunk = 8192;
  return (int)chunk;
}

// The block layouts' part of resolve_core: phase 1's CTAs (`chunk` 0: one wave, among which the call's units are dealt out on
// the device; else one for each piece of at most chunk tokens of every head) and the workspace of their partials.
kvq_status resolve_b64(kvq::AttendArgs &a, int chunk, size_t &need, void *ws) {
  const kvq::CacheView &c = a.cache;
  const int sms = kvq::sm_count();
  const long long rows = a.gqa * (long long)a.n_q;
  a.group = kvq::b64_group(c.D, rows);
  const long long heads = (long long)c.B * c.H * ((rows + a.group - 1) / a.group);
  const long long units = heads * (((long long)a.kv_len + 63) / 64);
  a.per = chunk / 64;
  const long long grid = chunk ? heads * ((((long long)a.kv_len + 63) / 64 + a.per - 1) / a.per) : std::min((long long)sms * kvq::b64_ctas(c.D, rows), units);
  if (grid + heads > INT_MAX / a.group) return fail(KVQ_ESHAPE, "too many rows and chunks for one call");
  a.grid = (int)grid;
  const size_t parts = (size_t)(grid + heads);
  size_t off = 0;
  const size_t o_m = off; off = round_up(off + parts * a.group * sizeof(float), 256);
  const size_t o_l = off; off = round_up(off + parts * a.group * sizeof(float), 256);
  const size_t o_s = off; off = round_up(off + (size_t)heads * sizeof(int2), 256);
  const size_t o_o = off; off = round_up(off + parts * a.group * c.D * sizeof(float), 256);
  need = off;
  if (ws) {
    char *w = static_cast<char *>(ws);
    a.part_m = reinterpret_cast<float *>(w + o_m);
    a.part_l = reinterpret_cast<float *>(w + o_l);
    a.spans = reinterpret_cast<int2 *>(w + o_s);
    a.part_o = reinterpret_cast<float *>(w + o_o);
    a.q8 = nullptr;
    a.s_q = a.q_rot = nullptr;
  }
  return KVQ_OK;
}

// Resolve the attention arguments and the workspace layout for a checked cache view `a.cache`
// (kv_len: the call's length, or the largest per-sequence length of a paged call). When `ws` is
// NULL only sizes are computed (returned through `need`).
kvq_status resolve_core(int n_q_heads, int n_q, int kv_len, int causal, int q_pos0, bool paged, int chunk,
                        kvq::AttendArgs &a, size_t &need, void *ws, long long work = 0) {
  const kvq::CacheView &c = a.cache;
  if (n_q_heads < 1 || n_q < 1) return fail(KVQ_EINVAL, "n_q_heads and n_q must be >= 1");
  if (n_q_heads % c.H) return fail(KVQ_ESHAPE, "n_q_heads %d not a multiple of n_kv_heads %d", n_q_heads, c.H);
  if (kv_len < 1) return fail(KVQ_EINVAL, "kv_len must be >= 1");
  if (kv_len > c.cap) return fail(KVQ_ECAPACITY, "kv_len %d > capacity %d", kv_len, c.cap);
  if (!paged && causal && (q_pos0 < 0 || (long long)q_pos0 + n_q > kv_len))
    return fail(KVQ_EINVAL, "causal call needs 0 <= q_pos0 and q_pos0 + n_q <= kv_len");
  const int given = chunk;
  if (chunk == 0)
  {
    const int n_win = kvq::is_hadamard(c.layout) ? (c.n_recent < kv_len ? c.n_recent : kv_len) : 0;
    chunk = auto_chunk(c, (n_q_heads / c.H) * n_q, kv_len - n_win, c.B * c.H, work,
                       (n_win + kvq::kWinChunk - 1) / kvq::kWinChunk);
  }
  if (chunk < 64 || chunk > 8192 || chunk % 64) return fail(KVQ_ESHAPE, "chunk %d not a multiple of 64 in [64, 8192]", chunk);
  a.Hq = n_q_heads; a.gqa = n_q_heads / c.H; a.n_q = n_q;
  a.kv_len = kv_len;
  a.n_win = kvq::is_hadamard(c.layout) ? (c.n_recent < kv_len ? c.n_recent : kv_len) : 0;
  a.n_body = kv_len - a.n_win;
  a.causal = causal ? 1 : 0;
  a.q_pos0 = causal ? q_pos0 : 0;
  a.chunk = chunk;
  a.n_chunks = (a.n_body + chunk - 1) / chunk;
  a.n_wchunks = (a.n_win + kvq::kWinChunk - 1) / kvq::kWinChunk;
  a.C = a.n_chunks + a.n_wchunks;
  a.win_in_reduce = 0;
  a.y_base = 0;
  a.q_prepped = 0;
  a.fresh_lo = 0;
  a.fresh_hi = INT_MAX;
  a.seq_lens = nullptr;
  a.fresh_tail = 0;
  a.cap_scores = nullptr;
  a.cap_sq = nullptr;
  a.lse = nullptr;
  a.part_s = nullptr;
  a.s_rows = a.s_tokens = 0;
  a.held = false;
  a.out_nq = 1;
  a.grid = a.per = 0;
  a.group = 8;
  a.spans = nullptr;
  if (kvq::is_b64(c.layout)) return resolve_b64(a, given, need, ws);
  const size_t rows = (size_t)c.B * n_q_heads * n_q;
  size_t off = 0;
  const size_t o_m = off; off = round_up(off + rows * a.C * sizeof(float), 256);
  const size_t o_l = off; off = round_up(off + rows * a.C * sizeof(float), 256);
  const size_t o_o = off; off = round_up(off + rows * a.C * (size_t)c.D * sizeof(float), 256);
  size_t o_q8 = 0, o_sq = 0, o_qr = 0;
  if (kvq::is_hadamard(c.layout)) {
    o_q8 = off; off = round_up(off + rows * (size_t)c.D, 256);
    o_sq = off; off = round_up(off + rows * sizeof(float), 256);
    o_qr = off; off = round_up(off + rows * (size_t)c.D * sizeof(float), 256);
  }
  need = off;
  if (ws) {
    char *w = static_cast<char *>(ws);
    a.part_m = reinterpret_cast<float *>(w + o_m);
    a.part_l = reinterpret_cast<float *>(w + o_l);
    a.part_o = reinterpret_cast<float *>(w + o_o);
    a.q8 = kvq::is_hadamard(c.layout) ? reinterpret_cast<int8_t *>(w + o_q8) : nullptr;
    a.s_q = kvq::is_hadamard(c.layout) ? reinterpret_cast<float *>(w + o_sq) : nullptr;
    a.q_rot = kvq::is_hadamard(c.layout) ? reinterpret_cast<float *>(w + o_qr) : nullptr;
  }
  return KVQ_OK;
}

kvq_status resolve_attend(const kvq_cache *cache, int n_q_heads, int n_q, int kv_len, int causal, int q_pos0,
                          int chunk, kvq::AttendArgs &a, size_t &need, void *ws) {
  kvq_status st = check_cache(cache, a.cache);
  if (st != KVQ_OK) return st;
  return resolve_core(n_q_heads, n_q, kv_len, causal, q_pos0, false, chunk, a, need, ws);
}

// Paged call: the grid is sized for max_kv_len; per-sequence lengths are read on the device.
kvq_status resolve_paged(const kvq_paged_cache *cache, int n_q_heads, int n_q, int max_kv_len, int causal, int chunk,
                         kvq::AttendArgs &a, size_t &need, void *ws, long long total_kv_len = 0) {
  kvq_status st = check_paged_cache(cache, a.cache);
  if (st != KVQ_OK) return st;
  long long work = 0;                                    // body tokens over all sequences and kv heads
  if (total_kv_len > 0) {
    const long long win = kvq::is_hadamard(cache->layout & 0xFF) ? (long long)cache->n_recent * cache->batch : 0;
    work = (total_kv_len > win ? total_kv_len - win : 1) * cache->n_kv_heads;
  }
  return resolve_core(n_q_heads, n_q, max_kv_len, causal, 0, true, chunk, a, need, ws, work);
}

}  // namespace

extern "C" {

size_t kvq_row_bytes(int32_t layout, int32_t head_dim) { return row_bytes_of(layout, head_dim); }

kvq_status kvq_cache_bytes(int32_t layout, int32_t batch, int32_t n_kv_heads, int32_t head_dim, int32_t capacity,
                           int32_t n_recent, size_t out_sizes[4]) {
  g_last_error[0] = 0;
  if (!out_sizes) return fail(KVQ_EINVAL, "out_sizes is NULL");
  const size_t rb = row_bytes_of(layout, head_dim);
  if (layout < KVQ_Q4_0 || layout > kvq::kLastLayout) return fail(KVQ_EINVAL, "unknown layout %d", layout);
  if (!rb) return fail(KVQ_ESHAPE, "head_dim %d not 128/256", head_dim);
  if (batch < 1 || n_kv_heads < 1 || capacity < 1 || n_recent < 0) return fail(KVQ_EINVAL, "bad sizes");
  if (kvq::is_b64(layout) && capacity % 64) return fail(KVQ_ESHAPE, "capacity %d not a multiple of 64 (block layouts)", capacity);
  const size_t rows = (size_t)batch * n_kv_heads * capacity;
  const size_t nb = (size_t)head_dim / kvq::kBlock;
  out_sizes[0] = rows * rb;
  out_sizes[1] = scale_bytes_of(layout, rows, head_dim);
  out_sizes[2] = layout == KVQ_ASYM4_G32 ? rows * nb * 2 : 0;
  out_sizes[3] = kvq::is_hadamard(layout) ? (size_t)batch * n_kv_heads * n_recent * head_dim * sizeof(float) : 0;
  return KVQ_OK;
}

kvq_status kvq_store_q4_0(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype, int32_t n_new,
                          int32_t pos0, kvq_stream_t stream) {
  return store_common(KVQ_Q4_0, cache, k_new, v_new, dtype, n_new, pos0, stream);
}
kvq_status kvq_store_q6_0(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype, int32_t n_new,
                          int32_t pos0, kvq_stream_t stream) {
  return store_common(KVQ_Q6_0, cache, k_new, v_new, dtype, n_new, pos0, stream);
}
kvq_status kvq_store_hadamard_int4(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype,
                                   int32_t n_new, int32_t pos0, kvq_stream_t stream) {
  return store_common(KVQ_HAD_INT4, cache, k_new, v_new, dtype, n_new, pos0, stream);
}
kvq_status kvq_store_asym4_g32(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype,
                               int32_t n_new, int32_t pos0, kvq_stream_t stream) {
  return store_common(KVQ_ASYM4_G32, cache, k_new, v_new, dtype, n_new, pos0, stream);
}
kvq_status kvq_store_q8_0(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype, int32_t n_new,
                          int32_t pos0, kvq_stream_t stream) {
  return store_common(KVQ_Q8_0, cache, k_new, v_new, dtype, n_new, pos0, stream);
}
kvq_status kvq_store_hadamard_int2(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype,
                                   int32_t n_new, int32_t pos0, kvq_stream_t stream) {
  return store_common(KVQ_HAD_INT2, cache, k_new, v_new, dtype, n_new, pos0, stream);
}
kvq_status kvq_store(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t dtype, int32_t n_new,
                     int32_t pos0, kvq_stream_t stream) {
  return store_common(-1, cache, k_new, v_new, dtype, n_new, pos0, stream);
}

size_t kvq_attend_workspace_bytes(const kvq_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t kv_len,
                                  int32_t chunk) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (resolve_attend(cache, n_q_heads, n_q, kv_len, 0, 0, chunk, a, need, nullptr) != KVQ_OK) return 0;
  return need;
}

int32_t kvq_attend_chunk(const kvq_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t kv_len, int32_t chunk) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (resolve_attend(cache, n_q_heads, n_q, kv_len, 0, 0, chunk, a, need, nullptr) != KVQ_OK) return 0;
  return a.chunk;
}

namespace {

// The query, output, workspace and scale arguments of an attention call.
kvq_status check_call(size_t need, const void *q, int32_t q_dtype, float attn_scale, const float *out,
                      const void *workspace, size_t workspace_bytes) {
  if (q_dtype < KVQ_F32 || q_dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown q dtype %d", q_dtype);
  if (!q || !out || !workspace) return fail(KVQ_EINVAL, "q/out/workspace is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_EALIGN, "q/out not 16-byte aligned");
  if (!aligned(workspace, 256)) return fail(KVQ_EALIGN, "workspace not 256-byte aligned");
  if (workspace_bytes < need) return fail(KVQ_EWORKSPACE, "workspace %zu < required %zu", workspace_bytes, need);
  if (!(attn_scale == attn_scale) || attn_scale > 3.0e38f || attn_scale < -3.0e38f)
    return fail(KVQ_EINVAL, "attn_scale must be finite");
  return KVQ_OK;
}

// Validation of an attention call and its workspace; on success `a` is fully resolved.
kvq_status prepare_attend(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads, int32_t n_q,
                          int32_t kv_len, int32_t causal, int32_t q_pos0, float attn_scale, int32_t chunk,
                          float *out, void *workspace, size_t workspace_bytes, kvq::AttendArgs &a) {
  size_t need = 0;
  kvq_status st = resolve_attend(cache, n_q_heads, n_q, kv_len, causal, q_pos0, chunk, a, need, nullptr);
  if (st != KVQ_OK) return st;
  st = check_call(need, q, q_dtype, attn_scale, out, workspace, workspace_bytes);
  if (st != KVQ_OK) return st;
  resolve_attend(cache, n_q_heads, n_q, kv_len, causal, q_pos0, chunk, a, need, workspace);
  a.q = q;
  a.q_dtype = q_dtype;
  a.scale = attn_scale;
  a.out = out;
  return KVQ_OK;
}

// Phase 1 (tensor-core or CUDA-core kernel) and phase 2 on `s`, with the optional phase-1 events.
cudaError_t launch_attend_sequence(kvq::AttendArgs &a, cudaStream_t s, bool events) {
  cudaError_t e = cudaSuccess;
  const bool b64 = kvq::is_b64(a.cache.layout);
  const bool mma = b64 || kvq::mma_supported(a);
  // the decode tensor-core kernels (and the row-side kernel's decode form) cover the body chunks only
  a.win_in_reduce = mma && a.n_win > 0 &&
                    (!kvq::prefill_supported(a) ||
                     kvq::dec_shape(a.cache.layout, a.cache.v_layout, a.cache.D, a.gqa * a.n_q));
  // the tensor-core kernels prepare the Hadamard query themselves; the CUDA-core one reads it
  if (kvq::is_hadamard(a.cache.layout) && !mma) {
    a.fresh_lo = 0;                                      // its predecessor is then the prep kernel
    a.fresh_hi = INT_MAX;
    a.fresh_tail = 0;
    e = kvq::launch_had_prep(a, s);
  }
  const bool prof = events && g_ev_begin && g_ev_end;
  // Under stream capture an event record must be external to become a graph node.
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (e == cudaSuccess && prof) e = cudaStreamIsCapturing(s, &cap);
  const unsigned rec_flags = cap == cudaStreamCaptureStatusActive ? cudaEventRecordExternal : cudaEventRecordDefault;
  if (e == cudaSuccess && prof) e = cudaEventRecordWithFlags(g_ev_begin, s, rec_flags);
  if (e == cudaSuccess) e = b64 ? kvq::launch_attend_b64(a, s) : mma ? kvq::launch_attend_mma(a, s) : kvq::launch_attend_generic(a, s);
  if (e == cudaSuccess && prof) e = cudaEventRecordWithFlags(g_ev_end, s, rec_flags);
  if (e == cudaSuccess) e = b64 ? kvq::launch_join_b64(a, s) : kvq::launch_attend_reduce(a, s, true);
  return e;
}

// The append (when n_new > 0) and the attention of a validated append + attend call.
cudaError_t launch_append_attend(const kvq::CacheView &v, kvq::AttendArgs &a, const void *k_new, const void *v_new,
                                 int kv_dtype, int n_new, int pos0, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (n_new > 0) {
    e = kvq::launch_store(v, k_new, v_new, kv_dtype, n_new, pos0, s);
    // the rows (and window slots) it writes; a block layout's append may touch the rows in front of them too
    a.fresh_lo = kvq::is_b64(v.layout) ? pos0 / 64 * 64 : pos0;
    a.fresh_hi = pos0 + n_new;
  }
  if (e == cudaSuccess) e = launch_attend_sequence(a, s, true);
  return e;
}

size_t dtype_bytes(int32_t dt) { return dt == KVQ_F32 ? 4 : 2; }

// Device staging of a host-buffer call, in the caller's workspace after the attention partials:
// k_new, v_new, q, out and (paged) seq_lens, each from a 256-byte boundary.
struct HostStaging {
  size_t k = 0, v = 0, q = 0, out = 0, lens = 0, total = 0;
  size_t kv_bytes = 0, q_bytes = 0, out_bytes = 0, lens_bytes = 0;
};

HostStaging host_staging(size_t attend_need, int batch, int n_kv_heads, int head_dim, int kv_dtype, int n_new,
                         int q_dtype, int n_q_heads, int n_q, bool paged) {
  HostStaging h;
  h.kv_bytes = n_new > 0 ? (size_t)batch * n_kv_heads * n_new * head_dim * dtype_bytes(kv_dtype) : 0;
  h.q_bytes = (size_t)batch * n_q_heads * n_q * head_dim * dtype_bytes(q_dtype);
  h.out_bytes = (size_t)batch * n_q_heads * n_q * head_dim * sizeof(float);
  h.lens_bytes = paged ? (size_t)batch * sizeof(int32_t) : 0;
  // k_new, v_new and q back to back (each size is a multiple of 256 bytes: head_dim 128 or 256), so
  // host inputs that are back to back too arrive with one copy
  h.k = round_up(attend_need, 256);
  h.v = h.k + h.kv_bytes;
  h.q = h.v + h.kv_bytes;
  h.out = h.q + round_up(h.q_bytes, 256);
  h.lens = h.out + round_up(h.out_bytes, 256);
  h.total = h.lens + round_up(h.lens_bytes, 256);
  return h;
}

// The element types and row count that size a host-buffer call's staging.
kvq_status check_host_sizes(int kv_dtype, int n_new, int q_dtype) {
  if (q_dtype < KVQ_F32 || q_dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown q dtype %d", q_dtype);
  if (kv_dtype < KVQ_F32 || kv_dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown dtype %d", kv_dtype);
  if (n_new < 0) return fail(KVQ_EINVAL, "n_new must be >= 0");
  return KVQ_OK;
}

// The host-side arguments of a host-buffer call that the device entry points cannot see.
kvq_status check_host_args(int kv_dtype, int n_new, int q_dtype, const void *k_new, const void *v_new, const void *q,
                           const float *out, const void *workspace) {
  const kvq_status st = check_host_sizes(kv_dtype, n_new, q_dtype);
  if (st != KVQ_OK) return st;
  if (n_new > 0 && (!k_new || !v_new)) return fail(KVQ_EINVAL, "k_new/v_new is NULL");
  if (!q || !out || !workspace) return fail(KVQ_EINVAL, "q/out/workspace is NULL");
  return KVQ_OK;
}

// The device address of a host buffer that the GPU reads and writes in place: pinned memory
// (cudaHostAlloc / cudaMallocHost, or registered), which unified addressing maps into every
// device's address space, and 16-byte aligned like the device-buffer calls require; nullptr for
// anything else (pageable memory goes through the staging copies).
void *device_view(const void *p) {
  if (!p || !aligned(p, 16)) return nullptr;
  cudaPointerAttributes pa;
  if (cudaPointerGetAttributes(&pa, p) != cudaSuccess) {
    cudaGetLastError();                                  // not a CUDA-known pointer: clear the error
    return nullptr;
  }
  return pa.type == cudaMemoryTypeHost ? pa.devicePointer : nullptr;
}

// Where a host-buffer call's kernels find their inputs and put their output. Pinned caller
// buffers are used in place where that saves a copy operation: the store kernel reads k_new /
// v_new over the host link (each element once) and the reduce writes the result there. q is
// always staged in device memory, since every phase-1 CTA of a kv head reads it (reading it over
// the link measured slower than one small copy). Pageable buffers go through the staging area of
// the workspace with a copy each way.
struct HostIo {
  const void *k, *v, *q;
  float *out;
  bool copy_in, copy_out;                                // copy_in: k_new and v_new staged with q
};
HostIo host_io(const HostStaging &h, char *ws, int n_new, const void *k_new, const void *v_new, float *out) {
  HostIo io;
  const void *kd = n_new > 0 ? device_view(k_new) : nullptr, *vd = n_new > 0 ? device_view(v_new) : nullptr;
  io.copy_in = !(n_new == 0 || (kd && vd));
  io.k = io.copy_in ? ws + h.k : kd;
  io.v = io.copy_in ? ws + h.v : vd;
  io.q = ws + h.q;
  float *od = static_cast<float *>(device_view(out));
  io.copy_out = od == nullptr;
  io.out = io.copy_out ? reinterpret_cast<float *>(ws + h.out) : od;
  return io;
}

// Host -> staging copies of the inputs (cudaMemcpyDefault: pinned or pageable host memory).
cudaError_t copy_in(const HostStaging &h, char *ws, const void *k_new, const void *v_new, const void *q,
                    const void *seq_lens, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const char *kb = static_cast<const char *>(k_new), *vb = static_cast<const char *>(v_new);
  if (h.kv_bytes && vb == kb + h.kv_bytes && static_cast<const char *>(q) == vb + h.kv_bytes) {
    e = cudaMemcpyAsync(ws + h.k, k_new, 2 * h.kv_bytes + h.q_bytes, cudaMemcpyDefault, s);   // one copy
  } else if (h.kv_bytes) {
    e = cudaMemcpyAsync(ws + h.k, k_new, h.kv_bytes, cudaMemcpyDefault, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(ws + h.v, v_new, h.kv_bytes, cudaMemcpyDefault, s);
  }
  if (e == cudaSuccess && !(h.kv_bytes && vb == kb + h.kv_bytes && static_cast<const char *>(q) == vb + h.kv_bytes))
    e = cudaMemcpyAsync(ws + h.q, q, h.q_bytes, cudaMemcpyDefault, s);
  if (e == cudaSuccess && h.lens_bytes) e = cudaMemcpyAsync(ws + h.lens, seq_lens, h.lens_bytes, cudaMemcpyDefault, s);
  return e;
}

// Staging -> host copy of the output, then wait for the stream.
cudaError_t copy_out_and_wait(const HostStaging &h, const char *ws, float *out, cudaStream_t s) {
  cudaError_t e = cudaMemcpyAsync(out, ws + h.out, h.out_bytes, cudaMemcpyDefault, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e;
}

}  // namespace

kvq_status kvq_decode_attend(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads, int32_t n_q,
                             int32_t kv_len, int32_t causal, int32_t q_pos0, float attn_scale, int32_t chunk,
                             float *out, void *workspace, size_t workspace_bytes, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  kvq_status st = prepare_attend(cache, q, q_dtype, n_q_heads, n_q, kv_len, causal, q_pos0, attn_scale, chunk, out,
                                 workspace, workspace_bytes, a);
  if (st != KVQ_OK) return st;
  cudaError_t e = launch_attend_sequence(a, reinterpret_cast<cudaStream_t>(stream), true);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_append_decode_attend(const kvq_cache *cache, const void *k_new, const void *v_new, int32_t kv_dtype,
                                    int32_t n_new, int32_t pos0, const void *q, int32_t q_dtype, int32_t n_q_heads,
                                    int32_t n_q, int32_t kv_len, int32_t causal, int32_t q_pos0, float attn_scale,
                                    int32_t chunk, float *out, void *workspace, size_t workspace_bytes,
                                    kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq_status st = check_store(-1, cache, k_new, v_new, kv_dtype, n_new, pos0, v);
  if (st != KVQ_OK) return st;
  kvq::AttendArgs a;
  st = prepare_attend(cache, q, q_dtype, n_q_heads, n_q, kv_len, causal, q_pos0, attn_scale, chunk, out, workspace,
                      workspace_bytes, a);
  if (st != KVQ_OK) return st;
  const cudaError_t e = launch_append_attend(v, a, k_new, v_new, kv_dtype, n_new, pos0,
                                             reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "append/attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// ------------------------------------------------------------------ paged pool
kvq_status kvq_paged_cache_bytes(int32_t layout, int32_t n_pages, int32_t n_kv_heads, int32_t head_dim,
                                 int32_t page_size, int32_t batch, int32_t n_recent, size_t out_sizes[4]) {
  g_last_error[0] = 0;
  if (!out_sizes) return fail(KVQ_EINVAL, "out_sizes is NULL");
  if (layout < KVQ_Q4_0 || layout > kvq::kLastLayout) return fail(KVQ_EINVAL, "unknown layout %d", layout);
  const size_t rb = row_bytes_of(layout, head_dim);
  if (!rb) return fail(KVQ_ESHAPE, "head_dim %d not 128/256", head_dim);
  if (n_pages < 1 || n_kv_heads < 1 || page_size < 1 || batch < 1 || n_recent < 0) return fail(KVQ_EINVAL, "bad sizes");
  if (kvq::is_b64(layout) && page_size % 64) return fail(KVQ_ESHAPE, "page_size %d not a multiple of 64 (block layouts)", page_size);
  const size_t rows = (size_t)n_pages * n_kv_heads * page_size;
  const size_t nb = (size_t)head_dim / kvq::kBlock;
  out_sizes[0] = rows * rb;
  out_sizes[1] = scale_bytes_of(layout, rows, head_dim);
  out_sizes[2] = layout == KVQ_ASYM4_G32 ? rows * nb * 2 : 0;
  out_sizes[3] = kvq::is_hadamard(layout) ? (size_t)batch * n_kv_heads * n_recent * head_dim * sizeof(float) : 0;
  return KVQ_OK;
}

namespace {

kvq_status check_paged_store(const kvq_paged_cache *cache, const void *k_new, const void *v_new, int dtype, int n_new,
                             const void *positions, kvq::CacheView &v) {
  kvq_status st = check_paged_cache(cache, v);
  if (st != KVQ_OK) return st;
  if (dtype < KVQ_F32 || dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown dtype %d", dtype);
  if (n_new < 0) return fail(KVQ_EINVAL, "n_new must be >= 0");
  if (n_new > v.cap) return fail(KVQ_ECAPACITY, "n_new %d > sequence capacity %d", n_new, v.cap);
  if (n_new == 0) return KVQ_OK;
  if (!k_new || !v_new || !positions) return fail(KVQ_EINVAL, "k_new/v_new/positions is NULL");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(positions, 16))
    return fail(KVQ_EALIGN, "k_new/v_new/positions not 16-byte aligned");
  return KVQ_OK;
}

kvq_status prepare_paged(const kvq_paged_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads, int32_t n_q,
                         const int32_t *seq_lens, int32_t max_kv_len, int32_t causal, float attn_scale, int32_t chunk,
                         float *out, void *workspace, size_t workspace_bytes, kvq::AttendArgs &a) {
  size_t need = 0;
  kvq_status st = resolve_paged(cache, n_q_heads, n_q, max_kv_len, causal, chunk, a, need, nullptr);
  if (st != KVQ_OK) return st;
  if (!seq_lens) return fail(KVQ_EINVAL, "seq_lens is NULL");
  if (!aligned(seq_lens, 16)) return fail(KVQ_EALIGN, "seq_lens not 16-byte aligned");
  st = check_call(need, q, q_dtype, attn_scale, out, workspace, workspace_bytes);
  if (st != KVQ_OK) return st;
  resolve_paged(cache, n_q_heads, n_q, max_kv_len, causal, chunk, a, need, workspace);
  a.seq_lens = seq_lens;
  a.q = q;
  a.q_dtype = q_dtype;
  a.scale = attn_scale;
  a.out = out;
  return KVQ_OK;
}

cudaError_t launch_paged_append_attend(const kvq::CacheView &v, kvq::AttendArgs &a, const void *k_new,
                                       const void *v_new, int kv_dtype, int n_new, const int32_t *seq_lens,
                                       cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (n_new > 0) {
    // the new tokens end each sequence: positions seq_lens[b] - n_new + j
    e = kvq::launch_store(v, k_new, v_new, kv_dtype, n_new, 0, s, seq_lens, -n_new);
    a.fresh_tail = kvq::is_b64(v.layout) ? n_new + 63 : n_new;   // the rows (and window slots) it writes, and their blocks
  }
  if (e == cudaSuccess) e = launch_attend_sequence(a, s, true);
  return e;
}

}  // namespace

kvq_status kvq_paged_store(const kvq_paged_cache *cache, const void *k_new, const void *v_new, int32_t dtype,
                           int32_t n_new, const int32_t *positions, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq_status st = check_paged_store(cache, k_new, v_new, dtype, n_new, positions, v);
  if (st != KVQ_OK || n_new == 0) return st;
  cudaError_t e = kvq::launch_store(v, k_new, v_new, dtype, n_new, 0, reinterpret_cast<cudaStream_t>(stream),
                                    positions, 0);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "store launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

namespace {

// Resident CTAs per SM of the phase-1 kernel a call with these shapes runs, and how many of its
// CTAs one (batch, kv head, chunk) unit takes (the row-side kernel: one per 64-query-row block).
void phase1_capacity(const kvq::CacheView &c, int rows, int q_dtype, int &ctas_per_sm, int &ctas_per_unit,
                     bool &window_ctas) {
  ctas_per_unit = 1;
  window_ctas = false;                                   // the decode kernels leave the window to phase 2
  if (kvq::is_b64(c.layout)) {
    ctas_per_sm = kvq::b64_ctas(c.D, rows);
    ctas_per_unit = (rows + kvq::b64_group(c.D, rows) - 1) / kvq::b64_group(c.D, rows);
  } else if (c.layout == KVQ_Q6_0 && c.v_layout == KVQ_Q6_0 && kvq::mma_q6_shape(c.D, rows) &&
      !(kvq::prefill_shape(c.layout, c.v_layout, c.D, rows) && q_dtype != KVQ_F32)) {
    ctas_per_sm = kvq::kMmaQ6CtasPerSm(c.D);
    ctas_per_unit = (rows + 3) / 4;
  } else if (kvq::tc_prefill_shape(c.layout, c.v_layout, c.D, rows)) {
    ctas_per_sm = 1;                                     // the tcgen05 kernel: one CTA of 256 rows per SM
    ctas_per_unit = (rows + kvq::kTcRows - 1) / kvq::kTcRows;
  } else if (kvq::prefill_shape(c.layout, c.v_layout, c.D, rows) &&
             (kvq::is_hadamard(c.layout) || q_dtype != KVQ_F32)) {
    ctas_per_sm = kvq::is_hadamard(c.layout) ? kvq::kPrefillCtasPerSm : 2;
    const bool dec = rows <= 16 && !kvq::decode_kernel(c.layout, c.v_layout);
    ctas_per_unit = dec ? 1 : (rows + kvq::kPrefillRows - 1) / kvq::kPrefillRows;
    window_ctas = kvq::is_hadamard(c.layout) && !dec;    // the row-side kernel scores the window chunks
  } else if (c.layout == c.v_layout && kvq::uses_mma4(c.layout)) {
    ctas_per_sm = kvq::kMma4CtasPerSm;
  } else {
    ctas_per_sm = kvq::kMmaWarpsPerSm / 4;
  }
}

}  // namespace

int32_t kvq_paged_attend_plan_chunk(const kvq_paged_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t q_dtype,
                                    const int32_t *host_seq_lens) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  if (check_paged_cache(cache, v) != KVQ_OK) return 0;
  if (!host_seq_lens || n_q_heads < 1 || n_q < 1 || n_q_heads % v.H) {
    fail(KVQ_EINVAL, "host_seq_lens is NULL or bad head counts");
    return 0;
  }
  if ((long long)(n_q_heads / v.H) * n_q > INT_MAX) {
    fail(KVQ_ESHAPE, "more than INT_MAX query rows of a kv head");
    return 0;
  }
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int per_sm = 1, per_unit = 1;
  bool window_ctas = false;
  phase1_capacity(v, (n_q_heads / v.H) * n_q, q_dtype, per_sm, per_unit, window_ctas);
  const long long ctas = (long long)sms * per_sm, capacity = ctas / per_unit;   // (head, chunk) units in one wave
  const int cap_len = v.cap;
  auto units = [&](int ch) {
    long long u = 0;
    for (int b = 0; b < v.B; ++b) {
      const int L = host_seq_lens[b] < 0 ? 0 : (host_seq_lens[b] > cap_len ? cap_len : host_seq_lens[b]);
      const int nw = kvq::is_hadamard(v.layout) ? (v.n_recent < L ? v.n_recent : L) : 0;
      const int nb = L - nw;
      u += nb > 0 ? (nb + ch - 1) / ch : 0;
      if (window_ctas) u += (nw + kvq::kWinChunk - 1) / kvq::kWinChunk;
    }
    return u * v.H;
  };
  // the shortest chunk whose units fit one wave: every CTA then has at most that many tokens
  for (int ch = 64; ch <= 8192; ch += 64)
    if (units(ch) <= capacity) return ch;
  // more work than one wave at the longest chunk: the least (waves x chunk)
  long long best = -1;
  int best_ch = 8192;
  for (int ch = 64; ch <= 8192; ch += 64) {
    // (a unit of more CTAs than a wave holds: counted by CTAs)
    const long long waves = capacity > 0 ? (units(ch) + capacity - 1) / capacity : (units(ch) * per_unit + ctas - 1) / ctas;
    const long long cost = waves * ch;
    if (best < 0 || cost < best) {
      best = cost;
      best_ch = ch;
    }
  }
  return best_ch;
}

size_t kvq_paged_attend_workspace_bytes(const kvq_paged_cache *cache, int32_t n_q_heads, int32_t n_q,
                                        int32_t max_kv_len, int32_t chunk) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (resolve_paged(cache, n_q_heads, n_q, max_kv_len, 0, chunk, a, need, nullptr) != KVQ_OK) return 0;
  return need;
}

int32_t kvq_paged_attend_chunk(const kvq_paged_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t max_kv_len,
                               int64_t total_kv_len, int32_t chunk) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (total_kv_len < 0) return 0;
  if (resolve_paged(cache, n_q_heads, n_q, max_kv_len, 0, chunk, a, need, nullptr, total_kv_len) != KVQ_OK) return 0;
  return a.chunk;
}

kvq_status kvq_paged_decode_attend(const kvq_paged_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads,
                                   int32_t n_q, const int32_t *seq_lens, int32_t max_kv_len, int32_t causal,
                                   float attn_scale, int32_t chunk, float *out, void *workspace,
                                   size_t workspace_bytes, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  kvq_status st = prepare_paged(cache, q, q_dtype, n_q_heads, n_q, seq_lens, max_kv_len, causal, attn_scale, chunk,
                                out, workspace, workspace_bytes, a);
  if (st != KVQ_OK) return st;
  cudaError_t e = launch_attend_sequence(a, reinterpret_cast<cudaStream_t>(stream), true);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_paged_append_decode_attend(const kvq_paged_cache *cache, const void *k_new, const void *v_new,
                                          int32_t kv_dtype, int32_t n_new, const void *q, int32_t q_dtype,
                                          int32_t n_q_heads, int32_t n_q, const int32_t *seq_lens,
                                          int32_t max_kv_len, int32_t causal, float attn_scale, int32_t chunk,
                                          float *out, void *workspace, size_t workspace_bytes,
                                          kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq_status st = check_paged_store(cache, k_new, v_new, kv_dtype, n_new, seq_lens, v);
  if (st != KVQ_OK) return st;
  kvq::AttendArgs a;
  st = prepare_paged(cache, q, q_dtype, n_q_heads, n_q, seq_lens, max_kv_len, causal, attn_scale, chunk, out,
                     workspace, workspace_bytes, a);
  if (st != KVQ_OK) return st;
  const cudaError_t e = launch_paged_append_attend(v, a, k_new, v_new, kv_dtype, n_new, seq_lens,
                                                   reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "append/attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// ------------------------------------------------------------------ rotary positions
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

kvq_status check_rot_dim(int rot_dim, int max_dim) {
  if (rot_dim < 16 || rot_dim > max_dim || rot_dim % 16)
    return fail(KVQ_ESHAPE, "rot_dim %d not a multiple of 16 in [16, %d]", rot_dim, max_dim);
  return KVQ_OK;
}

// Rows read by their strides: pointer and strides 16-byte aligned (the kernels load 16 bytes at a time).
kvq_status check_rows(const char *name, const kvq_rows *r, int dtype, kvq::RowsIn &in) {
  if (!r || !r->data) return fail(KVQ_EINVAL, "%s is NULL", name);
  const int64_t st[] = {r->batch_stride, r->head_stride, r->token_stride};
  for (int64_t x : st) {
    if (x < 0) return fail(KVQ_EINVAL, "%s has a negative stride", name);
    if (x % 16 * (int64_t)dtype_bytes(dtype) % 16) return fail(KVQ_EALIGN, "%s: a stride is not a multiple of 16 bytes", name);
  }
  if (!aligned(r->data, 16)) return fail(KVQ_EALIGN, "%s not 16-byte aligned", name);
  in = {r->data, r->batch_stride, r->head_stride, r->token_stride};
  return KVQ_OK;
}

// The arguments both rotary appends share, for a checked cache view.
kvq_status check_rope_store(const kvq::CacheView &v, const kvq_rope *rope, const kvq_rows *k_new, const kvq_rows *v_new,
                            const kvq_rows *q, int dtype, int n_q_heads, int n_new, void *q_out, kvq::RopeStore &g) {
  if (!rope || !rope->table) return fail(KVQ_EINVAL, "rope or its table is NULL");
  if (kvq::is_b64(v.layout)) return fail(KVQ_EUNSUPPORTED, "the rotary append has no block layouts (rotate, then kvq_store)");
  if (dtype < KVQ_F32 || dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown dtype %d", dtype);
  if (n_new < 0) return fail(KVQ_EINVAL, "n_new must be >= 0");
  if (n_q_heads < 0) return fail(KVQ_EINVAL, "n_q_heads must be >= 0");
  kvq_status st = check_rot_dim(rope->rot_dim, v.D);
  if (st != KVQ_OK) return st;
  if (rope->n_pos < 1) return fail(KVQ_EINVAL, "the rotary table has no positions");
  if (!aligned(rope->table, 16) || !aligned(rope->positions, 16))
    return fail(KVQ_EALIGN, "rotary table/positions not 16-byte aligned");
  if ((q != nullptr) != (n_q_heads > 0)) return fail(KVQ_EINVAL, "q and n_q_heads go together");
  if (n_q_heads % v.H) return fail(KVQ_ESHAPE, "n_q_heads %d not a multiple of n_kv_heads %d", n_q_heads, v.H);
  if ((long double)v.B * (2.0L * v.H + n_q_heads) * n_new * 32 > 256.0L * INT_MAX)
    return fail(KVQ_ESHAPE, "too many rows for one launch");
  if (n_new == 0) return KVQ_OK;                         // (buffers of no rows have no address)
  if (q && !q_out) return fail(KVQ_EINVAL, "q_out is NULL");
  if (q && !aligned(q_out, 16)) return fail(KVQ_EALIGN, "q_out not 16-byte aligned");
  st = check_rows("k_new", k_new, dtype, g.in[0]);
  if (st == KVQ_OK) st = check_rows("v_new", v_new, dtype, g.in[1]);
  g.in[2] = {nullptr, 0, 0, 0};
  if (st == KVQ_OK && q) st = check_rows("q", q, dtype, g.in[2]);
  if (st != KVQ_OK) return st;
  g.dtype = dtype; g.Hq = n_q_heads; g.n_new = n_new; g.pos0 = 0; g.slots = nullptr;
  g.table = rope->table; g.n_pos = rope->n_pos; g.rot = rope->rot_dim; g.interleaved = rope->interleaved ? 1 : 0;
  g.positions = rope->positions;
  g.q_out = q_out;
  g.k_rows = g.v_rows = g.q_rows = 0;
  g.row_bytes = 0;
  return KVQ_OK;
}

// q_out is written while other rows, and the other halves of its own, are still to be read: it lies outside the run
// of bytes from an input's first row to its last.
kvq_status check_q_out(const kvq::CacheView &v, const kvq::RopeStore &g) {
  const size_t size = dtype_bytes(g.dtype), out = (size_t)v.B * g.Hq * g.n_new * v.D * size;
  const char *const names[] = {"k_new", "v_new", "q"};
  for (int i = 0; i < 3; ++i) {
    const kvq::RowsIn &in = g.in[i];
    const int heads = i == 2 ? g.Hq : v.H;
    const size_t last = (size_t)(v.B - 1) * in.batch + (size_t)(heads - 1) * in.head + (size_t)(g.n_new - 1) * in.token;
    if (overlap(g.q_out, out, in.data, (last + v.D) * size)) return fail(KVQ_EINVAL, "q_out overlaps %s", names[i]);
  }
  return KVQ_OK;
}

}  // namespace

kvq_status kvq_rope_frequencies(const kvq_rope_config *config, double *inv_freq, float *magnitude) {
  g_last_error[0] = 0;
  if (!config || !inv_freq || !magnitude) return fail(KVQ_EINVAL, "config/inv_freq/magnitude is NULL");
  const kvq_rope_config &c = *config;
  const kvq_status st = check_rot_dim(c.rot_dim, 2 * kvq::kMaxRotHalf);
  if (st != KVQ_OK) return st;
  if (c.scaling < KVQ_ROPE_NONE || c.scaling > KVQ_ROPE_YARN) return fail(KVQ_EINVAL, "unknown scaling %d", c.scaling);
  if (!(c.base > 1.0) || std::isinf(c.base)) return fail(KVQ_EINVAL, "base must be finite and > 1");
  if (c.scaling != KVQ_ROPE_NONE && (!(c.factor > 0.0) || std::isinf(c.factor)))
    return fail(KVQ_EINVAL, "factor must be finite and > 0");
  const bool bands = c.scaling == KVQ_ROPE_BANDED || c.scaling == KVQ_ROPE_YARN;
  if (bands && (!(c.original_len > 0.0) || std::isinf(c.original_len) || !(c.low > 0.0) || !(c.high > c.low) || std::isinf(c.high)))
    return fail(KVQ_EINVAL, "original_len > 0 and 0 < low < high are needed");
  const int n = c.rot_dim / 2;
  const double base = c.scaling == KVQ_ROPE_NTK ? c.base * std::pow(c.factor, (double)c.rot_dim / (c.rot_dim - 2)) : c.base;
  if (!(base > 0.0) || std::isinf(base)) return fail(KVQ_EINVAL, "the scaled base is out of range");
  double lo = 0.0, hi = 0.0;
  if (c.scaling == KVQ_ROPE_YARN) {
    const double k = c.rot_dim / (2.0 * std::log(c.base));
    lo = std::fmin(std::fmax(std::floor(k * std::log(c.original_len / (c.high * kTwoPi))), 0.0), c.rot_dim - 1.0);
    hi = std::fmin(std::fmax(std::ceil(k * std::log(c.original_len / (c.low * kTwoPi))), 0.0), c.rot_dim - 1.0);
    if (hi <= lo) hi = lo + 0.001;                       // a step instead of a ramp
  }
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(base, -2.0 * i / c.rot_dim);
    double own = 1.0;                                    // the share of the unscaled frequency
    if (c.scaling == KVQ_ROPE_LINEAR) own = 0.0;
    if (c.scaling == KVQ_ROPE_BANDED)
      own = std::fmin(std::fmax((c.original_len * f / kTwoPi - c.low) / (c.high - c.low), 0.0), 1.0);
    if (c.scaling == KVQ_ROPE_YARN) own = 1.0 - std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
    inv_freq[i] = own == 1.0 ? f : f / c.factor * (1.0 - own) + f * own;
  }
  *magnitude = c.scaling == KVQ_ROPE_YARN && c.factor > 1.0 ? (float)(0.1 * std::log(c.factor) + 1.0) : 1.0f;
  return KVQ_OK;
}

kvq_status kvq_rope_table(const double *inv_freq, int32_t rot_dim, int32_t pos0, int32_t n_pos, float magnitude,
                          float *table, kvq_stream_t stream) {
  g_last_error[0] = 0;
  const kvq_status st = check_rot_dim(rot_dim, 2 * kvq::kMaxRotHalf);
  if (st != KVQ_OK) return st;
  if (pos0 < 0 || n_pos < 0 || (long long)pos0 + n_pos > INT_MAX)
    return fail(KVQ_EINVAL, "positions [%d, %lld) out of range", pos0, (long long)pos0 + n_pos);
  if (!std::isfinite(magnitude)) return fail(KVQ_EINVAL, "magnitude must be finite");
  if (n_pos == 0) return KVQ_OK;
  if (!inv_freq || !table) return fail(KVQ_EINVAL, "inv_freq/table is NULL");
  if (!aligned(table, 16)) return fail(KVQ_EALIGN, "table not 16-byte aligned");
  kvq::RopeTurns f = {};
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!(inv_freq[i] >= 0.0 && inv_freq[i] <= 65536.0)) return fail(KVQ_EINVAL, "inv_freq[%d] not in [0, 65536]", i);
    // inv_freq / 2 pi to 2^-64 of a turn: 1 / 2 pi as two doubles, the first product's rounding by an fma;
    // whole turns change nothing
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double turns = inv_freq[i] * kHi, rest = std::fma(inv_freq[i], kHi, -turns) + inv_freq[i] * kLo;
    f.turn[i] = (unsigned long long)std::ldexp(turns - std::floor(turns), 64) +
                (unsigned long long)std::llrint(std::ldexp(rest, 64));
  }
  const cudaError_t e = kvq::launch_rope_table(f, rot_dim, pos0, n_pos, magnitude, table, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "rope table launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_rope_store(const kvq_cache *cache, const kvq_rope *rope, const kvq_rows *k_new, const kvq_rows *v_new,
                          const kvq_rows *q, int32_t dtype, int32_t n_q_heads, int32_t n_new, int32_t pos0, void *q_out,
                          kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq::RopeStore g;
  kvq_status st = check_cache(cache, v);
  if (st == KVQ_OK) st = check_rope_store(v, rope, k_new, v_new, q, dtype, n_q_heads, n_new, q_out, g);
  if (st != KVQ_OK) return st;
  if (pos0 < 0) return fail(KVQ_EINVAL, "pos0 must be >= 0");
  if ((long long)pos0 + n_new > v.cap) return fail(KVQ_ECAPACITY, "pos0 + n_new = %lld > capacity %d", (long long)pos0 + n_new, v.cap);
  if (n_new == 0) return KVQ_OK;
  if ((st = check_q_out(v, g)) != KVQ_OK) return st;
  g.pos0 = pos0;
  const cudaError_t e = kvq::launch_rope_store(v, g, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "rope store launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_paged_rope_store(const kvq_paged_cache *cache, const kvq_rope *rope, const kvq_rows *k_new,
                                const kvq_rows *v_new, const kvq_rows *q, int32_t dtype, int32_t n_q_heads, int32_t n_new,
                                const int32_t *slots, void *q_out, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq::RopeStore g;
  kvq_status st = check_paged_cache(cache, v);
  if (st == KVQ_OK) st = check_rope_store(v, rope, k_new, v_new, q, dtype, n_q_heads, n_new, q_out, g);
  if (st != KVQ_OK) return st;
  if (n_new > v.cap) return fail(KVQ_ECAPACITY, "n_new %d > sequence capacity %d", n_new, v.cap);
  if (n_new == 0) return KVQ_OK;
  if (!slots) return fail(KVQ_EINVAL, "slots is NULL");
  if (!aligned(slots, 16)) return fail(KVQ_EALIGN, "slots not 16-byte aligned");
  if ((st = check_q_out(v, g)) != KVQ_OK) return st;
  g.slots = slots;
  const cudaError_t e = kvq::launch_rope_store(v, g, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "rope store launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// ------------------------------------------------------------------ a cache inside a budget
namespace {

constexpr int kMaxEvictTokens = 1 << 27;

// Chunk of an attention call that also scores the tokens, for chunk 0: the attention's own choice, but for four
// kinds.
//   Paged pools with up to two (sequence, kv head) per SM: up to 128 rows (whose partials are then at most 43 bytes
//     per token and kv head, less than a third of its packed row) at most 1536 tokens, since chunks that leave scores
//     behind take longer and the sequences' lengths differ (16 sequences of up to 16379 tokens, 8 kv heads: Q8_0 81 us
//     against 93 at the attention's 4608, asymmetric 101 against 140 at 8192; 64 sequences of 1000 to 4000, which fill
//     the SMs by themselves: 117 against 97). One long sequence, or equal ones, would gain by longer chunks, but what
//     the call knows is an upper bound of the lengths.
//   The tcgen05 kernel: as many chunks as fill the SMs beside the window's CTAs (it takes at most eight by itself:
//     64 CTAs for 128 rows and 8 kv heads; window CTAs in a second wave cost 13 us). Sequences of a paged batch count
//     as five eighths of the longest, here and below (4 of up to 16379 tokens, 256 rows, 8 kv heads 175 us; 210 without).
//   The row-side kernel with more rows than its decode form: the fewest waves of two CTAs per SM times the tokens of
//     a chunk and 256 more for what a CTA costs beside them, over one to four whole waves, so that the partials of a
//     call stay bounded whatever its length (four waves of 64 rows, or chunks of 8192 tokens). Q4_0, 128 rows, 8 kv
//     heads of 8000 tokens 70 us (the attention's own four to six waves: 108); Q8_0, 256 rows, 8 of 32768 333 (380;
//     chunks of 512 tokens 412); Q4_0, 256 rows, 8 of 131072 1114 (1475 at 512); 16 rows, 128 of 4096 174 (221).
//   The CUDA-core kernel, whose time goes with the chunk: 64 tokens where chunks of 128 leave SMs idle (Q4_0, d256,
//     4 kv heads of 5947 tokens: 29 against 44 us).
int weights_chunk(const kvq::CacheView &c, int n_q_heads, int n_q, int kv_len, int auto_chunk, bool f32_queries) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int chunk = auto_chunk;
  const long long heads = (long long)c.B * c.H;
  const int rows = n_q_heads / c.H * n_q;
  if (c.page_shift >= 0 && heads <= 2LL * sms && rows <= 128) chunk = std::min(chunk, 1536);
  const bool had = kvq::is_hadamard(c.layout), decode = kvq::decode_kernel(c.layout, c.v_layout);
  const int window = had ? std::min(c.n_recent, kv_len) : 0;
  const long long body = kv_len > window ? kv_len - window : 1;
  const long long n_win = (window + kvq::kWinChunk - 1) / kvq::kWinChunk;
  auto split = [&](long long n) { return (int)std::min(8192LL, ((body + n - 1) / n + 63) / 64 * 64); };   // into n chunks
  // CTAs of `per` query rows that one chunk of every sequence takes
  auto units = [&](int per) {
    const long long n = (long long)((rows + per - 1) / per) * heads;
    return c.page_shift >= 0 && c.B > 1 ? (5 * n + 7) / 8 : n;
  };
  if (kvq::tc_prefill_shape(c.layout, c.v_layout, c.D, rows)) {
    const long long n = (sms - heads * n_win) / units(kvq::kTcRows);
    if (n > 1) chunk = std::min(chunk, split(n));
  } else if (kvq::prefill_shape(c.layout, c.v_layout, c.D, rows) && (had || !f32_queries)) {
    if (rows > 16 || decode) {
      const long long slots = 2LL * sms, ctas = units(kvq::kPrefillRows);
      auto cost = [&](long long n) { return (ctas * (n + n_win) + slots - 1) / slots * (split(n) + 256); };
      long long best = (body + 8191) / 8192;
      for (long long waves = 1; waves <= 4; ++waves) {
        const long long n = waves * slots / ctas - n_win;
        if (n > (body + 8191) / 8192 && cost(n) < cost(best)) best = n;
      }
      chunk = split(best);
    }
  } else if (!(decode && c.D == 128 && rows <= 8) && !(c.layout == KVQ_Q6_0 && c.v_layout == c.layout && kvq::mma_q6_shape(c.D, rows))) {
    if (heads * ((body + 127) / 128) < 2LL * sms) chunk = 64;
  }
  return chunk;
}
int contiguous_chunk(const kvq_cache *cache, int n_q_heads, int n_q, int kv_len, int chunk, bool f32_queries) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (chunk || resolve_attend(cache, n_q_heads, n_q, kv_len, 0, 0, 0, a, need, nullptr) != KVQ_OK) return chunk;
  return weights_chunk(a.cache, n_q_heads, n_q, kv_len, a.chunk, f32_queries);
}
int paged_chunk(const kvq_paged_cache *cache, int n_q_heads, int n_q, int max_kv_len, int chunk, bool f32_queries) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (chunk || resolve_paged(cache, n_q_heads, n_q, max_kv_len, 0, 0, a, need, nullptr) != KVQ_OK) return chunk;
  return weights_chunk(a.cache, n_q_heads, n_q, max_kv_len, a.chunk, f32_queries);
}

// A weights call's workspace behind the attention's: the rows' log-sum-exp, then the scores that phase 1
// leaves behind on the kernels that can (score_rows).
struct WeightsSpace {
  size_t lse, scores, total;
  int rows, tokens;
};
WeightsSpace weights_space(const kvq::AttendArgs &a, size_t attend_need) {
  const kvq::CacheView &c = a.cache;
  WeightsSpace w;
  w.rows = kvq::score_rows(c.layout, c.v_layout, c.D, a.gqa * a.n_q);
  w.tokens = (a.n_body + 63) / 64 * 64;
  w.lse = round_up(attend_need, 256);
  w.scores = w.lse + round_up((size_t)c.B * a.Hq * a.n_q * sizeof(float), 256);
  w.total = w.scores + (size_t)c.B * c.H * w.tokens * w.rows * sizeof(float);
  return w;
}

// `rows`: of scores, batch * n_kv_heads
kvq_status check_scores(const float *scores_in, const float *scores_out, int64_t stride, int kv_len, float decay,
                        int64_t rows) {
  if (!scores_out) return fail(KVQ_EINVAL, "scores_out is NULL");
  if (!aligned(scores_in, 16) || !aligned(scores_out, 16)) return fail(KVQ_EALIGN, "scores not 16-byte aligned");
  if (stride < kv_len) return fail(KVQ_ESHAPE, "scores_stride %lld < kv_len %d", (long long)stride, kv_len);
  if (!std::isfinite(decay)) return fail(KVQ_EINVAL, "decay must be finite");
  if (scores_in && scores_in != scores_out && decay != 0.0f) {
    // scores_out starts k rows and r entries behind scores_in: one of its rows meets row k or row k + 1 of scores_in
    const int64_t d = (int64_t)((intptr_t)scores_out - (intptr_t)scores_in) / (int64_t)sizeof(float);
    const int64_t k = d >= 0 ? d / stride : -((stride - 1 - d) / stride), r = d - k * stride;
    if ((r < kv_len && std::abs(k) < rows) || (stride - r < kv_len && std::abs(k + 1) < rows))
      return fail(KVQ_EINVAL, "scores_in and scores_out overlap without being the same");
  }
  return KVQ_OK;
}

kvq_status run_weights(kvq::AttendArgs &a, size_t attend_need, void *workspace, size_t workspace_bytes, const float *scores_in,
                       float *scores_out, int64_t stride, float decay, cudaStream_t s) {
  const WeightsSpace w = weights_space(a, attend_need);
  if (workspace_bytes < w.total) return fail(KVQ_EWORKSPACE, "workspace %zu < required %zu", workspace_bytes, w.total);
  char *ws = static_cast<char *>(workspace);
  a.lse = reinterpret_cast<float *>(ws + w.lse);
  a.held = true;
  if (w.rows > 0 && w.tokens > 0) {
    a.part_s = reinterpret_cast<float *>(ws + w.scores);
    a.s_rows = w.rows;
    a.s_tokens = w.tokens;
  }
  cudaError_t e = launch_attend_sequence(a, s, true);
  if (e == cudaSuccess) e = kvq::launch_attend_weights(a, scores_in, scores_out, stride, decay, s);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "attend weights launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status check_evict(const int32_t *keep, int n_keep, int kv_len, const int32_t *seq_lens) {
  if (!keep) return fail(KVQ_EINVAL, "keep is NULL");
  if (!aligned(keep, 16) || !aligned(seq_lens, 16)) return fail(KVQ_EALIGN, "keep/seq_lens not 16-byte aligned");
  if (n_keep < 1) return fail(KVQ_EINVAL, "n_keep must be >= 1");
  if (kv_len < 1) return fail(KVQ_EINVAL, "kv_len must be >= 1");
  if (kv_len > kMaxEvictTokens) return fail(KVQ_ECAPACITY, "kv_len %d > %d", kv_len, kMaxEvictTokens);
  return KVQ_OK;
}

// The planes of a compaction, and its launch. Both views are checked; scores may be NULL.
kvq_status run_compact(const kvq::CacheView &src, const kvq::CacheView &dst, bool in_place, const int32_t *keep, int n_keep,
                       int kv_len, const int32_t *seq_lens, float *scores, int64_t scores_stride, float *scores_out,
                       int64_t out_stride, cudaStream_t s) {
  if (kvq::is_b64(src.layout)) return fail(KVQ_EUNSUPPORTED, "rows of a block layout share their block's scale: they do not move one by one");
  if (n_keep < src.n_recent) return fail(KVQ_EINVAL, "n_keep %d < n_recent %d: the window's tokens stay", n_keep, src.n_recent);
  const int most = n_keep < kv_len ? n_keep : kv_len;
  if (scores) {
    if (!aligned(scores, 16) || !aligned(scores_out, 16)) return fail(KVQ_EALIGN, "scores not 16-byte aligned");
    if (scores_stride < kv_len) return fail(KVQ_ESHAPE, "scores_stride %lld < kv_len %d", (long long)scores_stride, kv_len);
    if (out_stride < most) return fail(KVQ_ESHAPE, "out_stride %lld < %d kept tokens", (long long)out_stride, most);
    const size_t rows = (size_t)src.B * src.H - 1;
    if (scores_out != scores && overlap(scores, (rows * scores_stride + kv_len) * sizeof(float), scores_out,
                                        (rows * out_stride + std::min<int64_t>(out_stride, kv_len)) * sizeof(float)))
      return fail(KVQ_EINVAL, "scores and scores_out overlap");
  }
  kvq::CompactArgs a;
  a.src = src;
  a.dst = dst;
  a.keep = keep;
  a.seq_lens = seq_lens;
  a.n_keep = n_keep;
  a.kv_len = kv_len;
  a.ranks = 1;
  a.scores = scores;
  a.scores_out = scores_out;
  a.scores_stride = scores_stride;
  a.out_stride = out_stride;
  const cudaError_t e = kvq::launch_evict_compact(a, in_place, s);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "compact launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

}  // namespace

size_t kvq_attend_weights_workspace_bytes(const kvq_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t kv_len,
                                          int32_t chunk) {
  size_t most = 0;
  for (const bool f32_queries : {false, true}) {         // the queries' type is not known here
    kvq::AttendArgs a;
    size_t need = 0;
    const int ch = contiguous_chunk(cache, n_q_heads, n_q, kv_len, chunk, f32_queries);
    if (resolve_attend(cache, n_q_heads, n_q, kv_len, 0, 0, ch, a, need, nullptr) != KVQ_OK) return 0;
    most = std::max(most, weights_space(a, need).total);
  }
  return most;
}

size_t kvq_paged_attend_weights_workspace_bytes(const kvq_paged_cache *cache, int32_t n_q_heads, int32_t n_q,
                                                int32_t max_kv_len, int32_t chunk) {
  size_t most = 0;
  for (const bool f32_queries : {false, true}) {
    kvq::AttendArgs a;
    size_t need = 0;
    const int ch = paged_chunk(cache, n_q_heads, n_q, max_kv_len, chunk, f32_queries);
    if (resolve_paged(cache, n_q_heads, n_q, max_kv_len, 0, ch, a, need, nullptr) != KVQ_OK) return 0;
    most = std::max(most, weights_space(a, need).total);
  }
  return most;
}

kvq_status kvq_decode_attend_weights(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads,
                                     int32_t n_q, int32_t kv_len, int32_t causal, int32_t q_pos0, float attn_scale,
                                     int32_t chunk, float *out, const float *scores_in, float *scores_out,
                                     int64_t scores_stride, float decay, void *workspace, size_t workspace_bytes,
                                     kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  chunk = contiguous_chunk(cache, n_q_heads, n_q, kv_len, chunk, q_dtype == KVQ_F32);
  kvq_status st = prepare_attend(cache, q, q_dtype, n_q_heads, n_q, kv_len, causal, q_pos0, attn_scale, chunk, out,
                                 workspace, workspace_bytes, a);
  if (st == KVQ_OK && kvq::is_b64(a.cache.layout)) st = fail(KVQ_EUNSUPPORTED, "token weights are not provided for the block layouts");
  if (st == KVQ_OK) st = check_scores(scores_in, scores_out, scores_stride, kv_len, decay, (int64_t)a.cache.B * a.cache.H);
  if (st != KVQ_OK) return st;
  const size_t need = kvq_attend_workspace_bytes(cache, n_q_heads, n_q, kv_len, chunk);   // of the same chunk
  return run_weights(a, need, workspace, workspace_bytes, scores_in, scores_out, scores_stride, decay,
                     reinterpret_cast<cudaStream_t>(stream));
}

kvq_status kvq_paged_decode_attend_weights(const kvq_paged_cache *cache, const void *q, int32_t q_dtype,
                                           int32_t n_q_heads, int32_t n_q, const int32_t *seq_lens, int32_t max_kv_len,
                                           int32_t causal, float attn_scale, int32_t chunk, float *out,
                                           const float *scores_in, float *scores_out, int64_t scores_stride, float decay,
                                           void *workspace, size_t workspace_bytes, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  chunk = paged_chunk(cache, n_q_heads, n_q, max_kv_len, chunk, q_dtype == KVQ_F32);
  kvq_status st = prepare_paged(cache, q, q_dtype, n_q_heads, n_q, seq_lens, max_kv_len, causal, attn_scale, chunk, out,
                                workspace, workspace_bytes, a);
  if (st == KVQ_OK && kvq::is_b64(a.cache.layout)) st = fail(KVQ_EUNSUPPORTED, "token weights are not provided for the block layouts");
  if (st == KVQ_OK) st = check_scores(scores_in, scores_out, scores_stride, max_kv_len, decay, (int64_t)a.cache.B * a.cache.H);
  if (st != KVQ_OK) return st;
  const size_t need = kvq_paged_attend_workspace_bytes(cache, n_q_heads, n_q, max_kv_len, chunk);
  return run_weights(a, need, workspace, workspace_bytes, scores_in, scores_out, scores_stride, decay,
                     reinterpret_cast<cudaStream_t>(stream));
}

kvq_status kvq_evict_select(const float *scores, int32_t batch, int32_t n_kv_heads, int64_t scores_stride, int32_t kv_len,
                            const int32_t *seq_lens, int32_t n_keep, int32_t n_sink, int32_t n_recent, int32_t *keep,
                            int32_t *new_lens, kvq_stream_t stream) {
  g_last_error[0] = 0;
  const kvq_status st = check_evict(keep, n_keep, kv_len, seq_lens);
  if (st != KVQ_OK) return st;
  if (!scores) return fail(KVQ_EINVAL, "scores is NULL");
  if (!aligned(scores, 16) || !aligned(new_lens, 16)) return fail(KVQ_EALIGN, "scores/new_lens not 16-byte aligned");
  if (batch < 1 || n_kv_heads < 1) return fail(KVQ_EINVAL, "batch and n_kv_heads must be >= 1");
  if ((long long)batch * n_kv_heads > 1 << 24) return fail(KVQ_ESHAPE, "batch * n_kv_heads > 2^24");
  if (scores_stride < kv_len) return fail(KVQ_ESHAPE, "scores_stride %lld < kv_len %d", (long long)scores_stride, kv_len);
  if (n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > n_keep)
    return fail(KVQ_EINVAL, "n_sink and n_recent must be >= 0 and together at most n_keep");
  if (overlap(new_lens, batch * sizeof(int32_t), seq_lens, batch * sizeof(int32_t)))
    return fail(KVQ_EINVAL, "new_lens must not be seq_lens");
  const size_t rows = (size_t)batch * n_kv_heads;
  if (overlap(keep, rows * n_keep * sizeof(int32_t), scores, ((rows - 1) * scores_stride + kv_len) * sizeof(float)))
    return fail(KVQ_EINVAL, "keep overlaps the scores");
  kvq::SelectArgs a = {batch, n_kv_heads, kv_len, n_keep, n_sink, n_recent, scores_stride, scores, seq_lens, keep, new_lens};
  const cudaError_t e = kvq::launch_evict_select(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "select launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_evict_compact(const kvq_cache *cache, const kvq_cache *dst, const int32_t *keep, int32_t n_keep,
                             int32_t kv_len, float *scores, int64_t scores_stride, float *scores_out, int64_t out_stride,
                             kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v, d;
  kvq_status st = check_cache(cache, v);
  if (st == KVQ_OK) st = check_cache(dst ? dst : cache, d);
  if (st == KVQ_OK) st = check_evict(keep, n_keep, kv_len, nullptr);
  if (st != KVQ_OK) return st;
  if (kv_len > v.cap) return fail(KVQ_ECAPACITY, "kv_len %d > capacity %d", kv_len, v.cap);
  if (v.layout != d.layout || v.v_layout != d.v_layout || v.B != d.B || v.H != d.H || v.D != d.D || v.n_recent != d.n_recent)
    return fail(KVQ_ESHAPE, "dst differs from the cache in layout, batch, heads, head_dim or n_recent");
  // the same cache means every plane; a plane shared between two caches would be overwritten while it is read
  int same = 0, planes = 0;
  for (int t = 0; t < 2; ++t) {
    const int layout = t ? v.v_layout : v.layout;
    same += v.payload[t] == d.payload[t];
    same += v.scale[t] == d.scale[t];
    planes += 2;
    if (layout == KVQ_ASYM4_G32) same += v.zero[t] == d.zero[t], ++planes;
    if (v.n_recent > 0) same += v.ring[t] == d.ring[t], ++planes;
  }
  const bool in_place = same == planes && v.cap == d.cap;
  if (!in_place && same) return fail(KVQ_EINVAL, "dst shares planes with the cache");
  const int most = n_keep < kv_len ? n_keep : kv_len;
  if (most > d.cap) return fail(KVQ_ECAPACITY, "%d kept tokens > dst capacity %d", most, d.cap);
  if (in_place) {
    if (scores_out && scores_out != scores) return fail(KVQ_EINVAL, "in place the scores move in place too");
    scores_out = scores;
    out_stride = scores_stride;
  } else if (scores ? !scores_out || scores_out == scores : scores_out != nullptr) {
    return fail(KVQ_EINVAL, "with another dst the scores go to a scores_out of their own");
  }
  return run_compact(v, d, in_place, keep, n_keep, kv_len, nullptr, scores, scores_stride, scores_out, out_stride,
                     reinterpret_cast<cudaStream_t>(stream));
}

kvq_status kvq_paged_evict_compact(const kvq_paged_cache *cache, const int32_t *keep, int32_t n_keep,
                                   const int32_t *seq_lens, int32_t max_kv_len, float *scores, int64_t scores_stride,
                                   kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq_status st = check_paged_cache(cache, v);
  if (st == KVQ_OK && !seq_lens) st = fail(KVQ_EINVAL, "seq_lens is NULL");
  if (st == KVQ_OK) st = check_evict(keep, n_keep, max_kv_len, seq_lens);
  if (st != KVQ_OK) return st;
  if (max_kv_len > v.cap) return fail(KVQ_ECAPACITY, "max_kv_len %d > capacity %d", max_kv_len, v.cap);
  return run_compact(v, v, true, keep, n_keep, max_kv_len, seq_lens, scores, scores_stride, scores, scores_stride,
                     reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ steps planned on the device
kvq_status kvq_page_plan(int32_t batch, int32_t page_size, int32_t max_pages_per_seq, const int32_t *seq_lens,
                         const int32_t *new_lens, int32_t *block_table, int32_t *free_pages, int32_t n_pool,
                         const int32_t *n_free, int32_t max_tokens, int32_t *lens_out, int32_t *granted,
                         int32_t *n_free_out, int32_t *cu_new, int64_t *slots, int32_t *positions, kvq_stream_t stream) {
  g_last_error[0] = 0;
  if (batch < 1 || batch > 1 << 20) return fail(KVQ_EINVAL, "batch %d not in [1, 2^20]", batch);
  if (max_pages_per_seq < 1 || n_pool < 1) return fail(KVQ_EINVAL, "max_pages_per_seq and n_pool must be >= 1");
  if (max_tokens < 0 || max_tokens > 1 << 30) return fail(KVQ_EINVAL, "max_tokens %d not in [0, 2^30]", max_tokens);
  const int shift = page_shift_of(page_size);
  if (shift < 0) return fail(KVQ_ESHAPE, "page_size %d is not a power of two in [64, 2^20]", page_size);
  if ((long long)max_pages_per_seq * page_size > INT_MAX)
    return fail(KVQ_ECAPACITY, "max_pages_per_seq * page_size exceeds INT_MAX tokens");
  const size_t n = sizeof(int32_t), b = batch;
  const struct { const char *name; const void *p; size_t bytes; } bufs[] = {
      {"seq_lens", seq_lens, n * b}, {"new_lens", new_lens, n * b}, {"n_free", n_free, n},
      {"block_table", block_table, n * b * max_pages_per_seq}, {"free_pages", free_pages, n * n_pool},
      {"lens_out", lens_out, n * b}, {"granted", granted, n * b}, {"n_free_out", n_free_out, n}, {"cu_new", cu_new, n * (b + 1)},
      {"slots", slots, sizeof(int64_t) * max_tokens}, {"positions", positions, n * max_tokens}};
  constexpr int kInputs = 3, kAll = sizeof(bufs) / sizeof(bufs[0]);
  for (const auto &x : bufs) {
    if (!x.p && x.bytes) return fail(KVQ_EINVAL, "%s is NULL", x.name);
    if (!aligned(x.p, 16)) return fail(KVQ_EALIGN, "%s not 16-byte aligned", x.name);
  }
  for (int i = kInputs; i < kAll; ++i)
    for (int j = 0; j < i; ++j) {
      // in place: lens_out = seq_lens, granted = new_lens, n_free_out = n_free
      if (j < kInputs && i == j + 5 && bufs[i].p == bufs[j].p) continue;
      if (overlap(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes))
        return fail(KVQ_EINVAL, "%s overlaps %s", bufs[i].name, bufs[j].name);
    }
  const kvq::PlanArgs a = {batch, shift, max_pages_per_seq, n_pool, max_tokens, seq_lens, new_lens, n_free,
                           block_table, free_pages, lens_out, granted, n_free_out, cu_new, slots, positions};
  const cudaError_t e = kvq::launch_page_plan(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "page plan launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_paged_store_slots(const kvq_paged_cache *cache, const kvq_rows *k_new, const kvq_rows *v_new, int32_t dtype,
                                 int32_t n_tokens, const int64_t *slots, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  kvq_status st = check_paged_cache(cache, v);
  if (st != KVQ_OK) return st;
  if (v.n_recent > 0) return fail(KVQ_EUNSUPPORTED, "a slot map has no sequences: a cache with a window takes kvq_paged_store");
  if (dtype < KVQ_F32 || dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown dtype %d", dtype);
  if (n_tokens < 0) return fail(KVQ_EINVAL, "n_tokens must be >= 0");
  if ((long double)v.H * n_tokens * 2 * 32 > 256.0L * INT_MAX) return fail(KVQ_ESHAPE, "too many rows for one launch");
  if (n_tokens == 0) return KVQ_OK;
  kvq::SlotRows g;
  st = check_rows("k_new", k_new, dtype, g.k);
  if (st == KVQ_OK) st = check_rows("v_new", v_new, dtype, g.v);
  if (st != KVQ_OK) return st;
  if (!slots) return fail(KVQ_EINVAL, "slots is NULL");
  if (!aligned(slots, 16)) return fail(KVQ_EALIGN, "slots not 16-byte aligned");
  g.dtype = dtype;
  g.n_tokens = n_tokens;
  g.slots = reinterpret_cast<const long long *>(slots);
  const cudaError_t e = kvq::launch_store_slots(v, g, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "store launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// ------------------------------------------------------------------ attention over selected blocks
namespace {

// What the calls over blocks ask of a checked cache view: whole blocks, one basis, grids that hold every list.
kvq_status check_blocks(const kvq::CacheView &v, int n_q_heads, int n_q) {
  if (v.n_recent > 0) return fail(KVQ_EUNSUPPORTED, "blocks of a cache with a recent window are not provided");
  if (v.page_shift < 0 && v.cap % 64) return fail(KVQ_ESHAPE, "capacity %d not a multiple of 64", v.cap);
  if (n_q_heads < 1 || n_q < 1) return fail(KVQ_EINVAL, "n_q_heads and n_q must be >= 1");
  if (n_q_heads % v.H) return fail(KVQ_ESHAPE, "n_q_heads %d not a multiple of n_kv_heads %d", n_q_heads, v.H);
  if ((long long)v.B * v.H * n_q > 65535) return fail(KVQ_ESHAPE, "batch * n_kv_heads * n_q > 65535");
  const long long rows = v.page_shift < 0 ? (long long)v.B * v.H * v.cap : ((long long)v.n_pages * v.H) << v.page_shift;
  if (rows / 64 > INT_MAX) return fail(KVQ_ESHAPE, "more than INT_MAX blocks");
  return KVQ_OK;
}

kvq_status check_lengths(const kvq::CacheView &v, int n_q, const int32_t *seq_lens, int kv_len, int causal, int q_pos0) {
  const bool paged = v.page_shift >= 0;
  if (paged && !seq_lens) return fail(KVQ_EINVAL, "seq_lens is NULL");
  if (!aligned(seq_lens, 16)) return fail(KVQ_EALIGN, "seq_lens not 16-byte aligned");
  if (kv_len < 1) return fail(KVQ_EINVAL, "kv_len must be >= 1");
  if (kv_len > v.cap) return fail(KVQ_ECAPACITY, "kv_len %d > capacity %d", kv_len, v.cap);
  if (!paged && causal && (q_pos0 < 0 || (long long)q_pos0 + n_q > kv_len))
    return fail(KVQ_EINVAL, "causal call needs 0 <= q_pos0 and q_pos0 + n_q <= kv_len");
  return KVQ_OK;
}

kvq_status check_bounds(const kvq_block_bounds *bounds) {
  if (!bounds || !bounds->codes || !bounds->scale) return fail(KVQ_EINVAL, "bounds or one of its planes is NULL");
  if (!aligned(bounds->codes, 16) || !aligned(bounds->scale, 16)) return fail(KVQ_EALIGN, "bounds not 16-byte aligned");
  return KVQ_OK;
}

kvq_status run_bounds(const kvq::CacheView &v, const kvq_block_bounds *bounds, int first, int kv_len, int n_fresh,
                      const int32_t *seq_lens, kvq_stream_t stream) {
  kvq_status st = check_blocks(v, v.H, 1);
  if (st == KVQ_OK) st = check_bounds(bounds);
  if (st != KVQ_OK) return st;
  const kvq::BoundsArgs a = {v, bounds->codes, bounds->scale, first, kv_len, n_fresh, seq_lens};
  const cudaError_t e = kvq::launch_block_bounds(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "block bounds launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status run_block_select(const kvq::CacheView &v, const kvq_block_bounds *bounds, const void *q, int q_dtype, int n_q_heads,
                            int n_q, const int32_t *seq_lens, int kv_len, int causal, int q_pos0, int n_sel, int n_sink,
                            int n_recent, int32_t *sel, kvq_stream_t stream) {
  kvq_status st = check_blocks(v, n_q_heads, n_q);
  if (st == KVQ_OK) st = check_lengths(v, n_q, seq_lens, kv_len, causal, q_pos0);
  if (st == KVQ_OK) st = check_bounds(bounds);
  if (st != KVQ_OK) return st;
  if (q_dtype < KVQ_F32 || q_dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown q dtype %d", q_dtype);
  if (!q || !sel) return fail(KVQ_EINVAL, "q/sel is NULL");
  if (!aligned(q, 16) || !aligned(sel, 16)) return fail(KVQ_EALIGN, "q/sel not 16-byte aligned");
  if (((long long)kv_len + 63) / 64 > kvq::kMaxSelectBlocks) return fail(KVQ_ECAPACITY, "kv_len %d > 2^24", kv_len);
  if (n_sel < 1) return fail(KVQ_EINVAL, "n_sel must be >= 1");
  if (n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > n_sel)
    return fail(KVQ_EINVAL, "n_sink and n_recent must be >= 0 and together at most n_sel");
  const kvq::BlockSelectArgs a = {v, bounds->codes, bounds->scale, q, q_dtype, n_q_heads / v.H, n_q, kv_len, causal ? 1 : 0,
                                  q_pos0, kvq::is_hadamard(v.layout) ? 1 : 0, seq_lens, n_sel, n_sink, n_recent, sel};
  const cudaError_t e = kvq::launch_block_select(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "block select launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// The cache as a pool of pages of 64 tokens of one head, read by one sequence per list.
kvq::CacheView list_view(const kvq::CacheView &v, int n_q, int n_sel) {
  kvq::CacheView c = v;
  const long long rows = v.page_shift < 0 ? (long long)v.B * v.H * v.cap : ((long long)v.n_pages * v.H) << v.page_shift;
  c.B = v.B * v.H * n_q;
  c.H = 1;
  c.cap = n_sel * 64;
  c.page_shift = 6;
  c.table_stride = n_sel;
  c.n_pages = (int)(rows / 64);
  return c;
}

// The attention's arguments and workspace (its own, then the tables, the lengths and the queries by list).
struct SparseSpace {
  size_t table, lens, queries, total;
};
kvq_status resolve_sparse(const kvq::CacheView &v, int n_q_heads, int n_q, int n_sel, int chunk, kvq::AttendArgs &a, SparseSpace &w,
                          void *ws) {
  if (n_sel < 1 || n_sel > INT_MAX / 64) return fail(KVQ_EINVAL, "n_sel %d not in [1, 2^25)", n_sel);
  a.cache = list_view(v, n_q, n_sel);
  size_t need = 0;
  const kvq_status st = resolve_core(n_q_heads / v.H, 1, n_sel * 64, 0, 0, true, chunk, a, need, ws);
  if (st != KVQ_OK) return st;
  const size_t lists = (size_t)a.cache.B;
  w.table = round_up(need, 256);
  w.lens = w.table + round_up(lists * n_sel * sizeof(int32_t), 256);
  w.queries = w.lens + round_up(lists * sizeof(int32_t), 256);
  w.total = w.queries + (n_q > 1 ? lists * (n_q_heads / v.H) * v.D * sizeof(float) : 0);
  // Held to float32 (probabilities 2^12 larger, rounded additions) in every layout and for every number of heads: Q8_0, 64 rows
  // of 32 blocks 1.0e-5 -> 7e-7 of the output's norm, 79 -> 87 us. Over 4096 tokens with values of 0.001: Q6_0 7e-4 -> 4e-7, the
  // row-side kernel in Hadamard int4 4e-5 -> 4e-7 (rows of 32 blocks, 12 or 16 heads each: 81.5 -> 82.9 us, 91.3 -> 92.1).
  a.held = true;
  return KVQ_OK;
}

kvq_status run_sparse(const kvq::CacheView &v, const void *q, int q_dtype, int n_q_heads, int n_q, const int32_t *seq_lens,
                      int kv_len, int causal, int q_pos0, float attn_scale, const int32_t *sel, int n_sel, int chunk, float *out,
                      void *workspace, size_t workspace_bytes, kvq_stream_t stream) {
  kvq::AttendArgs a;
  SparseSpace w;
  kvq_status st = check_blocks(v, n_q_heads, n_q);
  if (st == KVQ_OK) st = check_lengths(v, n_q, seq_lens, kv_len, causal, q_pos0);
  if (st == KVQ_OK) st = resolve_sparse(v, n_q_heads, n_q, n_sel, chunk, a, w, nullptr);
  if (st == KVQ_OK) st = check_call(w.total, q, q_dtype, attn_scale, out, workspace, workspace_bytes);
  if (st != KVQ_OK) return st;
  if (!sel) return fail(KVQ_EINVAL, "sel is NULL");
  if (!aligned(sel, 16)) return fail(KVQ_EALIGN, "sel not 16-byte aligned");
  resolve_sparse(v, n_q_heads, n_q, n_sel, chunk, a, w, workspace);
  char *ws = static_cast<char *>(workspace);
  const kvq::SparseArgs p = {v, q, reinterpret_cast<uint4 *>(ws + w.queries), q_dtype, n_q_heads / v.H, n_q, kv_len,
                             causal ? 1 : 0, q_pos0, seq_lens, sel, n_sel, reinterpret_cast<int32_t *>(ws + w.table),
                             reinterpret_cast<int32_t *>(ws + w.lens)};
  a.cache.table = p.table;
  a.seq_lens = p.lens;
  a.q = n_q > 1 ? static_cast<const void *>(ws + w.queries) : q;
  a.q_dtype = q_dtype;
  a.scale = attn_scale;
  a.out = out;
  a.out_nq = n_q;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = kvq::launch_sparse_prepare(p, s);
  if (e == cudaSuccess) e = launch_attend_sequence(a, s, false);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "sparse attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

}  // namespace

kvq_status kvq_block_bounds_update(const kvq_cache *cache, const kvq_block_bounds *bounds, int32_t first, int32_t kv_len,
                                   kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  const kvq_status st = check_cache(cache, v);
  if (st != KVQ_OK) return st;
  if (first < 0 || kv_len < first) return fail(KVQ_EINVAL, "0 <= first <= kv_len is needed");
  if (kv_len > v.cap) return fail(KVQ_ECAPACITY, "kv_len %d > capacity %d", kv_len, v.cap);
  if (kv_len == first) return KVQ_OK;
  return run_bounds(v, bounds, first, kv_len, 0, nullptr, stream);
}

kvq_status kvq_paged_block_bounds_update(const kvq_paged_cache *cache, const kvq_block_bounds *bounds, const int32_t *seq_lens,
                                         int32_t n_fresh, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  const kvq_status st = check_paged_cache(cache, v);
  if (st != KVQ_OK) return st;
  if (n_fresh < 0) return fail(KVQ_EINVAL, "n_fresh must be >= 0");
  if (n_fresh == 0) return KVQ_OK;
  if (!seq_lens) return fail(KVQ_EINVAL, "seq_lens is NULL");
  if (!aligned(seq_lens, 16)) return fail(KVQ_EALIGN, "seq_lens not 16-byte aligned");
  return run_bounds(v, bounds, 0, v.cap, n_fresh, seq_lens, stream);
}

kvq_status kvq_block_select(const kvq_cache *cache, const kvq_block_bounds *bounds, const void *q, int32_t q_dtype,
                            int32_t n_q_heads, int32_t n_q, int32_t kv_len, int32_t causal, int32_t q_pos0, int32_t n_sel,
                            int32_t n_sink, int32_t n_recent, int32_t *sel, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  const kvq_status st = check_cache(cache, v);
  if (st != KVQ_OK) return st;
  return run_block_select(v, bounds, q, q_dtype, n_q_heads, n_q, nullptr, kv_len, causal, q_pos0, n_sel, n_sink, n_recent, sel,
                          stream);
}
kvq_status kvq_paged_block_select(const kvq_paged_cache *cache, const kvq_block_bounds *bounds, const void *q, int32_t q_dtype,
                                  int32_t n_q_heads, int32_t n_q, const int32_t *seq_lens, int32_t max_kv_len, int32_t causal,
                                  int32_t n_sel, int32_t n_sink, int32_t n_recent, int32_t *sel, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  const kvq_status st = check_paged_cache(cache, v);
  if (st != KVQ_OK) return st;
  return run_block_select(v, bounds, q, q_dtype, n_q_heads, n_q, seq_lens, max_kv_len, causal, 0, n_sel, n_sink, n_recent, sel,
                          stream);
}

size_t kvq_sparse_attend_workspace_bytes(const kvq_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t n_sel, int32_t chunk) {
  kvq::CacheView v;
  kvq::AttendArgs a;
  SparseSpace w;
  if (check_cache(cache, v) != KVQ_OK || check_blocks(v, n_q_heads, n_q) != KVQ_OK ||
      resolve_sparse(v, n_q_heads, n_q, n_sel, chunk, a, w, nullptr) != KVQ_OK) return 0;
  return w.total;
}
size_t kvq_paged_sparse_attend_workspace_bytes(const kvq_paged_cache *cache, int32_t n_q_heads, int32_t n_q, int32_t n_sel,
                                               int32_t chunk) {
  kvq::CacheView v;
  kvq::AttendArgs a;
  SparseSpace w;
  if (check_paged_cache(cache, v) != KVQ_OK || check_blocks(v, n_q_heads, n_q) != KVQ_OK ||
      resolve_sparse(v, n_q_heads, n_q, n_sel, chunk, a, w, nullptr) != KVQ_OK) return 0;
  return w.total;
}

kvq_status kvq_sparse_attend(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads, int32_t n_q, int32_t kv_len,
                             int32_t causal, int32_t q_pos0, float attn_scale, const int32_t *sel, int32_t n_sel, int32_t chunk,
                             float *out, void *workspace, size_t workspace_bytes, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  const kvq_status st = check_cache(cache, v);
  if (st != KVQ_OK) return st;
  return run_sparse(v, q, q_dtype, n_q_heads, n_q, nullptr, kv_len, causal, q_pos0, attn_scale, sel, n_sel, chunk, out, workspace,
                    workspace_bytes, stream);
}
kvq_status kvq_paged_sparse_attend(const kvq_paged_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads, int32_t n_q,
                                   const int32_t *seq_lens, int32_t max_kv_len, int32_t causal, float attn_scale,
                                   const int32_t *sel, int32_t n_sel, int32_t chunk, float *out, void *workspace,
                                   size_t workspace_bytes, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::CacheView v;
  const kvq_status st = check_paged_cache(cache, v);
  if (st != KVQ_OK) return st;
  return run_sparse(v, q, q_dtype, n_q_heads, n_q, seq_lens, max_kv_len, causal, 0, attn_scale, sel, n_sel, chunk, out, workspace,
                    workspace_bytes, stream);
}

// ------------------------------------------------------------------ host-buffer calls
size_t kvq_append_decode_attend_host_workspace_bytes(const kvq_cache *cache, int32_t kv_dtype, int32_t n_new,
                                                     int32_t q_dtype, int32_t n_q_heads, int32_t n_q,
                                                     int32_t kv_len, int32_t chunk) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (resolve_attend(cache, n_q_heads, n_q, kv_len, 0, 0, chunk, a, need, nullptr) != KVQ_OK) return 0;
  if (check_host_sizes(kv_dtype, n_new, q_dtype) != KVQ_OK) return 0;
  return host_staging(need, cache->batch, cache->n_kv_heads, cache->head_dim, kv_dtype, n_new, q_dtype, n_q_heads,
                      n_q, false).total;
}

kvq_status kvq_append_decode_attend_host(const kvq_cache *cache, const void *k_new, const void *v_new,
                                         int32_t kv_dtype, int32_t n_new, int32_t pos0, const void *q,
                                         int32_t q_dtype, int32_t n_q_heads, int32_t n_q, int32_t kv_len,
                                         int32_t causal, int32_t q_pos0, float attn_scale, int32_t chunk,
                                         float *out, void *workspace, size_t workspace_bytes,
                                         kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  size_t need = 0;
  kvq_status st = resolve_attend(cache, n_q_heads, n_q, kv_len, causal, q_pos0, chunk, a, need, nullptr);
  if (st != KVQ_OK) return st;
  st = check_host_args(kv_dtype, n_new, q_dtype, k_new, v_new, q, out, workspace);
  if (st != KVQ_OK) return st;
  const HostStaging h = host_staging(need, cache->batch, cache->n_kv_heads, cache->head_dim, kv_dtype, n_new,
                                     q_dtype, n_q_heads, n_q, false);
  if (workspace_bytes < h.total)
    return fail(KVQ_EWORKSPACE, "workspace %zu < required %zu", workspace_bytes, h.total);
  char *ws = static_cast<char *>(workspace);
  const HostIo io = host_io(h, ws, n_new, k_new, v_new, out);
  // both parts validated against the addresses the kernels will use before anything is enqueued
  kvq::CacheView v;
  st = check_store(-1, cache, io.k, io.v, kv_dtype, n_new, pos0, v);
  if (st != KVQ_OK) return st;
  st = prepare_attend(cache, io.q, q_dtype, n_q_heads, n_q, kv_len, causal, q_pos0, attn_scale, chunk, io.out,
                      workspace, need, a);
  if (st != KVQ_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = io.copy_in ? copy_in(h, ws, k_new, v_new, q, nullptr, s)
                             : cudaMemcpyAsync(ws + h.q, q, h.q_bytes, cudaMemcpyDefault, s);   // q only
  if (e == cudaSuccess) e = launch_append_attend(v, a, io.k, io.v, kv_dtype, n_new, pos0, s);
  if (e == cudaSuccess) e = io.copy_out ? copy_out_and_wait(h, ws, out, s) : cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "host-buffer append/attend: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

size_t kvq_paged_append_decode_attend_host_workspace_bytes(const kvq_paged_cache *cache, int32_t kv_dtype,
                                                           int32_t n_new, int32_t q_dtype, int32_t n_q_heads,
                                                           int32_t n_q, int32_t max_kv_len, int32_t chunk) {
  kvq::AttendArgs a;
  size_t need = 0;
  if (resolve_paged(cache, n_q_heads, n_q, max_kv_len, 0, chunk, a, need, nullptr) != KVQ_OK) return 0;
  if (check_host_sizes(kv_dtype, n_new, q_dtype) != KVQ_OK) return 0;
  return host_staging(need, cache->batch, cache->n_kv_heads, cache->head_dim, kv_dtype, n_new, q_dtype, n_q_heads,
                      n_q, true).total;
}

kvq_status kvq_paged_append_decode_attend_host(const kvq_paged_cache *cache, const void *k_new, const void *v_new,
                                               int32_t kv_dtype, int32_t n_new, const void *q, int32_t q_dtype,
                                               int32_t n_q_heads, int32_t n_q, const int32_t *seq_lens,
                                               int32_t max_kv_len, int32_t causal, float attn_scale, int32_t chunk,
                                               float *out, void *workspace, size_t workspace_bytes,
                                               kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  size_t need = 0;
  kvq_status st = resolve_paged(cache, n_q_heads, n_q, max_kv_len, causal, chunk, a, need, nullptr);
  if (st != KVQ_OK) return st;
  st = check_host_args(kv_dtype, n_new, q_dtype, k_new, v_new, q, out, workspace);
  if (st != KVQ_OK) return st;
  if (!seq_lens) return fail(KVQ_EINVAL, "seq_lens is NULL");
  const HostStaging h = host_staging(need, cache->batch, cache->n_kv_heads, cache->head_dim, kv_dtype, n_new,
                                     q_dtype, n_q_heads, n_q, true);
  if (workspace_bytes < h.total)
    return fail(KVQ_EWORKSPACE, "workspace %zu < required %zu", workspace_bytes, h.total);
  char *ws = static_cast<char *>(workspace);
  const HostIo io = host_io(h, ws, n_new, k_new, v_new, out);
  // the sequence lengths are read by every CTA: always staged in device memory
  const int32_t *lens = reinterpret_cast<const int32_t *>(ws + h.lens);
  kvq::CacheView v;
  st = check_paged_store(cache, io.k, io.v, kv_dtype, n_new, lens, v);
  if (st != KVQ_OK) return st;
  st = prepare_paged(cache, io.q, q_dtype, n_q_heads, n_q, lens, max_kv_len, causal, attn_scale, chunk, io.out,
                     workspace, need, a);
  if (st != KVQ_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (io.copy_in) {
    e = copy_in(h, ws, k_new, v_new, q, seq_lens, s);
  } else {                                               // q and the lengths only
    e = cudaMemcpyAsync(ws + h.q, q, h.q_bytes, cudaMemcpyDefault, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(ws + h.lens, seq_lens, h.lens_bytes, cudaMemcpyDefault, s);
  }
  if (e == cudaSuccess) e = launch_paged_append_attend(v, a, io.k, io.v, kv_dtype, n_new, lens, s);
  if (e == cudaSuccess) e = io.copy_out ? copy_out_and_wait(h, ws, out, s) : cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "host-buffer paged append/attend: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_debug_scores_i32(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads,
                                int32_t n_q, int32_t kv_len, int32_t *scores_out, float *s_q_out,
                                kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  size_t need = 0;
  kvq_status st = resolve_attend(cache, n_q_heads, n_q, kv_len, 0, 0, 0, a, need, nullptr);
  if (st != KVQ_OK) return st;
  if (!kvq::is_hadamard(a.cache.layout)) return fail(KVQ_EUNSUPPORTED, "integer scores exist for the Hadamard layouts only");
  if (q_dtype < KVQ_F32 || q_dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown q dtype %d", q_dtype);
  if (!q || !scores_out || !s_q_out) return fail(KVQ_EINVAL, "q/scores_out/s_q_out is NULL");
  if (!aligned(q, 16) || !aligned(scores_out, 16) || !aligned(s_q_out, 16))
    return fail(KVQ_EALIGN, "q/scores_out/s_q_out not 16-byte aligned");
  cudaError_t e = kvq::launch_debug_scores(a.cache, q, q_dtype, n_q_heads, n_q, kv_len, a.n_body, scores_out, s_q_out,
                                           reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "debug scores launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status kvq_debug_attend_scores_i32(const kvq_cache *cache, const void *q, int32_t q_dtype, int32_t n_q_heads,
                                       int32_t n_q, int32_t kv_len, int32_t causal, int32_t q_pos0, float attn_scale,
                                       int32_t chunk, float *out, void *workspace, size_t workspace_bytes,
                                       int32_t *scores_out, float *s_q_out, kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  kvq_status st = prepare_attend(cache, q, q_dtype, n_q_heads, n_q, kv_len, causal, q_pos0, attn_scale, chunk, out,
                                 workspace, workspace_bytes, a);
  if (st != KVQ_OK) return st;
  if (!scores_out || !s_q_out) return fail(KVQ_EINVAL, "scores_out/s_q_out is NULL");
  if (!aligned(scores_out, 16) || !aligned(s_q_out, 16)) return fail(KVQ_EALIGN, "scores_out/s_q_out not 16-byte aligned");
  if (!kvq::capture_supported(a))
    return fail(KVQ_EUNSUPPORTED, "score capture needs a contiguous Hadamard cache (one layout in both planes) "
                                  "whose body is scored by a tensor-core kernel");
  a.cap_scores = scores_out;
  a.cap_sq = s_q_out;
  cudaError_t e = launch_attend_sequence(a, reinterpret_cast<cudaStream_t>(stream), false);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

const char *kvq_status_string(int32_t status) {
  switch (status) {
    case KVQ_OK: return "ok";
    case KVQ_EINVAL: return "invalid argument";
    case KVQ_ESHAPE: return "unsupported shape";
    case KVQ_ECAPACITY: return "beyond cache capacity";
    case KVQ_EUNSUPPORTED: return "unsupported layout or option";
    case KVQ_EALIGN: return "misaligned pointer";
    case KVQ_ECUDA: return "CUDA launch error";
    case KVQ_EWORKSPACE: return "workspace too small";
    default: return "unknown status";
  }
}

const char *kvq_last_error(void) { return g_last_error; }

kvq_status kvq_profile_phase1_events(void *phase1_begin, void *phase1_end) {
  g_ev_begin = static_cast<cudaEvent_t>(phase1_begin);
  g_ev_end = static_cast<cudaEvent_t>(phase1_end);
  return KVQ_OK;
}

}  // extern "C"

// ------------------------------------------------------------------ allocation-free attention
// kvq_decode_attend_static: the same two-phase attention as kvq_decode_attend, for callers that
// cannot hand the library a workspace of their own. Its scratch is one file-scope device array
// of KVQ_STATIC_SCRATCH_BYTES, present on every device that loads the library for the life of
// the process. Host code resolves the array's device address with cudaGetSymbolAddress (the
// array's name is only a host-side stand-in) once per device, on the first call made with that
// device current, and keeps it.
namespace {

static __device__ __align__(256) unsigned char g_static_scratch[KVQ_STATIC_SCRATCH_BYTES];
std::mutex g_static_mu;
void *g_static_ptr[kvq::kMaxDevices] = {};

cudaError_t static_scratch_of_current_device(void **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kvq::kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_static_mu);
  if (!g_static_ptr[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_static_scratch);
    if (e != cudaSuccess) return e;
    g_static_ptr[dev] = p;
  }
  *out = g_static_ptr[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" kvq_status kvq_decode_attend_static(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                               int32_t n_q_heads, int32_t n_q, int32_t kv_len, int32_t causal,
                                               int32_t q_pos0, float attn_scale, int32_t chunk, float *out,
                                               kvq_stream_t stream) {
  g_last_error[0] = 0;
  kvq::AttendArgs a;
  size_t need = 0;
  kvq_status st = resolve_attend(cache, n_q_heads, n_q, kv_len, causal, q_pos0, chunk, a, need, nullptr);
  if (st != KVQ_OK) return st;
  if (q_dtype < KVQ_F32 || q_dtype > KVQ_F16) return fail(KVQ_EINVAL, "unknown q dtype %d", q_dtype);
  if (!q || !out) return fail(KVQ_EINVAL, "q/out is NULL");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_EALIGN, "q/out not 16-byte aligned");
  if (!(attn_scale == attn_scale) || attn_scale > 3.0e38f || attn_scale < -3.0e38f)
    return fail(KVQ_EINVAL, "attn_scale must be finite");
  if (need > (size_t)KVQ_STATIC_SCRATCH_BYTES)
    return fail(KVQ_EWORKSPACE, "call needs %zu bytes of scratch; the built-in scratch holds %zu", need,
                (size_t)KVQ_STATIC_SCRATCH_BYTES);
  void *ws = nullptr;
  cudaError_t e = static_scratch_of_current_device(&ws);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "built-in scratch address: %s", cudaGetErrorString(e));
  resolve_attend(cache, n_q_heads, n_q, kv_len, causal, q_pos0, chunk, a, need, ws);
  a.q = q;
  a.q_dtype = q_dtype;
  a.scale = attn_scale;
  a.out = out;
  e = launch_attend_sequence(a, reinterpret_cast<cudaStream_t>(stream), false);
  if (e != cudaSuccess) return fail(KVQ_ECUDA, "attend launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}
