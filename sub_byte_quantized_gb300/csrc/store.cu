// Store (append) kernels: quantise new K/V rows and write them into the packed cache.
//
// Bit-exactness: every value is produced by one IEEE float32 operation at a time
// (__fdiv_rn / __fsub_rn / __fmul_rn, rintf = round half to even, __float2half_rn), and this
// file is compiled with -fmad=false so no multiply-add is ever contracted.
//
// Q4_0 / Q6_0 / Q8_0 / asymmetric: 4 threads per 32-value block, 8 values per thread; the
// block's amax (or min/max) is reduced over those 4 lanes with shuffles. Loads are 16-byte
// vectors, stores are the thread's 4 payload bytes (+ 2 high-plane bytes for Q6_0; 8 bytes for
// Q8_0).
// Hadamard int4 / int2: one warp per token row; the FWHT runs in registers and shuffles.
#include "store_quant.cuh"

namespace kvq {
namespace {

struct StoreGeom {
  int B, H, D, cap, n_new, pos0, row_bytes, nb;
  long long rows_per_tensor;   // B * H * n_new
  long long n_rows;            // rows of this launch: both planes (2 * rows_per_tensor) or one
  int kv_only;                 // -1: K and V in one launch; 0 / 1: this launch covers that plane only
  // per-sequence first position seq_pos[b] + pos_offset (device), or nullptr: pos0 for every one
  const int32_t *seq_pos;
  int pos_offset;
  // a ragged run of tokens: strides of k and v in elements, and each token's pool row
  long long head[2], token[2];
  const long long *slots;
};

// Row r of a ragged run: heads of one token are neighbours. False where the token has no row in the pool.
__device__ __forceinline__ bool slot_coords(const CacheView &c, const StoreGeom &g, long long r, int &kv, long long &elem,
                                            long long &crow) {
  kv = g.kv_only >= 0 ? g.kv_only : (r >= g.rows_per_tensor ? 1 : 0);
  const long long rr = g.kv_only >= 0 ? r : r - (long long)kv * g.rows_per_tensor;
  const long long t = rr / g.H;
  const int h = (int)(rr - t * g.H);
  const long long slot = __ldg(g.slots + t);
  elem = t * g.token[kv] + h * g.head[kv];
  const bool ok = slot >= 0 && slot < (long long)c.n_pages << c.page_shift;
  crow = ok ? ((((slot >> c.page_shift) * c.H + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1))) : 0;
  return ok;
}

// Decompose a global row id into (tensor, input row, plane row, row j of the append, position,
// batch * H + head). False when the position is outside [0, cap): a per-sequence position the
// host could not check; such a row is computed but not written.
__device__ __forceinline__ bool row_coords(const CacheView &c, const StoreGeom &g, long long r, int &kv,
                                           long long &in_row, long long &crow, int &j, int &pos, long long &bh) {
  kv = g.kv_only >= 0 ? g.kv_only : (r >= g.rows_per_tensor ? 1 : 0);
  const long long rr = g.kv_only >= 0 ? r : r - (long long)kv * g.rows_per_tensor;
  in_row = rr;
  int bb, kvh;
  if (g.rows_per_tensor <= 0x7FFFFFFFLL) {                // 32-bit index arithmetic (every realistic call)
    const unsigned ur = (unsigned)rr, nn = (unsigned)g.n_new, hh = (unsigned)g.H;
    const unsigned ubh = ur / nn, ubb = ubh / hh;
    j = (int)(ur - ubh * nn);
    bh = ubh;
    bb = (int)ubb;
    kvh = (int)(ubh - ubb * hh);
  } else {
    bh = rr / g.n_new;
    j = (int)(rr - bh * g.n_new);
    bb = (int)(bh / g.H);
    kvh = (int)(bh - (long long)bb * g.H);
  }
  pos = (g.seq_pos ? __ldg(g.seq_pos + bb) + g.pos_offset : g.pos0) + j;
  const bool ok = pos >= 0 && pos < g.cap;
  crow = ok ? (long long)cache_row(c, bb, kvh, pos) : 0;
  return ok;
}

// LAYOUT: KVQ_Q4_0, KVQ_Q6_0, KVQ_Q8_0 or KVQ_ASYM4_G32. SLOTS: rows of a ragged run by their pool rows.
template <int LAYOUT, bool SLOTS>
__global__ void __launch_bounds__(256) store_block_kernel(CacheView c, const void *__restrict__ k_new,
                                                          const void *__restrict__ v_new, int dtype,
                                                          StoreGeom g) {
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");   // attention may launch and wait on us
#endif
  const int tpr_shift = g.D == 128 ? 4 : 5;                // D / 8 threads per row
  const long long gt = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long r = gt >> tpr_shift;
  const int tr = (int)(gt & ((1 << tpr_shift) - 1));      // thread within row
  // Threads past the last row still take part in the quad shuffles (full-warp masks) but load
  // and store nothing.
  bool valid = r < g.n_rows;
  int kv = 0, j = 0, pos = 0;
  long long in_row = 0, crow = 0, bh = 0;
  if constexpr (SLOTS) {
    if (valid) valid = slot_coords(c, g, r, kv, in_row, crow);
  } else {
    if (valid) valid = row_coords(c, g, r, kv, in_row, crow, j, pos, bh);
  }
  const int blk = tr >> 2, lb = tr & 3;

  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (valid) load8_f32(kv ? v_new : k_new, dtype, (SLOTS ? (size_t)in_row : (size_t)in_row * g.D) + (size_t)tr * 8, v);
  quant_block<LAYOUT, 8>(c, kv, crow, g.row_bytes, g.nb, blk, lb, v, valid);
}

// Hadamard int4 (BITS 4: scale amax / 7, codes [-7, 7], two per byte) or int2 (BITS 2: scale
// amax, codes [-1, 1], four per byte): one warp per token row, V = D/32 values per lane.
template <int V, int BITS, bool SLOTS>
__global__ void __launch_bounds__(256) store_had_kernel(CacheView c, const void *__restrict__ k_new,
                                                        const void *__restrict__ v_new, int dtype,
                                                        StoreGeom g) {
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");   // attention may launch and wait on us
#endif
  const int lane = threadIdx.x & 31;
  const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (r >= g.n_rows) return;                               // whole warp exits together
  int kv, j = 0, pos = 0;
  long long in_row, crow, bh = 0;
  if constexpr (SLOTS) {                                   // (a ragged run has no window)
    if (!slot_coords(c, g, r, kv, in_row, crow)) return;
  } else {
    if (!row_coords(c, g, r, kv, in_row, crow, j, pos, bh)) return;   // whole warp (one row)
  }
  float x[V];
  const void *src = kv ? v_new : k_new;
  const size_t elem = SLOTS ? (size_t)in_row : (size_t)in_row * g.D;
  if (V == 4) {
    load4_f32(src, dtype, elem + lane * 4, x);
  } else {
    load8_f32(src, dtype, elem + lane * 8, x);
  }
  // Exact-f32 ring of the newest tokens: only the last min(n_new, n_recent) rows of this call,
  // so no two rows of one call write the same slot.
  quant_had<V, 32, BITS>(c, kv, crow, g.row_bytes, lane, x, c.n_recent > 0 && j >= g.n_new - c.n_recent, bh, pos, true);
}

}  // namespace

namespace {

// One launch of the store kernel for `layout` over both planes (kv_only < 0) or one plane.
template <bool SLOTS>
cudaError_t launch_store_plane(const CacheView &c, int layout, const void *k_new, const void *v_new, int dtype,
                               StoreGeom g, cudaStream_t st) {
  const long long rows = g.n_rows;
  if (is_hadamard(layout)) {
    const unsigned blocks = (unsigned)((rows * 32 + 255) / 256);
    const bool two = layout == KVQ_HAD_INT2;
    if (c.D == 128) {
      if (two) store_had_kernel<4, 2, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g);
      else store_had_kernel<4, 4, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g);
    } else {
      if (two) store_had_kernel<8, 2, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g);
      else store_had_kernel<8, 4, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g);
    }
  } else {
    const long long threads = rows * (c.D / 8);
    const unsigned blocks = (unsigned)((threads + 255) / 256);
    switch (layout) {
      case KVQ_Q4_0: store_block_kernel<KVQ_Q4_0, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g); break;
      case KVQ_Q6_0: store_block_kernel<KVQ_Q6_0, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g); break;
      case KVQ_Q8_0: store_block_kernel<KVQ_Q8_0, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g); break;
      default: store_block_kernel<KVQ_ASYM4_G32, SLOTS><<<blocks, 256, 0, st>>>(c, k_new, v_new, dtype, g); break;
    }
  }
  return cudaGetLastError();
}

}  // namespace

namespace {

// Both planes in one launch, or one launch per plane of a mixed cache, each with its own layout.
template <bool SLOTS>
cudaError_t launch_store_planes(const CacheView &c, const void *k_new, const void *v_new, int dtype, StoreGeom &g, cudaStream_t st) {
  g.B = c.B; g.H = c.H; g.D = c.D; g.cap = c.cap;
  g.nb = c.D / kBlock;
  if (c.layout == c.v_layout) {
    g.row_bytes = c.row_bytes;
    g.n_rows = 2 * g.rows_per_tensor;
    g.kv_only = -1;
    return launch_store_plane<SLOTS>(c, c.layout, k_new, v_new, dtype, g, st);
  }
  g.n_rows = g.rows_per_tensor;
  g.kv_only = 0;
  g.row_bytes = c.row_bytes;
  cudaError_t e = launch_store_plane<SLOTS>(c, c.layout, k_new, v_new, dtype, g, st);
  if (e != cudaSuccess) return e;
  g.kv_only = 1;
  g.row_bytes = c.v_row_bytes;
  return launch_store_plane<SLOTS>(c, c.v_layout, k_new, v_new, dtype, g, st);
}

}  // namespace

cudaError_t launch_store(const CacheView &c, const void *k_new, const void *v_new, int dtype, int n_new,
                         int pos0, cudaStream_t st, const int32_t *seq_pos, int pos_offset) {
  if (is_b64(c.layout)) return launch_store_b64(c, k_new, v_new, dtype, n_new, pos0, st, seq_pos, pos_offset);
  StoreGeom g = {};
  g.n_new = n_new; g.pos0 = pos0;
  g.seq_pos = seq_pos; g.pos_offset = pos_offset;
  g.rows_per_tensor = (long long)c.B * c.H * n_new;
  return launch_store_planes<false>(c, k_new, v_new, dtype, g, st);
}

cudaError_t launch_store_slots(const CacheView &c, const SlotRows &r, cudaStream_t st) {
  if (is_b64(c.layout)) return launch_store_b64_slots(c, r, st);
  StoreGeom g = {};
  g.head[0] = r.k.head; g.head[1] = r.v.head;
  g.token[0] = r.k.token; g.token[1] = r.v.token;
  g.slots = r.slots;
  g.rows_per_tensor = (long long)c.H * r.n_tokens;
  return launch_store_planes<true>(c, r.k.data, r.v.data, r.dtype, g, st);
}

}  // namespace kvq
