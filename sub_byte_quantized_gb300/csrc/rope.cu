// Rotary positions: the table of cosines and sines, and the append that rotates.
//
// Table. Row p holds cos(p f_i) m, i = 0 .. h-1, then sin(p f_i) m, h = rot_dim / 2. A far position's
// angle has lost its fraction of a turn in float32 (p f = 1e5 leaves 2^-7 of a radian), so the angle is
// counted in turns: f_i / 2 pi as a 64-bit binary fraction, and p times it in wrapping 64-bit integers,
// which takes whole turns off exactly. The upper 32 bits, rounded, are the angle (off by 2^-33 of a turn: 7e-10
// in the entry, an eightieth of a rounding of the entries near 1). The nearest quarter turn goes into signs and a
// swap; what is left, in [-1/8, 1/8) of a turn, is rounded to float32 and goes into two short polynomials.
//
// Append with rotary positions. One launch reads q, k and v from wherever their projection left them
// (any strides between batches, heads and tokens), rotates q and k, and writes q in its own type and k
// and v packed: nothing is rotated into memory and read again. Half layout: dims (i, i + h) are a pair;
// interleaved: dims (2 i, 2 i + 1); dims from rot_dim on stay as they are.
//   y_a = x_a c - x_b s,   y_b = x_b c + x_a s
// Each product and each sum is rounded to float32 by itself (this file is compiled with -fmad=false),
// so the packed bytes follow from the table's entries exactly. A thread holds 16 dims of a row (block
// layouts) or 8 (Hadamard); its partners' dims (half layout) are a second 16-byte load of the same row,
// which the L1 answers.
//
// 8192 tokens, 16 q and 8 kv heads of 256 dims (f16, asymmetric) move 224 MB, 33 us at the copy rate; 53.9 us. What
// limits them is open: issue slots 79 % busy and DRAM 44 %, yet fewer instructions did not help.
#include "mma_util.cuh"
#include "store_quant.cuh"

namespace kvq {
namespace {
using namespace mma;

constexpr int kTableThreads = 256;
constexpr int kTableRows = 8;        // positions per thread, a grid apart

// sin(pi u) and cos(pi u) for |u| <= 1/4, by their Taylor polynomials in u^2 (remainders below 2^-29);
// pi is split so that only u's own rounding and the last addition count.
__device__ __forceinline__ void sincos_pi(float u, float &s, float &c) {
  const float z = __fmul_rn(u, u);
  float p = 0.08214588661112823f;                        // pi^9 / 9!
  p = __fmaf_rn(p, z, -0.5992645293207921f);             // pi^7 / 7!
  p = __fmaf_rn(p, z, 2.550164039877345f);               // pi^5 / 5!
  p = __fmaf_rn(p, z, -5.16771278004997f);               // pi^3 / 3!
  p = __fmaf_rn(p, z, -8.742277657347586e-08f);          // pi - fl(pi)
  s = __fmaf_rn(u, 3.1415927410125732f, __fmul_rn(u, p));
  float q = -0.025806891390014061f;                      // pi^10 / 10!
  q = __fmaf_rn(q, z, 0.23533063035889321f);             // pi^8 / 8!
  q = __fmaf_rn(q, z, -1.3352627688545895f);             // pi^6 / 6!
  q = __fmaf_rn(q, z, 4.0587121264167682f);              // pi^4 / 4!
  q = __fmaf_rn(q, z, -4.9348022005446793f);             // pi^2 / 2!
  c = __fmaf_rn(q, z, 1.0f);
}

// Thread (frequency quad, first row) steps through its positions by adding rows * f to the angle: the
// frequencies, read at an index of its own per lane, are loaded once per thread. 16-byte stores.
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(RopeTurns f, int half, int pos0, int n_pos, int rows, float mag,
                                                                   float *__restrict__ table) {
  const int quads = half >> 2;
  const long long id = (long long)blockIdx.x * kTableThreads + threadIdx.x;
  const long long first = id / quads;
  if (first >= rows) return;
  const int i0 = 4 * (int)(id - first * quads);
  unsigned long long turn[4], step[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned long long t = f.turn[i0 + k];
    // in 2^-64 turns, whole turns gone; the half of 2^-32 rounds the upper word, which is what is read
    turn[k] = ((unsigned long long)pos0 + (unsigned long long)first) * t + (1ull << 31);
    step[k] = (unsigned long long)rows * t;
  }
  for (long long p = first; p < n_pos; p += rows) {
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned angle = (unsigned)(turn[k] >> 32);          // in 2^-32 turns
      const unsigned quarter = (angle + (1u << 29)) >> 30;       // nearest quarter turn (0 .. 3)
      const int rest = (int)(angle - (quarter << 30));           // [-2^29, 2^29)
      float sr, cr;
      sincos_pi(__int2float_rn(rest) * 0x1.0p-31f, sr, cr);      // in units of pi
      const float sv = (quarter & 1) ? cr : sr, cv = (quarter & 1) ? sr : cr;
      s[k] = __fmul_rn((quarter & 2) ? -sv : sv, mag);
      c[k] = __fmul_rn(((quarter + 1) & 2) ? -cv : cv, mag);     // cos is negative in quarters 1 and 2
      turn[k] += step[k];
    }
    float *row = table + (size_t)p * (2 * half) + i0;
    *reinterpret_cast<float4 *>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4 *>(row + half) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// n / d for n < 2^31 by one high product, (n + umulhi(n, mul)) >> shift, with the multiplier of Granlund and Montgomery
// ("Division by invariant integers using multiplication", 1994): 2^32 + mul = floor(2^(32 + shift) / d) + 1.
__device__ __forceinline__ unsigned divide(unsigned n, const FastDiv &d) { return (n + __umulhi(n, d.mul)) >> d.shift; }

// The row a group of threads works on: K rows first, then V, then q.
struct RopeRow {
  int what;                 // 0 = K, 1 = V, 2 = q
  int b, head, j, pos, at;  // batch, head (kv or query), row of the append, cache slot, table row
  long long crow;           // plane row (K and V)
};
// Grid column y of a LONG launch (many rows per head): K, V or q, batch entry and head. Columns run fastest:
// the heads of a token lie side by side in a fused projection's output.
__device__ __forceinline__ void rope_column(const CacheView &c, const RopeStore &g, unsigned y, RopeRow &w) {
  const unsigned kv = (unsigned)(c.B * c.H), k = g.k_rows ? kv : 0u, v = g.v_rows ? kv : 0u;
  w.what = y < k ? 0 : (y < k + v ? 1 : 2);
  const unsigned bh = y - (w.what == 0 ? 0u : (w.what == 1 ? k : k + v));
  w.b = (int)divide(bh, w.what == 2 ? g.by_q_heads : g.by_kv_heads);
  w.head = (int)(bh - (unsigned)w.b * (w.what == 2 ? (unsigned)g.Hq : (unsigned)c.H));
}
// Row r of a launch's rows in order: K, V or q, batch entry, head and row of the append.
__device__ __forceinline__ void rope_split(const CacheView &c, const RopeStore &g, long long group, RopeRow &w) {
  w.what = group < g.k_rows ? 0 : (group < g.k_rows + g.v_rows ? 1 : 2);
  const long long r = group - (w.what == 0 ? 0 : (w.what == 1 ? g.k_rows : g.k_rows + g.v_rows));
  const int heads = w.what == 2 ? g.Hq : c.H;
  if (r <= 0x7FFFFFFFLL) {
    const unsigned bh = divide((unsigned)r, g.by_new);
    w.j = (int)((unsigned)r - bh * (unsigned)g.n_new);
    w.b = (int)divide(bh, w.what == 2 ? g.by_q_heads : g.by_kv_heads);
    w.head = (int)(bh - (unsigned)w.b * (unsigned)heads);
  } else {
    const long long bh = r / g.n_new;
    w.j = (int)(r - bh * g.n_new);
    w.b = (int)(bh / heads);
    w.head = (int)(bh - (long long)w.b * heads);
  }
}
// The rest of row w.j: its slot, plane row and table row; false when there is nothing to write.
__device__ __forceinline__ bool rope_place(const CacheView &c, const RopeStore &g, RopeRow &w) {
  // a slot is 64-bit until it is known to lie inside the cache
  const long long slot = (g.slots ? (long long)__ldg(g.slots + w.b) : (long long)g.pos0) + w.j;
  const bool inside = slot >= 0 && slot < c.cap;
  w.pos = (int)min(max(slot, (long long)INT_MIN), (long long)INT_MAX);   // also the default rotary position
  if (w.what != 1) w.at = min(max(g.positions ? __ldg(g.positions + (size_t)w.b * g.n_new + w.j) : w.pos, 0), g.n_pos - 1);
  if (w.what == 2) return true;
  w.crow = inside ? (long long)cache_row(c, w.b, w.head, w.pos) : 0;
  return inside;
}

// Eight elements from the e-th of `in`, in global memory or (SM) in shared memory.
template <int DT, bool SM>
__device__ __forceinline__ void load8(const void *in, size_t e, float (&v)[8]) {
  if constexpr (!SM) {
    load8_f32(in, DT, e, v);
  } else if constexpr (DT == KVQ_F32) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(static_cast<const float *>(in) + e + i);
  } else {
    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(in) + e);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == KVQ_BF16) {
        v[2 * k] = bf16_bits_to_f32(u[k] & 0xFFFFu);
        v[2 * k + 1] = bf16_bits_to_f32(u[k] >> 16);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[k]));
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      }
    }
  }
}

// Eight consecutive dims from d0 of one row (at element `row` of `in`), rotated when the row is K or q and d0 < rot_dim (a multiple of
// 16: all eight are on the same side of rot_dim and of its half).
template <int DT, bool SM>
__device__ __forceinline__ void rope_load(const RopeStore &g, const RopeRow &w, const void *in, size_t row, int d0, float *y) {
  float x[8];
  load8<DT, SM>(in, row + d0, x);
  if (w.what == 1 || d0 >= g.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    return;
  }
  const float *t = g.table + (size_t)w.at * g.rot;
  const int half = g.rot >> 1;
  if (g.interleaved) {
    float c[4], s[4];
    load4_f32(t, KVQ_F32, d0 >> 1, c);
    load4_f32(t, KVQ_F32, half + (d0 >> 1), s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], c[i]), __fmul_rn(x[2 * i + 1], s[i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], c[i]), __fmul_rn(x[2 * i], s[i]));
    }
    return;
  }
  const bool second = d0 >= half;
  const int i0 = second ? d0 - half : d0;
  float p[8], c[8], s[8];
  load8<DT, SM>(in, row + (second ? i0 : d0 + half), p);
  load8_f32(t, KVQ_F32, i0, c);
  load8_f32(t, KVQ_F32, half + i0, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = __fmul_rn(x[i], c[i]), b = __fmul_rn(p[i], s[i]);
    y[i] = second ? __fadd_rn(a, b) : __fsub_rn(a, b);
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == KVQ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// q rows are written [batch][n_q_heads][n_new][head_dim], rounded once to their type
template <int DT>
__device__ __forceinline__ void write_q(const RopeStore &g, const RopeRow &w, int D, int d0, const float *y) {
  const size_t e = (((size_t)w.b * g.Hq + w.head) * g.n_new + w.j) * D + d0;
  if constexpr (DT == KVQ_F32) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(g.q_out) + e);
    o[0] = make_float4(y[0], y[1], y[2], y[3]);
    o[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(g.q_out) + e) =
        make_uint4(pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]), pack2<DT>(y[4], y[5]), pack2<DT>(y[6], y[7]));
  }
}

// Sixteen dims per thread (block layouts) or eight (Hadamard): rows per warp 4 or 2 at head_dim 128. Neither
// kernel lets a dependent launch start early: the attention call that follows reads q_out, and its query
// preparation does not wait for its predecessor.
// The threads of one row (TPR of them, `tr` this one's index): load, rotate, write q or quantise. Threads
// without a row take part in the shuffles (full-warp masks) but load and store nothing.
template <int LAYOUT, int D, int DT, bool SM>
__device__ __forceinline__ void rope_block_row(const CacheView &c, const RopeStore &g, RopeRow &w, bool valid, int tr,
                                               const void *in, size_t row) {
  if (valid) valid = rope_place(c, g, w);
  float y[16] = {};
  if (valid) {
    rope_load<DT, SM>(g, w, in, row, 16 * tr, y);
    rope_load<DT, SM>(g, w, in, row, 16 * tr + 8, y + 8);
    if (w.what == 2) {
      write_q<DT>(g, w, D, 16 * tr, y);
      write_q<DT>(g, w, D, 16 * tr + 8, y + 8);
    }
  }
  if (__all_sync(0xffffffffu, !valid || w.what == 2)) return;   // a warp of q rows has nothing to quantise
  quant_block<LAYOUT, 16>(c, w.what == 1, w.crow, g.row_bytes, D / kBlock, tr >> 1, tr & 1, y, valid && w.what != 2);
}
template <int LAYOUT, int D, int DT, bool SM>
__device__ __forceinline__ void rope_had_row(const CacheView &c, const RopeStore &g, RopeRow &w, bool valid, int lane,
                                             const void *in, size_t row) {
  if (valid) valid = rope_place(c, g, w);
  float y[8] = {};
  if (valid) {
    rope_load<DT, SM>(g, w, in, row, 8 * lane, y);
    if (w.what == 2) write_q<DT>(g, w, D, 8 * lane, y);
  }
  if (__all_sync(0xffffffffu, !valid || w.what == 2)) return;
  quant_had<8, D / 8, LAYOUT == KVQ_HAD_INT4 ? 4 : 2>(c, w.what == 1, w.crow, g.row_bytes, lane, y,
                                                      c.n_recent > 0 && w.j >= g.n_new - c.n_recent,
                                                      (long long)w.b * c.H + w.head, w.pos, valid && w.what != 2);
}

// LONG: a block takes the rows of one grid column, whose addresses are then the same but for the row; else the
// launch's rows are dealt out in order. The block layouts take four passes, whose input is on its way into shared
// memory (cp.async, each thread its own dims; partners are in the same warp) while the pass before is worked on:
// 8192 rows asymmetric, d256: 53.9 us, against 58.8 with four passes that load as they go, 57.6 with two and 58.9
// with eight. Hadamard, whose rotation hides its loads: one pass from memory, 255 rows of int4 15.2 us, against
// 16.2 with two and 17.4 with four from shared memory.
template <int LAYOUT>
constexpr int long_passes() { return is_hadamard(LAYOUT) ? 1 : 4; }
template <int LAYOUT, int D, int DT, bool LONG>
__global__ void __launch_bounds__(256, is_hadamard(LAYOUT) ? 6 : LONG ? 5 : 4) rope_store_kernel(CacheView c, RopeStore g) {
  constexpr int TPR = is_hadamard(LAYOUT) ? D / 8 : D / 16, ROWS = 256 / TPR;   // threads per row, rows per pass
  const int tr = threadIdx.x % TPR, own = threadIdx.x / TPR;
  RopeRow w = {};
  constexpr int PASSES = long_passes<LAYOUT>();
  if constexpr (LONG && PASSES > 1) {
    constexpr int E = DT == KVQ_F32 ? 4 : 2, BYTES = D / TPR * E;   // of a thread's dims
    __shared__ __align__(16) uint8_t ring[2][256 * BYTES];
    rope_column(c, g, blockIdx.x, w);
    const RowsIn &in = g.in[w.what];
    const int first = (int)blockIdx.y * (ROWS * PASSES);
    const uint8_t *src = static_cast<const uint8_t *>(in.data) + ((size_t)w.b * in.batch + (size_t)w.head * in.head) * E + tr * BYTES;
    auto fetch = [&](int k) {
      const int j = first + k * ROWS + own;
      if (k < PASSES && j < g.n_new) {
#pragma unroll
        for (int i = 0; i < BYTES; i += 16)
          cp_async16(smem_addr(ring[k & 1] + threadIdx.x * BYTES + i), src + (size_t)j * in.token * E + i, 16);
      }
      cp_async_commit();                                 // always one group per call
    };
    fetch(0);
#pragma unroll 1
    for (int k = 0; k < PASSES; ++k) {
      if (first + k * ROWS >= g.n_new) return;           // the whole block; the groups still open are empty
      fetch(k + 1);
      cp_async_wait<1>();
      __syncwarp();
      w.j = first + k * ROWS + own;
      rope_block_row<LAYOUT, D, DT, true>(c, g, w, w.j < g.n_new, tr, ring[k & 1], (size_t)own * D);
      __syncwarp();                                      // the buffer is read; the next fetch fills it
    }
  } else {
    bool valid;
    if constexpr (LONG) {
      rope_column(c, g, blockIdx.x, w);
      w.j = (int)blockIdx.y * ROWS + own;
      valid = w.j < g.n_new;
    } else {
      const long long group = (long long)blockIdx.x * ROWS + own;
      valid = group < g.k_rows + g.v_rows + g.q_rows;
      if (valid) rope_split(c, g, group, w);
    }
    const RowsIn &in = g.in[w.what];
    const size_t row = (size_t)w.b * in.batch + (size_t)w.head * in.head + (size_t)w.j * in.token;
    if constexpr (is_hadamard(LAYOUT)) rope_had_row<LAYOUT, D, DT, false>(c, g, w, valid, tr, in.data, row);
    else rope_block_row<LAYOUT, D, DT, false>(c, g, w, valid, tr, in.data, row);
  }
}

template <int LAYOUT, int D, int DT>
cudaError_t launch_typed(const CacheView &c, const RopeStore &g, cudaStream_t st) {
  constexpr int rows_per_pass = 256 / (is_hadamard(LAYOUT) ? D / 8 : D / 16), per_block = rows_per_pass * long_passes<LAYOUT>();
  const long long rows = g.k_rows + g.v_rows + g.q_rows, columns = rows / g.n_new;
  // at least a block of rows per head: a grid column per head
  const long long blocks_per_head = (g.n_new + per_block - 1) / per_block;
  if (g.n_new >= per_block && blocks_per_head <= 65535) {
    rope_store_kernel<LAYOUT, D, DT, true><<<dim3((unsigned)columns, (unsigned)blocks_per_head), 256, 0, st>>>(c, g);
  } else {
    const unsigned blocks = (unsigned)((rows + rows_per_pass - 1) / rows_per_pass);
    rope_store_kernel<LAYOUT, D, DT, false><<<blocks, 256, 0, st>>>(c, g);
  }
  return cudaGetLastError();
}
template <int LAYOUT>
cudaError_t launch_layout(const CacheView &c, const RopeStore &g, cudaStream_t st) {
  if (c.D == 128) {
    if (g.dtype == KVQ_F32) return launch_typed<LAYOUT, 128, KVQ_F32>(c, g, st);
    return g.dtype == KVQ_BF16 ? launch_typed<LAYOUT, 128, KVQ_BF16>(c, g, st) : launch_typed<LAYOUT, 128, KVQ_F16>(c, g, st);
  }
  if (g.dtype == KVQ_F32) return launch_typed<LAYOUT, 256, KVQ_F32>(c, g, st);
  return g.dtype == KVQ_BF16 ? launch_typed<LAYOUT, 256, KVQ_BF16>(c, g, st) : launch_typed<LAYOUT, 256, KVQ_F16>(c, g, st);
}
cudaError_t launch_plane(const CacheView &c, int layout, const RopeStore &g, cudaStream_t st) {
  switch (layout) {
    case KVQ_Q4_0: return launch_layout<KVQ_Q4_0>(c, g, st);
    case KVQ_Q6_0: return launch_layout<KVQ_Q6_0>(c, g, st);
    case KVQ_Q8_0: return launch_layout<KVQ_Q8_0>(c, g, st);
    case KVQ_ASYM4_G32: return launch_layout<KVQ_ASYM4_G32>(c, g, st);
    case KVQ_HAD_INT4: return launch_layout<KVQ_HAD_INT4>(c, g, st);
    default: return launch_layout<KVQ_HAD_INT2>(c, g, st);
  }
}

FastDiv fast_div(int d) {
  FastDiv f = {0, 0};
  while ((1ull << f.shift) < (unsigned long long)d) ++f.shift;
  f.mul = (unsigned)((((1ull << f.shift) - (unsigned long long)d) << 32) / (unsigned long long)d + 1);
  return f;
}

}  // namespace

cudaError_t launch_rope_table(const RopeTurns &f, int rot, int pos0, int n_pos, float mag, float *table, cudaStream_t st) {
  // short tables: a position per thread
  const int per = n_pos >= 32768 ? kTableRows : 1, rows = (n_pos + per - 1) / per;
  const long long threads = (long long)rows * (rot / 8);
  rope_table_kernel<<<(unsigned)((threads + kTableThreads - 1) / kTableThreads), kTableThreads, 0, st>>>(
      f, rot / 2, pos0, n_pos, rows, mag, table);
  return cudaGetLastError();
}

cudaError_t launch_rope_store(const CacheView &c, RopeStore g, cudaStream_t st) {
  const long long rows = (long long)c.B * c.H * g.n_new;
  g.by_new = fast_div(g.n_new);
  g.by_kv_heads = fast_div(c.H);
  g.by_q_heads = fast_div(g.Hq > 0 ? g.Hq : 1);
  g.k_rows = rows;
  g.v_rows = c.layout == c.v_layout ? rows : 0;
  g.q_rows = (long long)c.B * g.Hq * g.n_new;
  g.row_bytes = c.row_bytes;
  cudaError_t e = launch_plane(c, c.layout, g, st);
  if (e != cudaSuccess || g.v_rows) return e;
  // mixed K/V precision: the V plane's rows in a launch of their own layout
  g.k_rows = g.q_rows = 0;
  g.v_rows = rows;
  g.row_bytes = c.v_row_bytes;
  return launch_plane(c, c.v_layout, g, st);
}

}  // namespace kvq
