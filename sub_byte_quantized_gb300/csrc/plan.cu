// A step's pages and slots from the requests' lengths, on the device.
//
//   held_b = ceil(L_b / p),  need_b = ceil((L_b + n_b) / p) - held_b,  row of token at position t: table[b][t / p] p + t % p
//
// Which requests are served goes by prefix sums over them (64-bit: a sum of page counts or tokens can pass 2^31), so
// it hangs on nothing but their order. plan_pages_kernel is one CTA: thread i holds request i of a tile of 1024, a
// block scan gives each request its place, and the copies that a request brings (pages given back, pages taken) are
// spread over all threads by a binary search in the tile's prefix sums, so that one long request costs no more than
// many short ones. plan_slots_kernel writes the map of the step's tokens, one thread each, which finds its request
// by a binary search in cu_new.
//
// Bound: latency (a few dependent reads of lengths and free pages, then 12 bytes written per token). 256 decode rows 8.8 us with a
// copy of their inputs, 64 prompts of 262144 tokens 9.7.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

// Inclusive sum over the CTA; `total` gets the sum of all. `ws` holds kWarps values, free again on return.
__device__ __forceinline__ long long block_scan(long long x, long long *ws, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  long long w = ws[lane];                                // kWarps == 32: every warp scans the warps' sums
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, k);
    if (lane >= k) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return x + (warp > 0 ? before : 0);
}
static_assert(kWarps == 32, "one lane per warp's sum");

// The first of n ascending values that is greater than x (n where there is none).
template <class T>
__device__ __forceinline__ int first_above(const T *v, int n, T x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

struct Request {
  int len, fresh;              // tokens held (clamped into the table's room) and wanted; fresh < 0: it has ended
  int held, need;              // pages
  bool fits;
};
__device__ __forceinline__ Request request_of(const PlanArgs &a, int b) {
  Request r = {0, 0, 0, 0, false};
  if (b >= a.batch) return r;
  const int cap = a.max_pages << a.page_shift, page1 = (1 << a.page_shift) - 1;
  r.len = min(max(a.seq_lens[b], 0), cap);
  r.fresh = a.new_lens[b];
  r.held = (int)(((long long)r.len + page1) >> a.page_shift);
  r.fits = r.fresh >= 0 && (long long)r.len + r.fresh <= cap;
  r.need = r.fits ? (int)(((long long)r.len + r.fresh + page1) >> a.page_shift) - r.held : 0;
  return r;
}

__device__ __forceinline__ void write_slot(const PlanArgs &a, int i, int total, const int *cu, const int *lens, const int *table) {
  long long slot = -1;
  int pos = -1;
  if (i < total) {
    const int b = first_above(cu, a.batch + 1, i) - 1;   // the last request that begins at or before i: it has tokens
    pos = lens[b] - (cu[b + 1] - i);
    slot = ((long long)table[(size_t)b * a.max_pages + (pos >> a.page_shift)] << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  }
  a.slots[i] = slot;
  a.positions[i] = pos;
}

__global__ void __launch_bounds__(kThreads) plan_pages_kernel(PlanArgs a, bool with_slots) {
  __shared__ long long ws[kWarps];
  __shared__ long long upto[kThreads];                   // inclusive sums of what the tile's requests bring
  __shared__ int first[kThreads];                        // their first page index in the table
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");
#endif
  const int tid = threadIdx.x;
  long long n_free = min(max(*a.n_free, 0), a.n_pool);
  // pages of ended requests go behind the free ones
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const Request r = request_of(a, b0 + tid);
    long long total;
    const long long sum = block_scan(r.fresh < 0 ? r.held : 0, ws, total);
    if (total == 0) continue;                            // the same for every thread
    upto[tid] = sum;
    __syncthreads();
    const long long room = min(total, a.n_pool - n_free);
    for (long long i = tid; i < room; i += kThreads) {
      const int j = first_above(upto, kThreads, i);
      const long long k = i - (j ? upto[j - 1] : 0);
      a.free_pages[n_free + i] = a.table[(size_t)(b0 + j) * a.max_pages + k];
    }
    n_free += room;
    __syncthreads();
  }
  // In the requests' order: those that the table has room for, then those that the free pages last for, then those
  // whose tokens the step has room for.
  long long pages = 0, tokens = 0, taken = 0, given = 0; // sums of the tiles before, at each of the stages
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    const Request r = request_of(a, b);
    long long total;
    bool ok = r.fits;
    const long long p = pages + block_scan(r.need, ws, total);
    pages += total;
    ok = ok && (r.need == 0 || p <= n_free);
    const long long t = tokens + block_scan(ok ? r.fresh : 0, ws, total);
    tokens += total;
    ok = ok && (r.fresh == 0 || t <= a.max_tokens);
    const int got = ok ? r.fresh : 0, need = ok ? r.need : 0;
    const long long c = given + block_scan(got, ws, total);
    given += total;
    upto[tid] = block_scan(need, ws, total);
    first[tid] = r.held;
    if (b < a.batch) {
      a.lens_out[b] = r.fresh < 0 ? 0 : r.len + got;
      a.granted[b] = got;
      a.cu_new[b + 1] = (int)c;
    }
    __syncthreads();
    for (long long i = tid; i < total; i += kThreads) {
      const int j = first_above(upto, kThreads, i);
      const long long k = i - (j ? upto[j - 1] : 0);
      a.table[(size_t)(b0 + j) * a.max_pages + first[j] + k] = a.free_pages[n_free - 1 - (taken + i)];
    }
    taken += total;
    __syncthreads();
  }
  if (tid == 0) {
    a.cu_new[0] = 0;
    *a.n_free_out = (int)(n_free - taken);
  }
  if (!with_slots) return;
  __syncthreads();                                       // the table, the lengths and cu_new are this CTA's own writes
  for (int i = tid; i < a.max_tokens; i += kThreads) write_slot(a, i, (int)given, a.cu_new, a.lens_out, a.table);
}

__global__ void __launch_bounds__(256) plan_slots_kernel(PlanArgs a) {
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < a.max_tokens) write_slot(a, i, a.cu_new[a.batch], a.cu_new, a.lens_out, a.table);
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs &a, cudaStream_t st) {
  // Few tokens: the one CTA writes their map too, which saves a launch (64 requests, one CTA / two launches: 256 tokens
  // 4.8 / 6.5 us, 2048 6.6 / 7.5, 4096 8.2 / 7.3, 8192 11.1 / 7.4).
  const bool one = a.max_tokens <= 2 * kThreads;
  plan_pages_kernel<<<1, kThreads, 0, st>>>(a, one);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || one) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.max_tokens + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_slots_kernel, a);
}

}  // namespace kvq
