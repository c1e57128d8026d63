// Paged 4-bit memory: what its kernels share (the strip layout, a request's
// candidate and strip geometry, block scans).
//
// A strip is 16 tokens of one (page, kv head), P = 64 or 128 dims a row in
// G = P / 32 groups of one scale each.  It is laid out for the attention kernel's
// matrix fragments, so that a lane's share of it is a few 16-byte loads:
//   K codes  [token 16][c 4][group G] 32-bit words; nibble j is dim 32 g + 8 c + j
//   V codes  [half 2][lane 8][c 4][group G][odd 2] 16-bit units of token
//            8 half + 2 c + odd; nibble j is dim 32 g + 4 lane + j
//   scales   [token 16][K groups G, V groups G] bf16
#pragma once

#include "rba_internal.cuh"

struct rba_paged {
  rba_paged_desc d;
  rba_paged_buffers b;
  int32_t pitch;   // P
  int32_t strips;  // strips of one (page, kv head): ceil(page_size / 16)
};

namespace rba {

constexpr int kStrip = 16;           // tokens of a strip
constexpr int kMaxRequests = 4096;   // rows of a page table (scanned in one CTA's shared memory)
constexpr int kPagedMaxCandidates = 16384;  // scores one CTA selects from in shared memory

__host__ __device__ constexpr int strip_groups(int P) { return P / 32; }
__host__ __device__ constexpr int strip_bytes(int P) { return 16 * P + 64 * strip_groups(P); }
// byte offsets inside a strip
template <int P> __device__ __forceinline__ int k_unit_at(int t, int g, int lane) {
  // 16-bit unit of dims 32 g + 4 lane .. + 3 of token t
  return ((t * 4 + (lane >> 1)) * (P / 32) + g) * 4 + (lane & 1) * 2;
}
template <int P> __device__ __forceinline__ int v_unit_at(int t, int g, int lane) {
  const int half = t >> 3, c = (t & 7) >> 1, odd = t & 1;
  return 8 * P + (((half * 8 + lane) * 4 + c) * (P / 32) + g) * 4 + odd * 2;
}
template <int P> __device__ __forceinline__ int scale_at(int t, int which, int g) {
  return 16 * P + (t * 2 * (P / 32) + which * (P / 32) + g) * 2;
}

// x / d for 0 <= x < 2^31: with L = ceil(log2 d) and m = ceil(2^(31 + L) / d) (below 2^32 for
// d > 1), m d - 2^(31 + L) < d <= 2^L, so (x m) >> (31 + L) is the quotient.
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {d, 0, 0};
  if (d <= 1) return f;
  uint32_t L = 0;
  while ((uint64_t(1) << L) < d) ++L;
  f.m = static_cast<uint32_t>(((uint64_t(1) << (31 + L)) + d - 1) / d);
  f.s = L - 1;
  return f;
}
__device__ __forceinline__ int div(int x, const FastDiv& f) {
  return f.d <= 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), f.m) >> f.s);
}

// One request's attended set, in strips.  Page j is a candidate when it is full, ends past sink and
// begins before w0; the window always covers the partial last page.
struct PagedGeo {
  int T, w0, sink_end, first, nc;
};
__host__ __device__ inline PagedGeo paged_geo(int T, int full, int w0_page, int first, int bs,
                                              int sink, int window) {
  // full = T / bs, w0_page = w0 / bs, first = sink / bs
  PagedGeo g;
  const int open = T > window ? T - window : 0;
  g.T = T;
  g.w0 = open < full * bs ? open : full * bs;
  g.sink_end = sink < g.w0 ? sink : g.w0;
  g.first = first;
  int hi = w0_page + (g.w0 > w0_page * bs);
  hi = hi < full ? hi : full;
  g.nc = hi > first ? hi - first : 0;
  return g;
}
__host__ __device__ inline int paged_w0(int T, int full, int bs, int window) {
  const int open = T > window ? T - window : 0;
  return open < full * bs ? open : full * bs;
}
inline PagedGeo paged_geo(int T, int bs, int sink, int window) {
  const int full = T / bs;
  return paged_geo(T, full, paged_w0(T, full, bs, window) / bs, sink / bs, bs, sink, window);
}
__device__ __forceinline__ PagedGeo paged_geo(int T, const FastDiv& by_bs, int first, int sink,
                                              int window) {
  const int bs = by_bs.d, full = div(T, by_bs);
  return paged_geo(T, full, div(paged_w0(T, full, bs, window), by_bs), first, bs, sink, window);
}

// A request's length as the store holds it; a length outside the table is reported and
// taken as 0.
__device__ __forceinline__ int paged_len(const int32_t* lens, int r, int bs, int max_pages,
                                         int32_t* status) {
  const int T = lens[r];
  if (T < 0 || T > int64_t(max_pages) * bs) {
    report(status, RBA_ERR_BOUNDS, kWherePaged, r);
    return 0;
  }
  return T;
}

// Four elements of a row, in one load where rows start on their boundary (vec).
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool vec, float* x);
template <>
__device__ __forceinline__ void load4(const float* p, bool vec, float* x) {
  if (vec) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
    x[0] = p[0]; x[1] = p[1]; x[2] = p[2]; x[3] = p[3];
  }
}
template <>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, bool vec, float* x) {
  if (vec) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __bfloat162float(p[i]);
  }
}

// Exclusive block scan of one 64-bit value a thread (every thread calls it); *total is
// the sum.  s_w holds one word per warp.
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* s_w, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_w[warp] = incl;
  __syncthreads();
  int64_t base = 0, tot = 0;
  for (int w = 0; w < nw; ++w) {
    const int64_t x = s_w[w];
    if (w < warp) base += x;
    tot += x;
  }
  __syncthreads();
  *total = tot;
  return base + incl - v;
}

// Largest i in [0, n) with pre[i] <= x, for a non-decreasing pre with pre[0] <= x.
template <typename T>
__device__ __forceinline__ int last_at_most(const T* pre, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Every paged kernel is launched as a programmatic dependent of the one before it on the stream:
// its CTAs come up while that one runs and wait here, before their first access to memory, until
// it has completed.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... A>
cudaError_t launch_dependent(void (*kernel)(A...), unsigned grid, int threads, size_t smem,
                             cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// The host-side refusals of the calls of a decode step (RBA_OK: none): the library's limits, and
// the workspaces'.  Each call makes its own check; rba_paged_step_check makes all of them.
rba_status refuse_append(const rba_paged* s, int32_t n);
rba_status refuse_select(const rba_paged* s, int32_t n_requests, int32_t k, int32_t sink,
                         int32_t window, const void* workspace, size_t ws_bytes);
rba_status refuse_attend(const rba_paged* s, int32_t n_requests, int32_t k, int32_t sink,
                         int32_t window, const void* workspace, size_t ws_bytes);

// Top k per row of scores [rows][row_stride], row = request * heads + kv head: the request's
// candidates only, written as page numbers ascending, then -1.
rba_status launch_topk_paged(const float* scores, int row_stride, int rows, int heads,
                             const int32_t* lens, int bs, int max_pages, int sink, int window,
                             int k, int32_t* idx, cudaStream_t stream);

}  // namespace rba
