// Paged 4-bit memory: selection of each request's best pages.
//
// score(r, h, j) = sum over dims of (sum over the group's q heads of q) * rep[table[r][j]][h] for
// request r's candidate pages j, rounded once to 32 bits; the k best per (request, kv head), ties
// to the lower page.  A 32-bit accumulation would leave the order of near pages to the order of the
// sum, so it is held in 64.  (Only candidates near the k-th place need that; the others are summed so
// too, to have one pass.  In two 32-bit words, with exact products and sums, the same bits cost
// a fifth more time at 86 MB of page means: five times the instructions.)
#include "paged.cuh"
#include "paged_ring.cuh"

namespace rba {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreCtas = 3;  // per SM
constexpr int kBatch = 8;      // candidate rows that a lane has a share of at a time
constexpr int kRingPlaces = 2; // batches in a warp's ring: 4 KB each

struct SelectArgs {
  const void* q;
  int64_t q_req, q_head;
  const float* rep;
  const int32_t* table;
  const int32_t* lens;
  int32_t* status;
  float* scores;  // [R][Hkv][row]
  int R, heads, group, dim, bs, max_pages, n_pages, sink, window, row;
  int first;   // sink / bs
  bool q_vec;  // rows of q start on a boundary of four elements
  FastDiv by_bs, by_heads, by_warps;  // (warps of the grid)
};

// pre[r] = batches of `per` candidates of the requests before r (one kv head); returns their sum.
__device__ int scan_batches(const SelectArgs& a, int per, int32_t* pre, int32_t* ncand,
                                int64_t* s_w) {
  int run = 0;
  for (int base = 0; base < a.R; base += blockDim.x) {
    const int r = base + threadIdx.x;
    int nb = 0;
    if (r < a.R) {
      const int T = paged_len(a.lens, r, a.bs, a.max_pages, a.status);
      const PagedGeo g = paged_geo(T, a.by_bs, a.first, a.sink, a.window);
      ncand[r] = g.nc;
      nb = (g.nc + per - 1) / per;
    }
    int64_t tot;
    const int64_t ex = block_scan64(nb, s_w, &tot);
    if (r < a.R) pre[r] = run + static_cast<int>(ex);
    run += static_cast<int>(tot);
  }
  __syncthreads();
  return run;
}

// A warp takes a run of batches of PER candidates, through its own ring of bulk copies (a row is
// one run of bytes): 4 KB a batch, two batches on their way, whatever the warp is computing.
// The page numbers of the batch to be copied next are loaded one copy ahead.  The sums are added
// over lanes by halving exchanges (each step halves the rows a lane carries): two or three per row
// instead of five.  86 MB of page means and the choice among them take 27.4 us (28.2 with two CTAs
// an SM of three batches a warp), the means alone about 19 (4.5 TB/s); with rows loaded into
// registers a batch ahead, 16 warps an SM left the memory idle half the time (26 us for the means).
// What is left is the scan of the requests before the first copy (about 4 us) and the latency and
// issue slots of the 64-bit sums.
template <typename T, int P>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) paged_score_kernel(SelectArgs a) {
  constexpr int LPR = P / 4, RPW = 32 / LPR;  // lanes a row, rows a warp reads at once
  constexpr int PER = kBatch * RPW, ROW = P * 4, PLACE = PER * ROW;
  constexpr int kScoreWarps = kScoreThreads / 32;
  extern __shared__ __align__(128) char sm[];
  __shared__ int64_t s_w[kScoreWarps];
  __shared__ uint64_t s_bars[kScoreWarps][kRingPlaces];
  int32_t* pre = reinterpret_cast<int32_t*>(sm + kScoreWarps * kRingPlaces * PLACE);
  int32_t* ncand = pre + a.R;
  uint64_t* bars = s_bars[threadIdx.x >> 5];
  if ((threadIdx.x & 31) < kRingPlaces) mbar_init(bars + (threadIdx.x & 31), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  wait_for_stream();
  const int one = scan_batches(a, PER, pre, ncand, s_w);
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  // the warp's share of all batches (warps of one CTA lie far apart, so that few batches use every
  // SM).  With 64-bit and plain divisions here a selection over 86 MB took 2 us more.
  const int all = one * a.heads, w = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  const int share = div(all, a.by_warps), more = all - share * static_cast<int>(a.by_warps.d);
  const int b0 = w * share + min(w, more), batches = share + (w < more);
  if (batches == 0) return;
  struct Pos {
    int r, h, c0, nc;  // request, kv head, first candidate of the batch, the request's candidates
  } at;
  at.r = last_at_most(pre, a.R, div(b0, a.by_heads));
  at.nc = ncand[at.r];
  {
    const int nb = (at.nc + PER - 1) / PER;
    const int in = b0 - pre[at.r] * a.heads;
    at.h = in / nb;
    at.c0 = (in - at.h * nb) * PER;
  }
  const auto advance = [&](Pos p) {  // (called while a batch is left: a request with candidates is)
    p.c0 += PER;
    if (p.c0 < p.nc) return p;
    p.c0 = 0;
    if (++p.h < a.heads) return p;
    p.h = 0;
    do ++p.r;
    while (ncand[p.r] == 0);
    p.nc = ncand[p.r];
    return p;
  };
  const auto page_of = [&](const Pos& p) {  // lane i: page of candidate c0 + i, or -1
    if (lane >= PER || p.c0 + lane >= p.nc) return -1;
    const int page = a.table[int64_t(p.r) * a.max_pages + a.first + p.c0 + lane];
    if (page >= 0 && page < a.n_pages) return page;
    report(a.status, RBA_ERR_BOUNDS, kWherePaged, page);
    return -1;
  };
  double q[4];
  const auto load_q = [&](const Pos& p) {  // the group's sum
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = 0;
    if (l * 4 >= a.dim) return;
    const T* src = static_cast<const T*>(a.q) + p.r * a.q_req + int64_t(p.h) * a.group * a.q_head;
#pragma unroll 4
    for (int i = 0; i < a.group; ++i) {
      float f[4];
      load4(src + i * a.q_head + l * 4, a.q_vec, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] += static_cast<double>(f[e]);
    }
  };
  const char* ring = sm + (threadIdx.x >> 5) * kRingPlaces * PLACE;
  const uint32_t ring0 = smem_u32(ring) + lane * ROW, bar0 = smem_u32(bars);
  // copies run ahead of the sums: `ahead` is the next batch to copy, `page` its pages
  Pos ahead = at;
  int page = page_of(at);
  unsigned rows[kRingPlaces];  // lanes whose candidate's row is in the place
  const auto issue = [&](int n) {  // the warp's n-th batch into place n % kRingPlaces
    if (n >= batches) return;
    const int i = n % kRingPlaces;
    const unsigned there = __ballot_sync(0xffffffffu, page >= 0);
#pragma unroll
    for (int j = 0; j < kRingPlaces; ++j)
      if (j == i) rows[j] = there;
    arm_and_copy(bar0 + i * 8, lane == 0, ROW * __popc(there), ring0 + i * PLACE,
                 a.rep + (int64_t(page) * a.heads + ahead.h) * P, page >= 0 ? ROW : 0);
    if (n + 1 < batches) {
      ahead = advance(ahead);
      page = page_of(ahead);
    }
  };
#pragma unroll
  for (int n = 0; n < kRingPlaces; ++n) issue(n);
  load_q(at);
  for (int n = 0; n < batches; ++n) {
    const int i = n % kRingPlaces;
    if (!await_phase(bar0 + i * 8, (n / kRingPlaces) & 1)) {
      if (lane == 0) report(a.status, RBA_ERR_TIMEOUT, kWherePaged, n);
      for (int m = n; m < n + kRingPlaces && m < batches; ++m)  // copies in flight land first
        mbar_drain(bars + m % kRingPlaces, (m / kRingPlaces) & 1);
      return;
    }
    unsigned there = 0;
#pragma unroll
    for (int j = 0; j < kRingPlaces; ++j)
      if (j == i) there = rows[j];
    double s[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float4 x =
          *reinterpret_cast<const float4*>(ring + i * PLACE + (u * RPW + sub) * ROW + l * 16);
      s[u] = q[0] * x.x;
      s[u] = fma(q[1], double(x.y), s[u]);
      s[u] = fma(q[2], double(x.z), s[u]);
      s[u] = fma(q[3], double(x.w), s[u]);
    }
    const Pos done = at;
    __syncwarp();
    issue(n + kRingPlaces);
    if (n + 1 < batches) {
      at = advance(at);
      if (at.c0 == 0) load_q(at);
    }
    // after the steps of width 4, 2, 1 a lane carries row bits (l & 4, l & 2, l & 1) of the eight
#pragma unroll
    for (int w = kBatch / 2; w > 0; w >>= 1) {
      const bool up = (l & w) != 0;
#pragma unroll
      for (int u = 0; u < w; ++u) {
        const double give = up ? s[u] : s[u + w], keep = up ? s[u + w] : s[u];
        s[u] = keep + __shfl_xor_sync(0xffffffffu, give, w);
      }
    }
#pragma unroll
    for (int o = kBatch; o < LPR; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    const int r = (l % kBatch) * RPW + sub, c = done.c0 + r;
    if (l < kBatch && c < done.nc)  // (a page that is not in the pool scores 0)
      a.scores[(int64_t(done.r) * a.heads + done.h) * a.row + c] =
          (there >> r) & 1u ? static_cast<float>(s[0]) : 0.f;
  }
}

// candidates that a request can have at most
int most_candidates(const rba_paged* s, int sink, int window) {
  const int64_t most = int64_t(s->d.max_pages) * s->d.page_size;
  return paged_geo(static_cast<int>(most), s->d.page_size, sink, window).nc;
}

}  // namespace

rba_status refuse_select(const rba_paged* s, int32_t n_requests, int32_t k, int32_t sink,
                         int32_t window, const void* workspace, size_t ws_bytes) {
  if (s == nullptr || n_requests <= 0 || n_requests > s->d.max_requests || k < 0 || sink < 0 ||
      window < 0)
    return RBA_ERR_INVALID_ARG;
  if (k == 0) return RBA_OK;
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % alignof(float) != 0)
    return RBA_ERR_INVALID_ARG;
  const int row = most_candidates(s, sink, window);
  // (batches of scores are counted in 31 bits)
  if (row > kPagedMaxCandidates ||
      int64_t(n_requests) * s->d.n_kv_heads * (row / kBatch + 1) > INT32_MAX)
    return RBA_ERR_UNSUPPORTED;
  if (ws_bytes < size_t(n_requests) * s->d.n_kv_heads * row * sizeof(float))
    return RBA_ERR_WORKSPACE;
  return RBA_OK;
}

}  // namespace rba

extern "C" size_t rba_paged_select_workspace_size(const rba_paged* s) {
  if (s == nullptr) return 0;
  return size_t(s->d.max_requests) * s->d.n_kv_heads * s->d.max_pages * sizeof(float);
}

extern "C" rba_status rba_paged_select(const rba_paged* s, const void* q,
                                       int64_t q_request_stride, int64_t q_head_stride,
                                       int32_t n_requests, int32_t k, int32_t sink,
                                       int32_t window, int32_t* idx, void* workspace,
                                       size_t ws_bytes, cudaStream_t stream) {
  using namespace rba;
  if (k > 0 && (q == nullptr || idx == nullptr)) return RBA_ERR_INVALID_ARG;
  const rba_status refused = refuse_select(s, n_requests, k, sink, window, workspace, ws_bytes);
  if (refused != RBA_OK || k == 0) return refused;
  const int row = most_candidates(s, sink, window);
  SelectArgs a = {};
  a.q = q;
  a.q_req = q_request_stride;
  a.q_head = q_head_stride;
  a.rep = s->b.rep;
  a.table = s->b.table;
  a.lens = s->b.lens;
  a.status = s->b.status;
  a.scores = static_cast<float*>(workspace);
  a.R = n_requests;
  a.heads = s->d.n_kv_heads;
  a.group = s->d.n_q_heads / s->d.n_kv_heads;
  a.dim = s->d.head_dim;
  a.bs = s->d.page_size;
  a.max_pages = s->d.max_pages;
  a.n_pages = s->d.n_pages;
  a.sink = sink;
  a.window = window;
  a.row = row;
  a.first = sink / a.bs;
  a.by_bs = fast_div(a.bs);
  a.by_heads = fast_div(a.heads);
  const int grid = num_sms() * kScoreCtas;
  a.by_warps = fast_div(grid * (kScoreThreads / 32));
  a.q_vec = reinterpret_cast<uintptr_t>(q) % (4 * dtype_size(s->d.dtype)) == 0 &&
            ((q_request_stride | q_head_stride) & 3) == 0;
  if (row > 0) {
    const size_t smem = size_t(kScoreThreads / 32) * kRingPlaces * kBatch * 512 +
                        size_t(n_requests) * 8;
    const auto kernel =
        s->d.dtype == RBA_BF16
            ? (s->pitch == 128 ? paged_score_kernel<__nv_bfloat16, 128>
                               : paged_score_kernel<__nv_bfloat16, 64>)
            : (s->pitch == 128 ? paged_score_kernel<float, 128> : paged_score_kernel<float, 64>);
    RBA_CUDA_TRY(ensure_smem(reinterpret_cast<const void*>(kernel), smem));
    RBA_CUDA_TRY(launch_dependent(kernel, static_cast<unsigned>(grid), kScoreThreads, smem, stream,
                                  a));
  }
  return launch_topk_paged(a.scores, row, n_requests * s->d.n_kv_heads, s->d.n_kv_heads, a.lens,
                           a.bs, a.max_pages, sink, window, k, idx, stream);
}
