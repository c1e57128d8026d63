// Paged 4-bit memory: selection of each request's best pages.
//
// score(r, h, j) = sum over dims of (sum over the group's q heads of q) * rep[table[r][j]][h],
// accumulated in 64 bits and rounded once to 32, for request r's candidate pages j; the k best
// per (request, kv head), ties to the lower page.  A 32-bit accumulation would leave the order
// of near pages to the order of the sum.
#include "paged.cuh"

namespace rba {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreCtas = 2;  // per SM
constexpr int kBatch = 8;      // candidate rows in flight per lane

struct SelectArgs {
  const void* q;
  int64_t q_req, q_head;
  const float* rep;
  const int32_t* table;
  const int32_t* lens;
  int32_t* status;
  float* scores;  // [R][Hkv][row]
  int R, heads, group, dim, bs, max_pages, n_pages, sink, window, row;
};

// pre[r] = batches of `per` candidates of the requests before r (one kv head); returns their sum.
__device__ int64_t scan_batches(const SelectArgs& a, int per, int32_t* pre, int32_t* ncand,
                                int64_t* s_w) {
  int64_t run = 0;
  for (int base = 0; base < a.R; base += blockDim.x) {
    const int r = base + threadIdx.x;
    int nb = 0;
    if (r < a.R) {
      const int T = paged_len(a.lens, r, a.bs, a.max_pages, a.status);
      const PagedGeo g = paged_geo(T, a.bs, a.sink, a.window);
      ncand[r] = g.nc;
      nb = (g.nc + per - 1) / per;
    }
    int64_t tot;
    const int64_t ex = block_scan64(nb, s_w, &tot);
    if (r < a.R) pre[r] = static_cast<int32_t>(run + ex);
    run += tot;
  }
  __syncthreads();
  return run;
}

// A warp takes a run of batches of PER candidates: the page numbers of the next batch are loaded
// while this one's rows are; the rows' sums are added over lanes by halving exchanges (each step
// halves the rows a lane carries), two or three of a double per row instead of five.
template <typename T, int P>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) paged_score_kernel(SelectArgs a) {
  constexpr int LPR = P / 4, RPW = 32 / LPR;  // lanes a row, rows a warp reads at once
  constexpr int PER = kBatch * RPW;
  extern __shared__ int32_t sm[];
  __shared__ int64_t s_w[kScoreThreads / 32];
  wait_for_stream();
  int32_t* pre = sm;
  int32_t* ncand = sm + a.R;
  const int64_t one = scan_batches(a, PER, pre, ncand, s_w);
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int first = a.sink / a.bs;
  const int64_t all = one * a.heads;
  const int64_t nw = int64_t(gridDim.x) * (kScoreThreads / 32);
  // (warps of one CTA lie far apart, so that few batches use every SM)
  const int64_t w = int64_t(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  const int64_t b0 = all * w / nw, b1 = all * (w + 1) / nw;
  if (b0 >= b1) return;
  int r = last_at_most(pre, a.R, static_cast<int32_t>(b0 / a.heads));
  int nc = ncand[r], nb = (nc + PER - 1) / PER;
  int h, c0;
  {
    const int64_t in = b0 - int64_t(pre[r]) * a.heads;
    h = static_cast<int>(in / nb);
    c0 = static_cast<int>(in - int64_t(h) * nb) * PER;
  }
  const auto page_of = [&](int r_, int c0_, int nc_) {  // lane i: page of candidate c0 + i, or -1
    if (lane >= PER || c0_ + lane >= nc_) return -1;
    const int page = a.table[int64_t(r_) * a.max_pages + first + c0_ + lane];
    if (page >= 0 && page < a.n_pages) return page;
    report(a.status, RBA_ERR_BOUNDS, kWherePaged, page);
    return -1;
  };
  int page = page_of(r, c0, nc);
  bool fresh = true;
  double q[4] = {0, 0, 0, 0};
  for (int64_t b = b0; b < b1; ++b) {
    float4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int p = __shfl_sync(0xffffffffu, page, u * RPW + sub);
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p >= 0)
        x[u] = __ldg(reinterpret_cast<const float4*>(a.rep + (int64_t(p) * a.heads + h) * P) + l);
    }
    if (fresh) {
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = 0;
      if (l * 4 < a.dim) {
        const T* src = static_cast<const T*>(a.q) + r * a.q_req + int64_t(h) * a.group * a.q_head;
#pragma unroll 4
        for (int i = 0; i < a.group; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            q[e] += static_cast<double>(Elem<T>::to_f32(src[i * a.q_head + l * 4 + e]));
      }
    }
    // the batch after this one
    const int64_t unit = int64_t(r) * a.heads + h;
    const int at = c0, most = nc;
    if (b + 1 < b1) {
      c0 += PER;
      fresh = c0 >= nc;
      if (fresh) {
        c0 = 0;
        if (++h == a.heads) {
          h = 0;
          do ++r;
          while (ncand[r] == 0);  // (a batch is left, so a request with candidates is)
          nc = ncand[r];
        }
      }
      page = page_of(r, c0, nc);
    }
    double s[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      s[u] = q[0] * x[u].x;
      s[u] = fma(q[1], double(x[u].y), s[u]);
      s[u] = fma(q[2], double(x[u].z), s[u]);
      s[u] = fma(q[3], double(x[u].w), s[u]);
    }
    // after the steps of width 4, 2, 1 a lane carries row bits (l & 4, l & 2, l & 1) of the eight
#pragma unroll
    for (int n = kBatch / 2; n > 0; n >>= 1) {
      const bool up = (l & n) != 0;
#pragma unroll
      for (int u = 0; u < n; ++u) {
        const double give = up ? s[u] : s[u + n], keep = up ? s[u + n] : s[u];
        s[u] = keep + __shfl_xor_sync(0xffffffffu, give, n);
      }
    }
#pragma unroll
    for (int o = kBatch; o < LPR; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    const int c = at + (l % kBatch) * RPW + sub;
    if (l < kBatch && c < most) a.scores[unit * a.row + c] = static_cast<float>(s[0]);
  }
}

// candidates that a request can have at most
int most_candidates(const rba_paged* s, int sink, int window) {
  const int64_t most = int64_t(s->d.max_pages) * s->d.page_size;
  return paged_geo(static_cast<int>(most), s->d.page_size, sink, window).nc;
}

}  // namespace
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
  if (s == nullptr || n_requests <= 0 || n_requests > s->d.max_requests || k < 0 || sink < 0 ||
      window < 0)
    return RBA_ERR_INVALID_ARG;
  if (k == 0) return RBA_OK;
  if (q == nullptr || idx == nullptr || workspace == nullptr) return RBA_ERR_INVALID_ARG;
  const int row = most_candidates(s, sink, window);
  if (row > kPagedMaxCandidates) return RBA_ERR_UNSUPPORTED;
  if (ws_bytes < size_t(n_requests) * s->d.n_kv_heads * row * sizeof(float))
    return RBA_ERR_WORKSPACE;
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
  if (row > 0) {
    const size_t smem = size_t(n_requests) * 8;
    const auto kernel =
        s->d.dtype == RBA_BF16
            ? (s->pitch == 128 ? paged_score_kernel<__nv_bfloat16, 128>
                               : paged_score_kernel<__nv_bfloat16, 64>)
            : (s->pitch == 128 ? paged_score_kernel<float, 128> : paged_score_kernel<float, 64>);
    RBA_CUDA_TRY(launch_dependent(kernel, static_cast<unsigned>(num_sms() * kScoreCtas),
                                  kScoreThreads, smem, stream, a));
  }
  return launch_topk_paged(a.scores, row, n_requests * s->d.n_kv_heads, s->d.n_kv_heads, a.lens,
                           a.bs, a.max_pages, sink, window, k, idx, stream);
}
