// Paged 4-bit memory: description, page tables and slot maps.
#include <new>

#include "paged.cuh"

namespace rba {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kPer = kMaxRequests / kTableThreads;  // requests a thread scans at most

struct TableArgs {
  const int32_t* by;      // extend: new tokens a request; truncate: tokens it keeps
  int32_t* lens;
  int32_t* table;
  int32_t* free_pages;
  int32_t* n_free;
  int32_t* status;        // [4]: CTAs of the running call that are done reading
  int32_t* slots;
  int32_t* starts;
  int n_requests, bs, max_pages, n_pages, n_slots;
  int per;                // requests a thread scans: ceil(n_requests / kTableThreads)
  FastDiv by_bs;
};

__device__ __forceinline__ int pages_of(const TableArgs& a, int tokens) {
  const int full = div(tokens, a.by_bs);
  return full + (tokens > full * a.bs);
}

// Exclusive scans of two values a thread over the CTA; all[] receives the sums.
__device__ __forceinline__ void block_scan_two(int64_t* v, int64_t (*s_w)[32], int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl[2] = {v[0], v[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t t = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += t;
    }
  if (lane == 31) {
    s_w[0][warp] = incl[0];
    s_w[1][warp] = incl[1];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {  // (as many warps as lanes)
    const int64_t mine = s_w[k][lane];
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    all[k] = __shfl_sync(0xffffffffu, sum, 31);
    v[k] = __shfl_sync(0xffffffffu, sum - mine, warp) + incl[k] - v[k];
  }
}

// The last CTA of the call to arrive (thread 0 decides; every thread gets the answer).  The
// arrival count is left zero.
__device__ __forceinline__ bool last_cta(int32_t* count, int* s_last) {
  __syncthreads();
  if (gridDim.x == 1) return true;
  if (threadIdx.x == 0) {
    __threadfence();
    const int n = atomicAdd(count, 1);
    *s_last = n == static_cast<int>(gridDim.x) - 1;
    if (*s_last) {
      *count = 0;
      __threadfence();
    }
  }
  __syncthreads();
  return *s_last != 0;
}

// Page tables grown by n_r new tokens a request.  With held_r = ceil(len_r / bs) and
// need_r = ceil((len_r + n_r) / bs) - held_r, the i-th page needed (requests in order, pages
// ascending) is free_pages[n_free - 1 - i]; new token t of request r, at position
// pos = len_r + t, gets slot page * bs + pos % bs.  Every CTA scans the requests (at most
// 4096, one pass in shared memory) and maps its share of the tokens: no page is read from
// the table that this call writes, so the CTAs need no order among them, and the one that
// finishes last moves the lengths and the free count.  A call that cannot be served whole
// (too few pages, a table row too short, a bad count) changes nothing.
// Bound by latency, the chain lengths, scan, slots, lengths: with a truncate after it, 256 requests
// that grow by a token take 9.0 us, 33 that grow by 96K tokens in 24-token pages 12.3.
__global__ void __launch_bounds__(kTableThreads) extend_kernel(TableArgs a) {
  __shared__ int32_t s_start[kMaxRequests + 1], s_page[kMaxRequests + 1];
  __shared__ int64_t s_w[2][32];
  __shared__ int s_last;
  wait_for_stream();
  const int tid = threadIdx.x, R = a.n_requests, r0 = tid * a.per;
  int len[kPer], add[kPer], need[kPer];
  int64_t sum[2] = {0, 0}, all[2];  // tokens, pages
  int bad = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    len[i] = add[i] = 0;
    if (i < a.per && r0 + i < R) {
      len[i] = a.lens[r0 + i];
      add[i] = a.by[r0 + i];
    }
  }
  const int n_free = *a.n_free;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t room = int64_t(a.max_pages) * a.bs;
    if (len[i] < 0 || add[i] < 0 || int64_t(len[i]) + add[i] > room) {
      bad = 1;
      len[i] = add[i] = 0;
    }
    need[i] = pages_of(a, len[i] + add[i]) - pages_of(a, len[i]);
    sum[0] += add[i];
    sum[1] += need[i];
  }
  bad = __syncthreads_or(bad);
  block_scan_two(sum, s_w, all);
  bad |= all[0] > a.n_slots || all[1] > n_free || n_free > a.n_pages;
  if (!bad) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i < a.per && r0 + i < R) {
        s_start[r0 + i] = static_cast<int>(sum[0]);
        s_page[r0 + i] = static_cast<int>(sum[1]);
      }
      sum[0] += add[i];
      sum[1] += need[i];
    }
    if (tid == 0) s_start[R] = static_cast<int>(all[0]);
  }
  __syncthreads();
  const int total = bad ? 0 : static_cast<int>(all[0]);
  const int step = gridDim.x * kTableThreads;
  for (int i = blockIdx.x * kTableThreads + tid; i < a.n_slots; i += step) {
    int slot = -1;
    if (i < total) {
      const int r = last_at_most(s_start, R, i);
      const int len_r = a.lens[r], held = pages_of(a, len_r);
      const int pos = len_r + i - s_start[r], j = div(pos, a.by_bs), row = pos - j * a.bs;
      int page;
      if (j < held) {
        page = a.table[int64_t(r) * a.max_pages + j];
      } else {
        page = a.free_pages[n_free - 1 - (s_page[r] + j - held)];
        if (row == 0) a.table[int64_t(r) * a.max_pages + j] = page;
      }
      slot = page * a.bs + row;
    }
    a.slots[i] = slot;
  }
  for (int r = blockIdx.x * kTableThreads + tid; r <= R; r += step)
    a.starts[r] = bad ? 0 : s_start[r];
  if (!last_cta(a.status + 4, &s_last)) return;
  if (bad) {
    if (tid == 0) report(a.status, RBA_ERR_BOUNDS, kWherePaged, -1);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < a.per && r0 + i < R && add[i] != 0) a.lens[r0 + i] = len[i] + add[i];
  if (tid == 0) *a.n_free = n_free - static_cast<int>(all[1]);
}

// Requests cut back to min(len_r, keep_r) tokens.  The pages past them go back to the free
// list in the order opposite to extend's, so that a cut undoes the extension before it.
__global__ void __launch_bounds__(kTableThreads) truncate_kernel(TableArgs a) {
  __shared__ int32_t s_page[kMaxRequests + 1];
  __shared__ int64_t s_w[2][32];
  __shared__ int s_last;
  wait_for_stream();
  const int tid = threadIdx.x, R = a.n_requests, r0 = tid * a.per;
  int len[kPer], keep[kPer], kept[kPer], freed[kPer];
  int64_t sum[2] = {0, 0}, all[2];  // (the first unused), pages
  int bad = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    len[i] = keep[i] = 0;
    if (i < a.per && r0 + i < R) {
      len[i] = a.lens[r0 + i];
      keep[i] = a.by[r0 + i];
    }
  }
  const int n_free = *a.n_free;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (len[i] < 0 || keep[i] < 0 || len[i] > int64_t(a.max_pages) * a.bs) {
      bad = 1;
      len[i] = keep[i] = 0;
    }
    kept[i] = min(len[i], keep[i]);
    freed[i] = pages_of(a, len[i]) - pages_of(a, kept[i]);
    sum[1] += freed[i];
  }
  bad = __syncthreads_or(bad);
  block_scan_two(sum, s_w, all);
  bad |= n_free < 0 || n_free + all[1] > a.n_pages;
  if (!bad) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i < a.per && r0 + i < R) s_page[r0 + i] = static_cast<int>(sum[1]);
      sum[1] += freed[i];
    }
  }
  __syncthreads();
  const int total = bad ? 0 : static_cast<int>(all[1]);
  for (int i = blockIdx.x * kTableThreads + tid; i < total; i += gridDim.x * kTableThreads) {
    const int r = last_at_most(s_page, R, i);
    const int j = pages_of(a, min(a.lens[r], a.by[r])) + i - s_page[r];
    a.free_pages[n_free + total - 1 - i] = a.table[int64_t(r) * a.max_pages + j];
  }
  if (!last_cta(a.status + 4, &s_last)) return;
  if (bad) {
    if (tid == 0) report(a.status, RBA_ERR_BOUNDS, kWherePaged, -2);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < a.per && r0 + i < R) a.lens[r0 + i] = kept[i];
  if (tid == 0) *a.n_free = n_free + total;
}

TableArgs table_args(const rba_paged* s, const int32_t* by, int n_requests) {
  TableArgs a = {};
  a.by = by;
  a.lens = s->b.lens;
  a.table = s->b.table;
  a.free_pages = s->b.free_pages;
  a.n_free = s->b.n_free;
  a.status = s->b.status;
  a.n_requests = n_requests;
  a.bs = s->d.page_size;
  a.max_pages = s->d.max_pages;
  a.n_pages = s->d.n_pages;
  a.per = (n_requests + kTableThreads - 1) / kTableThreads;
  a.by_bs = fast_div(a.bs);
  return a;
}

}  // namespace
}  // namespace rba

extern "C" {

rba_status rba_paged_create(const rba_paged_desc* d, const rba_paged_buffers* b,
                            rba_paged** out) {
  if (d == nullptr || b == nullptr || out == nullptr) return RBA_ERR_INVALID_ARG;
  *out = nullptr;
  if (d->n_q_heads <= 0 || d->n_kv_heads <= 0 || d->n_q_heads % d->n_kv_heads != 0 ||
      d->page_size <= 0 || d->n_pages <= 0 || d->max_requests <= 0 || d->max_pages <= 0)
    return RBA_ERR_INVALID_ARG;
  if (d->dtype != RBA_F32 && d->dtype != RBA_BF16) return RBA_ERR_INVALID_ARG;
  if (rba::pool_pitch(d->head_dim) < 0 || d->max_requests > rba::kMaxRequests)
    return RBA_ERR_UNSUPPORTED;
  // token positions and slots are 32-bit
  if (int64_t(d->n_pages) * d->page_size > INT32_MAX ||
      int64_t(d->max_pages) * d->page_size > INT32_MAX)
    return RBA_ERR_UNSUPPORTED;
  if (b->pool == nullptr || b->rep == nullptr || b->table == nullptr || b->lens == nullptr ||
      b->free_pages == nullptr || b->n_free == nullptr || b->status == nullptr)
    return RBA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(b->pool) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(b->rep) % 16 != 0)
    return RBA_ERR_INVALID_ARG;
  rba_paged* s = new (std::nothrow) rba_paged;
  if (s == nullptr) return RBA_ERR_INVALID_ARG;
  s->d = *d;
  s->b = *b;
  s->pitch = rba::pool_pitch(d->head_dim);
  s->strips = (d->page_size + rba::kStrip - 1) / rba::kStrip;
  *out = s;
  return RBA_OK;
}

rba_status rba_paged_destroy(rba_paged* store) {
  delete store;
  return RBA_OK;
}

int32_t rba_paged_strip_bytes(int32_t head_dim) {
  const int p = rba::pool_pitch(head_dim);
  return p < 0 ? -1 : rba::strip_bytes(p);
}

rba_status rba_paged_extend(rba_paged* s, const int32_t* n_new, int32_t n_requests,
                            int32_t* slots, int32_t n_slots, int32_t* starts,
                            cudaStream_t stream) {
  using namespace rba;
  if (s == nullptr || n_new == nullptr || starts == nullptr || n_requests <= 0 ||
      n_requests > s->d.max_requests || n_slots < 0 || (n_slots > 0 && slots == nullptr))
    return RBA_ERR_INVALID_ARG;
  TableArgs a = table_args(s, n_new, n_requests);
  a.slots = slots;
  a.n_slots = n_slots;
  a.starts = starts;
  int grid = (n_slots + kTableThreads - 1) / kTableThreads;
  grid = grid < 1 ? 1 : grid > num_sms() ? num_sms() : grid;
  RBA_CUDA_TRY(launch_dependent(extend_kernel, static_cast<unsigned>(grid), kTableThreads, 0,
                                stream, a));
  return RBA_OK;
}

rba_status rba_paged_truncate(rba_paged* s, const int32_t* keep, int32_t n_requests,
                              cudaStream_t stream) {
  using namespace rba;
  if (s == nullptr || keep == nullptr || n_requests <= 0 || n_requests > s->d.max_requests)
    return RBA_ERR_INVALID_ARG;
  const TableArgs a = table_args(s, keep, n_requests);
  // at most a store's pages come back
  int grid = (s->d.n_pages + 4 * kTableThreads - 1) / (4 * kTableThreads);
  grid = grid > num_sms() ? num_sms() : grid;
  RBA_CUDA_TRY(launch_dependent(truncate_kernel, static_cast<unsigned>(grid), kTableThreads, 0,
                                stream, a));
  return RBA_OK;
}

rba_status rba_paged_check(const rba_paged* s, cudaStream_t stream) {
  if (s == nullptr) return RBA_ERR_INVALID_ARG;
  int32_t h[4] = {0, 0, 0, 0};
  if (cudaMemcpyAsync(h, s->b.status, sizeof(h), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return RBA_ERR_CUDA;
  if (h[0] != 0) {
    if (cudaMemsetAsync(s->b.status, 0, sizeof(h), stream) != cudaSuccess) return RBA_ERR_CUDA;
    return static_cast<rba_status>(h[0]);
  }
  return RBA_OK;
}

}  // extern "C"
