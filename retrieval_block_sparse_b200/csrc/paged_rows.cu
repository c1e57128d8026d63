// Paged 4-bit memory: rows written (quantised), read back, and the means of the pages that
// the new rows complete.
//
// A row of P dims is held as G = P / 32 groups.  With a = the largest |x| of a group,
//   s = bf16(a / 7), 0 where a / 7 rounds below 2^-100, NaN where a is not finite,
//   c = min(max(rint(x * fl(1 / s)), -7), 7)  (0 where s is 0 or NaN),   value = s c:
// symmetric, so that a zero stays zero and the attention kernel needs no offset per group; a
// bf16 scale has the range of the inputs, and its 2^-9 rounding moves a value by at most
// 7 * 2^-9 of a step.  Every operation is a correctly rounded 32-bit one, so the codes are a
// function of the inputs alone.
#include "paged.cuh"

namespace rba {
namespace {

constexpr int kRowThreads = 256;
constexpr float kLeastScale = 0x1p-100f;

struct RowArgs {
  const int32_t* slots;
  const void* k;
  const void* v;
  int64_t k_tok, k_head, v_tok, v_head;  // strides of the caller's rows, elements
  void* k_out;
  void* v_out;
  uint8_t* pool;
  float* rep;
  int32_t* status;
  int n, heads, dim, bs, strips, n_pages;
};

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
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

// The four codes (one 16-bit unit) of a lane's dims and the group's scale; the eight lanes of
// a group call it together.
__device__ __forceinline__ uint32_t quantise4(const float* x, __nv_bfloat16* scale) {
  float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  bool odd = !(isfinite(x[0]) && isfinite(x[1]) && isfinite(x[2]) && isfinite(x[3]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  const unsigned any = __ballot_sync(0xffffffffu, odd);
  odd = (any >> (threadIdx.x & 24)) & 0xffu;
  __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(a, 7.f));
  float sf = __bfloat162float(s);
  if (odd || !isfinite(sf)) {
    *scale = __ushort_as_bfloat16(0x7fff);
    return 0x8888u;
  }
  if (sf < kLeastScale) {
    *scale = __ushort_as_bfloat16(0);
    return 0x8888u;
  }
  *scale = s;
  const float inv = __frcp_rn(sf);
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = __float2int_rn(fminf(fmaxf(__fmul_rn(x[j], inv), -7.f), 7.f));
    u |= static_cast<uint32_t>(c + 8) << (4 * j);
  }
  return u;
}

__device__ __forceinline__ void values4(uint32_t unit, float s, float* x) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = __fmul_rn(static_cast<float>(static_cast<int>((unit >> (4 * j)) & 15u) - 8), s);
}

template <int P>
__device__ __forceinline__ uint8_t* strip_of(const RowArgs& a, int slot, int h, int* t) {
  const int page = slot / a.bs, row = slot - page * a.bs;
  *t = row % kStrip;
  return a.pool +
         ((int64_t(page) * a.heads + h) * a.strips + row / kStrip) * strip_bytes(P);
}

// One lane per four dims of one (token, head, K or V) row.
template <typename T, int P>
__global__ void __launch_bounds__(kRowThreads) append_kernel(RowArgs a, bool vec) {
  constexpr int LPR = P / 4;
  const int64_t item = (int64_t(blockIdx.x) * kRowThreads + threadIdx.x) / LPR;
  const int lane = threadIdx.x % LPR, g = lane / 8, l = lane % 8;
  const bool live = item < int64_t(a.n) * a.heads * 2;  // (whole rows; the shuffles need all lanes)
  const int which = static_cast<int>(item & 1);
  const int64_t th = item >> 1;
  const int i = live ? static_cast<int>(th / a.heads) : 0, h = static_cast<int>(th % a.heads);
  const int slot = live ? a.slots[i] : -1;
  const bool in = slot >= 0 && slot / a.bs < a.n_pages;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (in && lane * 4 < a.dim) {
    const T* src = which == 0
                       ? static_cast<const T*>(a.k) + i * a.k_tok + h * a.k_head
                       : static_cast<const T*>(a.v) + i * a.v_tok + h * a.v_head;
    load4(src + lane * 4, vec, x);
  }
  __nv_bfloat16 s;
  const uint32_t unit = quantise4(x, &s);
  if (!in) {
    if (slot >= 0 && lane == 0) report(a.status, RBA_ERR_BOUNDS, kWherePaged, slot);
    return;
  }
  int t;
  uint8_t* strip = strip_of<P>(a, slot, h, &t);
  const int at = which == 0 ? k_unit_at<P>(t, g, l) : v_unit_at<P>(t, g, l);
  *reinterpret_cast<uint16_t*>(strip + at) = static_cast<uint16_t>(unit);
  if (l == 0) *reinterpret_cast<__nv_bfloat16*>(strip + scale_at<P>(t, which, g)) = s;
}

// Means of the pages whose last row is among the slots: one CTA per 32 slots and head; the
// page's rows are split over the CTA's row groups and the partial sums added in a fixed order.
template <int P>
__global__ void __launch_bounds__(kRowThreads) page_mean_kernel(RowArgs a) {
  constexpr int LPR = P / 4, RG = kRowThreads / LPR;
  __shared__ float part[RG][P];
  const int lane = threadIdx.x % LPR, rg = threadIdx.x / LPR, g = lane / 8, l = lane % 8;
  const int h = blockIdx.y;
  const int i = blockIdx.x * 32 + (threadIdx.x & 31);
  const int mine = i < a.n ? a.slots[i] : -1;
  unsigned done = __ballot_sync(0xffffffffu, mine >= 0 && mine / a.bs < a.n_pages &&
                                                 mine % a.bs == a.bs - 1);
  while (done) {
    const int page = __shfl_sync(0xffffffffu, mine, __ffs(done) - 1) / a.bs;
    done &= done - 1;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int row = rg; row < a.bs; row += RG) {
      int t;
      const uint8_t* strip = strip_of<P>(a, page * a.bs + row, h, &t);
      float x[4];
      values4(*reinterpret_cast<const uint16_t*>(strip + k_unit_at<P>(t, g, l)),
              __bfloat162float(
                  *reinterpret_cast<const __nv_bfloat16*>(strip + scale_at<P>(t, 0, g))),
              x);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += x[j];
    }
    store4(&part[rg][lane * 4], acc);
    __syncthreads();
    if (threadIdx.x < P) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < RG; ++q) sum += part[q][threadIdx.x];
      a.rep[(int64_t(page) * a.heads + h) * P + threadIdx.x] = sum / static_cast<float>(a.bs);
    }
    __syncthreads();
  }
}

template <typename T, int P>
__global__ void __launch_bounds__(kRowThreads) read_kernel(RowArgs a) {
  constexpr int LPR = P / 4;
  const int64_t item = (int64_t(blockIdx.x) * kRowThreads + threadIdx.x) / LPR;
  const int lane = threadIdx.x % LPR, g = lane / 8, l = lane % 8;
  if (item >= int64_t(a.n) * a.heads * 2 || lane * 4 >= a.dim) return;
  const int which = static_cast<int>(item & 1);
  const int64_t th = item >> 1;
  const int i = static_cast<int>(th / a.heads), h = static_cast<int>(th % a.heads);
  const int slot = a.slots[i];
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (slot >= 0 && slot / a.bs < a.n_pages) {
    int t;
    const uint8_t* strip = strip_of<P>(a, slot, h, &t);
    values4(*reinterpret_cast<const uint16_t*>(
                strip + (which == 0 ? k_unit_at<P>(t, g, l) : v_unit_at<P>(t, g, l))),
            __bfloat162float(
                *reinterpret_cast<const __nv_bfloat16*>(strip + scale_at<P>(t, which, g))),
            x);
  } else if (slot >= 0 && lane == 0) {
    report(a.status, RBA_ERR_BOUNDS, kWherePaged, slot);
  }
  store4(static_cast<T*>(which == 0 ? a.k_out : a.v_out) + th * a.dim + lane * 4, x);
}

RowArgs row_args(const rba_paged* s, const int32_t* slots, int n) {
  RowArgs a = {};
  a.slots = slots;
  a.pool = static_cast<uint8_t*>(s->b.pool);
  a.rep = s->b.rep;
  a.status = s->b.status;
  a.n = n;
  a.heads = s->d.n_kv_heads;
  a.dim = s->d.head_dim;
  a.bs = s->d.page_size;
  a.strips = s->strips;
  a.n_pages = s->d.n_pages;
  return a;
}

bool rows_in_grid(int64_t n, int heads, int lanes) {
  return n * heads * 2 * lanes / kRowThreads < INT32_MAX - 1;
}

}  // namespace
}  // namespace rba

extern "C" rba_status rba_paged_append(rba_paged* s, const int32_t* slots, int32_t n,
                                       const void* k, int64_t k_token_stride,
                                       int64_t k_head_stride, const void* v,
                                       int64_t v_token_stride, int64_t v_head_stride,
                                       cudaStream_t stream) {
  using namespace rba;
  if (s == nullptr || n < 0) return RBA_ERR_INVALID_ARG;
  if (n == 0) return RBA_OK;
  if (slots == nullptr || k == nullptr || v == nullptr) return RBA_ERR_INVALID_ARG;
  const int lanes = s->pitch / 4;
  if (!rows_in_grid(n, s->d.n_kv_heads, lanes)) return RBA_ERR_UNSUPPORTED;
  RowArgs a = row_args(s, slots, n);
  a.k = k;
  a.v = v;
  a.k_tok = k_token_stride;
  a.k_head = k_head_stride;
  a.v_tok = v_token_stride;
  a.v_head = v_head_stride;
  // four dims in one load where every row starts on their boundary
  const uintptr_t unit = 4 * dtype_size(s->d.dtype);
  const bool vec = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % unit == 0 &&
                   ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 3) == 0;
  const int64_t rows = int64_t(n) * s->d.n_kv_heads * 2;
  const int grid = static_cast<int>((rows * lanes + kRowThreads - 1) / kRowThreads);
  const dim3 mean_grid((n + 31) / 32, s->d.n_kv_heads);
#define RBA_APPEND(T_, P_)                                                \
  do {                                                                    \
    append_kernel<T_, P_><<<grid, kRowThreads, 0, stream>>>(a, vec);      \
    RBA_LAUNCH_CHECK();                                                   \
    page_mean_kernel<P_><<<mean_grid, kRowThreads, 0, stream>>>(a);       \
  } while (0)
  if (s->d.dtype == RBA_BF16) {
    if (s->pitch == 128) RBA_APPEND(__nv_bfloat16, 128);
    else RBA_APPEND(__nv_bfloat16, 64);
  } else {
    if (s->pitch == 128) RBA_APPEND(float, 128);
    else RBA_APPEND(float, 64);
  }
#undef RBA_APPEND
  RBA_LAUNCH_CHECK();
  return RBA_OK;
}

extern "C" rba_status rba_paged_read(const rba_paged* s, const int32_t* slots, int32_t n,
                                     void* k, void* v, cudaStream_t stream) {
  using namespace rba;
  if (s == nullptr || n < 0) return RBA_ERR_INVALID_ARG;
  if (n == 0) return RBA_OK;
  if (slots == nullptr || k == nullptr || v == nullptr) return RBA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 != 0)
    return RBA_ERR_INVALID_ARG;
  const int lanes = s->pitch / 4;
  if (!rows_in_grid(n, s->d.n_kv_heads, lanes)) return RBA_ERR_UNSUPPORTED;
  RowArgs a = row_args(s, slots, n);
  a.k_out = k;
  a.v_out = v;
  const int64_t rows = int64_t(n) * s->d.n_kv_heads * 2;
  const int grid = static_cast<int>((rows * lanes + kRowThreads - 1) / kRowThreads);
  if (s->d.dtype == RBA_BF16) {
    if (s->pitch == 128) read_kernel<__nv_bfloat16, 128><<<grid, kRowThreads, 0, stream>>>(a);
    else read_kernel<__nv_bfloat16, 64><<<grid, kRowThreads, 0, stream>>>(a);
  } else {
    if (s->pitch == 128) read_kernel<float, 128><<<grid, kRowThreads, 0, stream>>>(a);
    else read_kernel<float, 64><<<grid, kRowThreads, 0, stream>>>(a);
  }
  RBA_LAUNCH_CHECK();
  return RBA_OK;
}
