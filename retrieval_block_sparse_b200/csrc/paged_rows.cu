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

constexpr float kLeastScale = 0x1p-100f;
constexpr float kToInt = 12582920.f;  // 1.5 2^23 + 8: adding it leaves rint(x) + 8 in the low bits

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
  int window;  // slots a CTA looks for runs in
  FastDiv by_bs, by_heads;
  bool vec;    // every row starts on a boundary of four elements
};

// Four elements of a row as they were loaded: their values, and the bits of the largest |x|
// (compared as integers: values that are not finite are the largest).
template <typename T> struct Four;
template <> struct Four<float> {
  float x[4];
  __device__ __forceinline__ void load(const float* p, bool vec) { load4(p, vec, x); }
  __device__ __forceinline__ void zero() { x[0] = x[1] = x[2] = x[3] = 0.f; }
  __device__ __forceinline__ float operator[](int i) const { return x[i]; }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
  }
};
template <> struct Four<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec) {
    if (vec) {
      u = *reinterpret_cast<const uint2*>(p);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      u.x = h[0] | uint32_t(h[1]) << 16;
      u.y = h[2] | uint32_t(h[3]) << 16;
    }
  }
  __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? u.x : u.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
};
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

// A group's scale and the factor of its codes (0 where the codes are all 0) from the bits of its
// largest |x| (as integers, values that are not finite are the largest).
__device__ __forceinline__ void scale_of_max(uint32_t bits, uint16_t* scale, float* inv) {
  const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(bits), 7.f));
  const float sf = __bfloat162float(s);
  const bool odd = bits >= 0x7f800000u, none = sf < kLeastScale;
  *scale = odd ? 0x7fff : none ? 0 : __bfloat16_as_ushort(s);
  *inv = odd || none ? 0.f : __frcp_rn(sf);
}
// Four codes, one 16-bit unit.  |x| inv <= 7 (1 + 2^-8) rounds to 7 at most: no clamp is needed.
template <typename R>
__device__ __forceinline__ uint32_t unit_of(const R& x, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(__fadd_rn(__fmul_rn(x[j], inv), kToInt));
  const uint32_t u = (b[0] + (b[1] << 4) + (b[2] << 8) + (b[3] << 12)) & 0xffffu;
  return inv == 0.f ? 0x8888u : u;
}
// c of the low nibble c + 8: as the low bits of 2^23 + c + 8
__device__ __forceinline__ float code_of(uint32_t nibble) {
  return __uint_as_float((nibble & 15u) | 0x4b000000u) - 8388616.f;
}
__device__ __forceinline__ void values4(uint32_t unit, float s, float* x) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = __fmul_rn(code_of(unit >> (4 * j)), s);
}

// Quantises eight tokens' K or V rows of one strip: tokens [t0, t0 + n) of the strip are slots
// i0 .. of the call, head h; this warp takes those of half `half`.  Lane (g, l) holds four dims of
// each row (P = 64: K in one half of the warp, V in the other).  The rows' largest values are
// found by halving exchanges that leave row l with lane l, so that the division and the reciprocal
// are computed once per group.  Everything goes to `to`, the strip or its copy in shared memory;
// v_pairs: the tokens' V units can be written two at a time.
template <typename T, int P>
__device__ __forceinline__ void write_half(const RowArgs& a, int64_t i0, int h, int t0, int n,
                                           int which, int half, uint8_t* to, bool v_pairs) {
  constexpr int LPR = P / 4;
  const int lane = threadIdx.x & 31, sub = lane % LPR, g = sub / 8, l = sub % 8;
  const int first = half * 8 - t0;  // run index of the half's token 0
  if (first + 8 <= 0 || first >= n) return;
  const T* base = which == 0 ? static_cast<const T*>(a.k) + i0 * a.k_tok + h * a.k_head
                             : static_cast<const T*>(a.v) + i0 * a.v_tok + h * a.v_head;
  const int64_t step = which == 0 ? a.k_tok : a.v_tok;
  Four<T> x[8];
  const T* p = base + first * step + sub * 4;
#pragma unroll
  for (int j = 0; j < 8; ++j, p += step) {
    const int i = first + j;
    if (i >= 0 && i < n && sub * 4 < a.dim) x[j].load(p, a.vec);
    else x[j].zero();
  }
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = x[j].top();
  // halving: after the step of width w a lane keeps the w rows that share its bit w
#pragma unroll
  for (int w = 4; w > 0; w >>= 1) {
    const bool up = (l & w) != 0;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const uint32_t give = up ? m[j] : m[j + w], keep = up ? m[j + w] : m[j];
      m[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  uint16_t scale;
  float inv;
  scale_of_max(m[0], &scale, &inv);
  if (first + l >= 0 && first + l < n)
    *reinterpret_cast<uint16_t*>(to + scale_at<P>(half * 8 + l, which, g)) = scale;
  uint32_t unit[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    unit[j] = unit_of(x[j], __shfl_sync(0xffffffffu, inv, (lane & 24) + j));
  if (v_pairs && which == 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint32_t*>(to + v_unit_at<P>(half * 8 + 2 * c, g, l)) =
          unit[2 * c] | unit[2 * c + 1] << 16;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = half * 8 + j;
      if (first + j >= 0 && first + j < n)
        *reinterpret_cast<uint16_t*>(
            to + (which == 0 ? k_unit_at<P>(t, g, l) : v_unit_at<P>(t, g, l))) =
            static_cast<uint16_t>(unit[j]);
    }
  }
}

// The runs whose first slot lies in this CTA's window of slots, each of consecutive slots of one
// strip: calls f(first slot's index, rows, strip, first row of the strip) for each, with every
// thread of the CTA.
template <int P, typename F>
__device__ __forceinline__ void for_runs(const RowArgs& a, int h, int64_t base, const F& f) {
  const int lane = threadIdx.x & 31;
  // lane i looks at slot base - 1 + i (window <= 16: a run's 16 slots stay within the warp)
  const int64_t i = base - 1 + lane;
  int slot = i >= 0 && i < a.n ? a.slots[i] : -1;
  int page = 0, row = 0;
  if (slot >= 0) {
    page = div(slot, a.by_bs);
    row = slot - page * a.bs;
    if (page >= a.n_pages) {
      if (h == 0 && threadIdx.x < 32 && lane >= 1 && lane <= a.window)
        report(a.status, RBA_ERR_BOUNDS, kWherePaged, slot);
      slot = -1;
    }
  }
  const int before = __shfl_up_sync(0xffffffffu, slot, 1);
  const bool next = slot >= 0 && lane > 0 && before == slot - 1 && row % kStrip != 0;
  const unsigned follows = __ballot_sync(0xffffffffu, next);
  unsigned firsts = __ballot_sync(0xffffffffu, slot >= 0 && !next && lane >= 1 && lane <= a.window);
  while (firsts) {
    const int k = __ffs(firsts) - 1;
    firsts &= firsts - 1;
    const int n = __ffs(~(follows >> (k + 1)));  // the first and those that follow it
    const int p = __shfl_sync(0xffffffffu, page, k), r = __shfl_sync(0xffffffffu, row, k);
    const int64_t strip = (int64_t(p) * a.heads + h) * a.strips + r / kStrip;
    f(base - 1 + k, n, a.pool + strip * strip_bytes(P), r % kStrip);
  }
}

// One CTA per (window of slots, head) writes the window's runs, a warp to each half strip of K and
// of V.  A whole strip is put together in shared memory and leaves it in 16-byte pieces; a part of
// one goes out unit by unit (the rows beside it belong to other calls).
// (Eight bf16 rows fit 40 registers a thread, 48 warps an SM; 32-bit rows take 64.)
template <int P> constexpr int run_warps() { return P == 128 ? 4 : 2; }
template <typename T, int P>
__global__ void __launch_bounds__(run_warps<P>() * 32,
                                  (sizeof(T) == 2 ? 1536 : 1024) / (run_warps<P>() * 32))
    append_kernel(RowArgs a) {
  constexpr int SB = strip_bytes(P), kThreads = run_warps<P>() * 32;
  __shared__ __align__(16) uint8_t s_stage[SB];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = P == 128 ? warp >> 1 : lane >> 4, half = warp & 1;
  const int w = div(blockIdx.x, a.by_heads), h = blockIdx.x - w * a.heads;
  for_runs<P>(a, h, int64_t(w) * a.window, [&](int64_t i0, int n, uint8_t* strip, int t0) {
    const bool whole = n == kStrip;
    write_half<T, P>(a, i0, h, t0, n, which, half, whole ? s_stage : strip, whole);
    if (!whole) return;
    __syncthreads();
    for (int o = threadIdx.x * 16; o < SB; o += kThreads * 16)
      *reinterpret_cast<uint4*>(strip + o) = *reinterpret_cast<const uint4*>(s_stage + o);
    __syncthreads();
  });
}

// Means of the pages whose last row is among the slots: one CTA per (32 slots, head), its warps
// each a share of a page's strips.  Lane (t, c) sums rows t and t + 8 over dims 8 c .. + 7 of each
// group; halving exchanges add the eight lanes of a c and leave G values with each; the warps' sums
// are added in order.
constexpr int kMeanWarps = 8;
template <int P>
__global__ void __launch_bounds__(kMeanWarps * 32) page_mean_kernel(RowArgs a) {
  constexpr int G = P / 32, SB = strip_bytes(P);
  __shared__ float s_sum[kMeanWarps][P];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane >> 2, c = lane & 3;
  const int w32 = div(blockIdx.x, a.by_heads), h = blockIdx.x - w32 * a.heads;
  const int64_t i = int64_t(w32) * 32 + lane;
  const int mine = i < a.n ? a.slots[i] : -1;
  const int at = mine >= 0 ? div(mine, a.by_bs) : 0;
  unsigned done = __ballot_sync(
      0xffffffffu, mine >= 0 && at < a.n_pages && mine - at * a.bs == a.bs - 1);
  for (; done; done &= done - 1) {
    const int page = __shfl_sync(0xffffffffu, at, __ffs(done) - 1);
    const uint8_t* strips = a.pool + (int64_t(page) * a.heads + h) * a.strips * SB;
    float acc[8 * G];
#pragma unroll
    for (int e = 0; e < 8 * G; ++e) acc[e] = 0.f;
    for (int s = warp; s < a.strips; s += kMeanWarps) {
      const uint8_t* strip = strips + int64_t(s) * SB;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t word[G];
        float sc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {  // (a strip's rows past the page exist: loaded, not added)
          word[g] = reinterpret_cast<const uint32_t*>(strip + half * 4 * P + lane * (G * 4))[g];
          sc[g] = __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(
                                      strip + scale_at<P>(half * 8 + t, 0, 0))[g]) << 16);
        }
        if (s * kStrip + half * 8 + t >= a.bs) continue;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[8 * g + j] = fmaf(code_of(word[g] >> (4 * j)), sc[g], acc[8 * g + j]);
      }
    }
    // lane (t, c) ends with values G t .. of its c's 8 G
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
      const bool up = (t & w) != 0;
#pragma unroll
      for (int e = 0; e < G * w; ++e) {
        const float give = up ? acc[e] : acc[e + G * w], keep = up ? acc[e + G * w] : acc[e];
        acc[e] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * w);
      }
    }
#pragma unroll
    for (int e = 0; e < G; ++e) {
      const int v = G * t + e;  // of (group, dim) = (v / 8, v % 8)
      s_sum[warp][32 * (v / 8) + 8 * c + v % 8] = acc[e];
    }
    __syncthreads();
    if (threadIdx.x < P) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kMeanWarps; ++w) sum += s_sum[w][threadIdx.x];
      a.rep[(int64_t(page) * a.heads + h) * P + threadIdx.x] = sum / static_cast<float>(a.bs);
    }
    __syncthreads();
  }
}

// One warp per slot and kHeads heads: lane (g, l) four dims of a row (P = 64: K in one half of
// the warp, V in the other).
constexpr int kReadWarps = 8, kHeads = 2;
template <typename T, int P>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(RowArgs a) {
  constexpr int LPR = P / 4, SB = strip_bytes(P);
  wait_for_stream();
  const int lane = threadIdx.x & 31, sub = lane % LPR, g = sub / 8, l = sub % 8;
  const int64_t w = int64_t(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
  const int chunks = (a.heads + kHeads - 1) / kHeads;
  const int64_t i = w / chunks;
  const int h0 = static_cast<int>(w - i * chunks) * kHeads;
  if (i >= a.n) return;
  const int slot = a.slots[i];
  const int page = slot >= 0 ? div(slot, a.by_bs) : 0, row = slot - page * a.bs, t = row % kStrip;
  const bool in = slot >= 0 && page < a.n_pages;
  if (slot >= 0 && !in && lane == 0 && h0 == 0) report(a.status, RBA_ERR_BOUNDS, kWherePaged, slot);
  if (sub * 4 >= a.dim) return;
  uint32_t unit[kHeads][2];
  uint16_t scale[kHeads][2];
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
#pragma unroll
    for (int pass = 0; pass < 2 * LPR / 32; ++pass) {
      unit[j][pass] = 0x8888u;
      scale[j][pass] = 0;
      if (!in || h0 + j >= a.heads) continue;
      const int which = P == 128 ? pass : lane / LPR;
      const uint8_t* strip =
          a.pool + ((int64_t(page) * a.heads + h0 + j) * a.strips + row / kStrip) * SB;
      unit[j][pass] = *reinterpret_cast<const uint16_t*>(
          strip + (which == 0 ? k_unit_at<P>(t, g, l) : v_unit_at<P>(t, g, l)));
      scale[j][pass] = *reinterpret_cast<const uint16_t*>(strip + scale_at<P>(t, which, g));
    }
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
#pragma unroll
    for (int pass = 0; pass < 2 * LPR / 32; ++pass) {
      if (h0 + j >= a.heads) continue;
      const int which = P == 128 ? pass : lane / LPR;
      float x[4];
      values4(unit[j][pass], __uint_as_float(uint32_t(scale[j][pass]) << 16), x);
      store4(static_cast<T*>(which == 0 ? a.k_out : a.v_out) +
                 (i * a.heads + h0 + j) * a.dim + sub * 4, x);
    }
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
  // a CTA per slot and head while that is at most one wave; else fewer CTAs look through more slots
  a.window = int64_t(n) * a.heads <= int64_t(num_sms()) * 16 ? 1 : 16;
  a.by_bs = fast_div(a.bs);
  a.by_heads = fast_div(a.heads);
  return a;
}
// CTAs of `slots` slots and one head each; 0 where a grid does not hold them.
unsigned run_grid(const RowArgs& a, int slots) {
  const int64_t grid = (int64_t(a.n) + slots - 1) / slots * a.heads;
  return grid <= INT32_MAX ? static_cast<unsigned>(grid) : 0;
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
  RowArgs a = row_args(s, slots, n);
  a.k = k;
  a.v = v;
  a.k_tok = k_token_stride;
  a.k_head = k_head_stride;
  a.v_tok = v_token_stride;
  a.v_head = v_head_stride;
  // four dims in one load where every row starts on their boundary
  const uintptr_t unit = 4 * dtype_size(s->d.dtype);
  a.vec = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % unit == 0 &&
          ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 3) == 0;
  const unsigned grid = run_grid(a, a.window);
  if (grid == 0) return RBA_ERR_UNSUPPORTED;
#define RBA_APPEND(T_, P_)                                                                      \
  do {                                                                                          \
    RBA_CUDA_TRY(launch_dependent(append_kernel<T_, P_>, grid, run_warps<P_>() * 32, 0, stream, \
                                  a));                                                          \
    RBA_CUDA_TRY(launch_dependent(page_mean_kernel<P_>, run_grid(a, 32), kMeanWarps * 32, 0,    \
                                  stream, a));                                                  \
  } while (0)
  if (s->d.dtype == RBA_BF16) {
    if (s->pitch == 128) RBA_APPEND(__nv_bfloat16, 128);
    else RBA_APPEND(__nv_bfloat16, 64);
  } else {
    if (s->pitch == 128) RBA_APPEND(float, 128);
    else RBA_APPEND(float, 64);
  }
#undef RBA_APPEND
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
  RowArgs a = row_args(s, slots, n);
  a.k_out = k;
  a.v_out = v;
  const int64_t grid =
      (int64_t(n) * ((a.heads + kHeads - 1) / kHeads) + kReadWarps - 1) / kReadWarps;
  if (grid > INT32_MAX) return RBA_ERR_UNSUPPORTED;
  const auto kernel = s->d.dtype == RBA_BF16
                          ? (s->pitch == 128 ? read_kernel<__nv_bfloat16, 128>
                                             : read_kernel<__nv_bfloat16, 64>)
                          : (s->pitch == 128 ? read_kernel<float, 128> : read_kernel<float, 64>);
  RBA_CUDA_TRY(
      launch_dependent(kernel, static_cast<unsigned>(grid), kReadWarps * 32, 0, stream, a));
  return RBA_OK;
}
