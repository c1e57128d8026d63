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
constexpr int kRowWarps = kRowThreads / 32;
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
  int window;  // slots a warp looks for strips in
  bool vec;    // every row starts on a boundary of four elements
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
__device__ __forceinline__ uint32_t unit_of(const float* x, float inv) {
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
__device__ __forceinline__ void write_half(const RowArgs& a, int i0, int h, int t0, int n,
                                           int which, int half, uint8_t* to, bool v_pairs) {
  constexpr int LPR = P / 4;
  const int lane = threadIdx.x & 31, sub = lane % LPR, g = sub / 8, l = sub % 8;
  const int first = half * 8 - t0;  // run index of the half's token 0
  if (first + 8 <= 0 || first >= n) return;
  const T* base = which == 0 ? static_cast<const T*>(a.k) + i0 * a.k_tok + h * a.k_head
                             : static_cast<const T*>(a.v) + i0 * a.v_tok + h * a.v_head;
  const int64_t step = which == 0 ? a.k_tok : a.v_tok;
  float x[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
    const int i = first + j;
    if (i >= 0 && i < n && sub * 4 < a.dim) load4(base + i * step + sub * 4, a.vec, x[j]);
  }
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m[j] = max(m[j], __float_as_uint(x[j][e]) & 0x7fffffffu);
  }
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

// One CTA per (window of slots, head): it writes the runs, each of consecutive slots of one
// strip, whose first slot lies in its window, a warp to each half strip of K and of V.  A whole
// strip is put together in shared memory and leaves it in 16-byte pieces; a part of one goes out
// unit by unit (the rows beside it belong to other calls).
template <int P> constexpr int append_warps() { return P == 128 ? 4 : 2; }
template <typename T, int P>
__global__ void __launch_bounds__(append_warps<P>() * 32) append_kernel(RowArgs a) {
  constexpr int SB = strip_bytes(P), kThreads = append_warps<P>() * 32;
  __shared__ __align__(16) uint8_t s_stage[SB];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = P == 128 ? warp >> 1 : lane >> 4, half = warp & 1;
  const int h = blockIdx.x % a.heads;
  const int64_t base = int64_t(blockIdx.x / a.heads) * a.window;
  // lane i looks at slot base - 1 + i (window <= 16: a run's 16 slots stay within the warp)
  const int64_t i = base - 1 + lane;
  int slot = i >= 0 && i < a.n ? a.slots[i] : -1;
  int page = 0, row = 0;
  if (slot >= 0) {
    page = slot / a.bs;
    row = slot - page * a.bs;
    if (page >= a.n_pages) {
      if (h == 0 && warp == 0 && lane >= 1 && lane <= a.window)
        report(a.status, RBA_ERR_BOUNDS, kWherePaged, slot);
      slot = -1;
    }
  }
  const int before = __shfl_up_sync(0xffffffffu, slot, 1);
  const bool next = slot >= 0 && lane > 0 && before == slot - 1 && row % kStrip != 0;
  const unsigned follows = __ballot_sync(0xffffffffu, next);
  unsigned firsts = __ballot_sync(0xffffffffu, slot >= 0 && !next && lane >= 1 && lane <= a.window);
  while (firsts) {
    const int f = __ffs(firsts) - 1;
    firsts &= firsts - 1;
    const int n = __ffs(~(follows >> (f + 1)));  // the first and those that follow it
    const int p = __shfl_sync(0xffffffffu, page, f), r = __shfl_sync(0xffffffffu, row, f);
    uint8_t* strip = a.pool + ((int64_t(p) * a.heads + h) * a.strips + r / kStrip) * SB;
    const bool whole = n == kStrip;
    write_half<T, P>(a, static_cast<int>(base) - 1 + f, h, r % kStrip, n, which, half,
                     whole ? s_stage : strip, whole);
    if (!whole) continue;
    __syncthreads();
    for (int o = threadIdx.x * 16; o < SB; o += kThreads * 16)
      *reinterpret_cast<uint4*>(strip + o) = *reinterpret_cast<const uint4*>(s_stage + o);
    __syncthreads();
  }
}

// Means of the pages whose last row is among the slots: one CTA per 32 slots and eight heads, one
// warp per head.  Lane (t, c) sums rows t, t + 8, .. over dims 8 c .. + 7 of each group in strip
// order; halving exchanges add the eight lanes of a c and leave four dims with each.
template <int P>
__global__ void __launch_bounds__(kRowThreads) page_mean_kernel(RowArgs a) {
  constexpr int G = P / 32, SB = strip_bytes(P);
  wait_for_stream();
  const int lane = threadIdx.x & 31, t = lane >> 2, c = lane & 3;
  const int chunks = (a.heads + kRowWarps - 1) / kRowWarps;
  const int h = blockIdx.x % chunks * kRowWarps + (threadIdx.x >> 5);
  const int64_t i = int64_t(blockIdx.x / chunks) * 32 + lane;
  const int mine = i < a.n ? a.slots[i] : -1;
  unsigned done = __ballot_sync(
      0xffffffffu, mine >= 0 && mine / a.bs < a.n_pages && mine % a.bs == a.bs - 1);
  if (h >= a.heads) return;
  for (; done; done &= done - 1) {
    const int page = __shfl_sync(0xffffffffu, mine, __ffs(done) - 1) / a.bs;
    const uint8_t* strip = a.pool + (int64_t(page) * a.heads + h) * a.strips * SB;
    float acc[8 * G];
#pragma unroll
    for (int e = 0; e < 8 * G; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.strips; ++s, strip += SB) {
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
    // lane (t, c) ends with values (8 G / 8) t .. of the c's 8 G
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
      const bool up = (t & w) != 0;
#pragma unroll
      for (int e = 0; e < G * w; ++e) {
        const float give = up ? acc[e] : acc[e + G * w], keep = up ? acc[e + G * w] : acc[e];
        acc[e] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * w);
      }
    }
    float* rep = a.rep + (int64_t(page) * a.heads + h) * P;
#pragma unroll
    for (int e = 0; e < G; ++e) {
      const int at = G * t + e;  // of (group, dim) = (at / 8, at % 8)
      rep[32 * (at / 8) + 8 * c + at % 8] = acc[e] / static_cast<float>(a.bs);
    }
  }
}

// One warp per slot and four heads: lane (g, l) four dims of a row (P = 64: K in one half of
// the warp, V in the other).
template <typename T, int P>
__global__ void __launch_bounds__(kRowThreads) read_kernel(RowArgs a) {
  constexpr int LPR = P / 4, SB = strip_bytes(P), kHeads = 4;
  wait_for_stream();
  const int lane = threadIdx.x & 31, sub = lane % LPR, g = sub / 8, l = sub % 8;
  const int64_t w = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int chunks = (a.heads + kHeads - 1) / kHeads;
  const int64_t i = w / chunks;
  const int h0 = static_cast<int>(w - i * chunks) * kHeads;
  if (i >= a.n) return;
  const int slot = a.slots[i];
  const int page = slot >= 0 ? slot / a.bs : 0, row = slot - page * a.bs, t = row % kStrip;
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
  return a;
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
  // a CTA per slot while that is at most one wave; else fewer CTAs look through more slots
  a.window = int64_t(n) * a.heads <= int64_t(num_sms()) * 16 ? 1 : 16;
  const int64_t grid = (int64_t(n) + a.window - 1) / a.window * a.heads;
  const int64_t means = (int64_t(n) + 31) / 32 * ((a.heads + kRowWarps - 1) / kRowWarps);
  if (grid > INT32_MAX || means > INT32_MAX) return RBA_ERR_UNSUPPORTED;
#define RBA_APPEND(T_, P_)                                                                       \
  do {                                                                                           \
    RBA_CUDA_TRY(launch_dependent(append_kernel<T_, P_>, static_cast<unsigned>(grid),            \
                                  append_warps<P_>() * 32, 0, stream, a));                       \
    RBA_CUDA_TRY(launch_dependent(page_mean_kernel<P_>, static_cast<unsigned>(means), kRowThreads, \
                                  0, stream, a));                                                \
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
  const int64_t blocks = (int64_t(n) * ((a.heads + 3) / 4) + kRowWarps - 1) / kRowWarps;
  if (blocks > INT32_MAX) return RBA_ERR_UNSUPPORTED;
  const auto kernel = s->d.dtype == RBA_BF16
                          ? (s->pitch == 128 ? read_kernel<__nv_bfloat16, 128>
                                             : read_kernel<__nv_bfloat16, 64>)
                          : (s->pitch == 128 ? read_kernel<float, 128> : read_kernel<float, 64>);
  RBA_CUDA_TRY(
      launch_dependent(kernel, static_cast<unsigned>(blocks), kRowThreads, 0, stream, a));
  return RBA_OK;
}
