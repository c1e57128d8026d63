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
//
// All three kernels are bound by the issue of instructions (56 to 75 % of its slots): 8192 tokens of 8
// heads of 128 in bf16 take 16.6 us to append, the means with it (43 MB), and 9.4 us to read back
// (43 MB, 4.6 TB/s); in 32 bits 20.7 and 12.1 us (77 MB).
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
  FastDiv by_bs, by_heads, by_chunks;
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
  // of eight rows over the eight lanes of a group, row l to lane l: after the step of width w a
  // lane keeps the w rows that share its bit w
  static __device__ __forceinline__ uint32_t top(const Four* r, int l) {
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m[j] = max(m[j], __float_as_uint(r[j].x[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
      const bool up = (l & w) != 0;
#pragma unroll
      for (int j = 0; j < w; ++j) {
        const uint32_t give = up ? m[j] : m[j + w], keep = up ? m[j + w] : m[j];
        m[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, w));
      }
    }
    return m[0];
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
  // the same with two rows to a word
  static __device__ __forceinline__ uint32_t top(const Four* r, int l) {
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = __vmaxu2(r[2 * j].u.x & 0x7fff7fffu, r[2 * j].u.y & 0x7fff7fffu);
      const uint32_t b = __vmaxu2(r[2 * j + 1].u.x & 0x7fff7fffu, r[2 * j + 1].u.y & 0x7fff7fffu);
      m[j] = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
#pragma unroll
    for (int w = 2; w > 0; w >>= 1) {
      const bool up = (l & (2 * w)) != 0;
#pragma unroll
      for (int j = 0; j < w; ++j) {
        const uint32_t give = up ? m[j] : m[j + w], keep = up ? m[j + w] : m[j];
        m[j] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, 2 * w));
      }
    }
    m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    return l & 1 ? m[0] & 0xffff0000u : m[0] << 16;
  }
};
// A group's scale and the factor of its codes (0 where the codes are all 0) from the bits of its
// largest |x|; whether it holds a value that is not finite.
__device__ __forceinline__ bool scale_of_max(uint32_t bits, uint16_t* scale, float* inv) {
  const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(bits), 7.f));
  const float sf = __bfloat162float(s);
  const bool odd = bits >= 0x7f800000u, none = sf < kLeastScale;
  *scale = odd ? 0x7fff : none ? 0 : __bfloat16_as_ushort(s);
  *inv = odd || none ? 0.f : __frcp_rn(sf);
  return odd;
}
// Four codes, one 16-bit unit (of finite x).  |x| inv <= 7 (1 + 2^-8) rounds to 7 at most: no clamp
// is needed.
template <typename R>
__device__ __forceinline__ uint32_t unit_of(const R& x, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(__fadd_rn(__fmul_rn(x[j], inv), kToInt));
  return (b[0] + (b[1] << 4) + (b[2] << 8) + (b[3] << 12)) & 0xffffu;
}
// c of nibble J < 5 of a word: left in its place as the low bits of 2^(23 - 4 J) + c + 8, less that
template <int J> __device__ __forceinline__ float code_of(uint32_t w) {
  static_assert(J < 5, "the nibble lies in a float's 23 bits");
  constexpr float base = float(1 << (23 - 4 * J));
  return __uint_as_float((w & (15u << (4 * J))) | uint32_t(150 - 4 * J) << 23) - (base + 8.f);
}
__device__ __forceinline__ void codes8(uint32_t w, float* x) {
  const uint32_t u = w >> 16;
  x[0] = code_of<0>(w); x[1] = code_of<1>(w); x[2] = code_of<2>(w); x[3] = code_of<3>(w);
  x[4] = code_of<0>(u); x[5] = code_of<1>(u); x[6] = code_of<2>(u); x[7] = code_of<3>(u);
}
// The four values of a 16-bit unit and its bf16 scale, to a row.  (A product of a code and a scale
// is exact in 32 bits, and rounded once to bf16 either way.)
__device__ __forceinline__ void store_values(float* p, uint32_t unit, uint32_t scale) {
  const float s = __uint_as_float(scale << 16);
  *reinterpret_cast<float4*>(p) = make_float4(
      __fmul_rn(code_of<0>(unit), s), __fmul_rn(code_of<1>(unit), s),
      __fmul_rn(code_of<2>(unit), s), __fmul_rn(code_of<3>(unit), s));
}
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t unit, uint32_t scale) {
  const uint32_t y = unit | unit << 12, s2 = scale | scale << 16;  // nibbles 1 and 3 above 0 and 2
  const auto two = [&](uint32_t w) {  // as the low bits of 128 + c + 8, twice
    const uint32_t n = (w & 0x000f000fu) | 0x43004300u, off = 0xc308c308u;
    const __nv_bfloat162 c = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&n),
                                        *reinterpret_cast<const __nv_bfloat162*>(&off));
    const __nv_bfloat162 v = __hmul2_rn(c, *reinterpret_cast<const __nv_bfloat162*>(&s2));
    return *reinterpret_cast<const uint32_t*>(&v);
  };
  *reinterpret_cast<uint2*>(p) = make_uint2(two(y), two(y >> 8));
}

// Quantises eight tokens' K or V rows of one strip: tokens [t0, t0 + n) of the strip are slots
// i0 .. of the call, head h; this warp takes those of half `half`.  Lane (g, l) holds four dims of
// each row (P = 64: K in one half of the warp, V in the other).  The rows' largest values are
// found by exchanges that leave row l with lane l, so that the division and the reciprocal are
// computed once per group.  A whole strip (kWhole: t0 = 0, n = 16) goes to its copy in shared
// memory, and its tokens' V units are written two at a time.
template <typename T, int P, bool kWhole>
__device__ __forceinline__ void write_half(const RowArgs& a, int64_t i0, int h, int t0, int n,
                                           int which, int half, uint8_t* to) {
  constexpr int LPR = P / 4;
  const int lane = threadIdx.x & 31, sub = lane % LPR, g = sub / 8, l = sub % 8;
  const int first = kWhole ? half * 8 : half * 8 - t0;  // run index of the half's token 0
  if (!kWhole && (first + 8 <= 0 || first >= n)) return;
  const auto there = [&](int j) { return kWhole || (first + j >= 0 && first + j < n); };
  const T* base = which == 0 ? static_cast<const T*>(a.k) + i0 * a.k_tok + h * a.k_head
                             : static_cast<const T*>(a.v) + i0 * a.v_tok + h * a.v_head;
  const int64_t step = which == 0 ? a.k_tok : a.v_tok;
  Four<T> x[8];
  const T* p = base + first * step + sub * 4;
#pragma unroll
  for (int j = 0; j < 8; ++j, p += step) {
    if (there(j) && sub * 4 < a.dim) x[j].load(p, a.vec);
    else x[j].zero();
  }
  uint16_t scale;
  float inv;
  const bool odd = scale_of_max(Four<T>::top(x, l), &scale, &inv);
  if (there(l)) *reinterpret_cast<uint16_t*>(to + scale_at<P>(half * 8 + l, which, g)) = scale;
  uint32_t unit[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    unit[j] = unit_of(x[j], __shfl_sync(0xffffffffu, inv, (lane & 24) + j));
  const unsigned odds = __ballot_sync(0xffffffffu, odd) >> (lane & 24);
  if (odds) {  // (a row of such values has codes 0)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (odds >> j & 1) unit[j] = 0x8888u;
  }
  if (kWhole && which == 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint32_t*>(to + v_unit_at<P>(half * 8 + 2 * c, g, l)) =
          unit[2 * c] | unit[2 * c + 1] << 16;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = half * 8 + j;
      if (there(j))
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
// (Eight bf16 rows fit 40 registers a thread, 48 warps an SM, with 40 bytes spilled, and are faster so
// than with 48 or 64; 32-bit rows take 64.)
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
    if (n != kStrip) {
      write_half<T, P, false>(a, i0, h, t0, n, which, half, strip);
      return;
    }
    write_half<T, P, true>(a, i0, h, 0, n, which, half, s_stage);
    __syncthreads();
    for (int o = threadIdx.x * 16; o < SB; o += kThreads * 16)
      *reinterpret_cast<uint4*>(strip + o) = *reinterpret_cast<const uint4*>(s_stage + o);
    __syncthreads();
  });
}

// Means of the pages whose last row is among the slots: one CTA per (`words` x 32 slots, head).
// Its warps find the pages, each for itself, and take them in groups of as many warps as a page has
// strips (the next power of two; all eight where there are more).  A lane holds one word of every
// second row (P = 64: every fourth), dims 32 g + 8 c .. + 7, so that its sums meet one other lane's
// (three others') in the end; the warps' sums are added in order.
constexpr int kMeanWarps = 8, kMeanWords = 4;  // up to 4 words of 32 slots
template <int P>
__global__ void __launch_bounds__(kMeanWarps * 32) page_mean_kernel(RowArgs a, int words,
                                                                    int log_warps) {
  constexpr int G = P / 32, SB = strip_bytes(P);
  constexpr int WORDS = 4 * G;                            // of a row
  constexpr int ROWS = 32 / WORDS, ITER = kStrip / ROWS;  // of a load; loads of a strip
  __shared__ __align__(16) float s_sum[kMeanWarps][P];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % WORDS / G, g = lane % G;
  const int window = div(blockIdx.x, a.by_heads), h = blockIdx.x - window * a.heads;
  int at[kMeanWords];  // the page that a slot completes, or -1; those before it in the window
  int before[kMeanWords], count = 0;
#pragma unroll
  for (int w = 0; w < kMeanWords; ++w) {
    const int64_t i = (int64_t(window) * words + w) * 32 + lane;
    at[w] = w < words && i < a.n ? a.slots[i] : -1;
  }
#pragma unroll
  for (int w = 0; w < kMeanWords; ++w) {
    const int page = at[w] >= 0 ? div(at[w], a.by_bs) : 0;
    const bool last = at[w] >= 0 && page < a.n_pages && at[w] - page * a.bs == a.bs - 1;
    at[w] = last ? page : -1;
    const unsigned done = __ballot_sync(0xffffffffu, last);
    before[w] = last ? count + __popc(done & ((1u << lane) - 1)) : -1;
    count += __popc(done);
  }
  const int warps_a_page = 1 << log_warps, pages_at_once = kMeanWarps >> log_warps;
  const int group = warp >> log_warps, in_group = warp & (warps_a_page - 1);
  for (int p0 = 0; p0 < count; p0 += pages_at_once) {
    int page = -1;
#pragma unroll
    for (int w = 0; w < kMeanWords; ++w) {
      const unsigned it = __ballot_sync(0xffffffffu, before[w] == p0 + group);
      if (it) page = __shfl_sync(0xffffffffu, at[w], __ffs(it) - 1);
    }
    if (page >= 0) {
      const uint8_t* strips = a.pool + (int64_t(page) * a.heads + h) * a.strips * SB;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int s = in_group; s < a.strips; s += warps_a_page) {
        const uint8_t* strip = strips + int64_t(s) * SB;
        uint32_t word[ITER];
        float sc[ITER];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {  // (a strip's rows past the page exist: loaded, not added)
          const int t = i * ROWS + lane / WORDS;
          word[i] = reinterpret_cast<const uint32_t*>(strip)[i * 32 + lane];
          sc[i] = __uint_as_float(
              uint32_t(*reinterpret_cast<const uint16_t*>(strip + scale_at<P>(t, 0, g))) << 16);
        }
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          if (s * kStrip + i * ROWS + lane / WORDS >= a.bs) continue;
          float x[8];
          codes8(word[i], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = fmaf(x[j], sc[i], acc[j]);
        }
      }
#pragma unroll
      for (int o = WORDS; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (lane < WORDS) {
        float4* to = reinterpret_cast<float4*>(&s_sum[warp][32 * g + 8 * c]);
        to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      }
    }
    __syncthreads();
    if (page >= 0) {
      for (int d = in_group * 32 + lane; d < P; d += warps_a_page * 32) {
        float sum = 0.f;
        for (int w = 0; w < warps_a_page; ++w) sum += s_sum[group * warps_a_page + w][d];
        a.rep[(int64_t(page) * a.heads + h) * P + d] = sum / static_cast<float>(a.bs);
      }
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
  const int w = blockIdx.x * kReadWarps + (threadIdx.x >> 5), i = div(w, a.by_chunks);
  const int h0 = (w - i * a.by_chunks.d) * kHeads;
  if (i >= a.n) return;
  const int slot = a.slots[i];
  const int page = slot >= 0 ? div(slot, a.by_bs) : 0, row = slot - page * a.bs, t = row % kStrip;
  const bool in = slot >= 0 && page < a.n_pages;
  if (slot >= 0 && !in && lane == 0 && h0 == 0) report(a.status, RBA_ERR_BOUNDS, kWherePaged, slot);
  if (sub * 4 >= a.dim) return;
  const int64_t head_bytes = int64_t(a.strips) * SB;
  const uint8_t* strip =
      a.pool + (int64_t(in ? page : 0) * a.heads + h0) * head_bytes + (in ? row / kStrip : 0) * SB;
  const int64_t out = (int64_t(i) * a.heads + h0) * a.dim + sub * 4;
  // the lane's unit and scale in a strip: of K and V in turn, or (P = 64) of its half warp's one
  constexpr int kPasses = 2 * LPR / 32;
  const int which0 = P == 128 ? 0 : lane / LPR;
  uint32_t unit[kHeads][kPasses], scale[kHeads][kPasses];
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int which = which0 + pass;
      unit[j][pass] = 0x8888u;
      scale[j][pass] = 0;
      if (in && (j == 0 || h0 + j < a.heads)) {
        const uint8_t* p = strip + j * head_bytes;
        unit[j][pass] = *reinterpret_cast<const uint16_t*>(
            p + (which == 0 ? k_unit_at<P>(t, g, l) : v_unit_at<P>(t, g, l)));
        scale[j][pass] = *reinterpret_cast<const uint16_t*>(p + scale_at<P>(t, which, g));
      }
    }
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass)
      if (j == 0 || h0 + j < a.heads)
        store_values(static_cast<T*>(which0 + pass == 0 ? a.k_out : a.v_out) + out + j * a.dim,
                     unit[j][pass], scale[j][pass]);
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
  // The fewest slots a CTA (up to 16, a whole strip's) with which the grid is at most one wave: its
  // runs go one after another, and rows far apart are a run each.  us, single rows far apart / rows
  // in a row, 8 bf16 heads of 128, with 1, 2, 4, 8, 16 slots a CTA:
  //    297 rows   8.0 / 6.3    9.3 / 5.9   11.8 / 6.1   14.3 / 5.8   20.9 / 6.7
  //   1024       17.6 / 12.4  17.2 / 8.8   18.5 / 7.8   22.5 / 7.5   35.8 / 8.4
  //   8192        112 / 73.9  99.6 / 40.4  95.5 / 24.3  94.8 / 18.2  99.5 / 16.5
  a.window = 1;
  while (a.window < kStrip && int64_t(n) * a.heads > int64_t(num_sms()) * 16 * a.window)
    a.window *= 2;
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

rba_status refuse_append(const rba_paged* s, int32_t n) {
  if (s == nullptr || n < 0) return RBA_ERR_INVALID_ARG;
  if (n == 0) return RBA_OK;
  const RowArgs a = row_args(s, nullptr, n);
  return run_grid(a, a.window) == 0 ? RBA_ERR_UNSUPPORTED : RBA_OK;
}

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
  const rba_status refused = refuse_append(s, n);
  if (refused != RBA_OK) return refused;
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
  // means: 128 slots a CTA, fewer where that would leave SMs without two (8192 tokens of 8 heads:
  // 24.9 us with their read-back, 25.8 with 64 slots; 777 of 32 heads: 20.2 and 18.8)
  int words = kMeanWords, log_warps = 0;  // (log_warps: of a page's warps)
  while (words > 1 && run_grid(a, words * 32) < 2u * num_sms()) words /= 2;
  while (1 << log_warps < kMeanWarps && 1 << log_warps < a.strips) ++log_warps;
#define RBA_APPEND(T_, P_)                                                                      \
  do {                                                                                          \
    RBA_CUDA_TRY(launch_dependent(append_kernel<T_, P_>, grid, run_warps<P_>() * 32, 0, stream, \
                                  a));                                                          \
    RBA_CUDA_TRY(launch_dependent(page_mean_kernel<P_>, run_grid(a, words * 32),                \
                                  kMeanWarps * 32, 0, stream, a, words, log_warps));            \
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
  const int chunks = (a.heads + kHeads - 1) / kHeads;
  const int64_t grid = (int64_t(n) * chunks + kReadWarps - 1) / kReadWarps;
  if (grid * kReadWarps > INT32_MAX) return RBA_ERR_UNSUPPORTED;
  a.by_chunks = fast_div(chunks);
  const auto kernel = s->d.dtype == RBA_BF16
                          ? (s->pitch == 128 ? read_kernel<__nv_bfloat16, 128>
                                             : read_kernel<__nv_bfloat16, 64>)
                          : (s->pitch == 128 ? read_kernel<float, 128> : read_kernel<float, 64>);
  RBA_CUDA_TRY(
      launch_dependent(kernel, static_cast<unsigned>(grid), kReadWarps * 32, 0, stream, a));
  return RBA_OK;
}
