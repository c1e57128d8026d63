// Paged 4-bit memory: decode attention over requests of different lengths.
//
// out = sum_t softmax_t(scale q . k_t) v_t over each request's sink tokens, selected pages and
// window, K and V held as codes c (a nibble, c + 8) and bf16 scales s per 32 dims.
//
// Mathematics.  q . k_t = sum_g s_tg sum_{d in g} q_d c_td, so the inner sums run on the codes
// and a scale enters once per group.  A nibble masked out of a word of two half-precision numbers
// is the number (c + 8) 2^-24 there (a subnormal half; 2^-20 for the nibble above it), and one
// fused multiply-add of halves turns it into c 2^-9, exactly: an AND and an HFMA2 for two codes,
// no conversion.  (Fed to the matrix unit as they are, subnormal operands cost it precision: it
// aligns products by their nominal exponents, and the outputs were off by 2^-17.)  q is scaled by
// a power of two per head and split into two halves (hi + lo, 22 bits); for the values the weight
// takes the scale, w = p s_tg 2^e, split the same way.  Softmax statistics, both products'
// accumulators and the merges are 32-bit.
//
// Layout.  One warp takes a strip of 16 tokens: K codes are the A operand of the first product
// (16 tokens x 16 dims), q its B; V codes, read in token pairs, are the A operand of the second
// (16 dims x 16 tokens), and the weights its B after 8 x 8 transposes in registers.  Up to four
// q heads to a kv head fill the eight columns with their hi and lo halves ("packed": one product
// for both); five to eight take a column each and a second product for the lo halves ("wide":
// the accumulators stay 32 registers); larger groups are cut into chunks of eight.
//
// The running maximum is lazy: weights are taken relative to a reference that moves only when
// a logit passes it by 2^4, so most strips need no cross-lane maximum and no rescale.
//
// Work.  All strips of all (request, kv head) units form one line, cut evenly over the CTAs
// whatever the requests' lengths; warps take a CTA's strips in turn, each through its own ring
// of bulk copies, which runs on across units.  A CTA's part of a unit that it does not hold
// whole goes to the workspace, and the last of the unit's CTAs to arrive merges the parts in
// order.
#include <cuda_fp16.h>

#include "decode_persist.cuh"
#include "paged.cuh"

namespace rba {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 2;
constexpr int kStages = 4;           // strips in flight per warp
constexpr int kLeast = 2 * kWarps;   // strips a CTA takes at least (or a whole unit)
constexpr float kToLog2 = 1.4426950408889634f;
constexpr float kToLn = 0.6931471805599453f;
constexpr float kSlack = 4.f;        // a logit may pass the reference by 2^4
constexpr int kScaleTop = 10;        // s 2^e stays below 2^10 when e is set, below 2^11 always

struct PagedAttendArgs {
  const void* q;
  int64_t q_req, q_head;
  const int32_t* idx;
  const uint8_t* pool;
  const int32_t* table;
  const int32_t* lens;
  int32_t* status;
  float* out;
  float* lse;
  uint32_t* tickets;  // one per unit, zero between calls
  float* parts;       // [CTA][2][heads of a unit][P + 4]
  float scale;
  int R, heads, group, dim, bs, strips, max_pages, n_pages, k, sink, window;
  int chunks;         // head chunks of a kv head
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^n for n in [-126, 127]
__device__ __forceinline__ float pow2(int n) { return __int_as_float((n + 127) << 23); }
// exponent of |x| (x finite, not subnormal; 0 and subnormals give -127)
__device__ __forceinline__ int exponent(float x) {
  return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127;
}
// Two codes, 2^-9 each, from the nibbles that the mask leaves: nibble 0 (or 1) of each half word.
template <int kNibble>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  const uint32_t x = w & (kNibble ? 0x00f000f0u : 0x000f000fu);
  const uint32_t up = kNibble ? 0x68006800u : 0x78007800u;  // 2^11 or 2^15, twice
  const uint32_t off = 0xa400a400u;                         // -8 2^-9, twice
  const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&x),
                            *reinterpret_cast<const __half2*>(&up),
                            *reinterpret_cast<const __half2*>(&off));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// A unit's strips as one line: sink, selected pages, window.
struct UnitMap {
  PagedGeo g;
  int ns, nk, nw, w_lin;  // strips of sink, of the selected pages, of the window; its first
  __device__ __forceinline__ int total() const { return ns + nk + nw; }
};
__device__ __forceinline__ int lin_strip(int pos, int bs, int strips) {
  const int j = pos / bs;
  return j * strips + (pos - j * bs) / kStrip;
}
__device__ __forceinline__ UnitMap unit_map(const PagedAttendArgs& a, int T) {
  UnitMap m;
  m.g = paged_geo(T, a.bs, a.sink, a.window);
  m.ns = m.g.sink_end > 0 ? lin_strip(m.g.sink_end - 1, a.bs, a.strips) + 1 : 0;
  m.nk = (a.k < m.g.nc ? a.k : m.g.nc) * a.strips;
  m.w_lin = lin_strip(m.g.w0, a.bs, a.strips);
  m.nw = T > m.g.w0 ? lin_strip(T - 1, a.bs, a.strips) - m.w_lin + 1 : 0;
  return m;
}

// Strip v of a unit: its address, and its valid rows [ra, rb) as ra + 32 rb (0 where nothing is
// attended).
__device__ __forceinline__ const uint8_t* locate(const PagedAttendArgs& a, const UnitMap& m, int r,
                                                 int h, int v, int sbytes, int* valid) {
  *valid = 0;
  int lin, lo, hi;
  if (v < m.ns) {
    lin = v;
    lo = 0;
    hi = m.g.sink_end;
  } else if (v < m.ns + m.nk) {
    const int i = (v - m.ns) / a.strips;
    const int j = a.idx[(int64_t(r) * a.heads + h) * a.k + i];
    if (j < m.g.first || j >= m.g.first + m.g.nc) {
      report(a.status, RBA_ERR_BOUNDS, kWherePaged, j);
      return a.pool;
    }
    lin = j * a.strips + (v - m.ns) - i * a.strips;
    lo = m.g.sink_end;
    hi = m.g.w0;
  } else {
    lin = m.w_lin + v - m.ns - m.nk;
    lo = m.g.w0;
    hi = m.g.T;
  }
  const int j = lin / a.strips, sp = lin - j * a.strips;
  const int page = a.table[int64_t(r) * a.max_pages + j];
  if (page < 0 || page >= a.n_pages) {
    report(a.status, RBA_ERR_BOUNDS, kWherePaged, page);
    return a.pool;
  }
  const int pos0 = j * a.bs + sp * kStrip;
  const int ra = max(lo - pos0, 0);
  const int rb = min(min(kStrip, hi - pos0), a.bs - sp * kStrip);
  if (rb > ra) *valid = ra + 32 * rb;
  return a.pool + ((int64_t(page) * a.heads + h) * a.strips + sp) * sbytes;
}
constexpr int kWholeStrip = 32 * kStrip;

// A lane's share of a strip.
template <int P> struct Frag {
  static constexpr int G = P / 32;
  uint32_t k[2][G];      // tokens lane / 4 and + 8: the words (lane % 4, g)
  uint32_t v[2][G];      // halves 0 and 1: unit pairs (lane / 4, lane % 4, g)
  uint32_t s[2][G];      // tokens lane / 4 and + 8: K scales, then V scales, two to a word
};

template <int P>
__device__ __forceinline__ void load_frag(const uint8_t* strip, int lane, Frag<P>& f) {
  constexpr int G = P / 32;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint8_t* kp = strip + half * 4 * P + lane * (G * 4);
    const uint8_t* vp = strip + 8 * P + half * 4 * P + lane * (G * 4);
    const uint8_t* sp = strip + 16 * P + (lane / 4 + 8 * half) * (G * 4);
    if constexpr (G == 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(kp);
      const uint4 b = *reinterpret_cast<const uint4*>(vp);
      const uint4 c = *reinterpret_cast<const uint4*>(sp);
      f.k[half][0] = a.x; f.k[half][1] = a.y; f.k[half][2] = a.z; f.k[half][3] = a.w;
      f.v[half][0] = b.x; f.v[half][1] = b.y; f.v[half][2] = b.z; f.v[half][3] = b.w;
      f.s[half][0] = c.x; f.s[half][1] = c.y; f.s[half][2] = c.z; f.s[half][3] = c.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(kp);
      const uint2 b = *reinterpret_cast<const uint2*>(vp);
      const uint2 c = *reinterpret_cast<const uint2*>(sp);
      f.k[half][0] = a.x; f.k[half][1] = a.y;
      f.v[half][0] = b.x; f.v[half][1] = b.y;
      f.s[half][0] = c.x; f.s[half][1] = c.y;
    }
  }
}
template <int G>
__device__ __forceinline__ float scale_of(const uint32_t* s, int i) {  // i-th of 2 G bf16 values
  const uint32_t w = s[i >> 1];
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}

// The q operand of a warp: for kWide with a lo part, hi then lo.
template <int P, bool kWide, bool kLo> struct QFrag {
  static constexpr int kParts = kWide && kLo ? 2 : 1;
  static constexpr int kWords = P / 8;  // 32-bit words a lane holds of one part
  uint32_t w[kParts][kWords];
};

// A warp's running state for the unit's heads; lane (t, c) = (lane / 4, lane % 4) holds head c
// (packed) or heads 2 c and 2 c + 1 (wide).
template <int P, bool kWide> struct State {
  static constexpr int HL = kWide ? 2 : 1, G = P / 32;
  float m[HL], l[HL];   // reference (log2 units); this lane's part of the sum
  float acc[2 * G][4];  // dims 32 g + 4 t + {0..3}: packed hi and lo columns, wide two heads
  int e;                // V scales are multiplied by 2^e
};

template <int P, bool kWide, bool kLo>
__device__ __forceinline__ void strip_step(const Frag<P>& f, int valid,
                                           const QFrag<P, kWide, kLo>& q, const float* fac,
                                           State<P, kWide>& st) {
  constexpr int G = P / 32, HL = kWide ? 2 : 1;
  const int t = (threadIdx.x & 31) >> 2;
  const bool whole = valid == kWholeStrip;
  // logits of tokens t and t + 8 for the lane's heads
  float x[HL][2];
#pragma unroll
  for (int i = 0; i < HL; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t w0 = f.k[0][g], w1 = f.k[1][g], u0 = w0 >> 8, u1 = w1 >> 8;
    const uint32_t a0[4] = {codes2<0>(w0), codes2<0>(w1), codes2<1>(w0), codes2<1>(w1)};
    const uint32_t a1[4] = {codes2<0>(u0), codes2<0>(u1), codes2<1>(u0), codes2<1>(u1)};
    const float s0 = scale_of<G>(f.s[0], g), s1 = scale_of<G>(f.s[1], g);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < QFrag<P, kWide, kLo>::kParts; ++p) {
      mma16816(d, a0, &q.w[p][4 * g]);
      mma16816(d, a1, &q.w[p][4 * g + 2]);
    }
    if constexpr (kWide) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i][0] = fmaf(s0, d[i], x[i][0]);
        x[i][1] = fmaf(s1, d[2 + i], x[i][1]);
      }
    } else {
      x[0][0] = fmaf(s0, d[0] + d[1], x[0][0]);
      x[0][1] = fmaf(s1, d[2] + d[3], x[0][1]);
    }
  }
  float sv[2][G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    sv[0][g] = scale_of<G>(f.s[0], G + g);
    sv[1][g] = scale_of<G>(f.s[1], G + g);
  }
  bool live0 = true, live1 = true;
  if (!whole) {
    const int ra = valid & 31, rb = valid >> 5;
    live0 = t >= ra && t < rb;
    live1 = t + 8 >= ra && t + 8 < rb;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      sv[0][g] = live0 ? sv[0][g] : 0.f;
      sv[1][g] = live1 ? sv[1][g] : 0.f;
    }
  }
  float smax = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) smax = fmaxf(smax, fmaxf(sv[0][g], sv[1][g]));
  // the reference moves where a logit or a scale outgrows it
  bool grow = smax * pow2(st.e) >= static_cast<float>(2 << kScaleTop);
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    x[i][0] = live0 ? x[i][0] * fac[i] : -INFINITY;
    x[i][1] = live1 ? x[i][1] * fac[i] : -INFINITY;
    grow |= fmaxf(x[i][0], x[i][1]) > st.m[i] + kSlack;
  }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, o));
    const int e = min(st.e, max(kScaleTop - 1 - exponent(smax), -120));
    const float fe = e == st.e ? 1.f : pow2(max(e - st.e, -126));
    st.e = e;
    float fm[HL];
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      float top = fmaxf(x[i][0], x[i][1]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m = fmaxf(st.m[i], top);
      fm[i] = m == st.m[i] ? 1.f : ex2(st.m[i] - m);
      st.m[i] = m;
      st.l[i] *= fm[i];
      fm[i] *= fe;
    }
#pragma unroll
    for (int b = 0; b < 2 * G; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.acc[b][j] *= fm[kWide ? (j & 1) : 0];
  }
  const float up = pow2(st.e);
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    float p0 = ex2(x[i][0] - st.m[i]), p1 = ex2(x[i][1] - st.m[i]);
    if (!whole) {
      p0 = live0 ? p0 : 0.f;
      p1 = live1 ? p1 : 0.f;
    }
    st.l[i] += p0 + p1;
    x[i][0] = p0 * up;
    x[i][1] = p1 * up;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    // codes of the group's two 16-dim tiles
    uint32_t a0[4], a1[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w = f.v[half][g], u = w >> 8;
      a0[2 * half] = codes2<0>(w);
      a0[2 * half + 1] = codes2<1>(w);
      a1[2 * half] = codes2<0>(u);
      a1[2 * half + 1] = codes2<1>(u);
    }
    // weights with the group's scale, hi + lo halves (11 + 11 bits)
    float hi[HL][2], lo[HL][2];
#pragma unroll
    for (int i = 0; i < HL; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float w = x[i][j] * sv[j][g];
        hi[i][j] = __uint_as_float(__float_as_uint(w) & 0xffffe000u);
        lo[i][j] = w - hi[i][j];
      }
    uint32_t b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      b[j] = transpose8x8(kWide ? pack_half2(hi[0][j], hi[HL - 1][j])
                                : pack_half2(hi[0][j], lo[0][j]));
    mma16816(st.acc[2 * g], a0, b);
    mma16816(st.acc[2 * g + 1], a1, b);
    if constexpr (kWide) {
#pragma unroll
      for (int j = 0; j < 2; ++j) b[j] = transpose8x8(pack_half2(lo[0][j], lo[HL - 1][j]));
      mma16816(st.acc[2 * g], a0, b);
      mma16816(st.acc[2 * g + 1], a1, b);
    }
  }
}

// Shared memory: rings | warp states | q operand | factors | strips' valid rows | barriers |
// strips before each request.
template <int P, bool kWide, bool kLo> struct Smem {
  static constexpr int H = kWide ? 8 : 4;
  static constexpr int kRow = P + 4;            // out, then m and l
  static constexpr int kSlot = H * kRow;
  static constexpr int kRing = kWarps * kStages * strip_bytes(P);
  static constexpr int kSlots = kRing;
  static constexpr int kQ = kSlots + kWarps * kSlot * 4;
  static constexpr int kFac = kQ + QFrag<P, kWide, kLo>::kParts * (P / 8) * 32 * 4;
  static constexpr int kInfo = kFac + 32;
  static constexpr int kBars = kInfo + kWarps * 64 * 2;
  static constexpr int kPre = kBars + kWarps * kStages * 8;
  static size_t bytes(int R) { return kPre + size_t(R + 1) * 4; }
};

// q of the unit's heads into the products' B operand: warp `hh` takes head hh, scaled by a power
// of two to a largest value in [2^14, 2^15), split hi + lo.  Word (part, 4 g + 2 ks + b) of lane
// (t, c) holds dims 32 g + 8 c + 2 ks + b and that + 4 of column t.
template <int P, bool kWide, bool kLo, typename T>
__device__ __forceinline__ void stage_q(const PagedAttendArgs& a, const T* q, bool live,
                                        uint32_t* qw, float* fac) {
  using S = Smem<P, kWide, kLo>;
  constexpr int WORDS = P / 8;
  const int hh = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (hh >= S::H) return;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (live && lane * 4 < a.dim) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = Elem<T>::to_f32(q[lane * 4 + e]);
  }
  float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int ex = top > 0.f ? 14 - exponent(top) : 0;
  // (two factors: 2^ex alone can leave the range of a float)
  const float up0 = pow2(ex / 2), up1 = pow2(ex - ex / 2);
  const int g = lane >> 3, c = (lane & 7) >> 1, odd = lane & 1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = x[e] * up0 * up1, hi = __half2float(__float2half_rn(v)), lo = v - hi;
    const float hi_n = __shfl_xor_sync(0xffffffffu, hi, 1), lo_n = __shfl_xor_sync(0xffffffffu, lo, 1);
    if (lane * 4 >= P) continue;
    // even lanes hold the first dim of a pair and write its hi part, odd lanes the lo part
    const uint32_t word = odd ? pack_half2(lo_n, lo) : pack_half2(hi, hi_n);
    const int w = 4 * g + e;  // e = 2 ks + b
    int part = 0, t;
    if (kWide) {
      if (odd && !kLo) continue;  // a bf16 q has no lo part
      part = odd;
      t = hh;
    } else {
      t = 2 * hh + odd;
    }
    qw[((part * (WORDS / 4) + w / 4) * 32 + t * 4 + c) * 4 + w % 4] = word;
  }
  if (lane == 0)
    fac[hh] = a.scale * kToLog2 * pow2((9 - ex) / 2) * pow2((9 - ex) - (9 - ex) / 2);
}

__device__ __forceinline__ void finish(const PagedAttendArgs& a, int64_t row, int d, float m,
                                       float l, float o) {
  if (d < a.dim) a.out[row * a.dim + d] = l == 0.f ? 0.f : o / l;
  if (d == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : kToLn * (m + log2f(l));
}

template <int P, bool kWide, typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_attend_kernel(PagedAttendArgs a) {
  constexpr bool kLo = sizeof(T) == 4;
  using S = Smem<P, kWide, kLo>;
  constexpr int G = P / 32, H = S::H, SB = strip_bytes(P), HL = kWide ? 2 : 1;
  extern __shared__ __align__(128) char sm[];
  float* slots = reinterpret_cast<float*>(sm + S::kSlots);
  uint32_t* qw = reinterpret_cast<uint32_t*>(sm + S::kQ);
  float* s_fac = reinterpret_cast<float*>(sm + S::kFac);
  int32_t* pre = reinterpret_cast<int32_t*>(sm + S::kPre);
  __shared__ int64_t s_w[kWarps];
  __shared__ int s_long;
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.heads * a.chunks;  // per request
  char* ring = sm + warp * kStages * SB;
  uint16_t* info = reinterpret_cast<uint16_t*>(sm + S::kInfo) + warp * 64;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBars) + warp * kStages;
  if (lane < kStages) mbar_init(bars + lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (tid == 0) s_long = 0;

  // strips before each request (of one unit), and the longest unit
  int64_t run = 0;
  for (int base = 0; base < a.R; base += kThreads) {
    const int r = base + tid;
    int n = 0;
    if (r < a.R) n = unit_map(a, paged_len(a.lens, r, a.bs, a.max_pages, a.status)).total();
    int64_t tot;
    const int64_t ex = block_scan64(n, s_w, &tot);  // (two barriers: s_long is set by now)
    if (r < a.R) pre[r] = static_cast<int32_t>(run + ex);
    if (n > 0) atomicMax(&s_long, n);
    run += tot;
  }
  if (tid == 0) pre[a.R] = static_cast<int32_t>(run);
  __syncthreads();
  // requests that attend to nothing
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    if (pre[r + 1] != pre[r]) continue;
    const int hq = a.heads * a.group;
    for (int i = tid; i < hq * a.dim; i += kThreads) a.out[int64_t(r) * hq * a.dim + i] = 0.f;
    if (a.lse != nullptr)
      for (int i = tid; i < hq; i += kThreads) a.lse[int64_t(r) * hq + i] = -INFINITY;
  }
  const uint32_t all = static_cast<uint32_t>(run) * units;
  const uint32_t chunk = max((all + gridDim.x - 1) / gridDim.x,
                             static_cast<uint32_t>(min(s_long, kLeast)));
  const uint64_t first = uint64_t(chunk) * blockIdx.x;
  if (first >= all) return;
  const uint32_t begin = static_cast<uint32_t>(first), end = min(all, begin + chunk);

  // the warp's strips: begin + warp, + 8, ..
  const int mine = static_cast<int>(end - begin) > warp
                       ? static_cast<int>(end - begin - warp + kWarps - 1) / kWarps : 0;
  const uint8_t* src = a.pool;  // of the lane's strip in the current round of 32
  int valid = 0;
  int dead_at = -1;             // the strip whose wait ran out: nothing is issued or awaited after
  auto find = [&](int j0) {     // lane i finds strip j0 + i
    valid = 0;
    const int j = j0 + lane;
    if (j < mine) {
      const uint32_t at = begin + warp + uint32_t(j) * kWarps;
      const int r = last_at_most(pre, a.R, static_cast<int32_t>(at / units));
      const uint32_t n = pre[r + 1] - pre[r], in = at - uint32_t(pre[r]) * units, u = in / n;
      src = locate(a, unit_map(a, a.lens[r]), r, static_cast<int>(u) / a.chunks,
                   static_cast<int>(in - u * n), SB, &valid);
    }
    info[(j0 + lane) & 63] = static_cast<uint16_t>(valid);
    __syncwarp();
  };
  auto issue = [&](int j) {  // strip j into its stage (which is free), by the lane that found it
    if (j >= mine) return;
    if ((j & 31) == 0) find(j);
    if (lane == (j & 31)) {
      uint64_t* bar = bars + j % kStages;
      if (valid != 0) {
        mbar_arrive_tx(bar, SB);
        bulk_g2s(ring + (j % kStages) * SB, src, SB, bar);
      } else {
        mbar_arrive(bar);
      }
    }
  };
#pragma unroll 1
  for (int j = 0; j < kStages; ++j) issue(j);

  int j = 0;  // the warp's next strip
  for (uint32_t at = begin; at < end;) {
    const int r = last_at_most(pre, a.R, static_cast<int32_t>(at / units));
    const uint32_t n = pre[r + 1] - pre[r], base = uint32_t(pre[r]) * units;
    const uint32_t u = (at - base) / n;
    const int h = static_cast<int>(u) / a.chunks, h0 = (static_cast<int>(u) - h * a.chunks) * H;
    const uint32_t u0 = base + u * n;             // the unit's first strip
    const uint32_t stop = min(end, u0 + n);
    const int nh = min(H, a.group - h0);
    {
      const int hh = warp;
      stage_q<P, kWide, kLo>(a,
                             static_cast<const T*>(a.q) + r * a.q_req +
                                 (int64_t(h) * a.group + h0 + hh) * a.q_head,
                             hh < nh, qw, s_fac);
    }
    __syncthreads();
    QFrag<P, kWide, kLo> qf;
#pragma unroll
    for (int p = 0; p < QFrag<P, kWide, kLo>::kParts; ++p)
#pragma unroll
      for (int w = 0; w < P / 32; ++w) {
        const uint4 x = *reinterpret_cast<const uint4*>(qw + ((p * (P / 32) + w) * 32 + lane) * 4);
        qf.w[p][4 * w] = x.x; qf.w[p][4 * w + 1] = x.y;
        qf.w[p][4 * w + 2] = x.z; qf.w[p][4 * w + 3] = x.w;
      }
    float fac[HL];
    State<P, kWide> st;
    st.e = 120;
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      fac[i] = s_fac[HL * (lane & 3) + i];
      st.m[i] = -INFINITY;
      st.l[i] = 0.f;
    }
#pragma unroll
    for (int b = 0; b < 2 * G; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.acc[b][i] = 0.f;

#pragma unroll 1
    for (; j < mine && begin + warp + uint32_t(j) * kWarps < stop; ++j) {
      const int stage = j % kStages;
      if (dead_at >= 0) continue;
      const uint32_t parity = (j / kStages) & 1;
      bool ok = mbar_try(bars + stage, parity);
      if (!__all_sync(0xffffffffu, ok)) {
        const unsigned long long t0 = now_ns();
        do {
          if (!ok) ok = mbar_try(bars + stage, parity);
        } while (!__all_sync(0xffffffffu, ok) &&
                 !__shfl_sync(0xffffffffu, now_ns() - t0 > kTimeoutNs, 0));
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) report(a.status, RBA_ERR_TIMEOUT, kWherePaged, j);
          dead_at = j;
          continue;
        }
      }
      const int v = info[j & 63];
      Frag<P> f;
      if (v != 0) load_frag<P>(reinterpret_cast<const uint8_t*>(ring + stage * SB), lane, f);
      __syncwarp();
      issue(j + kStages);
      if (v != 0) strip_step<P, kWide, kLo>(f, v, qf, fac, st);
    }

    // warp states to shared memory
    {
      const int t = lane >> 2, c = lane & 3;
      const float down = pow2(-st.e);
#pragma unroll
      for (int i = 0; i < HL; ++i) {
        float l = st.l[i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float* s = slots + warp * S::kSlot + (HL * c + i) * S::kRow;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float* d0 = st.acc[2 * g];
          const float* d1 = st.acc[2 * g + 1];
          float4 o;
          if constexpr (kWide) {
            o = make_float4(d0[i], d0[2 + i], d1[i], d1[2 + i]);
          } else {
            o = make_float4(d0[0] + d0[1], d0[2] + d0[3], d1[0] + d1[1], d1[2] + d1[3]);
          }
          *reinterpret_cast<float4*>(s + 32 * g + 4 * t) =
              make_float4(o.x * 0x1p9f * down, o.y * 0x1p9f * down, o.z * 0x1p9f * down,
                          o.w * 0x1p9f * down);
        }
        if (t == 0) {
          s[P] = st.m[i];
          s[P + 1] = l;
        }
      }
    }
    __syncthreads();

    const bool whole = at == u0 && stop == u0 + n;
    const int64_t row0 = (int64_t(r) * a.heads + h) * a.group + h0;
    float* part = a.parts + (int64_t(blockIdx.x) * 2 + (at == begin ? 0 : 1)) * S::kSlot;
    for (int i = tid; i < nh * P; i += kThreads) {
      const int hh = i / P, d = i % P;
      const float* s = slots + hh * S::kRow;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s[w * S::kSlot + P]);
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float pm = s[w * S::kSlot + P];
        const float f = pm == m ? 1.f : ex2(pm - m);
        l += f * s[w * S::kSlot + P + 1];
        o += f * s[w * S::kSlot + d];
      }
      if (whole) {
        finish(a, row0 + hh, d, m, l, o);
      } else {
        float* to = part + hh * S::kRow;
        to[d] = o;
        if (d == 0) {
          to[P] = m;
          to[P + 1] = l;
        }
      }
    }
    if (!whole) {
      // the unit's CTAs: i0 holds its first strip, i1 its last
      const int i0 = u0 / chunk, i1 = (u0 + n - 1) / chunk;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        uint32_t* ticket = a.tickets + int64_t(r) * units + u;
        s_last = atom_add_acq_rel(ticket, 1) == static_cast<uint32_t>(i1 - i0);
        if (s_last) *ticket = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        // i0's part is its second one unless its range starts with the unit
        const float* p0 = a.parts + (int64_t(i0) * 2 + (uint64_t(chunk) * i0 >= u0 ? 0 : 1)) * S::kSlot;
        const float* p1 = a.parts + int64_t(i0) * 2 * S::kSlot;
        for (int i = tid; i < nh * P; i += kThreads) {
          const int hh = i / P, d = i % P;
          const int off = hh * S::kRow;
          float m = __ldcg(p0 + off + P);
#pragma unroll 8
          for (int c = 1; c <= i1 - i0; ++c)
            m = fmaxf(m, __ldcg(p1 + int64_t(c) * 2 * S::kSlot + off + P));
          float l = 0.f, o = 0.f;
#pragma unroll 8
          for (int c = 0; c <= i1 - i0; ++c) {
            const float* s = (c == 0 ? p0 : p1 + int64_t(c) * 2 * S::kSlot) + off;
            const float pm = __ldcg(s + P), pl = __ldcg(s + P + 1), po = __ldcg(s + d);
            const float f = pm == m ? 1.f : ex2(pm - m);
            l += f * pl;
            o += f * po;
          }
          finish(a, row0 + hh, d, m, l, o);
        }
      }
    }
    at = stop;
  }
  if (dead_at >= 0) {  // copies in flight land before the CTA leaves
    const int last = min(mine, dead_at + kStages) - 1;
    for (int s = 0; s < kStages && s <= last; ++s)
      mbar_drain(bars + s, ((last - (last - s) % kStages) / kStages) & 1);
  }
}

// Groups of up to four q heads to a kv head take the packed form, larger ones the wide one.
bool wide_of(const rba_paged* s) { return s->d.n_q_heads / s->d.n_kv_heads > 4; }
int chunks_of(const rba_paged* s) {
  const int group = s->d.n_q_heads / s->d.n_kv_heads;
  return group <= 4 ? 1 : (group + 7) / 8;
}
size_t ticket_bytes(const rba_paged* s) {
  return align_up(size_t(s->d.max_requests) * s->d.n_kv_heads * chunks_of(s) * 4, 256);
}

template <int P, bool kWide, typename T>
rba_status launch(const PagedAttendArgs& a, cudaStream_t stream) {
  const size_t smem = Smem<P, kWide, sizeof(T) == 4>::bytes(a.R);
  const auto kernel = paged_attend_kernel<P, kWide, T>;
  RBA_CUDA_TRY(ensure_smem(reinterpret_cast<const void*>(kernel), smem));
  kernel<<<num_sms() * kCtasPerSm, kThreads, smem, stream>>>(a);
  RBA_LAUNCH_CHECK();
  return RBA_OK;
}

}  // namespace
}  // namespace rba

extern "C" size_t rba_paged_attend_workspace_size(const rba_paged* s) {
  using namespace rba;
  if (s == nullptr) return 0;
  return ticket_bytes(s) + size_t(num_sms()) * kCtasPerSm * 2 * (wide_of(s) ? 8 : 4) *
                               (s->pitch + 4) * sizeof(float);
}

extern "C" rba_status rba_paged_attend(const rba_paged* s, const void* q,
                                       int64_t q_request_stride, int64_t q_head_stride,
                                       int32_t n_requests, const int32_t* idx, int32_t k,
                                       int32_t sink, int32_t window, float scale, float* out,
                                       float* lse, void* workspace, size_t ws_bytes,
                                       cudaStream_t stream) {
  using namespace rba;
  if (s == nullptr || q == nullptr || out == nullptr || workspace == nullptr || n_requests <= 0 ||
      n_requests > s->d.max_requests || k < 0 || (k > 0 && idx == nullptr) || sink < 0 ||
      window < 0)
    return RBA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return RBA_ERR_INVALID_ARG;
  if (ws_bytes < rba_paged_attend_workspace_size(s)) return RBA_ERR_WORKSPACE;
  // the line of strips is counted in 32 bits (sink, selection and window can share two pages)
  const int64_t line = int64_t(n_requests) * (int64_t(s->d.max_pages) + 2) * s->strips;
  if (line > INT32_MAX || line * s->d.n_kv_heads * chunks_of(s) > INT32_MAX)
    return RBA_ERR_UNSUPPORTED;
  PagedAttendArgs a = {};
  a.q = q;
  a.q_req = q_request_stride;
  a.q_head = q_head_stride;
  a.idx = idx;
  a.pool = static_cast<const uint8_t*>(s->b.pool);
  a.table = s->b.table;
  a.lens = s->b.lens;
  a.status = s->b.status;
  a.out = out;
  a.lse = lse;
  a.tickets = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + ticket_bytes(s));
  a.scale = scale;
  a.R = n_requests;
  a.heads = s->d.n_kv_heads;
  a.group = s->d.n_q_heads / s->d.n_kv_heads;
  a.dim = s->d.head_dim;
  a.bs = s->d.page_size;
  a.strips = s->strips;
  a.max_pages = s->d.max_pages;
  a.n_pages = s->d.n_pages;
  a.k = k;
  a.sink = sink;
  a.window = window;
  a.chunks = chunks_of(s);
  const bool bf = s->d.dtype == RBA_BF16;
  if (s->pitch == 128) {
    if (wide_of(s))
      return bf ? launch<128, true, __nv_bfloat16>(a, stream) : launch<128, true, float>(a, stream);
    return bf ? launch<128, false, __nv_bfloat16>(a, stream) : launch<128, false, float>(a, stream);
  }
  if (wide_of(s))
    return bf ? launch<64, true, __nv_bfloat16>(a, stream) : launch<64, true, float>(a, stream);
  return bf ? launch<64, false, __nv_bfloat16>(a, stream) : launch<64, false, float>(a, stream);
}
