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
// Layout.  One warp takes a pair of strips of 16 tokens at a time.  K codes are the A operand of the first product
// (16 tokens x 16 dims), q its B; V codes, read in token pairs, are the A operand of the second
// (16 dims x 16 tokens), and the weights its B after 8 x 8 transposes in registers.  Up to four
// q heads to a kv head fill the eight columns with their hi and lo halves ("packed": one product
// for both); five to eight take a column each and a second product for the lo halves ("wide":
// the accumulators stay 32 registers); larger groups are cut into chunks of eight.
//
// The running maximum is lazy: weights are taken relative to a reference that moves only when
// a logit passes it by 2^4, so most strips need no cross-lane maximum and no rescale.
//
// Work.  All pairs of strips of all (request, kv head) units form one line, cut evenly over the
// CTAs whatever the requests' lengths; warps take a CTA's pairs in turn, each through its own ring
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
constexpr int kStages = 2;           // pairs of strips in a warp's ring
constexpr int kLeast = kWarps;       // pairs a CTA takes at least (or a whole unit)
constexpr float kToLog2 = 1.4426950408889634f;
constexpr float kToLn = 0.6931471805599453f;
constexpr float kSlack = 4.f;        // a logit may pass the reference by 2^4
constexpr int kScaleTop = 10;        // s 2^e stays below 2^10 when e is set, below 2^11 always
constexpr int kMostE = 100, kLeastE = -118;

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
__device__ __forceinline__ void mma16816_first(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
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

// The G words of a lane at p.
template <int G> __device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (G == 4) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x; w[1] = a.y;
  }
}
__device__ __forceinline__ float bf16_of(const uint32_t* s, int i) {  // i-th of packed bf16 values
  const uint32_t w = s[i >> 1];
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // (a NaN gives way)
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The q operand of a warp: for kWide with a lo part, hi then lo.
template <int P, bool kWide, bool kLo> struct QFrag {
  static constexpr int kParts = kWide && kLo ? 2 : 1;
  static constexpr int kWords = P / 8;  // 32-bit words a lane holds of one part
  uint32_t w[kParts][kWords];
};

// A warp's running state for the unit's heads; lane (t, c) = (lane / 4, lane % 4) holds head c
// (packed) or heads 2 c and 2 c + 1 (wide).  A weight is 2^(y - m), y the logit in log2 units;
// the values' scales are taken times 2^e, which keeps weight x scale within a half's range.
template <int P, bool kWide> struct State {
  static constexpr int HL = kWide ? 2 : 1, G = P / 32;
  float m[HL], l[HL];    // reference; this lane's part of the weights' sum
  float top[HL];         // a logit above it moves the reference
  float most;            // a scale above it moves e
  float acc[2 * G][4];   // dims 32 g + 4 t + {0..3}: packed hi and lo columns, wide two heads
  int e;
};

template <int P, bool kWide, bool kLo>
__device__ __forceinline__ void pair_step(const uint8_t* strips, int valid0, int valid1,
                                          const QFrag<P, kWide, kLo>& q, const float* fac,
                                          State<P, kWide>& st) {
  constexpr int G = P / 32, HL = kWide ? 2 : 1, SB = strip_bytes(P);
  const int lane = threadIdx.x & 31, t = lane >> 2;
  const bool whole = valid0 == kWholeStrip && valid1 == kWholeStrip;
  float y[HL][2][2];        // logits of tokens t and t + 8 of each strip for the lane's heads
  uint32_t sv[2][2][G / 2]; // their V scales, two to a word
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    uint32_t k[2][G], sc[2][G];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      load_words<G>(strips + n * SB + half * 4 * P + lane * (G * 4), k[half]);
      load_words<G>(strips + n * SB + 16 * P + (t + 8 * half) * (G * 4), sc[half]);
#pragma unroll
      for (int i = 0; i < G / 2; ++i) sv[n][half][i] = sc[half][G / 2 + i];
    }
#pragma unroll
    for (int i = 0; i < HL; ++i) y[i][n][0] = y[i][n][1] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t w0 = k[0][g], w1 = k[1][g], u0 = w0 >> 8, u1 = w1 >> 8;
      const uint32_t a0[4] = {codes2<0>(w0), codes2<0>(w1), codes2<1>(w0), codes2<1>(w1)};
      const uint32_t a1[4] = {codes2<0>(u0), codes2<0>(u1), codes2<1>(u0), codes2<1>(u1)};
      float d[4];
#pragma unroll
      for (int p = 0; p < QFrag<P, kWide, kLo>::kParts; ++p) {
        if (p == 0) mma16816_first(d, a0, &q.w[p][4 * g]);
        else mma16816(d, a0, &q.w[p][4 * g]);
        mma16816(d, a1, &q.w[p][4 * g + 2]);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float s = bf16_of(sc[half], g);
        if constexpr (kWide) {
          y[0][n][half] = fmaf(s, d[2 * half], y[0][n][half]);
          y[HL - 1][n][half] = fmaf(s, d[2 * half + 1], y[HL - 1][n][half]);
        } else {
          y[0][n][half] = fmaf(s, d[2 * half] + d[2 * half + 1], y[0][n][half]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < HL; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) y[i][n][half] *= fac[i];
  }
  if (!whole) {  // rows outside the attended set: no weight, and nothing of their scales
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int valid = n == 0 ? valid0 : valid1;
        if (t + 8 * half >= (valid & 31) && t + 8 * half < (valid >> 5)) continue;
#pragma unroll
        for (int i = 0; i < G / 2; ++i) sv[n][half][i] = 0;
#pragma unroll
        for (int i = 0; i < HL; ++i) y[i][n][half] = -INFINITY;
      }
  }
  // the reference moves where a logit or a scale outgrows it
  uint32_t s2 = 0;
#pragma unroll
  for (int i = 0; i < 2 * 2 * (G / 2); ++i)
    s2 = max_bf16x2(s2, sv[i / G][(i / (G / 2)) & 1][i % (G / 2)]);
  float smax = fmaxf(bf16_of(&s2, 0), bf16_of(&s2, 1));
  bool grow = smax > st.most;
  float ymax[HL];
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    ymax[i] = fmaxf(fmaxf(y[i][0][0], y[i][0][1]), fmaxf(y[i][1][0], y[i][1][1]));
    grow |= ymax[i] > st.top[i];
  }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, o));
    const int e = min(st.e, max(kScaleTop - 1 - exponent(smax), kLeastE));
    const float fe = pow2(max(e - st.e, -126));
    st.e = e;
    st.most = pow2(kScaleTop - e);
    float f[HL];
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      float m = ymax[i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = fmaxf(st.m[i], m);
      f[i] = m == st.m[i] ? 1.f : ex2(st.m[i] - m);
      st.m[i] = m;
      st.top[i] = m + kSlack;
      st.l[i] *= f[i];
      f[i] *= fe;
    }
#pragma unroll
    for (int b = 0; b < 2 * G; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.acc[b][j] *= f[kWide ? (j & 1) : 0];
  }
  const float up = pow2(st.e);
#pragma unroll
  for (int i = 0; i < HL; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float p = ex2(y[i][n][half] - st.m[i]);
        // (a row without weight before any row with one: -infinity against -infinity)
        if (!whole) p = y[i][n][half] == -INFINITY ? 0.f : p;
        st.l[i] += p;
        y[i][n][half] = p * up;
      }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    uint32_t v[2][G];
#pragma unroll
    for (int half = 0; half < 2; ++half)
      load_words<G>(strips + n * SB + 8 * P + half * 4 * P + lane * (G * 4), v[half]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // codes of the group's two 16-dim tiles
      const uint32_t w0 = v[0][g], w1 = v[1][g], u0 = w0 >> 8, u1 = w1 >> 8;
      const uint32_t a0[4] = {codes2<0>(w0), codes2<1>(w0), codes2<0>(w1), codes2<1>(w1)};
      const uint32_t a1[4] = {codes2<0>(u0), codes2<1>(u0), codes2<0>(u1), codes2<1>(u1)};
      // weights with the group's scale, hi + lo halves (11 + 11 bits)
      float hi[HL][2], lo[HL][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float s = bf16_of(sv[n][half], g);
#pragma unroll
        for (int i = 0; i < HL; ++i) {
          const float w = y[i][n][half] * s;
          hi[i][half] = __uint_as_float(__float_as_uint(w) & 0xffffe000u);
          lo[i][half] = w - hi[i][half];
        }
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
}

// Shared memory: rings | warp states | q operand | factors | strips' valid rows | barriers |
// strips before each request.
template <int P, bool kWide, bool kLo> struct Smem {
  static constexpr int H = kWide ? 8 : 4;
  static constexpr int kRow = P + 4;            // out, then m and l
  static constexpr int kSlot = H * kRow;
  static constexpr int kRing = kWarps * kStages * 2 * strip_bytes(P);
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
  char* ring = sm + warp * kStages * 2 * SB;
  uint16_t* info = reinterpret_cast<uint16_t*>(sm + S::kInfo) + warp * 64;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBars) + warp * kStages;
  if (lane < kStages) mbar_init(bars + lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (tid == 0) s_long = 0;
  wait_for_stream();

  // pairs of strips before each request (of one unit), and the longest unit
  int64_t run = 0;
  for (int base = 0; base < a.R; base += kThreads) {
    const int r = base + tid;
    int n = 0;
    if (r < a.R) n = (unit_map(a, paged_len(a.lens, r, a.bs, a.max_pages, a.status)).total() + 1) / 2;
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

  // the warp's pairs: begin + warp, + 8, ..
  const int mine = static_cast<int>(end - begin) > warp
                       ? static_cast<int>(end - begin - warp + kWarps - 1) / kWarps : 0;
  const uint8_t* src = a.pool;  // of the lane's strip in the current round of 16 pairs
  int valid = 0;
  unsigned some = 0;            // lanes whose strip has rows to attend to
  int dead_at = -1;             // the pair whose wait ran out: nothing is issued or awaited after
  auto find = [&](int j0) {     // lane i finds strip i % 2 of pair j0 + i / 2
    valid = 0;
    const int j = j0 + lane / 2;
    if (j < mine) {
      const uint32_t at = begin + warp + uint32_t(j) * kWarps;
      const int r = last_at_most(pre, a.R, static_cast<int32_t>(at / units));
      const uint32_t n = pre[r + 1] - pre[r], in = at - uint32_t(pre[r]) * units, u = in / n;
      const int v = 2 * static_cast<int>(in - u * n) + (lane & 1);
      const UnitMap map = unit_map(a, a.lens[r]);
      if (v < map.total())
        src = locate(a, map, r, static_cast<int>(u) / a.chunks, v, SB, &valid);
    }
    some = __ballot_sync(0xffffffffu, valid != 0);
    info[(2 * j0 + lane) & 63] = static_cast<uint16_t>(valid);
    __syncwarp();
  };
  auto issue = [&](int j) {  // pair j into its stage (which is free), by the lanes that found it
    if (j >= mine) return;
    if ((j & 15) == 0) find(j);
    if (lane / 2 == (j & 15)) {
      uint64_t* bar = bars + j % kStages;
      if ((lane & 1) == 0) mbar_arrive_tx(bar, SB * __popc((some >> lane) & 3u));
      if (valid != 0)
        bulk_g2s(ring + ((j % kStages) * 2 + (lane & 1)) * SB, src, SB, bar);
    }
  };
#pragma unroll 1
  for (int j = 0; j < kStages; ++j) issue(j);

  int j = 0;  // the warp's next pair
  for (uint32_t at = begin; at < end;) {
    const int r = last_at_most(pre, a.R, static_cast<int32_t>(at / units));
    const uint32_t n = pre[r + 1] - pre[r], base = uint32_t(pre[r]) * units;
    const uint32_t u = (at - base) / n;
    const int h = static_cast<int>(u) / a.chunks, h0 = (static_cast<int>(u) - h * a.chunks) * H;
    const uint32_t u0 = base + u * n;             // the unit's first pair
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
    st.e = kMostE;
    st.most = pow2(kScaleTop - kMostE);
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      fac[i] = s_fac[HL * (lane & 3) + i];
      st.m[i] = st.top[i] = -INFINITY;
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
      const int v0 = info[(2 * j) & 63], v1 = info[(2 * j + 1) & 63];
      if (v0 | v1)
        pair_step<P, kWide, kLo>(reinterpret_cast<const uint8_t*>(ring + stage * 2 * SB), v0, v1,
                                 qf, fac, st);
      __syncwarp();
      issue(j + kStages);
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
      // the unit's CTAs: i0 holds its first pair, i1 its last
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
        // Warps take rows and shares of the parts, eight parts' loads in flight; the shares meet
        // in shared memory.  (i0's part is its second one unless its range starts the unit.)
        const float* p0 = a.parts + (int64_t(i0) * 2 + (uint64_t(chunk) * i0 >= u0 ? 0 : 1)) * S::kSlot;
        const float* p1 = a.parts + int64_t(i0) * 2 * S::kSlot;
        constexpr int kShares = kWarps / H;
        const int hh = warp % H, share = warp / H, np = i1 - i0 + 1;
        if (hh < nh) {
          float m = -INFINITY, l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int kU = 8;
          for (int c0 = share; c0 < np; c0 += kU * kShares) {
            float pm[kU], pl[kU];
            float4 po[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
              const int c = c0 + i * kShares;
              pm[i] = -INFINITY;
              pl[i] = 0.f;
              po[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (c < np) {
                const float* s = (c == 0 ? p0 : p1 + int64_t(c) * 2 * S::kSlot) + hh * S::kRow;
                pm[i] = __ldcg(s + P);
                pl[i] = __ldcg(s + P + 1);
                if (lane * 4 < P) po[i] = __ldcg(reinterpret_cast<const float4*>(s) + lane);
              }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kU; ++i) top = fmaxf(top, pm[i]);
            const float f0 = m == top ? 1.f : ex2(m - top);
            l *= f0;
            o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
            m = top;
#pragma unroll
            for (int i = 0; i < kU; ++i) {
              const float f = pm[i] == top ? 1.f : ex2(pm[i] - top);
              l += f * pl[i];
              o.x += f * po[i].x; o.y += f * po[i].y; o.z += f * po[i].z; o.w += f * po[i].w;
            }
          }
          float* s = slots + (share * H + hh) * S::kRow;
          if (lane * 4 < P) *reinterpret_cast<float4*>(s + lane * 4) = o;
          if (lane == 0) {
            s[P] = m;
            s[P + 1] = l;
          }
        }
        __syncthreads();
        for (int i = tid; i < nh * P; i += kThreads) {
          const int row = i / P, d = i % P;
          const float* s = slots + row * S::kRow;
          float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
          for (int w = 0; w < kShares; ++w) m = fmaxf(m, s[w * S::kSlot + P]);
#pragma unroll
          for (int w = 0; w < kShares; ++w) {
            const float f = s[w * S::kSlot + P] == m ? 1.f : ex2(s[w * S::kSlot + P] - m);
            l += f * s[w * S::kSlot + P + 1];
            o += f * s[w * S::kSlot + d];
          }
          finish(a, row0 + row, d, m, l, o);
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
  void (*const kernel)(PagedAttendArgs) = paged_attend_kernel<P, kWide, T>;
  RBA_CUDA_TRY(ensure_smem(reinterpret_cast<const void*>(kernel), smem));
  RBA_CUDA_TRY(launch_dependent(kernel, static_cast<unsigned>(num_sms() * kCtasPerSm), kThreads,
                                smem, stream, a));
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
