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
// takes the scale, w = p s_tg 2^e, split the same way, with an e for each head and group that keeps
// the largest w in [2^7, 2^15): what a half cannot hold, 2^-25, is then at most 2^-32 of the group's
// largest term, whatever other groups and rows without weight hold.  Softmax statistics, both
// products' accumulators and the merges are 32-bit.
//
// Layout.  One warp takes a pair of strips of 16 tokens at a time.  K codes are the A operand of
// the first product (16 tokens x 16 dims), q its B; V codes, read in token pairs, are the A operand
// of the second (16 dims x 16 tokens), and the weights its B after 8 x 8 transposes in registers.
// Up to four q heads to a kv head fill the eight columns with their hi and lo halves ("packed": one
// product for both); five to eight take a column each and a second product for the lo halves
// ("wide": the accumulators stay 32 registers); larger groups are cut into chunks of eight.
//
// The running maximum is lazy: weights are taken relative to a reference, a whole number, that moves
// only when a weight passes 2^4 or a w 2^15, so most strips need no cross-lane maximum and no
// rescale.  Factors of a move are powers of two, and an e rises by what the reference rises.
//
// Work.  All pairs of strips of all (request, kv head) units form one line, cut evenly over
// workers whatever the requests' lengths, each unit counted with a few pairs more for what its
// start and end cost.  A worker is a CTA, whose warps take its pairs in turn, or, where units are
// short (a batch of short contexts, many kv heads), a single warp, which meets no barrier.  Each
// warp has its own ring of bulk copies, which runs on across units.  (Taking the next pair
// whenever there is room would even out the warps, but the sums' order, and with it the result,
// would change from run to run.)  A worker's part of a unit that it does not hold whole goes to
// the workspace, and a second kernel merges each unit's parts in order: cheaper than a ticket, a
// fence and a merge by the last worker to arrive, which few warps would then wait for.  Where no
// unit can be longer than kWholePairs, workers take whole units and there is no second kernel.
//
// Measured, with the merge: 4 requests of 128K tokens, 8 x 4 heads, bf16: 124.3 us, 4.8 TB/s of
// codes and scales, 73 % of a plain copy's rate (123.0 with one e for all heads and groups, which
// lost a small group's bits to a large one's); 64 requests to 8K tokens, 4 x 8 heads, 32-bit:
// 60.4 us (59.1), 2.4 TB/s.  335 and 510 instructions a strip (starts and ends of units included)
// keep 63 and 56 % of the issue slots busy: neither issue nor memory is full, the rest is warps that
// wait for a math pipe, for fixed latencies, for dispatch, and the wide form for code (16 warps an
// SM, 128 registers each: no more fit; the forms of 128 dims spill 12 to 56 bytes).  The same
// 4 x 128K in 32 bits: 124.1 us; with eight q heads to a kv head 165 (bf16) and 181 us (32-bit).
// 8192 attended tokens of one request: 12.9 us (12.6), bound by the chain launch, scan, table, copy,
// merge.
#include <cuda_fp16.h>

#include <algorithm>

#include "paged.cuh"
#include "paged_ring.cuh"

namespace rba {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kStages = 2;  // pairs of strips in a warp's ring (pair n takes place n % 2)
// What a unit's start and end cost, in pairs of its worker: a CTA's, a single warp's; and the pairs
// that a warp working alone takes at least (or a whole unit).  A CTA takes a multiple of kWarps, so
// that its warps have the same number: one each at 8192 of 128K tokens (8 kv heads) took 12.6 us,
// two each 14.3, 18 pairs to eight warps 14.8.
constexpr int kTeamCost = 10, kAloneCost = 3;
constexpr int kAloneLeast = 2;
// Warps work alone where the longest unit is then cut into at most this many parts.
constexpr int kAloneParts = 24;
constexpr int kFold = 16;  // pairs that a warp sums in the matrix unit's accumulators
// Units are taken whole where none can be longer than this: by single warps, or by CTAs where those
// suffice for one unit each.
constexpr int kWholePairs = 8;
constexpr float kToLog2 = 1.4426950408889634f;
constexpr float kToLn = 0.6931471805599453f;
constexpr float kSlack = 4.f;        // a logit may pass the reference by 2^4
constexpr int kTop = 7;              // exponent of a group's largest w when e is set
constexpr float kMostW = 32768.f;    // a w that may reach it sets e anew
constexpr int kMostScale = 11;       // s 2^e below 2^11 keeps w below it: 2^(11 + kSlack) = kMostW
constexpr int kMostE = 110;          // (scales are 0 or at least 2^-100)

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
  int2* units;        // per unit: its first part, and how many there are (1: nothing to merge)
  float* parts;       // [worker][2][heads of a unit][P + 4]
  float scale;
  int R, heads, group, dim, bs, strips, max_pages, n_pages, k, sink, window;
  int chunks;         // head chunks of a kv head
  int first;          // sink / bs
  int whole;          // workers take whole units
  bool q_vec;         // rows of q start on a boundary of four elements
  FastDiv by_bs, by_strips, by_units, by_chunks;
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
__device__ __forceinline__ UnitMap unit_map(const PagedAttendArgs& a, int T) {
  UnitMap m;
  const int full = div(T, a.by_bs);
  const int w0 = paged_w0(T, full, a.bs, a.window), w0_page = div(w0, a.by_bs);
  m.g = paged_geo(T, full, w0_page, a.first, a.bs, a.sink, a.window);
  const auto lin = [&](int pos, int page) {
    return page * a.strips + (pos - page * a.bs) / kStrip;
  };
  m.ns = m.g.sink_end > 0 ? lin(m.g.sink_end - 1, div(m.g.sink_end - 1, a.by_bs)) + 1 : 0;
  m.nk = (a.k < m.g.nc ? a.k : m.g.nc) * a.strips;
  m.w_lin = lin(w0, w0_page);
  m.nw = T > w0 ? lin(T - 1, div(T - 1, a.by_bs)) - m.w_lin + 1 : 0;
  return m;
}

// Strip v of a unit: its address, and its valid rows [ra, rb) as ra + 32 rb (0: nothing of it is
// attended to).
constexpr int kWholeStrip = 32 * kStrip, kWholePair = kWholeStrip << 16 | kWholeStrip;
__device__ __forceinline__ const uint8_t* locate(const PagedAttendArgs& a, const UnitMap& m, int r,
                                                 int h, int v, int sbytes, int* valid) {
  int lin, lo, hi;
  if (v < m.ns) {
    lin = v;
    lo = 0;
    hi = m.g.sink_end;
  } else if (v < m.ns + m.nk) {
    const int i = div(v - m.ns, a.by_strips);
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
  const int j = div(lin, a.by_strips), sp = lin - j * a.strips;
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

// The same for one byte of each half word (0: the low ones): the codes of its low nibbles, and
// low + 16 high in one number.  For a product's rows this saves the shift: the second row of a pair
// gathers the sum for low + 16 high, and the difference is taken once, at the end.
template <int kByte>
__device__ __forceinline__ void codes_of_bytes(uint32_t w, uint32_t* low, uint32_t* both) {
  const uint32_t b = __byte_perm(w, 0, kByte ? 0x4341 : 0x4240);
  const uint32_t up = 0x78007800u, off = 0xb440b440u;  // 2^15, -136 2^-9, twice
  const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&up),
                            *reinterpret_cast<const __half2*>(&off));
  *low = codes2<0>(b);
  *both = *reinterpret_cast<const uint32_t*>(&y);
}

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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Parts of the q operand (in shared memory, read group by group): hi, and for wide 32-bit q lo.
template <bool kWide, bool kLo> constexpr int q_parts() { return kWide && kLo ? 2 : 1; }

// A warp's running state for the unit's heads; lane (t, c) = (lane / 4, lane % 4) holds head c
// (packed) or heads 2 c and 2 c + 1 (wide).  A weight is 2^(y fac - m), y fac the logit in log2
// units, fac >= 0; the values' scales are taken times 2^e, e of the head and group, which keeps
// weight x scale within a half's range.
template <int P, bool kWide> struct State {
  static constexpr int HL = kWide ? 2 : 1, G = P / 32;
  float m[HL], l[HL];        // reference; this lane's part of the weights' sum
  uint32_t up[HL][G / 2];    // 2^e of two groups to a word, as bf16
  uint32_t most[G / 2];      // scales above it may pass kMostW with one of the heads' 2^e
  // dims 32 g + 4 t + {0, 1 (plus 16 times it), 2, 3 (the same)}: packed hi and lo columns, wide
  // two heads
  float acc[2 * G][4];
};

// Powers of two as bf16, two to a word: 2^n has the bits (n + 127) << 7, so words of them are added,
// subtracted and compared as pairs of 16-bit numbers.
constexpr uint32_t both(uint32_t x) { return x | x << 16; }
constexpr uint32_t kFirstUp = both((kMostE + 127) << 7);

template <int P, bool kWide> __device__ __forceinline__ void set_most(State<P, kWide>& st) {
#pragma unroll
  for (int j = 0; j < P / 64; ++j) {
    uint32_t up = st.up[0][j];
    if constexpr (kWide) up = __vmaxu2(up, st.up[1][j]);
    st.most[j] = both(((kMostScale + 2 * 127) << 7) - 1) - up;  // the number below 2^(kMostScale - e)
  }
}

// The reference moves to the largest logit so far and, for each head and group, e to where the
// largest weight x scale asks for it: sums so far are scaled by both (first: there are none).
// y, sv: logits and V scales of the lane's rows (-infinity and 0 for rows outside the attended set);
// ymax, smax: their largest.
template <int P, bool kWide, int kN>
__device__ __forceinline__ void move_reference(const float (*y)[kN][2], const float* ymax,
                                               const float* fac, const uint32_t (*sv)[2][P / 64],
                                               const uint32_t* smax, bool first,
                                               State<P, kWide>& st) {
  constexpr int G = P / 32, HL = kWide ? 2 : 1;
  constexpr uint32_t kExponents = both(0x7f80);
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    float m = ymax[i] * fac[i];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(st.m[i], ceilf(m));
    const float rise = m == st.m[i] ? 0.f : m - st.m[i];  // (infinite the first time)
    st.m[i] = m;
    uint32_t w[G / 2];  // the largest weight x scale, in bf16 (off by one in its exponent at most)
#pragma unroll
    for (int j = 0; j < G / 2; ++j) w[j] = 0;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // (-infinity times a factor of 0 is no number, and gives way)
        const __nv_bfloat162 p = __float2bfloat162_rn(ex2(fmaf(y[i][n][half], fac[i], -m)));
        const uint32_t p2 = *reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
        for (int j = 0; j < G / 2; ++j) w[j] = max_bf16x2(w[j], mul_bf16x2(sv[n][half][j], p2));
      }
    const float part = fminf(rise, 240.f), rest = ex2(part - rise);  // (an e ranges over 231)
    const uint32_t more = both(static_cast<uint32_t>(part) << 7);
#pragma unroll
    for (int j = 0; j < G / 2; ++j) {
      const uint32_t most = st.up[i][j] + more;
      uint32_t up = __vminu2(__vminu2(most, kFirstUp),
                             both((kTop + 2 * 127) << 7) - (w[j] & kExponents));
      // the largest scale times 2^e stays finite, so that a weight of 0 makes it 0
      up = __vminu2(up, both((126 + 2 * 127) << 7) - (smax[j] & kExponents));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) up = __vminu2(up, __shfl_xor_sync(0xffffffffu, up, o));
      st.up[i][j] = up;
      if (first) continue;
      // sums are scaled by 2^(e - rise), an e relative to the one before: at most 1
      const uint32_t f = both(127 << 7) - __vminu2(most - up, both(127 << 7));
#pragma unroll
      for (int g = 2 * j; g < 2 * j + 2; ++g) {
        const float scale = bf16_of(&f, g & 1) * rest;
#pragma unroll
        for (int b = 2 * g; b < 2 * g + 2; ++b)
#pragma unroll
          for (int x = kWide ? i : 0; x < 4; x += kWide ? 2 : 1) st.acc[b][x] *= scale;
      }
    }
    const uint32_t down = both(127 << 7) - __vminu2(more, both(127 << 7));
    st.l[i] *= bf16_of(&down, 0) * rest;
  }
  set_most(st);
}

// One step: kN strips, whose rows `valid` holds (16 bits each).  The packed form takes a pair, for
// one set of checks (123 us against 132, 128K tokens of 4 requests); a wide pair would be 13 KB of
// instructions and short of registers (60.6 us against 58.9, 64 requests to 8K tokens).
template <int P, bool kWide, bool kLo, int kN>
__device__ __forceinline__ void strips_step(const uint8_t* strips, int valid, const uint32_t* qw,
                                            const float* fac, bool first, State<P, kWide>& st) {
  constexpr int G = P / 32, HL = kWide ? 2 : 1, SB = strip_bytes(P);
  const int lane = threadIdx.x & 31, t = lane >> 2;
  const bool whole = valid == (kN == 2 ? kWholePair : kWholeStrip);
  float y[HL][kN][2];        // logits of tokens t and t + 8 of each strip for the lane's heads
  uint32_t sv[kN][2][G / 2]; // their V scales, two to a word
#pragma unroll
  for (int n = 0; n < kN; ++n) {
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
      for (int p = 0; p < q_parts<kWide, kLo>(); ++p) {
        uint32_t q[4];
        load_words<4>(reinterpret_cast<const uint8_t*>(qw + ((p * G + g) * 32 + lane) * 4), q);
        if (p == 0) mma16816_first(d, a0, q);
        else mma16816(d, a0, q);
        mma16816(d, a1, q + 2);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float s = bf16_of(sc[half], g);
        if constexpr (kWide) {
          y[0][n][half] = fmaf(s, d[2 * half], y[0][n][half]);
          y[HL - 1][n][half] = fmaf(s, d[2 * half + 1], y[HL - 1][n][half]);
        } else {
          // (a bf16 q has no lo part)
          y[0][n][half] = fmaf(s, kLo ? d[2 * half] + d[2 * half + 1] : d[2 * half], y[0][n][half]);
        }
      }
    }
  }
  if (!whole) {  // rows outside the attended set: no weight, and nothing of their scales
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int rows = valid >> (16 * n) & 0xffff;
        if (t + 8 * half >= (rows & 31) && t + 8 * half < (rows >> 5)) continue;
#pragma unroll
        for (int i = 0; i < G / 2; ++i) sv[n][half][i] = 0;
#pragma unroll
        for (int i = 0; i < HL; ++i) y[i][n][half] = -INFINITY;
      }
  }
  // the reference moves where a weight or weight x scale outgrows it: scales large enough for that
  // are seen first, their rows' weights only then
  uint32_t smax[G / 2];
#pragma unroll
  for (int j = 0; j < G / 2; ++j) {
    smax[j] = max_bf16x2(sv[0][0][j], sv[0][1][j]);
    if constexpr (kN == 2)
      smax[j] = max_bf16x2(smax[j], max_bf16x2(sv[kN - 1][0][j], sv[kN - 1][1][j]));
  }
  float ymax[HL];
  uint32_t large = 0;
#pragma unroll
  for (int j = 0; j < G / 2; ++j) large |= __vmaxu2(smax[j], st.most[j]) ^ st.most[j];
  bool grow = first || large != 0;
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    ymax[i] = fmaxf(y[i][0][0], y[i][0][1]);
    if constexpr (kN == 2) ymax[i] = fmaxf(ymax[i], fmaxf(y[i][kN - 1][0], y[i][kN - 1][1]));
    grow |= fmaf(ymax[i], fac[i], -st.m[i]) > kSlack;
  }
  if (__any_sync(0xffffffffu, grow)) {
    grow = first;
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      const float over = fmaf(ymax[i], fac[i], -st.m[i]);
      // (-infinity times a factor of 0 is no number: no weight)
      const float p = fmaxf(ex2(over), 0.f);
      uint32_t s = mul_bf16x2(smax[0], st.up[i][0]);
#pragma unroll
      for (int j = 1; j < G / 2; ++j) s = max_bf16x2(s, mul_bf16x2(smax[j], st.up[i][j]));
      // (a scale that 2^e makes infinite is to be met even by a weight of 0)
      grow |= over > kSlack || !(p * fmaxf(bf16_of(&s, 0), bf16_of(&s, 1)) < kMostW);
    }
    if (__any_sync(0xffffffffu, grow))
      move_reference<P, kWide, kN>(y, ymax, fac, sv, smax, first, st);
  }
#pragma unroll
  for (int i = 0; i < HL; ++i)
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float p = ex2(fmaf(y[i][n][half], fac[i], -st.m[i]));
        // (a row without weight before any row with one: -infinity against -infinity)
        if (!whole) p = y[i][n][half] == -INFINITY ? 0.f : p;
        st.l[i] += p;
        y[i][n][half] = p;
      }
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    uint32_t v[2][G], sc[HL][2][G / 2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      load_words<G>(strips + n * SB + 8 * P + half * 4 * P + lane * (G * 4), v[half]);
#pragma unroll
      for (int i = 0; i < HL; ++i)
#pragma unroll
        for (int j = 0; j < G / 2; ++j) sc[i][half][j] = mul_bf16x2(sv[n][half][j], st.up[i][j]);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // codes of the group's two 16-dim tiles
      uint32_t a0[4], a1[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        codes_of_bytes<0>(v[half][g], a0 + 2 * half, a0 + 2 * half + 1);
        codes_of_bytes<1>(v[half][g], a1 + 2 * half, a1 + 2 * half + 1);
      }
      // weights with the group's scale, hi + lo halves (11 + 11 bits)
      float hi[HL][2], lo[HL][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < HL; ++i) {
          const float w = y[i][n][half] * bf16_of(sc[i][half], g);
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

// Shared memory: rings | warp states (warps working alone: their q operands) | q operand |
// factors | barriers | pairs and units before each request.  (With up to 590 requests two CTAs fit
// an SM in every form.)
template <int P, bool kWide, bool kLo> struct Smem {
  static constexpr int H = kWide ? 8 : 4;
  static constexpr int kRow = P + 4;            // out, then m and l
  static constexpr int kSlot = H * kRow;
  static constexpr int kQBytes = q_parts<kWide, kLo>() * (P / 8) * 32 * 4;
  static constexpr int kRing = kWarps * kStages * 2 * strip_bytes(P);
  static constexpr int kSlots = kRing;
  static constexpr int kQ = kSlots + kWarps * kSlot * 4;
  static constexpr int kFac = kQ + kQBytes;
  static constexpr int kBars = kFac + kWarps * 32;
  static constexpr int kPre = kBars + kWarps * kStages * 8;
  static_assert(kQBytes <= kSlot * 4, "a warp's q operand fits its state's place");
  static size_t bytes(int R) { return kPre + size_t(R + 1) * 6; }
};

// q of the unit's heads into the products' B operand: a warp takes head hh, scaled by a power
// of two to a largest value in [2^14, 2^15), split hi + lo.  Word (part, 4 g + 2 ks + b) of lane
// (t, c) holds dims 32 g + 8 c + 2 ks + b and that + 4 of column t.
template <typename T>
__device__ __forceinline__ void load_q(const PagedAttendArgs& a, const T* q, bool live, float* x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = 0.f;
  if (live && lane * 4 < a.dim) load4(q + lane * 4, a.q_vec, x);
}
template <int P, bool kWide, bool kLo>
__device__ __forceinline__ void stage_q(const PagedAttendArgs& a, const float* x, int hh,
                                        uint32_t* qw, float* fac) {
  constexpr int WORDS = P / 8;
  const int lane = threadIdx.x & 31;
  float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int ex = top > 0.f ? 14 - exponent(top) : 0;
  // (two factors: 2^ex alone can leave the range of a float; the scale's sign goes with q)
  const float up0 = copysignf(pow2(ex / 2), a.scale), up1 = pow2(ex - ex / 2);
  const int g = lane >> 3, c = (lane & 7) >> 1, odd = lane & 1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = x[e] * up0 * up1, hi = __half2float(__float2half_rn(v)), lo = v - hi;
    const float hi_n = __shfl_xor_sync(0xffffffffu, hi, 1);
    const float lo_n = __shfl_xor_sync(0xffffffffu, lo, 1);
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
    fac[hh] = fabsf(a.scale) * kToLog2 * pow2((9 - ex) / 2) * pow2((9 - ex) - (9 - ex) / 2);
}

// The operand's columns of a head that is not there.
template <int P, bool kWide, bool kLo>
__device__ __forceinline__ void zero_q(int hh, uint32_t* qw, float* fac) {
  const int lane = threadIdx.x & 31, cols = kWide ? 1 : 2;
  for (int i = lane; i < q_parts<kWide, kLo>() * (P / 32) * cols * 4; i += 32) {
    const int c = i % 4, t = hh * cols + i / 4 % cols, w = i / 4 / cols;
    *reinterpret_cast<uint4*>(qw + (w * 32 + t * 4 + c) * 4) = make_uint4(0, 0, 0, 0);
  }
  if (lane == 0) fac[hh] = 0.f;
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : kToLn * (m + log2f(l));
}

// Where the line of pairs is at: unit u = (kv head, chunk) of request r, pairs [u0, u0 + n).
struct At {
  int r, h, h0, nh;
  uint32_t u, u0, n;
};

template <int P, bool kWide, typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_attend_kernel(PagedAttendArgs a) {
  constexpr bool kLo = sizeof(T) == 4;
  using S = Smem<P, kWide, kLo>;
  constexpr int G = P / 32, H = S::H, SB = strip_bytes(P), HL = kWide ? 2 : 1;
  extern __shared__ __align__(128) char sm[];
  float* slots = reinterpret_cast<float*>(sm + S::kSlots);
  int32_t* pre = reinterpret_cast<int32_t*>(sm + S::kPre);
  uint16_t* cnt = reinterpret_cast<uint16_t*>(pre + a.R + 1);
  __shared__ int64_t s_w[kWarps];
  __shared__ int s_long;
  __shared__ uint32_t s_chunk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t units = a.heads * a.chunks;  // per request
  char* ring = sm + warp * kStages * 2 * SB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBars) + warp * kStages;
  if (lane < kStages) mbar_init(bars + lane, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (tid == 0) s_long = 0;
  wait_for_stream();

  // pairs of strips (of one unit) and requests with any before each request; the longest unit
  int64_t run = 0;
  for (int base = 0; base < a.R; base += kThreads) {
    const int r = base + tid;
    int n = 0;
    if (r < a.R)
      n = (unit_map(a, paged_len(a.lens, r, a.bs, a.max_pages, a.status)).total() + 1) / 2;
    int64_t tot;
    const int64_t ex =  // (two barriers: s_long is set by now)
        run + block_scan64(int64_t(n) << 16 | int64_t(n > 0), s_w, &tot);
    if (r < a.R) {
      pre[r] = static_cast<int32_t>(ex >> 16);
      cnt[r] = static_cast<uint16_t>(ex & 0xffff);
    }
    if (n > 0) atomicMax(&s_long, n);
    run += tot;
  }
  const uint32_t pairs = static_cast<uint32_t>(run >> 16);
  const uint32_t some = static_cast<uint32_t>(run & 0xffff);
  if (tid == 0) {
    pre[a.R] = static_cast<int32_t>(pairs);
    cnt[a.R] = static_cast<uint16_t>(some);
  }
  __syncthreads();
  // requests that attend to nothing
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    if (pre[r + 1] != pre[r]) continue;
    const int hq = a.heads * a.group;
    for (int i = tid; i < hq * a.dim; i += kThreads) a.out[int64_t(r) * hq * a.dim + i] = 0.f;
    if (a.lse != nullptr)
      for (int i = tid; i < hq; i += kThreads) a.lse[int64_t(r) * hq + i] = -INFINITY;
    for (int i = tid; i < static_cast<int>(units); i += kThreads)
      a.units[int64_t(r) * units + i] = make_int2(0, 1);
  }
  if (pairs == 0) return;

  // (the same in every CTA)
  const uint32_t longest = s_long, all = pairs * units;
  const uint32_t share = (all + gridDim.x * kWarps - 1) / (gridDim.x * kWarps);
  const bool alone = a.whole ? some * units > gridDim.x : longest <= kAloneParts * share;
  const uint32_t extra = alone ? kAloneCost : kTeamCost;
  const uint32_t cost = (pairs + extra * some) * units;
  const uint32_t workers = alone ? gridDim.x * kWarps : gridDim.x;
  const uint32_t worker = alone ? blockIdx.x * kWarps + warp : blockIdx.x;
  uint32_t chunk = (cost + workers - 1) / workers;
  if (alone) chunk = max(chunk, min(longest, static_cast<uint32_t>(kAloneLeast)) + extra);
  else chunk = (chunk + kWarps - 1) / kWarps * kWarps;
  if (lane == 0) s_chunk = chunk;  // (every warp the same value: its own lanes read it back)

  const auto at_unit = [&](int r, uint32_t u) {
    At p;
    p.r = r;
    p.n = pre[r + 1] - pre[r];
    p.u = u;
    p.u0 = uint32_t(pre[r]) * units + u * p.n;
    p.h = div(static_cast<int>(u), a.by_chunks);
    p.h0 = (static_cast<int>(u) - p.h * a.chunks) * H;
    p.nh = min(H, a.group - p.h0);
    return p;
  };
  const auto place = [&](uint32_t at) {  // of a pair
    const int r = last_at_most(pre, a.R, div(static_cast<int>(at), a.by_units));
    return at_unit(r, (at - uint32_t(pre[r]) * units) / uint32_t(pre[r + 1] - pre[r]));
  };
  const auto unit_no = [&](const At& p) { return cnt[p.r] * units + p.u; };
  const auto cost_at = [&](const At& p) {  // of a unit's first pair
    return (uint32_t(pre[p.r]) + extra * cnt[p.r]) * units + p.u * (p.n + extra);
  };
  const auto pair_at = [&](uint32_t x) {  // the first pair whose cost is not below x
    if (x >= cost) return all;
    const uint32_t y = div(static_cast<int>(x), a.by_units);
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (uint32_t(pre[mid]) + extra * cnt[mid] <= y) lo = mid;
      else hi = mid;
    }
    const uint32_t n = pre[lo + 1] - pre[lo];
    const uint32_t in = x - (uint32_t(pre[lo]) + extra * cnt[lo]) * units;
    const uint32_t u = in / (n + extra);
    return uint32_t(pre[lo]) * units + u * n + min(in - u * (n + extra), n);
  };
  const auto unit_of = [&](uint32_t i) {  // the line's i-th unit
    const uint32_t k = div(static_cast<int>(i), a.by_units);
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cnt[mid] <= k) lo = mid;
      else hi = mid;
    }
    return at_unit(lo, i - k * units);
  };
  // the worker's pairs, and its CTA's: lane i finds the i-th bound
  uint32_t begin, end, cta_begin, cta_end;
  {
    const uint32_t w = lane < 2 ? worker + lane
                       : alone  ? blockIdx.x * kWarps + (lane & 1) * kWarps : worker + (lane & 1);
    uint32_t x = all;
    if (a.whole) {
      const uint32_t i = static_cast<uint32_t>(uint64_t(some) * units * w / workers);
      if (i < some * units) x = unit_of(i).u0;
    } else if (uint64_t(chunk) * w < cost) {
      x = pair_at(chunk * w);
    }
    begin = __shfl_sync(0xffffffffu, x, 0);
    end = __shfl_sync(0xffffffffu, x, 1);
    cta_begin = __shfl_sync(0xffffffffu, x, 2);
    cta_end = __shfl_sync(0xffffffffu, x, 3);
  }
  if (cta_begin >= cta_end) return;  // (no pair among what it was dealt)

  // the warp's pairs: begin + warp, + 8, .. of the CTA's, or all of its own
  const uint32_t turn = alone ? begin : begin + warp, stride = alone ? 1 : kWarps;
  const auto pairs_below = [&](uint32_t x) {  // how many of them lie before pair x of the line
    return x <= turn ? 0 : static_cast<int>(alone ? x - turn : (x - turn + kWarps - 1) / kWarps);
  };
  int mine = pairs_below(end);
  // lanes 2 i and 2 i + 1 hold the strips of pair i of the round of 16 pairs that is being issued:
  // the lane's strip and its bytes, and both strips' rows (rows0 | rows1 << 16); of the round
  // before, those rows
  const uint8_t* src = a.pool;
  uint32_t bytes = 0, bytes_both = 0;
  int rows = 0, rows_before = 0;
  const uint32_t bar0 = smem_u32(bars), place0 = smem_u32(ring) + (lane & 1) * SB;
  const auto find = [&](int n) {
    rows_before = rows;
    int valid = 0;
    const int i = n + lane / 2;
    if (i < mine) {
      const uint32_t at = turn + uint32_t(i) * stride;
      const At p = place(at);
      const int v = 2 * static_cast<int>(at - p.u0) + (lane & 1);
      const UnitMap map = unit_map(a, a.lens[p.r]);
      if (v < map.total()) src = locate(a, map, p.r, p.h, v, SB, &valid);
    }
    const int other = __shfl_xor_sync(0xffffffffu, valid, 1);
    bytes = valid ? SB : 0;
    bytes_both = bytes + (other ? SB : 0);
    rows = lane & 1 ? other | valid << 16 : valid | other << 16;
  };
  const auto issue = [&](int n) {  // the warp's n-th pair into stage n % 2, which is free
    if (n >= mine) return;
    if ((n & 15) == 0) find(n);
    const bool me = lane / 2 == (n & 15);
    arm_and_copy(bar0 + (n & 1) * 8, me && (lane & 1) == 0, bytes_both, place0 + (n & 1) * 2 * SB,
                 src, me ? bytes : 0);
  };
  // q operands: one for the CTA, or a place for each of the units in its warps' lines (for each of
  // its warps, where there are more units).  A unit of up to four heads is staged by one warp;
  // eight took one warp 7 us, so those are dealt out (61.8 -> 60.8 us, 64 requests to 8K tokens).
  const auto q_place = [&](int i) {
    return reinterpret_cast<uint32_t*>(alone ? sm + S::kSlots + i * S::kSlot * 4 : sm + S::kQ);
  };
  const auto fac_place = [&](int i) { return reinterpret_cast<float*>(sm + S::kFac) + 8 * i; };
  const auto fetch = [&](const At& p, int hh, float* x) {
    load_q(a, static_cast<const T*>(a.q) + p.r * a.q_req +
                  (int64_t(p.h) * a.group + p.h0 + hh) * a.q_head, hh < p.nh, x);
  };
  const auto stage = [&](const At& p, int hh) {  // one head of a CTA's unit
    float x[4];
    fetch(p, hh, x);
    stage_q<P, kWide, kLo>(a, x, hh, q_place(0), fac_place(0));
  };
  const auto stage_all = [&](const At& p, int i) {  // a unit's heads into place i
    float x[H][4];
#pragma unroll
    for (int hh = 0; hh < H; ++hh) fetch(p, hh, x[hh]);
#pragma unroll
    for (int hh = 0; hh < H; ++hh) {
      if (hh < p.nh) stage_q<P, kWide, kLo>(a, x[hh], hh, q_place(i), fac_place(i));
      else zero_q<P, kWide, kLo>(hh, q_place(i), fac_place(i));
    }
  };

  const auto stage_units = [&](uint32_t first, uint32_t n) {  // a warp takes one head of every unit
    const int hh = warp;
    const At p = unit_of(first + min(static_cast<uint32_t>(lane), n - 1));  // lane i: unit i
    const int64_t row = p.r * a.q_req + (int64_t(p.h) * a.group + p.h0) * a.q_head;
    float x[H][4];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int64_t at = __shfl_sync(0xffffffffu, row, i);
      const int nh = __shfl_sync(0xffffffffu, p.nh, i);
      load_q(a, static_cast<const T*>(a.q) + at + hh * a.q_head,
             i < static_cast<int>(n) && hh < nh, x[i]);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if (i >= static_cast<int>(n)) break;
      if (hh < __shfl_sync(0xffffffffu, p.nh, i))
        stage_q<P, kWide, kLo>(a, x[i], hh, q_place(i), fac_place(i));
      else
        zero_q<P, kWide, kLo>(hh, q_place(i), fac_place(i));
    }
  };

#pragma unroll 1
  for (int n = 0; n < kStages; ++n) issue(n);
  uint32_t first_unit = 0;
  bool shared_q = !alone;
  if (alone) {
    first_unit = unit_no(place(cta_begin));
    const uint32_t n = unit_no(place(cta_end - 1)) - first_unit + 1;
    shared_q = n <= kWarps;
    if constexpr (kWide) {
      if (shared_q) stage_units(first_unit, n);
    } else {
      if (shared_q && warp < static_cast<int>(n)) stage_all(unit_of(first_unit + warp), warp);
    }
  } else if (warp < H) {
    stage(place(begin), warp);
  }
  if (shared_q) __syncthreads();

  int j = 0;      // the warp's next pair
  int later = 0;  // not the worker's first unit
  for (uint32_t at = begin; at < end; later = 1) {
    uint32_t stop;
    int at_place;
    {
      const At p = place(at);
      stop = min(end, p.u0 + p.n);
      at_place = !alone ? 0 : shared_q ? static_cast<int>(unit_no(p) - first_unit) : warp;
      if (!shared_q) {
        __syncwarp();
        stage_all(p, warp);
        __syncwarp();
      }
    }
    const uint32_t* qw = q_place(at_place);
    float fac[HL];
#pragma unroll
    for (int i = 0; i < HL; ++i) fac[i] = fac_place(at_place)[HL * (lane & 3) + i];
    // Every kFold pairs the sums are added to their place in memory and start anew: the matrix unit
    // cuts its sums towards zero, which over a long line would add up.
    const auto part_of = [&] { return a.parts + (int64_t(worker) * 2 + later) * S::kSlot; };
    const int t = lane >> 2, c = lane & 3;
    State<P, kWide> st;
    float4 o[HL][G];  // the warp's state in its lanes: dims 32 g + 4 t + {0..3} of heads HL c ..
    int till = min(mine, pairs_below(stop));
    bool held = false, first = true;
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      st.m[i] = -INFINITY;
#pragma unroll
      for (int b = 0; b < G / 2; ++b) st.up[i][b] = kFirstUp;
    }
    set_most(st);
#pragma unroll 1
    while (true) {
#pragma unroll
      for (int i = 0; i < HL; ++i) st.l[i] = 0.f;
#pragma unroll
      for (int b = 0; b < 2 * G; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.acc[b][i] = 0.f;

      const int pause = min(till, j + kFold);
#pragma unroll 1
      for (; j < pause; ++j) {
        const uint32_t bar = bar0 + (j & 1) * 8, parity = (j >> 1) & 1;
        if (!await_phase(bar, parity)) {
          if (lane == 0) report(a.status, RBA_ERR_TIMEOUT, kWherePaged, j);
          // copies in flight land before the warp goes on without its pairs
          mbar_drain(bars + (j & 1), parity);
          if (j + 1 < mine) mbar_drain(bars + (~j & 1), ((j + 1) >> 1) & 1);
          mine = till = 0;
          break;
        }
        // (pair j + 1 was issued last: in j's round or the next)
        const int r2 = __shfl_sync(0xffffffffu, (j & 15) == 15 && j + 1 < mine ? rows_before : rows,
                                   2 * (j & 15));
        if (r2 != 0) {
          const uint8_t* pair = reinterpret_cast<const uint8_t*>(ring + (j & 1) * 2 * SB);
          if constexpr (kWide) {
#pragma unroll 1
            for (int n = 0; n < 2; ++n) {
              const int r1 = r2 >> (16 * n) & 0xffff;
              if (r1 == 0) continue;
              strips_step<P, kWide, kLo, 1>(pair + n * SB, r1, qw, fac, first, st);
              first = false;
            }
          } else {
            strips_step<P, kWide, kLo, 2>(pair, r2, qw, fac, first, st);
            first = false;
          }
        }
        __syncwarp();
        issue(j + kStages);
      }

      {
#pragma unroll
        for (int i = 0; i < HL; ++i) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], x);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float down = pow2(127 - static_cast<int>(st.up[i][g / 2] >> (g & 1 ? 23 : 7) & 255u));
            float y[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float* d = st.acc[2 * g + x / 2];
              y[x] = (kWide ? d[2 * (x % 2) + i] : d[2 * (x % 2)] + d[2 * (x % 2) + 1]) * 0x1p9f *
                     down;
            }
            // (the odd rows hold the even dim plus 16 times theirs)
            o[i][g] = make_float4(y[0], (y[1] - y[0]) * 0.0625f, y[2], (y[3] - y[2]) * 0.0625f);
          }
        }
      }
      float* to = alone ? part_of() : slots + warp * S::kSlot;
      if (held) {  // with what was put there before
#pragma unroll
        for (int i = 0; i < HL; ++i) {
          const float* s = to + (HL * c + i) * S::kRow;
          const float pm = s[P], pl = s[P + 1], m = fmaxf(st.m[i], pm);
          const float f0 = st.m[i] == m ? 1.f : ex2(st.m[i] - m), f1 = pm == m ? 1.f : ex2(pm - m);
          st.m[i] = m;
          st.l[i] = st.l[i] * f0 + pl * f1;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float4 x = *reinterpret_cast<const float4*>(s + 32 * g + 4 * t);
            o[i][g] = make_float4(o[i][g].x * f0 + x.x * f1, o[i][g].y * f0 + x.y * f1,
                                  o[i][g].z * f0 + x.z * f1, o[i][g].w * f0 + x.w * f1);
          }
        }
      }
      if (j >= till) break;
      __syncwarp();  // (read by every lane of a head, written by one)
#pragma unroll
      for (int i = 0; i < HL; ++i) {
        float* s = to + (HL * c + i) * S::kRow;
#pragma unroll
        for (int g = 0; g < G; ++g) *reinterpret_cast<float4*>(s + 32 * g + 4 * t) = o[i][g];
        if (t == 0) {
          s[P] = st.m[i];
          s[P + 1] = st.l[i];
        }
      }
      __syncwarp();
      held = true;
    }

    const bool more = stop < end;
    const At p = place(at);  // (again: nothing of it is kept over the loop)
    const bool whole = at == p.u0 && stop == p.u0 + p.n;
    const int64_t row0 = (int64_t(p.r) * a.heads + p.h) * a.group + p.h0;
    float* part = part_of();
    float* to = alone ? part : slots + warp * S::kSlot;
    if (held) __syncwarp();  // (as above)
    if (at == p.u0 && lane == 0 && (alone || warp == 0)) {
      // this worker holds the unit's first pair; the last one's holds its last
      const uint32_t x0 = cost_at(p);
      a.units[int64_t(p.r) * units + p.u] =
          whole ? make_int2(0, 1)
                : make_int2(static_cast<int>(worker) * 2 + later,
                            static_cast<int>((x0 + p.n - 1) / s_chunk - x0 / s_chunk) + 1);
    }
    if (!(alone && whole)) {
#pragma unroll
      for (int i = 0; i < HL; ++i) {
        if (alone && HL * c + i >= p.nh) continue;
        float* s = to + (HL * c + i) * S::kRow;
#pragma unroll
        for (int g = 0; g < G; ++g) *reinterpret_cast<float4*>(s + 32 * g + 4 * t) = o[i][g];
        if (t == 0) {
          s[P] = st.m[i];
          s[P + 1] = st.l[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < HL; ++i) {
        const int hh = HL * c + i;
        if (hh >= p.nh) continue;
        const float l = st.l[i], r = l == 0.f ? 0.f : 1.f / l;
        float* out = a.out + (row0 + hh) * a.dim;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int d = 32 * g + 4 * t;
          if (d >= a.dim) continue;
          out[d] = o[i][g].x * r;
          out[d + 1] = o[i][g].y * r;
          out[d + 2] = o[i][g].z * r;
          out[d + 3] = o[i][g].w * r;
        }
        if (t == 0 && a.lse != nullptr) a.lse[row0 + hh] = lse_of(st.m[i], l);
      }
    }
    if (!alone) {
      __syncthreads();
      if (more && warp < H) stage(place(stop), warp);  // (every warp is done with this unit's)
      for (int i = tid; i < p.nh * P; i += kThreads) {
        const int hh = i / P, d = i % P;
        const float* s = slots + hh * S::kRow;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s[w * S::kSlot + P]);
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float pm = s[w * S::kSlot + P];
          const float f = pm == m ? 1.f : ex2(pm - m);
          l += f * s[w * S::kSlot + P + 1];
          x += f * s[w * S::kSlot + d];
        }
        if (whole) {
          if (d < a.dim) a.out[(row0 + hh) * a.dim + d] = l == 0.f ? 0.f : x / l;
          if (d == 0 && a.lse != nullptr) a.lse[row0 + hh] = lse_of(m, l);
        } else {
          float* y = part + hh * S::kRow;
          y[d] = x;
          if (d == 0) {
            y[P] = m;
            y[P + 1] = l;
          }
        }
      }
    }
    at = stop;
    if (!alone && more) __syncthreads();  // the slots are read, q of the next unit is there
  }
}

// Merges the parts of one (request, q head): four warps take every fourth part, eight parts' loads
// in flight, and meet in shared memory.  The first part of a unit may be its worker's second; the
// others are the following workers' first.
constexpr int kMergeWarps = 4;
template <int P>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(PagedAttendArgs a, int H) {
  constexpr int kRow = P + 4, kU = 8;
  __shared__ __align__(16) float s_part[kMergeWarps][kRow];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = a.heads * a.group, r = blockIdx.x / hq, head = blockIdx.x - r * hq;
  const int h = head / a.group, in = head - h * a.group, chunk = in / H, hh = in - chunk * H;
  const int2 u = a.units[int64_t(r) * a.heads * a.chunks + h * a.chunks + chunk];
  if (u.y <= 1) return;
  const float* p0 = a.parts + (int64_t(u.x) * H + hh) * kRow;
  const float* p1 = a.parts + (int64_t(u.x / 2) * 2 * H + hh) * kRow;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = warp; c0 < u.y; c0 += kU * kMergeWarps) {
    float pm[kU], pl[kU];
    float4 po[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int c = c0 + i * kMergeWarps;
      pm[i] = -INFINITY;
      pl[i] = 0.f;
      po[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < u.y) {
        const float* s = c == 0 ? p0 : p1 + int64_t(c) * 2 * H * kRow;
        pm[i] = s[P];
        pl[i] = s[P + 1];
        if (lane * 4 < P) po[i] = reinterpret_cast<const float4*>(s)[lane];
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
  if (lane * 4 < P) *reinterpret_cast<float4*>(&s_part[warp][lane * 4]) = o;
  if (lane == 0) {
    s_part[warp][P] = m;
    s_part[warp][P + 1] = l;
  }
  __syncthreads();
  const int d = threadIdx.x;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, s_part[w][P]);
  float x = 0.f;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float f = s_part[w][P] == m ? 1.f : ex2(s_part[w][P] - m);
    l += f * s_part[w][P + 1];
    x += f * (d < P ? s_part[w][d] : 0.f);
  }
  const int64_t row = int64_t(r) * hq + head;
  if (d < a.dim) a.out[row * a.dim + d] = l == 0.f ? 0.f : x / l;
  if (d == 0 && a.lse != nullptr) a.lse[row] = lse_of(m, l);
}

// Groups of up to four q heads to a kv head take the packed form, larger ones the wide one.
bool wide_of(const rba_paged* s) { return s->d.n_q_heads / s->d.n_kv_heads > 4; }
int chunks_of(const rba_paged* s) {
  const int group = s->d.n_q_heads / s->d.n_kv_heads;
  return group <= 4 ? 1 : (group + 7) / 8;
}
size_t unit_bytes(const rba_paged* s) {
  return align_up(size_t(s->d.max_requests) * s->d.n_kv_heads * chunks_of(s) * sizeof(int2), 256);
}

template <int P, bool kWide, typename T>
rba_status launch(const PagedAttendArgs& a, cudaStream_t stream) {
  const size_t smem = Smem<P, kWide, sizeof(T) == 4>::bytes(a.R);
  void (*const kernel)(PagedAttendArgs) = paged_attend_kernel<P, kWide, T>;
  RBA_CUDA_TRY(ensure_smem(reinterpret_cast<const void*>(kernel), smem));
  RBA_CUDA_TRY(launch_dependent(kernel, static_cast<unsigned>(num_sms() * kCtasPerSm), kThreads,
                                smem, stream, a));
  if (!a.whole)
    RBA_CUDA_TRY(launch_dependent(paged_merge_kernel<P>,
                                  static_cast<unsigned>(a.R * a.heads * a.group), kMergeWarps * 32,
                                  0, stream, a, kWide ? 8 : 4));
  return RBA_OK;
}

}  // namespace

rba_status refuse_attend(const rba_paged* s, int32_t n_requests, int32_t k, int32_t sink,
                         int32_t window, const void* workspace, size_t ws_bytes) {
  if (s == nullptr || workspace == nullptr || n_requests <= 0 ||
      n_requests > s->d.max_requests || k < 0 || sink < 0 || window < 0)
    return RBA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return RBA_ERR_INVALID_ARG;
  if (ws_bytes < rba_paged_attend_workspace_size(s)) return RBA_ERR_WORKSPACE;
  // the line of pairs, with what units cost, is counted in 31 bits (sink, selection and window can
  // share two pages)
  const int64_t unit = ((int64_t(s->d.max_pages) + 2) * s->strips + 1) / 2 + kTeamCost;
  const int64_t units = int64_t(n_requests) * s->d.n_kv_heads * chunks_of(s);
  if (unit > INT32_MAX || unit * units > INT32_MAX ||
      int64_t(n_requests) * s->d.n_q_heads > INT32_MAX)
    return RBA_ERR_UNSUPPORTED;
  return RBA_OK;
}

}  // namespace rba

extern "C" size_t rba_paged_attend_workspace_size(const rba_paged* s) {
  using namespace rba;
  if (s == nullptr) return 0;
  return unit_bytes(s) + size_t(num_sms()) * kCtasPerSm * kWarps * 2 *
                               (wide_of(s) ? 8 : 4) * (s->pitch + 4) * sizeof(float);
}

extern "C" rba_status rba_paged_step_check(const rba_paged* s, int32_t n_requests, int32_t n_rows,
                                           int32_t k, int32_t sink, int32_t window,
                                           const void* select_workspace, size_t select_bytes,
                                           const void* attend_workspace, size_t attend_bytes) {
  using namespace rba;
  rba_status r = refuse_append(s, n_rows);
  if (r == RBA_OK)
    r = refuse_select(s, n_requests, k, sink, window, select_workspace, select_bytes);
  if (r == RBA_OK)
    r = refuse_attend(s, n_requests, k, sink, window, attend_workspace, attend_bytes);
  return r;
}

extern "C" rba_status rba_paged_attend(const rba_paged* s, const void* q,
                                       int64_t q_request_stride, int64_t q_head_stride,
                                       int32_t n_requests, const int32_t* idx, int32_t k,
                                       int32_t sink, int32_t window, float scale, float* out,
                                       float* lse, void* workspace, size_t ws_bytes,
                                       cudaStream_t stream) {
  using namespace rba;
  if (q == nullptr || out == nullptr || (k > 0 && idx == nullptr)) return RBA_ERR_INVALID_ARG;
  const rba_status refused = refuse_attend(s, n_requests, k, sink, window, workspace, ws_bytes);
  if (refused != RBA_OK) return refused;
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
  a.units = static_cast<int2*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + unit_bytes(s));
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
  a.q_vec = reinterpret_cast<uintptr_t>(q) % (4 * dtype_size(s->d.dtype)) == 0 &&
            ((q_request_stride | q_head_stride) & 3) == 0;
  a.first = sink / a.bs;
  // the longest unit there can be: what sink, selection and window ask for (each may begin and end
  // inside a page), or the whole table.  (A page that two of them share is counted once here, so a
  // unit of a short table can be two pages longer than kWholePairs: that costs its warp time only.)
  const auto strips_of = [&](int n) { return int64_t(n / a.bs) * s->strips + n % a.bs / kStrip; };
  const int64_t strips =
      std::min(strips_of(sink) + (int64_t(k) + 4) * s->strips + strips_of(window),
               int64_t(s->d.max_pages) * s->strips);
  a.whole = (strips + 1) / 2 <= kWholePairs;
  a.by_bs = fast_div(a.bs);
  a.by_strips = fast_div(a.strips);
  a.by_units = fast_div(a.heads * a.chunks);
  a.by_chunks = fast_div(a.chunks);
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
