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
// a power of two per head and split into two halves (hi + lo, 22 bits), in neighbouring columns
// of the product: 8 columns are 4 q heads, exactly a GQA group of 4.  For the values the weight
// takes the scale, w = p s_tg 2^e, again split into hi + lo columns.  Softmax statistics, both
// products' accumulators and the merges are 32-bit.
//
// Layout.  One warp takes a strip of 16 tokens: K codes are the A operand of the first product
// (16 tokens x 16 dims), q its B; V codes, read in token pairs, are the A operand of the second
// (16 dims x 16 tokens), and the weights its B after one 8 x 8 transpose in registers.
//
// The running maximum is lazy: weights are taken relative to a reference that moves only when
// a logit passes it by 2^4, so most strips need no cross-lane maximum and no rescale.
//
// Work.  All strips of all (request, kv head) units form one line, cut evenly over the CTAs
// whatever the requests' lengths; a CTA's part of a unit that it does not hold whole goes to
// the workspace, and the last of the unit's CTAs to arrive merges the parts in order.
#include <cuda_fp16.h>

#include "paged.cuh"

namespace rba {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 4.f;        // a logit may pass the reference by 2^4
constexpr int kScaleTop = 10;        // s 2^e stays below 2^10 when e is set, below 2^11 always

struct AttendArgs {
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
  float* parts;       // [CTA][2][heads of a unit][P + 2]
  float scale;
  int R, heads, group, dim, bs, strips, max_pages, n_pages, k, sink, window;
  int chunks;         // head chunks of a kv head: ceil(group / (4 NT))
  int bf16;
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1,
                                         const float* c) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
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
// Two codes, 2^-9 each, from the nibbles that `mask` leaves: nibble 0 (or 1) of each half word.
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
__device__ __forceinline__ UnitMap unit_map(const AttendArgs& a, int T) {
  UnitMap m;
  m.g = paged_geo(T, a.bs, a.sink, a.window);
  m.ns = m.g.sink_end > 0 ? lin_strip(m.g.sink_end - 1, a.bs, a.strips) + 1 : 0;
  m.nk = (a.k < m.g.nc ? a.k : m.g.nc) * a.strips;
  m.w_lin = lin_strip(m.g.w0, a.bs, a.strips);
  m.nw = T > m.g.w0 ? lin_strip(T - 1, a.bs, a.strips) - m.w_lin + 1 : 0;
  return m;
}

// Strip v of a unit: its address and its valid rows [ra, rb) (none where nothing is attended).
__device__ __forceinline__ const uint8_t* locate(const AttendArgs& a, const UnitMap& m, int r,
                                                 int h, int v, int sbytes, int* ra, int* rb) {
  *ra = *rb = 0;
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
  *ra = max(lo - pos0, 0);
  *rb = min(min(kStrip, hi - pos0), a.bs - sp * kStrip);
  if (*rb <= *ra) *ra = *rb = 0;
  return a.pool + ((int64_t(page) * a.heads + h) * a.strips + sp) * sbytes;
}

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

// A warp's running state for the unit's 4 NT heads; lane (t, c) = (lane / 4, lane % 4) holds
// head 4 i + c of column tile i.
template <int P, int NT> struct State {
  static constexpr int G = P / 32;
  float m[NT], l[NT];       // reference (log2 units); this lane's part of the sum
  float acc[NT][2 * G][4];  // out: dims 32 g + 4 (lane / 4) + {0..3}, hi and lo columns
  int e;                    // V scales are multiplied by 2^e
};

template <int P, int NT>
__device__ __forceinline__ void strip_step(const Frag<P>& f, bool whole, int ra, int rb,
                                           const uint32_t (&qf)[NT][P / 16][2],
                                           const float (&fac)[NT], State<P, NT>& st) {
  constexpr int G = P / 32;
  const int lane = threadIdx.x & 31, t = lane >> 2;
  // logits of tokens t and t + 8 for the lane's heads
  float x[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t w0 = f.k[0][g], w1 = f.k[1][g], u0 = w0 >> 8, u1 = w1 >> 8;
    const uint32_t a0[4] = {codes2<0>(w0), codes2<0>(w1), codes2<1>(w0), codes2<1>(w1)};
    const uint32_t a1[4] = {codes2<0>(u0), codes2<0>(u1), codes2<1>(u0), codes2<1>(u1)};
    const float s0 = scale_of<G>(f.s[0], g), s1 = scale_of<G>(f.s[1], g);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma16816(d, a0, qf[i][2 * g][0], qf[i][2 * g][1], d);
      mma16816(d, a1, qf[i][2 * g + 1][0], qf[i][2 * g + 1][1], d);
      x[i][0] = fmaf(s0, d[0] + d[1], x[i][0]);
      x[i][1] = fmaf(s1, d[2] + d[3], x[i][1]);
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
  for (int i = 0; i < NT; ++i) {
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
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float top = fmaxf(x[i][0], x[i][1]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m = fmaxf(st.m[i], top);
      const float fm = m == st.m[i] ? 1.f : ex2(st.m[i] - m);
      st.m[i] = m;
      st.l[i] *= fm;
#pragma unroll
      for (int b = 0; b < 2 * G; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.acc[i][b][j] *= fm * fe;
    }
  }
  const float up = pow2(st.e);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
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
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      // weights with the group's scale, hi + lo halves (11 + 11 bits)
      uint32_t b[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float w = x[i][j] * sv[j][g];
        const float hi = __uint_as_float(__float_as_uint(w) & 0xffffe000u);
        b[j] = transpose8x8(pack_half2(hi, w - hi));
      }
      mma16816(st.acc[i][2 * g], a0, b[0], b[1], st.acc[i][2 * g]);
      mma16816(st.acc[i][2 * g + 1], a1, b[0], b[1], st.acc[i][2 * g + 1]);
    }
  }
}

// Shared memory: [R] strips before a request | per warp merge slots | q rows.
template <int P, int NT> struct Smem {
  static constexpr int H = 4 * NT;
  static constexpr int kSlot = H * (P + 2);
  static size_t bytes(int R) {
    return size_t(kWarps) * kSlot * 4 + size_t(H) * P * 4 + size_t(R + 1) * 4;
  }
};

// Writes a merged state: whole units to the outputs, parts to the workspace.
template <int P, int NT, bool kBf16>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) paged_attend_kernel(AttendArgs a) {
  constexpr int G = P / 32, H = 4 * NT, SB = strip_bytes(P), SLOT = Smem<P, NT>::kSlot;
  extern __shared__ __align__(16) float smf[];
  float* slots = smf;                       // [warp][H][P + 2]: out, m, l
  float* qs = smf + kWarps * SLOT;          // [H][P]
  int32_t* pre = reinterpret_cast<int32_t*>(qs + H * P);
  __shared__ int64_t s_w[kWarps];
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.heads * a.chunks;     // per request

  int64_t run = 0;
  for (int base = 0; base < a.R; base += kThreads) {
    const int r = base + tid;
    int n = 0;
    if (r < a.R) n = unit_map(a, paged_len(a.lens, r, a.bs, a.max_pages, a.status)).total();
    int64_t tot;
    const int64_t ex = block_scan64(n, s_w, &tot);
    if (r < a.R) pre[r] = static_cast<int32_t>(run + ex);
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
  const int64_t all = run * units;
  const int64_t chunk = (all + gridDim.x - 1) / gridDim.x;
  const int64_t begin = chunk * blockIdx.x, end = min(all, begin + chunk);

  for (int64_t at = begin; at < end;) {
    const int r = last_at_most(pre, a.R, static_cast<int32_t>(at / units));
    const int n = pre[r + 1] - pre[r];
    const int64_t base = int64_t(pre[r]) * units;
    const int u = static_cast<int>((at - base) / n);
    const int h = u / a.chunks, h0 = (u - h * a.chunks) * H;  // first head of the chunk
    const int64_t u0 = base + int64_t(u) * n;                  // the unit's first strip
    const int v0 = static_cast<int>(at - u0);
    const int v1 = static_cast<int>(min(end - u0, int64_t(n)));
    const int nh = min(H, a.group - h0);
    const int T = a.lens[r];
    const UnitMap map = unit_map(a, T);

    // q rows of the unit, in 32 bits
    __syncthreads();
    for (int i = tid; i < H * P; i += kThreads) {
      const int hh = i / P, d = i % P;
      float x = 0.f;
      if (hh < nh && d < a.dim) {
        const int64_t o = r * a.q_req + (int64_t(h) * a.group + h0 + hh) * a.q_head + d;
        x = kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[o])
                  : static_cast<const float*>(a.q)[o];
      }
      qs[i] = x;
    }
    __syncthreads();

    // each head scaled by a power of two to a largest value in [2^14, 2^15)
    uint32_t qf[NT][P / 16][2];
    float fac[NT];
    State<P, NT> st;
    st.e = 120;
    {
      const int t = lane >> 2, c = lane & 3;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        // column t of the tile: head t / 2 of it, its hi (even) or lo part; this lane's factor
        // is that of head c
        float top[4];
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
          float x = 0.f;
          for (int d = lane; d < P; d += 32) x = fmaxf(x, fabsf(qs[(i * 4 + hh) * P + d]));
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          top[hh] = x;
        }
        int ex[4];
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) ex[hh] = top[hh] > 0.f ? 14 - exponent(top[hh]) : 0;
        const int et = (t >> 1) == 0 ? ex[0] : (t >> 1) == 1 ? ex[1] : (t >> 1) == 2 ? ex[2] : ex[3];
        const int ec = c == 0 ? ex[0] : c == 1 ? ex[1] : c == 2 ? ex[2] : ex[3];
        // (two factors: 2^ec alone can leave the range of a float)
        const float up0 = pow2(et / 2), up1 = pow2(et - et / 2);
        const float* row = qs + (i * 4 + (t >> 1)) * P;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              // nibbles 2 ks + b and + 4 of the word
              const int d = 32 * g + 8 * c + 2 * ks + b;
              const float x0 = row[d] * up0 * up1, x1 = row[d + 4] * up0 * up1;
              const float h0f = __half2float(__float2half_rn(x0));
              const float h1f = __half2float(__float2half_rn(x1));
              qf[i][2 * g + ks][b] = (t & 1) ? pack_half2(x0 - h0f, x1 - h1f) : pack_half2(h0f, h1f);
            }
        fac[i] = a.scale * kLog2e * pow2((9 - ec) / 2) * pow2((9 - ec) - (9 - ec) / 2);
        st.m[i] = -INFINITY;
        st.l[i] = 0.f;
#pragma unroll
        for (int b = 0; b < 2 * G; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) st.acc[i][b][j] = 0.f;
      }
    }

    // the warp's strips: lane i of a round finds the i-th of them
    for (int v = v0 + warp; v < v1; v += 32 * kWarps) {
      const int mine = v + lane * kWarps;
      int ra = 0, rb = 0;
      const uint8_t* p = a.pool;
      if (mine < v1) p = locate(a, map, r, h, mine, SB, &ra, &rb);
      const int count = min(32, (v1 - v + kWarps - 1) / kWarps);
      for (int i = 0; i < count; ++i) {
        const uint8_t* strip = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), i));
        const int lo = __shfl_sync(0xffffffffu, ra, i), hi = __shfl_sync(0xffffffffu, rb, i);
        if (hi == 0) continue;
        Frag<P> f;
        load_frag<P>(strip, lane, f);
        strip_step<P, NT>(f, lo == 0 && hi == kStrip, lo, hi, qf, fac, st);
      }
    }

    // warp states to shared memory
    {
      const int t = lane >> 2, c = lane & 3;
      const float down = pow2(-st.e);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float l = st.l[i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float* s = slots + warp * SLOT + (i * 4 + c) * (P + 2);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float* d0 = st.acc[i][2 * g];
          const float* d1 = st.acc[i][2 * g + 1];
          float* o = s + 32 * g + 4 * t;
          o[0] = (d0[0] + d0[1]) * 0x1p9f * down;
          o[1] = (d0[2] + d0[3]) * 0x1p9f * down;
          o[2] = (d1[0] + d1[1]) * 0x1p9f * down;
          o[3] = (d1[2] + d1[3]) * 0x1p9f * down;
        }
        if (t == 0) {
          s[P] = st.m[i];
          s[P + 1] = l;
        }
      }
    }
    __syncthreads();

    const bool whole = v0 == 0 && v1 == n;
    const int64_t ostride = int64_t(a.heads) * a.group;
    const int64_t orow = r * ostride + int64_t(h) * a.group + h0;
    float* part = a.parts + (int64_t(blockIdx.x) * 2 + (at == begin ? 0 : 1)) * SLOT;
    for (int i = tid; i < nh * P; i += kThreads) {
      const int hh = i / P, d = i % P;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, slots[w * SLOT + hh * (P + 2) + P]);
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* s = slots + w * SLOT + hh * (P + 2);
        const float f = s[P] == m ? 1.f : ex2(s[P] - m);
        l += f * s[P + 1];
        o += f * s[d];
      }
      if (whole) {
        if (d < a.dim) a.out[(orow + hh) * a.dim + d] = l == 0.f ? 0.f : o / l;
        if (d == 0 && a.lse != nullptr) a.lse[orow + hh] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
      } else {
        float* s = part + hh * (P + 2);
        s[d] = o;
        if (d == 0) {
          s[P] = m;
          s[P + 1] = l;
        }
      }
    }
    if (!whole) {
      // the unit's CTAs: i0 holds its first strip, i1 its last
      const int64_t i0 = u0 / chunk, i1 = (u0 + n - 1) / chunk;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        uint32_t* ticket = a.tickets + int64_t(r) * units + u;
        uint32_t old;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(old) : "l"(ticket) : "memory");
        s_last = old == static_cast<uint32_t>(i1 - i0);
        if (s_last) *ticket = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int i = tid; i < nh * P; i += kThreads) {
          const int hh = i / P, d = i % P;
          float m = -INFINITY, l = 0.f, o = 0.f;
          for (int64_t c = i0; c <= i1; ++c) {
            const float* s = a.parts + (c * 2 + (chunk * c >= u0 ? 0 : 1)) * SLOT + hh * (P + 2);
            const float pm = __ldcg(s + P), pl = __ldcg(s + P + 1), po = __ldcg(s + d);
            const float nm = fmaxf(m, pm);
            const float fo = m == nm ? 1.f : ex2(m - nm), fp = pm == nm ? 1.f : ex2(pm - nm);
            l = l * fo + pl * fp;
            o = o * fo + po * fp;
            m = nm;
          }
          if (d < a.dim) a.out[(orow + hh) * a.dim + d] = l == 0.f ? 0.f : o / l;
          if (d == 0 && a.lse != nullptr)
            a.lse[orow + hh] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
        }
      }
    }
    at = u0 + v1;
  }
}

// Column tiles: groups of up to four q heads fill one, larger ones take two.
int column_tiles(const rba_paged* s) { return s->d.n_q_heads / s->d.n_kv_heads <= 4 ? 1 : 2; }
int grid_of(int nt) { return num_sms() * (nt == 1 ? 2 : 1); }
size_t ticket_bytes(const rba_paged* s) {
  const int h = 4 * column_tiles(s), group = s->d.n_q_heads / s->d.n_kv_heads;
  return align_up(size_t(s->d.max_requests) * s->d.n_kv_heads * ((group + h - 1) / h) * 4, 256);
}

}  // namespace
}  // namespace rba

extern "C" size_t rba_paged_attend_workspace_size(const rba_paged* s) {
  using namespace rba;
  if (s == nullptr) return 0;
  const int nt = column_tiles(s);
  return ticket_bytes(s) + size_t(grid_of(nt)) * 2 * 4 * nt * (s->pitch + 2) * sizeof(float);
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
  const int group = s->d.n_q_heads / s->d.n_kv_heads, nt = column_tiles(s);
  // the line of strips of one head chunk is counted in 32 bits
  if (int64_t(n_requests) * s->d.max_pages * s->strips > INT32_MAX / 2) return RBA_ERR_UNSUPPORTED;
  AttendArgs a = {};
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
  a.group = group;
  a.dim = s->d.head_dim;
  a.bs = s->d.page_size;
  a.strips = s->strips;
  a.max_pages = s->d.max_pages;
  a.n_pages = s->d.n_pages;
  a.k = k;
  a.sink = sink;
  a.window = window;
  a.chunks = (group + 4 * nt - 1) / (4 * nt);
#define RBA_ATTEND(P_, NT_, B_)                                                              \
  do {                                                                                       \
    const size_t smem = Smem<P_, NT_>::bytes(n_requests);                                    \
    RBA_CUDA_TRY(                                                                            \
        ensure_smem(reinterpret_cast<const void*>(paged_attend_kernel<P_, NT_, B_>), smem)); \
    paged_attend_kernel<P_, NT_, B_><<<grid_of(NT_), kThreads, smem, stream>>>(a);           \
  } while (0)
#define RBA_ATTEND_T(P_, NT_)                          \
  do {                                                 \
    if (s->d.dtype == RBA_BF16) RBA_ATTEND(P_, NT_, true); \
    else RBA_ATTEND(P_, NT_, false);                   \
  } while (0)
  if (s->pitch == 128) {
    if (nt == 1) RBA_ATTEND_T(128, 1);
    else RBA_ATTEND_T(128, 2);
  } else {
    if (nt == 1) RBA_ATTEND_T(64, 1);
    else RBA_ATTEND_T(64, 2);
  }
#undef RBA_ATTEND_T
#undef RBA_ATTEND
  RBA_LAUNCH_CHECK();
  return RBA_OK;
}
