// Decode attention over the paged 3-bit cache: the arithmetic on one block
// (page, cache head) by one warp, for a group of query rows. The walk over the
// pages is paged_attn.cu's.
#pragma once
#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace blt {
namespace paged {

constexpr int kStageRows4 = 3;  // 4-bit rows of a page that travel with it; pools with more are read from global memory

// A piece: [cols][D] value sums, then [cols] maxima, then [cols] sums.
__host__ __device__ constexpr int piece_floats(int D, int cols) { return cols * (D + 2); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ int cut_len(const AttnArgs& a, int b, bool* bad) {
  const int64_t cap = static_cast<int64_t>(a.n_shared + a.W) * PT;
  const int len = __ldg(a.lens + b);
  *bad = len < 0 || len > cap;
  return len < 0 ? 0 : len > cap ? static_cast<int>(cap) : len;
}
__device__ __forceinline__ int own_pages(const AttnArgs& a, int b) {
  bool bad;
  return max(0, pages_of(cut_len(a, b, &bad)) - a.n_shared);
}
// What beginning and ending a segment costs, in pages. Measured with 2 columns (digits, flush): 64 ragged
// sequences of up to 4096 tokens take 116 us with 0, 96 with 2, 92 with 3, 96 with 4.
__host__ __device__ constexpr int segment_overhead(int cols) { return cols == 2 ? 3 : 1; }

// A segment: the pages of one (sequence, cache head) for one group of its rows.
struct Segment {
  int tok0;   // first query token (of B Sq) of its rows
  int r0;     // first row of the group
  int rows;   // of the (sequence, head)
  int h, G;   // cache head, query heads to a cache head
  bool front; // the shared pages (all sequences' rows), or a sequence's own
};

__device__ __forceinline__ const uint16_t* query_row(const AttnArgs& a, const Segment& s, int r) {
  return a.q + (s.tok0 + r / s.G) * a.ldq + static_cast<int64_t>(s.h * s.G + r % s.G) * a.D;
}

__device__ __forceinline__ uint16_t* output_row(const AttnArgs& a, const Segment& s, int r) {
  return a.out + (static_cast<int64_t>(s.tok0 + r / s.G) * a.Hq + s.h * s.G + r % s.G) * a.D;
}

// Tokens that row r sees, from the segment's first page on; a row that is none: all, so that nothing is masked for it.
__device__ __forceinline__ int row_sees(const AttnArgs& a, const Segment& s, int r) {
  if (r >= s.rows) return 0x7FFFFFFF;
  const int tok = s.tok0 + r / s.G;
  bool bad;
  const int len = cut_len(a, tok / a.Sq, &bad);
  if (bad && s.front) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
  const int sees = max(0, len - a.Sq + 1 + tok % a.Sq);
  return s.front ? sees : max(0, sees - PT * a.n_shared);
}

// ----------------------------------------------------------------- operands
// A 3-bit code c at bit j <= 7 of a 16-bit half, the other bits cleared, IS the
// fp16 subnormal c 2^(j - 24); one paired fma makes (c - 4) 2^(j - 9) of it,
// exact and normal. Two codes 16 bits apart (give or take what keeps both in
// the halves' low 10 bits) are so one operand register of the m16n8k16 fp16
// MMA, for a mask, an fma and a share of a shift. The 2^j go into the queries
// (a power of two: exact) for K, and leave at the end for V.
// Without the fma (the subnormals as operands, the offset of 4 taken off the
// sums) it would be 256 of 1000 instructions a page less, but the MMA lines its
// products up by the operands' exponents, where all subnormals have 2^-14:
// with small j, 8 bits of its sums were lost.

// A lane's 32 codes (96 bits) in 16 pairs, 16 codes (48 bits) in 8: the pair's
// codes and the stream bit that lands at bit 0. Found by search: the fewest
// windows that are no word of the stream (4 of 7).
struct Pair { int lo, hi, n; };
__host__ __device__ constexpr Pair pair32(int p) {
  constexpr Pair t[16] = {{0, 6, 0}, {1, 7, 0}, {2, 8, 4}, {3, 9, 4}, {4, 10, 10}, {5, 11, 10}, {12, 17, 32}, {13, 18, 32},
                          {14, 19, 41}, {15, 20, 41}, {16, 21, 41}, {22, 27, 64}, {23, 28, 64}, {24, 29, 71}, {25, 30, 71}, {26, 31, 71}};
  return t[p];
}
__host__ __device__ constexpr Pair pair16(int p) {
  constexpr Pair t[8] = {{0, 3, -7}, {1, 4, -4}, {2, 7, 0}, {5, 11, 13}, {6, 12, 13}, {8, 13, 23}, {9, 14, 23}, {10, 15, 23}};
  return t[p];
}
template <int D>
__host__ __device__ constexpr Pair k_pair(int p) { return D == 64 ? pair16(p) : pair32(p & 15); }

// 32 bits of the stream X from bit n on
template <int NW>
__device__ __forceinline__ uint32_t window(const uint32_t (&X)[NW], int n) {
  if (n < 0) return X[0] << (-n);
  if ((n & 31) == 0) return X[n >> 5];
  return (n >> 5) + 1 < NW ? __funnelshift_r(X[n >> 5], X[(n >> 5) + 1], n & 31) : X[n >> 5] >> (n & 31);
}

// fp16 c 2^(j - 24) -> (c - 4) 2^(j - 9) in both halves
__device__ __forceinline__ uint32_t less4(uint32_t x, int jl, int jh) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0x78007800u), "r"(0x80008000u | (jl + 8) << 10 | (jh + 8) << 26));
  return r;
}

template <int NW>
__device__ __forceinline__ uint32_t k_operand(const uint32_t (&X)[NW], Pair p) {
  const int jl = 3 * p.lo - p.n, jh = 3 * p.hi - p.n;
  return less4(window(X, p.n) & ((7u << jl) | (7u << jh)), jl, jh - 16);
}

// bit of code e (0..7) in its 16-bit half as v_pair leaves it
__host__ __device__ constexpr int v_bit(int e) { return e == 0 ? 0 : e == 1 ? 3 : e == 2 ? 6 : e == 3 ? 1 : e == 4 ? 4 : e == 5 ? 7 : e == 6 ? 2 : 5; }

// Code e of 8 consecutive dimensions for 4 tokens; w[i] holds byte i of the 4
// tokens' three bytes, x[i] = w[i] >> 8. r0: tokens 0 and 2, r1: tokens 1 and 3,
// as fp16 (c - 4) 2^(v_bit - 9).
template <int E>
__device__ __forceinline__ void v_operand(const uint32_t (&w)[3], const uint32_t (&x)[3], uint32_t& r0, uint32_t& r1) {
  constexpr int B = 3 * E / 8, j = v_bit(E);
  constexpr uint32_t full = 0x00070007u << j;
  if constexpr (E == 2 || E == 5) {  // the code's upper bits are the next byte's lowest
    constexpr uint32_t up = E == 2 ? 0x01000100u : 0x03000300u, low = full & 0x00FF00FFu;
    r0 = (w[B] & low) | ((w[B + 1] << 8) & up);
    r1 = (x[B] & low) | (w[B + 1] & up);
  } else {
    r0 = w[B] & full;
    r1 = x[B] & full;
  }
  r0 = less4(r0, j, j);
  r1 = less4(r1, j, j);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// a number's upper 11 bits, which are an fp16 number where it is no smaller than 2^-14
__device__ __forceinline__ float f16_top(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// What weights p = 2^(score - reference) are taken relative to, for a largest score: not below it (p <= 1), and 8 above
// it, so that scores a little larger do not move it. Far out, where 8 would be lost, the score itself.
__device__ __forceinline__ float reference(float score) { return fabsf(score) < 1048576.f ? ceilf(score) + 8.f : score; }
// The exponent e for a largest weight w = p x (V scale): w 2^-e lies in [2^7, 2^8). It grows with w, to kMostWeight;
// weights that are next to nothing beside p (2^-100) need none of their own.
constexpr float kLeastExp = -100.f, kMostWeight = 32768.f;
__device__ __forceinline__ float weight_exp(float w) { return fmaxf(static_cast<float>((__float_as_int(w) >> 23) - 134), kLeastExp); }

// The page's tokens kept at 4 bits among its first `most`, a bit each.
__device__ __forceinline__ uint64_t tokens4(const float* ksc, int most) {
  const int lane = threadIdx.x & 31;
  const uint32_t lo = __ballot_sync(0xFFFFFFFFu, lane < most && signbit(ksc[lane]));
  const uint32_t hi = __ballot_sync(0xFFFFFFFFu, lane + 32 < most && signbit(ksc[lane + 32]));
  return static_cast<uint64_t>(hi) << 32 | lo;
}
// 2^(e - 127) of a biased exponent 1..254
__device__ __forceinline__ float pow2_biased(int e) { return __int_as_float(e << 23); }

// ------------------------------------------------- up to 4 or 8 rows, fp16
// Tokens are the rows of the scores' product (K codes x queries) and the
// contracted index of the values' (V codes^T x weights); query rows are the 8
// columns of both. QC: columns of a lane that are queries: 1: 4 rows a group
// (columns 2 q and 2 q + 1 are both row q, of which one is kept: half the
// softmax), 2: 8. A weight goes into the value product as two fp16 numbers, its
// upper 11 bits and what is left of it, so that 2^-22 of it is lost. (With one number,
// 2^-11, the outputs of 8 sequences behind 4096 tokens were 8e-4 from those of 32-bit
// weights, now 5e-5; 8 rows of 64 sequences of up to 4096 tokens 135 us -> 151.)
// The second part of 4 rows lies in the columns that would be empty, that of 8
// takes products of its own.
// Two references a row: weights of the sum are relative to 2^m_run, a bound of
// the scores so far; those of the values, p x (V scale), are besides relative to
// 2^w_exp, which follows the largest of THEM: the largest V scale may be that of a
// token without weight. The largest is 2^7 to 2^15, so what is lost of the others
// for want of exponents (2^-24) is 2^-31 of it or less. References move when a
// score or a weight outgrows them, for which no lane needs the others' on most pages.
template <int D, int QC>
struct F16Page {
  static constexpr int COLS = 4 * QC;
  static constexpr int RB = row_bytes(D), NB = D / 64 * 4;  // NB: MMAs of a score
  static constexpr int LD = D / 8;                          // dimensions of a lane in the value product
  static constexpr int NM = D / 16;                         // and its MMAs
  static constexpr int KW = D == 64 ? 2 : 3;                // stream words of a lane's chunk

  uint32_t qb[2 * NB];   // query operands: pair i of this lane's chunk of column g
  float kq[QC];          // what makes of (sum) x (K scale) x c0 a score in base 2: a power of two, so that the
                         // largest score is exactly what its weight's exponent has taken off
  float c0;
  int sees[QC], n_all;   // tokens that the lane's columns see; pages before n_all are seen whole by all columns
  const uint16_t* qrow[QC];
  float m_run[QC], l_run[QC], w_exp[QC], acc[NM][4];  // acc: value sums / 2^(m_run + w_exp)

  __device__ __forceinline__ void begin(const AttnArgs& a, const Segment& sg, float*) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    {
      const int rq = sg.r0 + (QC == 1 ? g >> 1 : g);
      uint32_t x[D / 8];  // D / 4 dimensions of the row
#pragma unroll
      for (int i = 0; i < D / 8; ++i) x[i] = 0u;
      if (rq < sg.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(query_row(a, sg, rq)) + D / 32 * t4;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = __ldg(src + i);
          x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
      }
      uint32_t am = 0u;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) am = max(am, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      // the row's largest value goes to [2^14, 2^15): what is 2^-25 of it or more is exact in fp16
      const int fb = min(268 - max(1, static_cast<int>(am >> 7)), 254);
      const float f = pow2_biased(fb);
      auto qf = [&](int d) { return __uint_as_float((d & 1) ? (x[d >> 1] & 0xFFFF0000u) : (x[d >> 1] << 16)) * f; };
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) {
        const Pair pr = k_pair<D>(i);
        const int d0 = D == 64 ? 0 : 32 * (i >> 4);
        const int jl = 3 * pr.lo - pr.n, jh = 3 * pr.hi - pr.n - 16;
        qb[i] = pack_f16x2(qf(d0 + pr.lo) * (1.f / (1 << jl)), qf(d0 + pr.hi) * (1.f / (1 << jh)));
      }
      c0 = a.qk_scale * 1.4426950408889634f;
      const float kr = pow2_biased(263 - fb);  // 2^(9 + 127 - fb)
#pragma unroll
      for (int c = 0; c < QC; ++c) {
        const int src = QC == 1 ? 8 * t4 : 4 * (2 * t4 + c);  // a lane of the column's row
        kq[c] = __shfl_sync(0xFFFFFFFFu, kr, src);
        const int r = sg.r0 + (QC == 1 ? t4 : 2 * t4 + c);
        sees[c] = row_sees(a, sg, r);
        qrow[c] = r < sg.rows ? query_row(a, sg, r) : nullptr;
      }
    }
#pragma unroll
    for (int c = 0; c < QC; ++c) { m_run[c] = -INFINITY; l_run[c] = 0.f; w_exp[c] = kLeastExp; }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    n_all = sees[0];
    if constexpr (QC == 2) n_all = min(n_all, sees[QC - 1]);
    n_all = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<unsigned>(n_all)) / PT);
  }

  // A score in base 2 above m_run: takes the sum along; returns the factor of the value sums.
  __device__ __forceinline__ float more_score(int q, float score) {
    if (!(score > m_run[q])) return 1.f;
    const float m = reference(score), d = m_run[q] - m;
    l_run[q] *= ex2(d);
    m_run[q] = m;
    w_exp[q] += d;  // the value sums stay as they are
    if (w_exp[q] >= kLeastExp) return 1.f;
    const float f = ex2(w_exp[q] - kLeastExp);
    w_exp[q] = kLeastExp;
    return f;
  }
  // The same for a weight p x (V scale) that 2^w_exp does not hold.
  __device__ __forceinline__ float more_weight(int q, float w) {
    const float e = weight_exp(w);
    if (!(e > w_exp[q])) return 1.f;
    const float f = ex2(w_exp[q] - e);
    w_exp[q] = e;
    return f;
  }
  __device__ __forceinline__ void scale_values(int q, float f) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (QC == 1 || (i & 1) == q) acc[m][i] *= f;
  }

  // page number j of the segment; c4_bytes: of the page's 4-bit rows behind the block (0: none, or in global memory)
  __device__ __forceinline__ void page(const AttnArgs& a, const Segment& sg, const uint8_t* blk, int page, int j, int c4_bytes) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const float* ksc = reinterpret_cast<const float*>(blk + off_ks(D));
    const float* vsc = reinterpret_cast<const float*>(blk + off_vs(D));
    // ---- scores; C row g is token 16 u + 2 g, row g + 8 the one after it
    float s[4][2][QC], vs[4][2];
    uint32_t sign = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint8_t* row = blk + (16 * u + 2 * g) * RB;
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < (D == 256 ? 2 : 1); ++h) {
        uint32_t X[2][KW];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (D == 64) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(row + r * RB) + ((3 * t4) >> 1);
            const int sh = 16 * (t4 & 1);
            X[r][0] = __funnelshift_r(w[0], w[1], sh);
            X[r][1] = w[1] >> sh;
          } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(row + r * RB) + 3 * (D == 256 ? 2 * t4 + h : t4);
#pragma unroll
            for (int i = 0; i < 3; ++i) X[r][i] = w[i];
          }
        }
        constexpr int NH = D == 64 ? 4 : 8;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          const Pair x = k_pair<D>(2 * i), y = k_pair<D>(2 * i + 1);
          mma_f16(c, k_operand(X[0], x), k_operand(X[1], x), k_operand(X[0], y), k_operand(X[1], y),
                  qb[16 * h + 2 * i], qb[16 * h + 2 * i + 1]);
        }
      }
      const float2 ks = *reinterpret_cast<const float2*>(ksc + 16 * u + 2 * g);
      const float2 v2 = *reinterpret_cast<const float2*>(vsc + 16 * u + 2 * g);
      vs[u][0] = v2.x;
      vs[u][1] = v2.y;
      sign |= __float_as_uint(ks.x) | __float_as_uint(ks.y);
#pragma unroll
      for (int q = 0; q < QC; ++q) {
        s[u][0][q] = c[q] * (ks.x * c0);
        s[u][1][q] = c[2 + q] * (ks.y * c0);
      }
    }
    const bool part = j >= n_all, has4 = __any_sync(0xFFFFFFFFu, sign >> 31);
    int lim[QC], most = PT;
#pragma unroll
    for (int c = 0; c < QC; ++c) lim[c] = PT;
    if (part) {
      most = 0;
#pragma unroll
      for (int c = 0; c < QC; ++c) {
        lim[c] = max(0, min(PT, sees[c] - j * PT));
        if (qrow[c] != nullptr) most = max(most, lim[c]);
      }
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int o = 16 * u + 2 * g + r;
#pragma unroll
          for (int q = 0; q < QC; ++q)
            if (o >= lim[q]) s[u][r][q] = -INFINITY;
          if (o >= most) vs[u][r] = 0.f;  // not a token: whatever is there
        }
    }
    if (has4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 ks = *reinterpret_cast<const float2*>(ksc + 16 * u + 2 * g);
#pragma unroll
        for (int q = 0; q < QC; ++q) {
          if (signbit(ks.x)) s[u][0][q] = -INFINITY;
          if (signbit(ks.y)) s[u][1][q] = -INFINITY;
        }
      }
    }
    // ---- references, in base 2
    float vm = vs[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) vm = fmaxf(vm, vs[i >> 1][i & 1]);
    float mt[QC];
    bool more = false;
#pragma unroll
    for (int q = 0; q < QC; ++q) {
      mt[q] = s[0][0][q];
#pragma unroll
      for (int i = 1; i < 8; ++i) mt[q] = fmaxf(mt[q], s[i >> 1][i & 1][q]);
      mt[q] *= kq[q];  // (exact)
      more = more || mt[q] > m_run[q] || (mt[q] > -INFINITY && !(ex2(mt[q] - m_run[q]) * vm * ex2(-w_exp[q]) < kMostWeight));
    }
    if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
      for (int q = 0; q < QC; ++q) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mt[q] = fmaxf(mt[q], __shfl_xor_sync(0xFFFFFFFFu, mt[q], o));
        float f = more_score(q, mt[q]), top = 0.f;
        const float mr = m_run[q] == -INFINITY ? 0.f : m_run[q];
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, ex2(fmaf(s[i >> 1][i & 1][q], kq[q], -mr)) * vs[i >> 1][i & 1]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        f *= more_weight(q, top);
        scale_values(q, f);
      }
    }
    float mr[QC], wf[QC];
#pragma unroll
    for (int q = 0; q < QC; ++q) {
      mr[q] = m_run[q] == -INFINITY ? 0.f : m_run[q];
      wf[q] = ex2(-w_exp[q]);
    }
    // ---- weights and values; B's token 2 t4 (+ 1) of rows 0..7 is token 4 t4 (+ 2)
    // of the 16, of rows 8..15 token 4 t4 + 1 (+ 2): the lane's words of 4 tokens
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t b[QC][2];  // 8 rows: the weights' upper parts, then the lower ones
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = ex2(fmaf(s[u][r][0], kq[0], -mr[0]));
        l_run[0] += p0;
        const float w0 = p0 * vs[u][r] * wf[0], h0 = f16_top(w0);
        if constexpr (QC == 1) {
          b[0][r] = transpose8x8(pack_f16x2(h0, w0 - h0));
        } else {
          const float p1 = ex2(fmaf(s[u][r][QC - 1], kq[QC - 1], -mr[QC - 1]));
          l_run[QC - 1] += p1;
          const float w1 = p1 * vs[u][r] * wf[QC - 1], h1 = f16_top(w1);
          b[0][r] = transpose8x8(pack_f16x2(h0, h1));
          b[QC - 1][r] = transpose8x8(pack_f16x2(w0 - h0, w1 - h1));
        }
      }
      const uint8_t* vw = blk + off_v(D) + (4 * u + t4) * 4 * RB + 4 * (3 * LD / 8) * g;
      uint32_t vc[LD / 8][3];
      if constexpr (D == 64) {
#pragma unroll
        for (int i = 0; i < 3; ++i) vc[0][i] = reinterpret_cast<const uint32_t*>(vw)[i];
      } else if constexpr (D == 128) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint2 x = reinterpret_cast<const uint2*>(vw)[i];
          vc[(2 * i) / 3][(2 * i) % 3] = x.x;
          vc[(2 * i + 1) / 3][(2 * i + 1) % 3] = x.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint4 x = reinterpret_cast<const uint4*>(vw)[i];
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) vc[(4 * i + c) / 3][(4 * i + c) % 3] = y[c];
        }
      }
#define BLT_V(E_)                                                                    \
      {                                                                        \
        uint32_t x0, x1, y0, y1;                                               \
        v_operand<E_>(vc[i], x, x0, x1);                                       \
        v_operand<E_ + 1>(vc[i], x, y0, y1);                                   \
        mma_f16(acc[4 * i + E_ / 2], x0, y0, x1, y1, b[0][0], b[0][1]);        \
        if constexpr (QC == 2) mma_f16(acc[4 * i + E_ / 2], x0, y0, x1, y1, b[QC - 1][0], b[QC - 1][1]); \
      }
#pragma unroll
      for (int i = 0; i < LD / 8; ++i) {
        const uint32_t x[3] = {vc[i][0] >> 8, vc[i][1] >> 8, vc[i][2] >> 8};
        BLT_V(0) BLT_V(2) BLT_V(4) BLT_V(6)
      }
#undef BLT_V
    }
    // ---- the page's 4-bit tokens, one after the other: lane (g, t4) has dimensions
    // LD g .. LD g + LD - 1 of the rows and its columns' queries
    if (has4) {
      const int C4 = a.C4;
      for (uint64_t set = tokens4(ksc, most); set; set &= set - 1) {
        const int o = __ffsll(static_cast<long long>(set)) - 1;
        const int j4 = blk[o * RB];
        if (j4 >= C4) {
          if (lane == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
          continue;
        }
        const uint8_t* r4 = c4_bytes ? blk + block_bytes(D) + j4 * D
                                     : a.codes4 + ((static_cast<int64_t>(page) * a.H + sg.h) * C4 + j4) * D;
        uint32_t kc[LD / 8], vc[LD / 8];
#pragma unroll
        for (int c = 0; c < LD / 8; ++c) {
          kc[c] = reinterpret_cast<const uint32_t*>(r4 + LD / 2 * g)[c];
          vc[c] = reinterpret_cast<const uint32_t*>(r4 + D / 2 + LD / 2 * g)[c];
        }
        const float k4 = fabsf(ksc[o]) * c0, v4 = vsc[o];
        float sc[QC];
        bool more = false;
#pragma unroll
        for (int q = 0; q < QC; ++q) {
          float dot = 0.f;
          if (qrow[q] != nullptr) {
#pragma unroll
            for (int c = 0; c < LD / 8; ++c) {
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(qrow[q] + LD * g) + c);
              const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int d = 0; d < 8; ++d)
                dot = fmaf(__uint_as_float((d & 1) ? (y[d >> 1] & 0xFFFF0000u) : (y[d >> 1] << 16)),
                           static_cast<float>(static_cast<int>((kc[c] >> (4 * d)) & 15u) - 8), dot);
            }
          }
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
          sc[q] = o < lim[q] ? dot * k4 : -INFINITY;
          more = more || sc[q] > m_run[q] || !(v4 * ex2(-w_exp[q]) < 0x1p60f);  // (its weight is not rounded to fewer bits)
        }
        if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
          for (int q = 0; q < QC; ++q) {
            const float f = more_score(q, sc[q]);
            scale_values(q, f * more_weight(q, sc[q] == -INFINITY ? 0.f : ex2(sc[q] - m_run[q]) * v4));
          }
        }
#pragma unroll
        for (int q = 0; q < QC; ++q) {
          const float pe = sc[q] == -INFINITY ? 0.f : ex2(sc[q] - m_run[q]);
          if (g == 0) l_run[q] += pe;
          const float v = pe * v4 * ex2(-w_exp[q]) * (1.f / 512.f);
#pragma unroll
          for (int d = 0; d < LD; ++d) {
            const float x = static_cast<float>(static_cast<int>((vc[d >> 3] >> (4 * (d & 7))) & 15u) - 8) *
                            static_cast<float>(1 << v_bit(d & 7));
            float& y = acc[d >> 1][2 * (d & 1) + q];
            y = fmaf(v, x, y);
          }
        }
      }
    }
  }

  // The piece, or the rows themselves.
  __device__ __forceinline__ void finish(const AttnArgs& a, const Segment& sg, float* out, bool whole) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int q = 0; q < QC; ++q) {
      const int col = QC == 1 ? t4 : 2 * t4 + q;
      float l = l_run[q];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      if (qrow[q] == nullptr) continue;
      const float vf = ex2(w_exp[q]) * (!whole ? 1.f : l > 0.f ? 1.f / l : 0.f);
      uint16_t* row = output_row(a, sg, sg.r0 + col) + LD * g;
#pragma unroll
      for (int c = 0; c < LD / 4; ++c) {
        float x[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int dl = 4 * c + d, at = 2 * (dl & 1);
          x[d] = (QC == 1 ? acc[dl >> 1][at] + acc[dl >> 1][at + 1] : acc[dl >> 1][at + q]) *
                 (512.f / static_cast<float>(1 << v_bit(dl & 7))) * vf;
        }
        if (whole) reinterpret_cast<uint2*>(row)[c] = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        else reinterpret_cast<float4*>(out + col * D + LD * g)[c] = make_float4(x[0], x[1], x[2], x[3]);
      }
      if (!whole && g == 0) {
        out[COLS * D + col] = m_run[q];
        out[COLS * D + COLS + col] = l;
      }
    }
  }
};

// ------------------------------------------------- up to 2 rows, integers
// One or two rows leave most of an fp16 MMA's columns empty, and a page costs
// what taking its codes apart costs. In 8-bit integers that is a mask alone:
// a byte with all bits but those of one code (or of the part of a code that
// lies in this byte) cleared is an unsigned operand, 4 bytes a register:
//   byte 0 of 3: bits 0-2 code 0 | 3-5 code 1 | 6-7 low bits of code 2
//   byte 1:      bit 0 high bit of code 2 | 1-3 code 3 | 4-6 code 4 | 7 low bit of code 5
//   byte 2:      bits 0-1 high bits of code 5 | 2-4 code 6 | 5-7 code 7
// 10 fields for 8 codes; a field's place and the part's weight in its code are
// powers of two that go into the queries (K: the contracted index is the
// dimension) or are taken out of the whole numbers at the end (V: the rows of
// the product are the fields). The other operands are 32-bit fixed-point
// numbers in 4 digits of 8 bits, a column each: 8 columns are 2 rows.
//   * queries: a field at bit b takes q 2^-b as a whole number, with the row's largest q
//     in [2^27, 2^28): 2^(b - 1) is lost, 2^-25 of the largest or less at bits 0 to 3,
//     2^-21 at bit 7 (the lowest bit of code 5);
//   * weights p x (V scale): whole numbers below 2^32, 2^32 being 4 to 8 times
//     the largest so far: sums of codes x weights are exact, zeros add zero.
// When a weight outgrows that, or the score by 2^20 the one that weights are
// relative to, the sums so far are added to the piece in global memory as
// floats, and new ones begin (once or twice a segment).
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_u8u8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The field that K operand kind k (0, 1: of the word as it is, 2: of the word >> 4,
// 3: bit 7 of byte 1) takes from a byte of type b % 3: code of the 8, lowest bit, bits, weight 2^up in the code.
struct Field { int code, bit, bits, up; };
__host__ __device__ constexpr Field k_field(int type, int k) {
  constexpr Field t[3][4] = {{{0, 0, 3, 0}, {1, 3, 3, 0}, {2, 2, 2, 0}, {0, 0, 0, 0}},
                             {{2, 0, 1, 2}, {3, 1, 3, 0}, {4, 0, 3, 0}, {5, 7, 1, 0}},
                             {{5, 0, 2, 1}, {6, 2, 3, 0}, {7, 1, 3, 0}, {0, 0, 0, 0}}};
  return t[type][k];
}
__host__ __device__ constexpr uint32_t field_mask(Field f) { return ((1u << f.bits) - 1u) << f.bit; }
// of kind k in word i of a chunk of n bytes
__host__ __device__ constexpr uint32_t k_mask(int i, int k, int n) {
  uint32_t m = 0u;
  for (int p = 0; p < 4; ++p)
    if (4 * i + p < n) m |= field_mask(k_field((4 * i + p) % 3, k)) << (8 * p);
  return m;
}

template <int D, bool FOUR>
struct I8Page {
  static constexpr int COLS = 2;
  static constexpr int RB = row_bytes(D), LD = D / 8;
  static constexpr int NC = D == 256 ? 2 : 1;            // chunks of a lane in a K row
  static constexpr int KW = D == 64 ? 2 : 3;             // words of a chunk
  static constexpr int CB = D == 64 ? 6 : 12;            // its bytes
  static constexpr int NK = D == 64 ? 8 : 10;            // and operands (D = 64: 7, one of them nothing)
  static constexpr int NF = 5 * (D / 64);                // MMAs of the value product: 10 fields a unit of 8 dimensions, 2 each
  static constexpr int kFlushPages = 512;                // 64 tokens x 255 x 224 a page: below 2^31

  uint32_t qb[NC * NK];
  float kq, f_mul, f_add;  // row t4 / 2: sums -> score / K scale / kq: digits 0, 1 (t4 even) and 2, 3 meet, less 4 sum q;
                           // kq is a power of two, so that a largest score is exactly what its weight's exponent has taken off
  int sees, n_all;
  const uint16_t* qrow;
  float m_ref, l_run, to_int;  // weights are relative to 2^m_ref, and to_int x as whole numbers
  int acc[NF][4], off[4];
  float o4[FOUR ? LD / 2 : 1];  // 4-bit tokens' part: this lane's half of the dimensions
  uint32_t q4[2][FOUR ? D / 64 : 1];  // and D / 32 dimensions of both rows' queries for their scores
  int held, w_exp;              // pages in acc; biased exponent behind to_int
  bool any;                     // the piece has been written to
  float* piece;

  __device__ __forceinline__ void begin(const AttnArgs& a, const Segment& sg, float* out) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    piece = out;
    {
      const int rq = sg.r0 + (g >> 2), dig = g & 3;
      uint32_t x[D / 8];  // D / 4 dimensions of the row
#pragma unroll
      for (int i = 0; i < D / 8; ++i) x[i] = 0u;
      if (rq < sg.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(query_row(a, sg, rq)) + D / 32 * t4;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = __ldg(src + i);
          x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
      }
      uint32_t am = 0u;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) am = max(am, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      // the row's largest value goes to [2^27, 2^28), 4 times that fits the digits
      const int fb = min(281 - max(1, static_cast<int>(am >> 7)), 253);
      const float f = pow2_biased(fb);
      auto qf = [&](int d) { return __uint_as_float((d & 1) ? (x[d >> 1] & 0xFFFF0000u) : (x[d >> 1] << 16)) * f; };
      float sum = 0.f;
#pragma unroll
      for (int d = 0; d < D / 4; ++d) sum += qf(d);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
#pragma unroll
      for (int i = 0; i < NC * NK; ++i) qb[i] = 0u;
      // a digit of q 2^(up - bit): carries make the lower three digits signed
      auto digit = [&](int d, Field fl) {
        const int v = __float2int_rn(qf(d) * (fl.up == 2 ? 4.f : fl.up == 1 ? 2.f : 1.f / static_cast<float>(1 << fl.bit)));
        const uint32_t y = static_cast<uint32_t>(v) + 0x00808080u;
        return ((y >> (8 * dig)) ^ (dig < 3 ? 0x80u : 0u)) & 255u;
      };
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int b = 0; b < CB; ++b) {  // byte b of the chunk
          const int d0 = D / 4 / NC * c + 8 * (b / 3);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const Field fl = k_field(b % 3, k);
            qb[c * NK + 3 * (b / 4) + k] |= digit(d0 + fl.code, fl) << (8 * (b & 3));
          }
          if (b % 3 == 1) qb[c * NK + 3 * KW] |= digit(d0 + 5, k_field(1, 3)) << (8 * (b & 3));
        }
      // (2^27 of the sums' size is taken off them and put here: they lie below 2^11, and a K scale of up to 2^117 fits)
      const float kr = pow2_biased(281 - fb);
      const int src = 16 * (t4 >> 1);  // a lane of the row's columns
      kq = __shfl_sync(0xFFFFFFFFu, kr, src);
      sum = __shfl_sync(0xFFFFFFFFu, sum, src);
      const float c0 = a.qk_scale * 1.4426950408889634f;
      f_mul = (t4 & 1) ? 0x1p-11f * c0 : 0x1p-27f * c0;
      f_add = (t4 & 1) ? 0.f : -0x1p-25f * c0 * sum;
      const int r = sg.r0 + (t4 >> 1);
      sees = row_sees(a, sg, r);
      qrow = r < sg.rows ? query_row(a, sg, r) : nullptr;
    }
    if constexpr (FOUR) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          q4[r][i] = sg.r0 + r < sg.rows ? __ldg(reinterpret_cast<const uint32_t*>(query_row(a, sg, sg.r0 + r)) + D / 64 * (threadIdx.x & 31) + i) : 0u;
    }
    n_all = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<unsigned>(sees)) / PT);
    m_ref = -INFINITY;
    l_run = 0.f;
    w_exp = 31;
    to_int = pow2_biased(285 - 31);
    held = 0;
    any = false;
    clear();
#pragma unroll
    for (int i = 0; i < (FOUR ? LD / 2 : 1); ++i) o4[i] = 0.f;
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) off[c] = 0;
    held = 0;
  }

  // The sums so far go to the piece, which is then relative to 2^m_new: a lane of
  // the two that have a row's digits writes half of their dimensions.
  // With `row`, the row itself: what there is, times inv.
  __device__ __forceinline__ void flush(float m_new, uint16_t* row = nullptr, float inv = 1.f) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const float f = m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
    const float us = pow2_biased(127 - 16) * pow2_biased(max(w_exp - 15, 1)) * f;  // 2^(w_exp - 158) in two steps
    const float dig = (t4 & 1) ? 65536.f : 1.f;
    float* dst = piece + (t4 >> 1) * D + LD * g + (t4 & 1) * (LD / 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int q = 0; q < LD / 8; ++q) {  // 4 dimensions LD / 2 h + 4 q ..
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int dl = LD / 2 * h + 4 * q + e, i = 5 * (dl >> 3), c = dl & 7;
          float v[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int o = off[n];
            int y;
            if (c == 0) y = acc[i][n];
            else if (c == 1) y = acc[i][2 + n] >> 3;
            else if (c == 2) y = (acc[i + 1][n] >> 6) + (acc[i + 1][2 + n] << 2);
            else if (c == 3) y = acc[i + 2][n] >> 1;
            else if (c == 4) y = acc[i + 2][2 + n] >> 4;
            else if (c == 5) y = (acc[i + 3][n] >> 7) + (acc[i + 3][2 + n] << 1);
            else if (c == 6) y = acc[i + 4][n] >> 2;
            else y = acc[i + 4][2 + n] >> 5;
            v[n] = static_cast<float>(y - o);
          }
          x[e] = fmaf(v[1], 256.f, v[0]) * dig;
          x[e] += __shfl_xor_sync(0xFFFFFFFFu, x[e], 1);
          x[e] *= us;
        }
        if ((t4 & 1) == h && qrow != nullptr) {
          if constexpr (FOUR) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fmaf(o4[4 * q + e], f, x[e]);
          }
          float4* d4 = reinterpret_cast<float4*>(dst) + q;
          if (any) {
            const float4 old = *d4;
            x[0] = fmaf(old.x, f, x[0]); x[1] = fmaf(old.y, f, x[1]);
            x[2] = fmaf(old.z, f, x[2]); x[3] = fmaf(old.w, f, x[3]);
          }
          if (row != nullptr)
            reinterpret_cast<uint2*>(row + LD * g + (t4 & 1) * (LD / 2))[q] =
                make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
          else
            *d4 = make_float4(x[0], x[1], x[2], x[3]);
        }
      }
    }
    if constexpr (FOUR) {
#pragma unroll
      for (int i = 0; i < LD / 2; ++i) o4[i] = 0.f;
    }
    l_run *= f;
    m_ref = m_new;
    any = true;
    clear();
  }

  __device__ __forceinline__ void page(const AttnArgs& a, const Segment& sg, const uint8_t* blk, int page, int j, int c4_bytes) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const float* ksc = reinterpret_cast<const float*>(blk + off_ks(D));
    const float* vsc = reinterpret_cast<const float*>(blk + off_vs(D));
    // ---- scores; C row g is token 16 u + 2 g, row g + 8 the one after it
    float s[4][2], vs[4][2];
    uint32_t sign = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint8_t* row = blk + (16 * u + 2 * g) * RB;
      int c[4] = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < NC; ++h) {
        uint32_t o[2][NK];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t X[3];
          if constexpr (D == 64) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(row + r * RB) + ((3 * t4) >> 1);
            const int sh = 16 * (t4 & 1);
            X[0] = __funnelshift_r(w[0], w[1], sh);
            X[1] = w[1] >> sh;
            X[2] = 0u;
            o[r][7] = 0u;
          } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(row + r * RB) + 3 * (NC * t4 + h);
#pragma unroll
            for (int i = 0; i < 3; ++i) X[i] = w[i];
          }
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            o[r][3 * i] = X[i] & k_mask(i, 0, CB);
            o[r][3 * i + 1] = X[i] & k_mask(i, 1, CB);
            o[r][3 * i + 2] = (X[i] >> 4) & k_mask(i, 2, CB);
          }
          o[r][3 * KW] = (X[0] & k_mask(0, 3, CB)) | (X[1] & k_mask(1, 3, CB)) | (X[2] & k_mask(2, 3, CB));
        }
#pragma unroll
        for (int i = 0; i < NK / 2; ++i)
          mma_u8s8(c, o[0][2 * i], o[1][2 * i], o[0][2 * i + 1], o[1][2 * i + 1], qb[h * NK + 2 * i], qb[h * NK + 2 * i + 1]);
      }
      const float2 ks = *reinterpret_cast<const float2*>(ksc + 16 * u + 2 * g);
      const float2 v2 = *reinterpret_cast<const float2*>(vsc + 16 * u + 2 * g);
      vs[u][0] = v2.x;
      vs[u][1] = v2.y;
      sign |= __float_as_uint(ks.x) | __float_as_uint(ks.y);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float f = fmaf(static_cast<float>(c[2 * r] + (c[2 * r + 1] << 8)), f_mul, f_add);
        f += __shfl_xor_sync(0xFFFFFFFFu, f, 1);
        s[u][r] = f * (r ? ks.y : ks.x);
      }
    }
    const bool part = j >= n_all, has4 = __any_sync(0xFFFFFFFFu, sign >> 31);
    int lim = PT, most = PT;
    if (part) {
      lim = max(0, min(PT, sees - j * PT));
      most = qrow != nullptr ? lim : 0;
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      lim = min(lim, most);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int o = 16 * u + 2 * g + r;
          if (o >= lim) s[u][r] = -INFINITY;
          if (o >= most) vs[u][r] = 0.f;  // not a token: whatever is there
        }
    }
    if (has4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 ks = *reinterpret_cast<const float2*>(ksc + 16 * u + 2 * g);
        if (signbit(ks.x)) s[u][0] = -INFINITY;
        if (signbit(ks.y)) s[u][1] = -INFINITY;
      }
    }
    // ---- weights p x (V scale) as whole numbers; base 2
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i >> 1][i & 1]);
    float mr = m_ref == -INFINITY ? 0.f : m_ref;
    float pe[4][2], w[4][2];
    int wm = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        pe[u][r] = ex2(fmaf(s[u][r], kq, -mr));
        w[u][r] = pe[u][r] * (vs[u][r] * to_int);
        wm = max(wm, __float_as_int(w[u][r]));  // not negative: ordered as whole numbers are; infinities and NaN above all
      }
    if (__any_sync(0xFFFFFFFFu, wm >= 0x4F800000 || top * kq > m_ref + 20.f) || held >= kFlushPages) {
      float mt = top;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, o));
      const float m_new = fmaxf(m_ref, mt * kq);
      if (held > 0 || any) flush(m_new); else m_ref = m_new;
      mr = m_new == -INFINITY ? 0.f : m_new;
      float wf = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          pe[u][r] = ex2(fmaf(s[u][r], kq, -mr));
          w[u][r] = pe[u][r] * vs[u][r];
          wf = fmaxf(wf, w[u][r]);
        }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) wf = fmaxf(wf, __shfl_xor_sync(0xFFFFFFFFu, wf, o));
      w_exp = min(max((__float_as_int(wf) >> 23) + 2, 31), 254);  // room for weights 4 to 8 times as large
      to_int = pow2_biased(285 - w_exp);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) w[u][r] *= to_int;
    }
    uint32_t b[4];
    const uint32_t sel = (t4 & 1) ? 0x7362u : 0x5140u;  // digits 2, 3 or 0, 1 of two tokens side by side
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      l_run += pe[u][0] + pe[u][1];
      b[u] = transpose8x8(prmt(__float2uint_rn(w[u][0]), __float2uint_rn(w[u][1]), sel));
    }
    // ---- values: digits x 32 tokens a step; the lane's words of 4 tokens of group 4 u + t4
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t x[2][LD / 8][3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* vw = blk + off_v(D) + (8 * t + 4 * e + t4) * 4 * RB + 4 * (3 * LD / 8) * g;
        if constexpr (D == 64) {
#pragma unroll
          for (int i = 0; i < 3; ++i) x[e][0][i] = reinterpret_cast<const uint32_t*>(vw)[i];
        } else if constexpr (D == 128) {
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint2 y = reinterpret_cast<const uint2*>(vw)[i];
            x[e][(2 * i) / 3][(2 * i) % 3] = y.x;
            x[e][(2 * i + 1) / 3][(2 * i + 1) % 3] = y.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint4 y = reinterpret_cast<const uint4*>(vw)[i];
            const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) x[e][(4 * i + c) / 3][(4 * i + c) % 3] = z[c];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < LD / 8; ++i) {
        constexpr uint32_t ones = 0x01010101u;
        const uint32_t (&p)[3] = x[0][i], (&q)[3] = x[1][i];
        const uint32_t b0 = b[2 * t], b1 = b[2 * t + 1];
        mma_u8u8(acc[5 * i], p[0] & 7u * ones, p[0] & 56u * ones, q[0] & 7u * ones, q[0] & 56u * ones, b0, b1);
        mma_u8u8(acc[5 * i + 1], p[0] & 192u * ones, p[1] & ones, q[0] & 192u * ones, q[1] & ones, b0, b1);
        mma_u8u8(acc[5 * i + 2], p[1] & 14u * ones, p[1] & 112u * ones, q[1] & 14u * ones, q[1] & 112u * ones, b0, b1);
        mma_u8u8(acc[5 * i + 3], p[1] & 128u * ones, p[2] & 3u * ones, q[1] & 128u * ones, q[2] & 3u * ones, b0, b1);
        mma_u8u8(acc[5 * i + 4], p[2] & 28u * ones, p[2] & 224u * ones, q[2] & 28u * ones, q[2] & 224u * ones, b0, b1);
      }
      mma_u8u8(off, 0x04040404u, 0x04040404u, 0x04040404u, 0x04040404u, b[2 * t], b[2 * t + 1]);
    }
    ++held;
    if (has4) four_bit(a, sg, blk, page, tokens4(ksc, most), lim, c4_bytes);
  }

  // The page's 4-bit tokens, one after the other: a lane has D / 32 dimensions of
  // the K row for both rows, and half of LD dimensions of the V row for its own.
  __device__ __forceinline__ void four_bit(const AttnArgs& a, const Segment& sg, const uint8_t* blk, int page, uint64_t set,
                                           int lim, int c4_bytes) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll 1
    for (; set; set &= set - 1) {
      const int o = __ffsll(static_cast<long long>(set)) - 1;
      const int j4 = blk[o * RB];
      if (!FOUR || j4 >= a.C4) {
        if (lane == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
        continue;
      }
      if constexpr (FOUR) {
        const uint8_t* r4 = c4_bytes ? blk + block_bytes(D) + j4 * D
                                     : a.codes4 + ((static_cast<int64_t>(page) * a.H + sg.h) * a.C4 + j4) * D;
        const uint32_t kc = D == 64 ? r4[lane] : D == 128 ? reinterpret_cast<const uint16_t*>(r4)[lane] : reinterpret_cast<const uint32_t*>(r4)[lane];
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          const float c = static_cast<float>(static_cast<int>((kc >> (4 * d)) & 15u) - 8);
          d0 = fmaf(__uint_as_float((d & 1) ? (q4[0][d >> 1] & 0xFFFF0000u) : (q4[0][d >> 1] << 16)), c, d0);
          d1 = fmaf(__uint_as_float((d & 1) ? (q4[1][d >> 1] & 0xFFFF0000u) : (q4[1][d >> 1] << 16)), c, d1);
        }
        // even lanes sum the first row's, odd lanes the second's; then each takes its row's
        float dot = (lane & 1) ? d1 : d0;
        dot += __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? d0 : d1, 1);
#pragma unroll
        for (int x = 2; x < 32; x <<= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
        dot = __shfl_sync(0xFFFFFFFFu, dot, t4 >> 1);
        const float k4 = fabsf(reinterpret_cast<const float*>(blk + off_ks(D))[o]) * a.qk_scale * 1.4426950408889634f;
        const float v4 = reinterpret_cast<const float*>(blk + off_vs(D))[o];
        const float sc = o < lim ? dot * k4 : -INFINITY;
        if (__any_sync(0xFFFFFFFFu, sc > m_ref + 20.f)) {
          flush(fmaxf(m_ref, sc));
          to_int = INFINITY;  // found anew on the next page
        }
        const float e = sc == -INFINITY ? 0.f : ex2(sc - m_ref);
        if (g == 0) l_run += e;
        const float ev = e * v4;
        const uint8_t* vr = r4 + D / 2 + LD / 2 * g + (t4 & 1) * (LD / 4);
#pragma unroll
        for (int d = 0; d < LD / 2; d += 2) {
          const uint32_t c = vr[d / 2];
          o4[d] = fmaf(ev, static_cast<float>(static_cast<int>(c & 15u) - 8), o4[d]);
          o4[d + 1] = fmaf(ev, static_cast<float>(static_cast<int>(c >> 4) - 8), o4[d + 1]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(const AttnArgs& a, const Segment& sg, float* out, bool whole) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    float l = l_run;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    uint16_t* row = whole && qrow != nullptr ? output_row(a, sg, sg.r0 + (t4 >> 1)) : nullptr;
    flush(m_ref, row, l > 0.f ? 1.f / l : 0.f);
    if (g == 0 && (t4 & 1) == 0 && qrow != nullptr && !whole) {
      out[COLS * D + (t4 >> 1)] = m_ref;
      out[COLS * D + COLS + (t4 >> 1)] = l;
    }
  }
};

}  // namespace paged
}  // namespace blt
