// Decode attention over the paged 3-bit cache (layout: paged.cuh).
//
// Query i of sequence b (length n_b, its Sq newest tokens the queries' own)
// sees the tokens t < n_b - Sq + 1 + i: token t lies in page shared[t / 64]
// while t < 64 n_shared, in page tables[b][t / 64 - n_shared] after that.
//   s_t = (q . k_t) / sqrt(D),  p = softmax_t(s),  o = sum_t p_t v_t
//
// Two walks over the pages and a join:
//   * the sequences' own pages: the Sq Hq / H rows of a sequence that read
//     one cache head are the columns of its pages' products;
//   * the shared pages: the rows of ALL sequences are their columns, so a
//     shared page is read once for the batch (once for every 8 rows);
//   * a walk leaves, for each stretch of pages that a warp took of one (head,
//     group of columns), the running maximum, sum and value sums ("a piece");
//     the join adds a row's pieces of both walks.
#include <cmath>

#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace blt {
namespace paged {

// ----------------------------------------------------------------- operands
// A 3-bit code c at bit j <= 7 of a 16-bit half, the other bits cleared, IS the
// fp16 subnormal c 2^(j - 24); one paired fma makes (c - 4) 2^(j - 9) of it,
// exact and normal. Two codes 16 bits apart (give or take what keeps both in
// the halves' low 10 bits) are so one operand register of the m16n8k16 fp16
// MMA, for a mask, an fma and a share of a shift. The 2^j go into the queries
// (a power of two: exact) for K, and leave at the end for V.
// Without the fma (the subnormals as operands, the offset of 4 taken off the
// sums) it would be 256 of 900 instructions a page less, but the MMA lines its
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
__device__ __forceinline__ float f16lo(uint32_t v) {
  float f;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l; }" : "=f"(f) : "r"(v));
  return f;
}
__device__ __forceinline__ float f16hi(uint32_t v) {
  float f;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, h; }" : "=f"(f) : "r"(v));
  return f;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(e - 127) of a biased exponent 1..254
__device__ __forceinline__ float pow2_biased(int e) { return __int_as_float(e << 23); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// --------------------------------------------------------------------- walk
// A unit is (page, cache head, group of columns). The units of one (sequence,
// head, group) lie side by side, warp w of NW takes the units
// [U w / NW, U (w + 1) / NW): equal shares whatever the lengths are. Each warp
// streams its pages' blocks (one bulk copy a block) through a ring of its own
// and shares nothing with its neighbours.
//
// Its piece of segment s = (sequence, head, group) goes to slot s + w: along
// the units either s or w grows from one piece to the next, so no two pieces
// have one slot.
constexpr int kStageRows4 = 3;  // 4-bit rows of a page that travel with it; pools with more are read from global memory

struct WalkArgs {
  AttnArgs a;
  int front;        // 1: the shared pages, all sequences' rows; 0: the own pages
  int groups;       // groups of columns of a (sequence, head)
  int stage_bytes;
  int late_wait;    // an earlier kernel of this call has waited for what the call depends on
  float* parts;     // pieces
  int64_t* cum;     // [B + 1] own pages before sequence b (written)
};

__host__ __device__ constexpr int piece_floats(int D, int cols) { return cols * (D + 2); }

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
// warps that have units (each one at least), the first unit of warp w, and the warp that has unit u
__device__ __forceinline__ int64_t walkers(int64_t U, int64_t NW) { return U < NW ? U : NW; }
__device__ __forceinline__ int64_t first_unit(int64_t U, int64_t w, int64_t NW) { return U * w / NW; }
__device__ __forceinline__ int64_t warp_of(int64_t U, int64_t u, int64_t NW) { return ((u + 1) * NW - 1) / U; }

struct Cursor {  // a unit: page j of P of segment seg = (b heads + h) groups + group
  int b, h, grp, j, P;
};

// QC: columns of a lane that are queries: 1: 4 queries a group (columns 2 q and
// 2 q + 1 are both query q, of which one is kept: half the softmax), 2: 8.
// The weights are rounded to fp16 for the value product: 2^-11 of a weight, a
// quarter of what the output's own rounding may take.
template <int D, int QC, int WARPS, int NS>
__global__ void __launch_bounds__(32 * WARPS, 1) walk_kernel(const __grid_constant__ WalkArgs p) {
  constexpr int RB = row_bytes(D), NB = D / 64 * 4;  // NB: fp16 MMAs of a score
  constexpr int LD = D / 8;                          // dimensions of a lane in the value product
  constexpr int NM = D / 16;                         // and its MMAs
  constexpr int COLS = 4 * QC;
  constexpr int KW = D == 64 ? 2 : 3;                // stream words of a lane's chunk
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[WARPS][NS];
  __shared__ int s_page[WARPS][NS];
  __shared__ int64_t s_cum[32 * WARPS + 1];
  __shared__ int64_t s_sum[WARPS];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init();
  }
  if (!p.late_wait) pdl_wait();
  pdl_trigger();

  // ---- units: pages before each chunk of sequences, then this warp's share
  const int chunk = (a.B + 32 * WARPS - 1) / (32 * WARPS);
  int64_t U;
  if (p.front) {
    __syncthreads();
    U = static_cast<int64_t>(a.n_shared) * a.H * p.groups;
  } else {
    int64_t mine = 0;
    const int b0 = tid * chunk, b1 = min(a.B, b0 + chunk);
    for (int b = b0; b < b1; ++b) {
      bool bad;
      const int len = cut_len(a, b, &bad);
      if (bad && blockIdx.x == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
      mine += max(0, pages_of(len) - a.n_shared);
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += s_sum[w];
    s_cum[tid + 1] = upto;
    if (tid == 0) s_cum[0] = 0;
    __syncthreads();
    U = s_cum[32 * WARPS] * a.H * p.groups;
    if (blockIdx.x == 0) {  // for the join
      int64_t c = upto - mine;
      for (int b = b0; b < b1; ++b) {
        p.cum[b] = c;
        c += own_pages(a, b);
      }
      if (tid == 0) p.cum[a.B] = s_cum[32 * WARPS];
    }
  }
  // few units: one a warp, over all SMs (neighbouring numbers lie on neighbouring SMs)
  const int64_t NW = walkers(U, static_cast<int64_t>(gridDim.x) * WARPS);
  const int64_t wid = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  const int64_t u0 = wid < NW ? first_unit(U, wid, NW) : 0;
  const int n_units = wid < NW ? static_cast<int>(first_unit(U, wid + 1, NW) - u0) : 0;
  if (n_units > 0) {
    Cursor take;
    int64_t seg;
    if (p.front) {
      seg = u0 / a.n_shared;
      take.b = 0;
      take.P = a.n_shared;
      take.j = static_cast<int>(u0 - seg * a.n_shared);
      take.h = static_cast<int>(seg / p.groups);
      take.grp = static_cast<int>(seg - static_cast<int64_t>(take.h) * p.groups);
    } else {
      const int64_t hg = static_cast<int64_t>(a.H) * p.groups;
      const int64_t pg = u0 / hg;
      int lo = 0, hi = 32 * WARPS - 1;  // the last chunk that begins at or before pg
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cum[mid] <= pg) lo = mid; else hi = mid - 1;
      }
      int64_t c = s_cum[lo];
      int b = lo * chunk, P = own_pages(a, b);
      while (c + P <= pg) { c += P; P = own_pages(a, ++b); }
      const int64_t v = u0 - c * hg, s = v / P;
      take.b = b;
      take.P = P;
      take.j = static_cast<int>(v - s * P);
      take.h = static_cast<int>(s / p.groups);
      take.grp = static_cast<int>(s - static_cast<int64_t>(take.h) * p.groups);
      seg = static_cast<int64_t>(b) * hg + s;
    }
    auto advance = [&](Cursor& c) {
      if (++c.j < c.P) return;
      c.j = 0;
      if (++c.grp < p.groups) return;
      c.grp = 0;
      if (++c.h < a.H) return;
      c.h = 0;
      do { c.P = own_pages(a, ++c.b); } while (c.P == 0);  // called only while units are left
    };

    uint8_t* ring = smem + static_cast<size_t>(warp) * NS * p.stage_bytes;
    const int c4_bytes = p.stage_bytes - block_bytes(D);  // 0: no 4-bit rows, or read from global memory
    // ---- the copying side: page ids 32 at a time, a lane each
    Cursor put = take;
    int id_b = -1, id_j = -1, ids = 0, n_put = 0, put_st = 0;
    auto issue = [&]() {
      if (put.b != id_b || (put.j & ~31) != id_j) {
        id_b = put.b;
        id_j = put.j & ~31;
        const int j = id_j + lane;
        ids = j < put.P ? (p.front ? __ldg(a.shared + j) : __ldg(a.tables + id_b * a.ldt + j)) : 0;
      }
      const int page = __shfl_sync(0xFFFFFFFFu, ids, put.j & 31);
      const int st = put_st;
      put_st = put_st + 1 == NS ? 0 : put_st + 1;
      if (lane == 0) {
        const bool good = page >= 0 && page < a.n_pages;
        s_page[warp][st] = good ? page : -1;
        if (good) {
          const int64_t at = static_cast<int64_t>(page) * a.H + put.h;
          uint8_t* dst = ring + st * p.stage_bytes;
          mbar_arrive_expect_tx(&s_full[warp][st], static_cast<uint32_t>(p.stage_bytes));
          bulk_load(dst, a.pages + at * block_bytes(D), block_bytes(D), &s_full[warp][st]);
          if (c4_bytes) bulk_load(dst + block_bytes(D), a.codes4 + at * c4_bytes, static_cast<uint32_t>(c4_bytes), &s_full[warp][st]);
        } else {
          report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
        }
      }
      ++n_put;
      if (n_put < n_units) advance(put);
    };
    while (n_put < min(NS, n_units)) issue();

    const int G = a.Hq / a.H;
    const int rows = (p.front ? a.B : 1) * a.Sq * G;  // of a (sequence, head)
    uint32_t parity = 0u;                             // bit per stage
    int st = 0;
    bool ok = true;
    for (int k = 0; k < n_units && ok;) {
      // ---- a segment: its columns' queries
      const int r0 = take.grp * COLS, tok0 = p.front ? 0 : take.b * a.Sq;
      uint32_t qb[2 * NB];   // query operands: pair i of this lane's chunk of column g
      float kq[QC];          // what makes of (sum) x (K scale) a score in base 2
      int sees[QC];          // tokens that the lane's columns see, from the segment's first page on
      const uint16_t* qrow[QC];
      {
        const int rq = r0 + (QC == 1 ? g >> 1 : g);
        uint32_t x[D / 8];  // D / 4 dimensions of the row
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = 0u;
        if (rq < rows) {
          const uint4* src = reinterpret_cast<const uint4*>(a.q + (tok0 + rq / G) * a.ldq + static_cast<int64_t>(take.h * G + rq % G) * D) + D / 32 * t4;
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
        const float kr = a.qk_scale * 1.4426950408889634f * pow2_biased(263 - fb);  // 2^(9 + 127 - fb)
#pragma unroll
        for (int c = 0; c < QC; ++c) {
          const int src = QC == 1 ? 8 * t4 : 4 * (2 * t4 + c);  // a lane of the column's row
          kq[c] = __shfl_sync(0xFFFFFFFFu, kr, src);
          const int r = r0 + (QC == 1 ? t4 : 2 * t4 + c);
          sees[c] = 0x7FFFFFFF;  // no row: nothing is masked, nothing kept
          qrow[c] = nullptr;
          if (r < rows) {
            const int tok = tok0 + r / G;
            bool bad;
            const int len = cut_len(a, tok / a.Sq, &bad);
            if (bad && p.front) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
            sees[c] = max(0, len - a.Sq + 1 + tok % a.Sq);
            if (!p.front) sees[c] = max(0, sees[c] - PT * a.n_shared);
            qrow[c] = a.q + tok * a.ldq + static_cast<int64_t>(take.h * G + r % G) * D;
          }
        }
      }
      float m_run[QC], l_run[QC], acc[NM][4];
#pragma unroll
      for (int c = 0; c < QC; ++c) { m_run[c] = -INFINITY; l_run[c] = 0.f; }
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
      int ve = 14;  // biased exponent that value scales are taken relative to (at least that of 2^-113)

      // ---- the segment's pages; those before page n_all are seen whole by all columns
      int n_all = sees[0];
      if constexpr (QC == 2) n_all = min(n_all, sees[QC - 1]);
      n_all = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<unsigned>(n_all)) / PT);
      const int last = min(n_units - k, take.P - take.j);
      for (int e = 0; e < last; ++e, ++k) {
        const uint8_t* blk = ring + st * p.stage_bytes;
        __syncwarp();  // s_page is lane 0's
        const int page = s_page[warp][st];
        if (page >= 0) {
          if (!mbar_wait(&s_full[warp][st], (parity >> st) & 1u, a.timeout_ns, nullptr)) ok = false;
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          parity ^= 1u << st;
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
              s[u][0][q] = c[q] * ks.x;
              s[u][1][q] = c[2 + q] * ks.y;
            }
          }
          const bool plain = __all_sync(0xFFFFFFFFu, !(sign >> 31)) && take.j + e < n_all;
          uint32_t four = 0u;  // bit 2 u + r: the lane's token is kept at 4 bits
          int lim[QC], most = 0;
          if (!plain) {
#pragma unroll
            for (int c = 0; c < QC; ++c) {
              lim[c] = max(0, min(PT, sees[c] - (take.j + e) * PT));
              if (qrow[c] != nullptr) most = max(most, lim[c]);
            }
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int o = 16 * u + 2 * g + r;
                const bool is4 = signbit(ksc[o]);
                if (is4) four |= 1u << (2 * u + r);
#pragma unroll
                for (int q = 0; q < QC; ++q)
                  if (is4 || o >= lim[q]) s[u][r][q] = -INFINITY;
                if (o >= most) { vs[u][r] = 0.f; four &= ~(1u << (2 * u + r)); }  // not a token: whatever is there
              }
          }
          // ---- online softmax, in base 2; value scales relative to 2^(ve - 127)
          float m_new[QC];
          bool grew = false;
#pragma unroll
          for (int q = 0; q < QC; ++q) {
            float mt = s[0][0][q];
#pragma unroll
            for (int i = 1; i < 8; ++i) mt = fmaxf(mt, s[i >> 1][i & 1][q]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, o));
            m_new[q] = fmaxf(m_run[q], mt * kq[q]);
            grew = grew || m_new[q] > m_run[q];
          }
          float vm = vs[0][0];
#pragma unroll
          for (int i = 1; i < 8; ++i) vm = fmaxf(vm, vs[i >> 1][i & 1]);
          const int vb = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(vm)) >> 23;
          if (__any_sync(0xFFFFFFFFu, grew || vb > ve)) {
            const int vn = max(ve, vb);
            const float fv = vn - ve > 126 ? 0.f : pow2_biased(127 - (vn - ve));
            ve = vn;
#pragma unroll
            for (int q = 0; q < QC; ++q) {
              const float f = m_new[q] == -INFINITY ? 1.f : ex2(m_run[q] - m_new[q]);
              m_run[q] = m_new[q];
              l_run[q] *= f;
#pragma unroll
              for (int m = 0; m < NM; ++m) {
                acc[m][q] *= f * fv;
                acc[m][2 + q] *= f * fv;
              }
            }
          }
          const float vf = pow2_biased(min(268 - ve, 254));  // value scales below 2^15
          float mr[QC];
#pragma unroll
          for (int q = 0; q < QC; ++q) mr[q] = m_run[q] == -INFINITY ? 0.f : m_run[q];
          // ---- weights and values; B's token 2 t4 (+ 1) of rows 0..7 is token 4 t4 (+ 2)
          // of the 16, of rows 8..15 token 4 t4 + 1 (+ 2): the lane's words of 4 tokens
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t b[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float v = vs[u][r] * vf;
              const float p0 = ex2(fmaf(s[u][r][0], kq[0], -mr[0]));
              l_run[0] += p0;
              if constexpr (QC == 1) {
                b[r] = pack_f16x2(p0 * v, 0.f);
              } else {
                const float p1 = ex2(fmaf(s[u][r][QC - 1], kq[QC - 1], -mr[QC - 1]));
                l_run[QC - 1] += p1;
                b[r] = pack_f16x2(p0 * v, p1 * v);
              }
              b[r] = transpose8x8(b[r]);
            }
            const uint8_t* vw = blk + off_v(D) + (4 * u + t4) * 4 * RB + 4 * (3 * LD / 8) * g;
            uint32_t w[LD / 8][3];
            if constexpr (D == 64) {
#pragma unroll
              for (int i = 0; i < 3; ++i) w[0][i] = reinterpret_cast<const uint32_t*>(vw)[i];
            } else if constexpr (D == 128) {
#pragma unroll
              for (int i = 0; i < 3; ++i) {
                const uint2 x = reinterpret_cast<const uint2*>(vw)[i];
                w[(2 * i) / 3][(2 * i) % 3] = x.x;
                w[(2 * i + 1) / 3][(2 * i + 1) % 3] = x.y;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 3; ++i) {
                const uint4 x = reinterpret_cast<const uint4*>(vw)[i];
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) w[(4 * i + c) / 3][(4 * i + c) % 3] = y[c];
              }
            }
#define BLT_V(E_)                                                                    \
            {                                                                        \
              uint32_t x0, x1, y0, y1;                                               \
              v_operand<E_>(w[i], x, x0, x1);                                        \
              v_operand<E_ + 1>(w[i], x, y0, y1);                                    \
              mma_f16(acc[4 * i + E_ / 2], x0, y0, x1, y1, b[0], b[1]);              \
            }
#pragma unroll
            for (int i = 0; i < LD / 8; ++i) {
              const uint32_t x[3] = {w[i][0] >> 8, w[i][1] >> 8, w[i][2] >> 8};
              BLT_V(0) BLT_V(2) BLT_V(4) BLT_V(6)
            }
#undef BLT_V
          }
          // ---- the page's 4-bit tokens, one after the other: lane (g, t4) has dimensions
          // LD g .. LD g + LD - 1 of the rows and its columns' queries
          if (!plain) {
            const int C4 = a.C4;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              uint32_t set = __ballot_sync(0xFFFFFFFFu, t4 == 0 && ((four >> i) & 1u));
              for (; set; set &= set - 1u) {
                const int o = 16 * (i >> 1) + (__ffs(set) - 1) / 2 + (i & 1);
                const int j4 = blk[o * RB];
                if (j4 >= C4) {
                  if (lane == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
                  continue;
                }
                const uint8_t* r4 = c4_bytes ? blk + block_bytes(D) + j4 * D
                                             : a.codes4 + ((static_cast<int64_t>(page) * a.H + take.h) * C4 + j4) * D;
                uint32_t kc[LD / 8], vc[LD / 8];
#pragma unroll
                for (int c = 0; c < LD / 8; ++c) {
                  kc[c] = reinterpret_cast<const uint32_t*>(r4 + LD / 2 * g)[c];
                  vc[c] = reinterpret_cast<const uint32_t*>(r4 + D / 2 + LD / 2 * g)[c];
                }
                const float k4 = fabsf(ksc[o]) * a.qk_scale * 1.4426950408889634f, v4 = vsc[o];
                const int vb4 = __float_as_int(v4) >> 23;
                float fv = 1.f;
                if (vb4 > ve) {
                  fv = vb4 - ve > 126 ? 0.f : pow2_biased(127 - (vb4 - ve));
                  ve = vb4;
                }
                const float v = v4 * pow2_biased(min(268 - ve, 254)) * (1.f / 512.f);
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
                  const float sc = o < lim[q] ? dot * k4 : -INFINITY;
                  const float mn = fmaxf(m_run[q], sc);
                  const float f = mn == -INFINITY ? 1.f : ex2(m_run[q] - mn);
                  const float pe = mn == -INFINITY ? 0.f : ex2(sc - mn);
                  m_run[q] = mn;
                  l_run[q] = fmaf(l_run[q], f, g == 0 ? pe : 0.f);
#pragma unroll
                  for (int d = 0; d < LD; ++d) {
                    const float x = static_cast<float>(static_cast<int>((vc[d >> 3] >> (4 * (d & 7))) & 15u) - 8) *
                                    static_cast<float>(1 << v_bit(d & 7));
                    float& y = acc[d >> 1][2 * (d & 1) + q];
                    y = fmaf(pe * v, x, y * (f * fv));
                  }
                }
              }
            }
          }
        }
        __syncwarp();  // all lanes are done with the stage
        if (n_put < n_units) issue();
        st = st + 1 == NS ? 0 : st + 1;
      }

      // ---- the piece
      if (ok) {
        float* out = p.parts + (seg + wid) * piece_floats(D, COLS);
#pragma unroll
        for (int q = 0; q < QC; ++q) {
          const int col = QC == 1 ? t4 : 2 * t4 + q;
          float l = l_run[q];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
          if (qrow[q] != nullptr) {
            float4* dst = reinterpret_cast<float4*>(out + col * D + LD * g);
#pragma unroll
            for (int c = 0; c < LD / 4; ++c) {
              float x[4];
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const int dl = 4 * c + d;
                x[d] = acc[dl >> 1][2 * (dl & 1) + q] * (1.f / static_cast<float>(32 << v_bit(dl & 7))) *
                       pow2_biased(ve);  // 2^(9 - 14 + ve - 127 - v_bit)
              }
              dst[c] = make_float4(x[0], x[1], x[2], x[3]);
            }
            if (g == 0) {
              out[COLS * D + col] = m_run[q];
              out[COLS * D + COLS + col] = l;
            }
          }
        }
      }
      // the next segment
      if (ok && k < n_units) {
        take.j = take.P - 1;
        const int b = take.b;
        advance(take);
        seg += 1 + static_cast<int64_t>(take.b - (b == take.b ? b : b + 1)) * a.H * p.groups;  // sequences without pages
      }
    }
    if (!ok) {  // copies still in flight land before the block's shared memory is released
      report_status(a.status, BITLINEAR_STATUS_TIMEOUT);
      for (int i = 0; i < NS; ++i)
        if (lane == 0 && i < n_put && s_page[warp][i] >= 0) mbar_wait(&s_full[warp][i], (parity >> i) & 1u, a.timeout_ns, nullptr);
    }
  }
  if (p.late_wait) pdl_wait();  // the kernel before this one is done when this one is
}

// --------------------------------------------------------------------- join
// A block a row (query, head): its warps take the row's pieces in turn, a lane
// D / 32 dimensions, then the warps' sums meet.
struct JoinArgs {
  AttnArgs a;
  const float* own;      // null: no own pages
  const float* front;    // null: no shared pages
  const int64_t* cum;
  int64_t own_nw, front_nw;
  int own_groups, front_groups, own_cols, front_cols;
};

template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ JoinArgs p) {
  constexpr int DL = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int tok = blockIdx.y, hq = blockIdx.x;
  const int G = a.Hq / a.H, h = hq / G, gg = hq % G;
  float m = -INFINITY, l = 0.f, o[DL];
#pragma unroll
  for (int i = 0; i < DL; ++i) o[i] = 0.f;
  auto add = [&](const float* base, int cols, int col, int64_t first, int64_t n) {
    for (int64_t i = warp; i < n; i += 4) {
      const float* x = base + (first + i) * piece_floats(D, cols);
      const float pm = x[cols * D + col], pl = x[cols * D + cols + col];
      float v[DL];
#pragma unroll
      for (int d = 0; d < DL; ++d) v[d] = x[col * D + lane + 32 * d];
      const float mn = fmaxf(m, pm);
      const float f0 = mn == -INFINITY ? 0.f : ex2(m - mn), f1 = mn == -INFINITY ? 0.f : ex2(pm - mn);
      m = mn;
      l = l * f0 + pl * f1;
#pragma unroll
      for (int d = 0; d < DL; ++d) o[d] = o[d] * f0 + v[d] * f1;
    }
  };
  if (p.own != nullptr) {
    const int b = tok / a.Sq, r = (tok % a.Sq) * G + gg, grp = r / p.own_cols;
    const int64_t c = p.cum[b], P = p.cum[b + 1] - c, hg = static_cast<int64_t>(a.H) * p.own_groups;
    if (P > 0) {
      const int64_t U = p.cum[a.B] * hg, u = c * hg + (static_cast<int64_t>(h) * p.own_groups + grp) * P;
      const int64_t nw = walkers(U, p.own_nw), w0 = warp_of(U, u, nw), w1 = warp_of(U, u + P - 1, nw);
      add(p.own, p.own_cols, r % p.own_cols, static_cast<int64_t>(b) * hg + static_cast<int64_t>(h) * p.own_groups + grp + w0, w1 - w0 + 1);
    }
  }
  if (p.front != nullptr) {
    const int r = tok * G + gg, grp = r / p.front_cols;
    const int64_t seg = static_cast<int64_t>(h) * p.front_groups + grp, U = static_cast<int64_t>(a.n_shared) * a.H * p.front_groups;
    const int64_t nw = walkers(U, p.front_nw), w0 = warp_of(U, seg * a.n_shared, nw), w1 = warp_of(U, (seg + 1) * a.n_shared - 1, nw);
    add(p.front, p.front_cols, r % p.front_cols, seg + w0, w1 - w0 + 1);
  }
  if (p.own == nullptr && p.front == nullptr && threadIdx.x == 0 && __ldg(a.lens + tok / a.Sq) != 0)
    report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);  // no page at all
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int d = 0; d < DL; ++d) s_o[warp][lane + 32 * d] = o[d];
  __syncthreads();
  const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float f[4], L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - M);
    L = fmaf(f[w], s_l[w], L);
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float O = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) O = fmaf(f[w], s_o[w][d], O);
    a.out[(static_cast<int64_t>(tok) * a.Hq + hq) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(L > 0.f ? O / L : 0.f));
  }
}

// --------------------------------------------------------------------- plan
struct Plan {
  struct Walk { int cols, groups, grid; int64_t nw, slots; };
  Walk own, front;
  int64_t off_front, off_cum, bytes;
};

constexpr int walk_warps(int D) { return D == 256 ? 8 : 16; }
constexpr int walk_stages(int D) { return D == 64 ? 3 : 2; }

static Plan::Walk plan_walk(int64_t D, int64_t rows, int64_t segs_per_group, int64_t max_units_per_group, bool any) {
  Plan::Walk w{};
  w.cols = rows <= 4 ? 4 : 8;
  w.groups = static_cast<int>((rows + w.cols - 1) / w.cols);
  if (!any) return w;
  const int64_t units = max_units_per_group * w.groups;
  w.grid = static_cast<int>(units < num_sms() ? units : num_sms());
  w.nw = static_cast<int64_t>(w.grid) * walk_warps(static_cast<int>(D));
  w.slots = segs_per_group * w.groups + w.nw;
  return w;
}

static Plan make_plan(int64_t B, int64_t Sq, int64_t Hq, int64_t H, int64_t D, int64_t n_shared, int64_t W) {
  Plan p{};
  const int64_t rows = Sq * (Hq / H);
  p.own = plan_walk(D, rows, B * H, B * W * H, W > 0);
  p.front = plan_walk(D, B * rows, H, n_shared * H, n_shared > 0);
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  p.off_front = up(p.own.slots * piece_floats(static_cast<int>(D), p.own.cols) * 4);
  p.off_cum = p.off_front + up(p.front.slots * piece_floats(static_cast<int>(D), p.front.cols) * 4);
  p.bytes = p.off_cum + (W > 0 ? up((B + 1) * 8) : 0);
  return p;
}

// As launch_kernel, and may always start before the kernel ahead of it has ended.
template <typename K, typename... A>
static cudaError_t launch_behind(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int QC>
static cudaError_t launch_walk(const AttnArgs& a, const Plan::Walk& w, bool front, bool behind, float* parts, int64_t* cum,
                               cudaStream_t s) {
  constexpr int kWarps = walk_warps(D);
  auto kern = walk_kernel<D, QC, kWarps, walk_stages(D)>;
  WalkArgs p{};
  p.a = a;
  p.front = front;
  p.groups = w.groups;
  p.late_wait = behind;
  p.parts = parts;
  p.cum = cum;
  p.stage_bytes = block_bytes(D) + (a.C4 <= kStageRows4 ? a.C4 * D : 0);
  const int smem = walk_stages(D) * kWarps * p.stage_bytes;
  cudaError_t e = set_smem_limit(kern, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(w.grid));
  if (behind) return launch_behind(kern, grid, dim3(32 * kWarps), smem, s, p);
  return launch_kernel(kern, grid, dim3(32 * kWarps), smem, s, 0u, p);
}

template <int D>
static cudaError_t launch_all(const AttnArgs& a, cudaStream_t s) {
  const Plan pl = make_plan(a.B, a.Sq, a.Hq, a.H, D, a.n_shared, a.W);
  JoinArgs j{};
  j.a = a;
  j.own_nw = pl.own.nw;
  j.front_nw = pl.front.nw;
  j.own_groups = pl.own.groups;
  j.front_groups = pl.front.groups;
  j.own_cols = pl.own.cols;
  j.front_cols = pl.front.cols;
  int64_t* cum = reinterpret_cast<int64_t*>(a.work + pl.off_cum);
  j.cum = cum;
  bool behind = false;
  auto walk = [&](const Plan::Walk& w, bool front, float* parts) {
    const cudaError_t e = w.cols == 4 ? launch_walk<D, 1>(a, w, front, behind, parts, cum, s)
                                      : launch_walk<D, 2>(a, w, front, behind, parts, cum, s);
    behind = true;
    return e;
  };
  cudaError_t e = cudaSuccess;
  if (a.n_shared > 0) {
    float* parts = reinterpret_cast<float*>(a.work + pl.off_front);
    j.front = parts;
    e = walk(pl.front, true, parts);
  }
  if (e == cudaSuccess && a.W > 0) {
    float* parts = reinterpret_cast<float*>(a.work);
    j.own = parts;
    e = walk(pl.own, false, parts);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.Hq), static_cast<unsigned>(a.B * a.Sq));
  if (behind) return launch_behind(join_kernel<D>, grid, dim3(128), 0, s, j);
  return launch_kernel(join_kernel<D>, grid, dim3(128), 0, s, 0u, j);
}

}  // namespace paged

int64_t paged_attention_workspace(int64_t B, int64_t Sq, int64_t Hq, int64_t H, int64_t D, int64_t n_shared,
                                  int64_t W) {
  return paged::make_plan(B, Sq, Hq, H, D, n_shared, W).bytes;
}

cudaError_t launch_paged_attention(const paged::AttnArgs& a, cudaStream_t s, const char** why) {
  if (a.D == 64) return paged::launch_all<64>(a, s);
  if (a.D == 128) return paged::launch_all<128>(a, s);
  return paged::launch_all<256>(a, s);
}

}  // namespace blt
