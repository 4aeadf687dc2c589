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
//     shared page is read once for the batch (once for every 8 rows; from
//     tile_rows() on paged_front.cu has them, 128 a tile);
//   * a walk leaves, for each stretch of pages that a warp took of one (head,
//     group of columns), the running maximum, sum and value sums ("a piece");
//     the join adds a row's pieces of both walks.
#include <cmath>

#include "launch.h"
#include "paged.cuh"
#include "paged_front.cuh"
#include "paged_mma.cuh"
#include "ptx.cuh"

namespace blt {
namespace paged {

// --------------------------------------------------------------------- walk
// The pages of one (sequence, head, group of columns) are a segment. Segments
// lie one behind the other, each as long as its pages and segment_overhead()
// more (what beginning and ending one costs, in pages: without it a warp among one-page
// sequences took 27 segments where others took one), and warp w of NW takes
// the pages that lie in [U w / NW, U (w + 1) / NW): equal shares whatever the
// lengths are. Each warp streams its pages' blocks (one bulk copy a block)
// through a ring of its own and shares nothing with its neighbours.
//
// Its piece of segment s goes to slot s + w: along the line either s or w
// grows from one piece to the next, so no two pieces have one slot.

struct WalkArgs {
  AttnArgs a;
  int front;        // 1: the shared pages, all sequences' rows; 0: the own pages
  int groups;       // groups of columns of a (sequence, head)
  int stage_bytes;
  int late_wait;    // an earlier kernel of this call has waited for what the call depends on
  float* parts;     // pieces
  int64_t* cum;     // [B + 1] length of one head's and group's segments before sequence b (written)
};

// warps with a share of a line of U (each one unit at least), where that of warp w begins, and the warp that has unit u
__device__ __forceinline__ int64_t walkers(int64_t U, int64_t NW) { return U < NW ? U : NW; }
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {  // of numbers that are not negative
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}
__device__ __forceinline__ int64_t first_unit(int64_t U, int64_t w, int64_t NW) { return quot(U * w, NW); }
__device__ __forceinline__ int64_t warp_of(int64_t U, int64_t u, int64_t NW) { return quot((u + 1) * NW - 1, U); }

struct Cursor {  // page j of P of a segment, at place x of the warp's share
  int b, h, grp, j, P, x;
};

// Page: the arithmetic on a page's block (paged_mma.cuh).
template <int D, typename Page, int WARPS, int NS>
__global__ void __launch_bounds__(32 * WARPS, 2) walk_kernel(const __grid_constant__ WalkArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[WARPS][NS];
  __shared__ int s_page[WARPS][NS];
  __shared__ int64_t s_cum[32 * WARPS + 1];
  __shared__ int64_t s_sum[WARPS];
  constexpr int OV = segment_overhead(Page::COLS);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init();
  }
  if (!p.late_wait) pdl_wait();
  pdl_trigger();

  // ---- the line: its length before each chunk of sequences, then this warp's share
  const int chunk = (a.B + 32 * WARPS - 1) / (32 * WARPS);
  int64_t U;
  if (p.front) {
    __syncthreads();
    U = static_cast<int64_t>(a.n_shared + OV) * a.H * p.groups;
  } else {
    int64_t mine = 0;
    const int b0 = tid * chunk, b1 = min(a.B, b0 + chunk);
    for (int b = b0; b < b1; ++b) {
      bool bad;
      const int len = cut_len(a, b, &bad);
      if (bad && blockIdx.x == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
      const int P = pages_of(len) - a.n_shared;
      if (P > 0) mine += P + OV;
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
        const int P = own_pages(a, b);
        if (P > 0) c += P + OV;
      }
      if (tid == 0) p.cum[a.B] = s_cum[32 * WARPS];
    }
  }
  // few pages: one a warp, over all SMs (neighbouring numbers lie on neighbouring SMs)
  const int64_t NW = walkers(U, static_cast<int64_t>(gridDim.x) * WARPS);
  const int64_t wid = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  const int64_t x0 = wid < NW ? first_unit(U, wid, NW) : 0;
  const int limit = wid < NW ? static_cast<int>(first_unit(U, wid + 1, NW) - x0) : 0;
  if (limit > 0) {
    Cursor take;
    int64_t seg;
    int off;  // place in the segment
    const int64_t hg = static_cast<int64_t>(a.H) * p.groups;
    if (p.front) {
      seg = quot(x0, a.n_shared + OV);
      take.b = 0;
      take.P = a.n_shared;
      off = static_cast<int>(x0 - seg * (a.n_shared + OV));
      take.h = static_cast<int>(quot(seg, p.groups));
      take.grp = static_cast<int>(seg - static_cast<int64_t>(take.h) * p.groups);
    } else {
      const int64_t at = quot(x0, hg);
      int lo = 0, hi = 32 * WARPS - 1;  // the last chunk that begins at or before that
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cum[mid] <= at) lo = mid; else hi = mid - 1;
      }
      int64_t c = s_cum[lo];
      int b = lo * chunk, P = own_pages(a, b);
      while (P == 0 || c + P + OV <= at) {
        if (P > 0) c += P + OV;
        P = own_pages(a, ++b);
      }
      const int64_t v = x0 - c * hg, s = quot(v, P + OV);
      take.b = b;
      take.P = P;
      off = static_cast<int>(v - s * (P + OV));
      take.h = static_cast<int>(quot(s, p.groups));
      take.grp = static_cast<int>(s - static_cast<int64_t>(take.h) * p.groups);
      seg = static_cast<int64_t>(b) * hg + s;
    }
    take.j = max(off - OV, 0);
    take.x = max(OV - off, 0);
    auto advance = [&](Cursor& c) {
      ++c.x;
      if (++c.j < c.P) return;
      c.x += OV;
      if (c.x >= limit) return;
      c.j = 0;
      if (++c.grp < p.groups) return;
      c.grp = 0;
      if (++c.h < a.H) return;
      c.h = 0;
      do { c.P = own_pages(a, ++c.b); } while (c.P == 0);  // the line goes on: there is one
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
      advance(put);
    };
    while (n_put < NS && put.x < limit) issue();

    const int G = a.Hq / a.H;
    const int rows = (p.front ? a.B : 1) * a.Sq * G;  // of a (sequence, head)
    uint32_t parity = 0u;                             // bit per stage
    int st = 0;
    bool ok = true;
    while (take.x < limit && ok) {
      Segment sg{p.front ? 0 : take.b * a.Sq, take.grp * Page::COLS, rows, take.h, G, p.front != 0};
      float* out = p.parts + (seg + wid) * piece_floats(D, Page::COLS);
      Page pg;
      pg.begin(a, sg, out);
      const int last = min(limit - take.x, take.P - take.j);
      for (int e = 0; e < last; ++e) {
        const uint8_t* blk = ring + st * p.stage_bytes;
        __syncwarp();  // s_page is lane 0's
        const int page = s_page[warp][st];
        if (page >= 0) {
          if (!mbar_wait(&s_full[warp][st], (parity >> st) & 1u, a.timeout_ns, nullptr)) ok = false;
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          parity ^= 1u << st;
          pg.page(a, sg, blk, page, take.j + e, c4_bytes);
        }
        __syncwarp();  // all lanes are done with the stage
        if (put.x < limit) issue();
        st = st + 1 == NS ? 0 : st + 1;
      }

      // a whole segment, and nothing in front of it: the rows are done
      if (ok) pg.finish(a, sg, out, !p.front && a.n_shared == 0 && take.j == 0 && last == take.P);
      // the next segment
      take.j += last - 1;
      take.x += last - 1;
      const int b = take.b;
      advance(take);
      seg += 1 + static_cast<int64_t>(take.b - (b == take.b ? b : b + 1)) * hg;  // sequences without pages
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
// WPR warps a row (query, head), D / 32 dimensions a lane; lane i reads the
// maximum and sum of the warp's i-th piece, then all pieces' values come with
// their factors known, so that their loads do not wait for one another.
struct JoinArgs {
  AttnArgs a;
  const float* own;      // null: no own pages
  const float* front;    // null: no shared pages
  const int64_t* cum;
  int64_t own_nw, front_nw;
  int own_groups, front_groups, own_cols, front_cols;
  FrontPlan tiles;       // k > 0: the tensor-core kernel's pieces
};

template <int D, int WPR>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ JoinArgs p) {
  constexpr int DL = D / 32, VL = DL < 4 ? DL : 4;  // VL: dimensions side by side
  __shared__ float s_m[4], s_l[4], s_o[WPR == 1 ? 1 : 4][D];
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x * (4 / WPR) + (WPR == 1 ? warp : 0);
  if (row >= a.B * a.Sq * a.Hq) return;
  const int sub = WPR == 1 ? 0 : warp;
  const int tok = row / a.Hq, hq = row - tok * a.Hq;
  const int G = a.Hq / a.H, h = hq / G, gg = hq - h * G;
  float m = -INFINITY, l = 0.f, o[DL];
#pragma unroll
  for (int i = 0; i < DL; ++i) o[i] = 0.f;
  auto add = [&](const float* base, int cols, int col, int64_t first, int64_t n, int step = 1) {
    const int64_t size = piece_floats(D, cols);
    for (int64_t i0 = sub; i0 < n; i0 += 32 * WPR) {
      float pm = -INFINITY, pl = 0.f;
      if (i0 + WPR * lane < n) {
        const float* x = base + (first + (i0 + WPR * lane) * step) * size + cols * D + col;
        pm = x[0];
        pl = x[cols];
      }
      float mn = fmaxf(m, pm);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, x));
      const float f0 = m == -INFINITY ? 0.f : ex2(m - mn), f = pm == -INFINITY ? 0.f : ex2(pm - mn);
      m = mn;
      pl *= f;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) pl += __shfl_xor_sync(0xFFFFFFFFu, pl, x);
      l = fmaf(l, f0, pl);
#pragma unroll
      for (int d = 0; d < DL; ++d) o[d] *= f0;
      const int cnt = static_cast<int>(min(static_cast<int64_t>(32), (n - i0 + WPR - 1) / WPR));
      const float* v = base + (first + i0 * step) * size + col * D + lane * VL;
#pragma unroll 4
      for (int j = 0; j < cnt; ++j) {
        const float fj = __shfl_sync(0xFFFFFFFFu, f, j);
        if (fj == 0.f) continue;  // nothing seen there, or nothing that counts: its values may be anything
#pragma unroll
        for (int c = 0; c < DL / VL; ++c) {
          float y[VL];
          if constexpr (VL == 4) {
            const float4 t = *reinterpret_cast<const float4*>(v + j * (WPR * step * size) + 128 * c);
            y[0] = t.x; y[1] = t.y; y[2] = t.z; y[3] = t.w;
          } else {
            const float2 t = *reinterpret_cast<const float2*>(v + j * (WPR * step * size));
            y[0] = t.x; y[1] = t.y;
          }
#pragma unroll
          for (int e = 0; e < VL; ++e) o[VL * c + e] = fmaf(fj, y[e], o[VL * c + e]);
        }
      }
    }
  };
  if (p.own != nullptr) {
    const int b = tok / a.Sq, r = (tok % a.Sq) * G + gg, grp = r / p.own_cols;
    const int64_t c = p.cum[b], len = p.cum[b + 1] - c, hg = static_cast<int64_t>(a.H) * p.own_groups;
    if (len > 0) {
      const int64_t U = p.cum[a.B] * hg, u = c * hg + (static_cast<int64_t>(h) * p.own_groups + grp) * len;
      const int64_t nw = walkers(U, p.own_nw), w0 = warp_of(U, u + segment_overhead(p.own_cols), nw), w1 = warp_of(U, u + len - 1, nw);
      if (p.front == nullptr && w0 == w1) return;  // the walk has written the row
      add(p.own, p.own_cols, r % p.own_cols, static_cast<int64_t>(b) * hg + static_cast<int64_t>(h) * p.own_groups + grp + w0, w1 - w0 + 1);
    }
  }
  if (p.front != nullptr && p.tiles.k > 0) {
    const int r = tok * G + gg, tile = r >> 7, k = p.tiles.k;
    const int64_t item = static_cast<int64_t>(h) * (2 * k * p.tiles.pairs + k * p.tiles.singles);
    if (front_streams(D) == 1) add(p.front, 128, r & 127, item + tile * k, k);
    else if (tile < 2 * p.tiles.pairs) add(p.front, 128, r & 127, 2 * (item + (tile >> 1) * 2 * k) + (tile & 1), 2 * k, 2);
    else add(p.front, 128, r & 127, 2 * (item + p.tiles.pairs * 2 * k), 2 * k);
  } else if (p.front != nullptr) {
    const int r = tok * G + gg, grp = r / p.front_cols;
    const int64_t ov = segment_overhead(p.front_cols), len = a.n_shared + ov;
    const int64_t seg = static_cast<int64_t>(h) * p.front_groups + grp, U = len * a.H * p.front_groups;
    const int64_t nw = walkers(U, p.front_nw), w0 = warp_of(U, seg * len + ov, nw), w1 = warp_of(U, (seg + 1) * len - 1, nw);
    add(p.front, p.front_cols, r % p.front_cols, seg + w0, w1 - w0 + 1);
  }
  if (p.own == nullptr && p.front == nullptr && lane == 0 && __ldg(a.lens + tok / a.Sq) != 0)
    report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);  // no page at all
  uint16_t* out = a.out + static_cast<int64_t>(row) * D;
  if constexpr (WPR == 1) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int c = 0; c < DL / VL; ++c) {
      uint32_t x[VL / 2];
#pragma unroll
      for (int e = 0; e < VL / 2; ++e) x[e] = pack_bf16x2(o[VL * c + 2 * e] * inv, o[VL * c + 2 * e + 1] * inv);
      if constexpr (VL == 4) reinterpret_cast<uint2*>(out + 128 * c)[lane] = make_uint2(x[0], x[1]);
      else reinterpret_cast<uint32_t*>(out)[lane] = x[0];
    }
  } else {
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
    for (int d = 0; d < DL; ++d) s_o[warp][VL * lane + 128 * (d / VL) + d % VL] = o[d];
    __syncthreads();
    const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float f[4], L = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f[w] = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - M);
      L = fmaf(f[w], s_l[w], L);
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    for (int d = threadIdx.x; d < D; d += 128) {
      float O = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) O = fmaf(f[w], s_o[w][d], O);
      out[d] = __bfloat16_as_ushort(__float2bfloat16_rn(O * inv));
    }
  }
}

// --------------------------------------------------------------------- plan
struct Plan {
  struct Walk { int cols, groups, grid; int64_t nw, slots; };
  Walk own, front;
  FrontPlan tiles;  // k > 0: the tensor-core kernel has the shared pages
  int64_t off_front, off_cum, bytes;
};

// Two CTAs an SM: of one walk, or one of each where both walks run (the second is launched behind the
// first and runs beside it).
constexpr int walk_warps(int D) { return D == 256 ? 4 : 8; }
constexpr int walk_stages(int D) { return D == 64 ? 3 : 2; }

static Plan::Walk plan_walk(int64_t D, int64_t rows, int64_t segs_per_group, int64_t max_units_per_group, bool any, int per_sm) {
  Plan::Walk w{};
  w.cols = rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
  w.groups = static_cast<int>((rows + w.cols - 1) / w.cols);
  if (!any) return w;
  const int64_t units = (max_units_per_group + segs_per_group * segment_overhead(w.cols)) * w.groups;
  const int64_t most = static_cast<int64_t>(per_sm) * num_sms();
  w.grid = static_cast<int>(units < most ? units : most);
  w.nw = static_cast<int64_t>(w.grid) * walk_warps(static_cast<int>(D));
  w.slots = segs_per_group * w.groups + w.nw;
  return w;
}

// Fewest rounds of CTAs x (pages of one + what beginning and ending cost, about 8).
static FrontPlan plan_tiles(int64_t D, int64_t rows, int64_t H, int64_t n) {
  const int64_t tiles = (rows + 127) / 128;
  FrontPlan p{};
  p.pairs = static_cast<int>(front_streams(static_cast<int>(D)) == 2 ? tiles / 2 : 0);
  p.singles = static_cast<int>(tiles - 2 * p.pairs);
  int64_t best = -1;
  for (int64_t k = 1; k <= n && k <= 64; ++k) {
    const int64_t items = H * (2 * p.pairs + p.singles) * k;
    const int64_t cost = (items + num_sms() - 1) / num_sms() * ((n + k - 1) / k + 8);
    if (best < 0 || cost < best) {
      best = cost;
      p.k = static_cast<int>(k);
      p.items = items;
    }
  }
  return p;
}

// Rows from which the tensor-core kernel takes the shared pages. Walk / tiles, whole call in us:
//   D = 128, 64 pages x 32 heads   24 rows 39 / 45, 32 rows 42 / 46, 40 rows 47 / 46, 56 rows 58 / 48
//   D = 128, 256 pages x 8 heads   24 rows 37 / 42, 32 rows 39 / 42, 40 rows 44 / 44, 56 rows 55 / 45
//   D = 64, 64 pages x 32 heads    24 rows 29 / 37, 32 rows 31 / 37, 40 rows 33 / 38, 56 rows 42 / 39
//   D = 256, 64 pages x 32 heads   17 rows 59 / 61, 32 rows 72 / 63; with a 4-bit token a page 85 / 66, 106 / 68
constexpr int64_t tile_rows(int64_t D) { return D == 256 ? 17 : 33; }

static Plan make_plan(int64_t B, int64_t Sq, int64_t Hq, int64_t H, int64_t D, int64_t n_shared, int64_t W) {
  Plan p{};
  const int64_t rows = Sq * (Hq / H);
  const bool tiled = n_shared > 0 && B * rows >= tile_rows(D);
  const int per_sm = W > 0 && n_shared > 0 && !tiled ? 1 : 2;
  p.own = plan_walk(D, rows, B * H, B * W * H, W > 0, per_sm);
  if (tiled) p.tiles = plan_tiles(D, B * rows, H, n_shared);
  p.front = plan_walk(D, B * rows, H, n_shared * H, n_shared > 0 && !tiled, per_sm);
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  p.off_front = up(p.own.slots * piece_floats(static_cast<int>(D), p.own.cols) * 4);
  p.off_cum = p.off_front + up(tiled ? p.tiles.items * front_streams(static_cast<int>(D)) * piece_floats(static_cast<int>(D), 128) * 4
                                     : p.front.slots * piece_floats(static_cast<int>(D), p.front.cols) * 4);
  p.bytes = p.off_cum + (W > 0 ? up((B + 1) * 8) : 0);
  return p;
}

template <int D, typename Page>
static cudaError_t launch_walk(const AttnArgs& a, const Plan::Walk& w, bool front, bool behind, float* parts, int64_t* cum,
                               cudaStream_t s) {
  constexpr int kWarps = walk_warps(D);
  auto kern = walk_kernel<D, Page, kWarps, walk_stages(D)>;
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
  j.tiles = pl.tiles;
  int64_t* cum = reinterpret_cast<int64_t*>(a.work + pl.off_cum);
  j.cum = cum;
  bool behind = false;
  auto walk = [&](const Plan::Walk& w, bool front, float* parts) {
    const cudaError_t e = w.cols == 8   ? launch_walk<D, F16Page<D, 2>>(a, w, front, behind, parts, cum, s)
                          : w.cols == 4 ? launch_walk<D, F16Page<D, 1>>(a, w, front, behind, parts, cum, s)
                          : a.C4 > 0    ? launch_walk<D, I8Page<D, true>>(a, w, front, behind, parts, cum, s)
                                        : launch_walk<D, I8Page<D, false>>(a, w, front, behind, parts, cum, s);
    behind = true;
    return e;
  };
  cudaError_t e = cudaSuccess;
  if (a.n_shared > 0) {
    float* parts = reinterpret_cast<float*>(a.work + pl.off_front);
    j.front = parts;
    if (pl.tiles.k > 0) {
      e = launch_front(a, pl.tiles, parts, s);
      behind = true;
    } else {
      e = walk(pl.front, true, parts);
    }
  }
  if (e == cudaSuccess && a.W > 0) {
    float* parts = reinterpret_cast<float*>(a.work);
    j.own = parts;
    e = walk(pl.own, false, parts);
  }
  if (e != cudaSuccess) return e;
  // A warp a row while a row has few pieces (64 sequences of up to 4096 tokens, 2 pieces: 4 us against
  // 7.7 with a block a row); four where one sequence's pages went to many warps.
  const int64_t rows = static_cast<int64_t>(a.B) * a.Sq * a.Hq;
  const int64_t pieces = (j.own ? pl.own.nw / (static_cast<int64_t>(a.B) * a.H * pl.own.groups) + 1 : 0) +
                         (pl.tiles.k > 0 ? 2 * pl.tiles.k : j.front ? pl.front.nw / (static_cast<int64_t>(a.H) * pl.front.groups) + 1 : 0);
  const bool wide = pieces > 16;
  const dim3 grid(static_cast<unsigned>(wide ? rows : (rows + 3) / 4));
  auto join = wide ? join_kernel<D, 4> : join_kernel<D, 1>;
  if (behind) return launch_behind(join, grid, dim3(128), 0, s, j);
  return launch_kernel(join, grid, dim3(128), 0, s, 0u, j);
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
