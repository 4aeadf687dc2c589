// The paged 3-bit KV cache: appending tokens, and copying, forking, growing,
// freeing and compacting pages. The layout is in paged.cuh.
#include <cuda_bf16.h>

#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace blt {
namespace paged {

// ------------------------------------------------------------------ append
// One warp quantises TT = 32 / GP tokens of one head of K or of V, GP = D / 32
// lanes a row, each with 32 consecutive dimensions: the arithmetic of the
// contiguous cache's quantiser (absmax over the row, one IEEE division, codes
// by multiply, then add), written into the tokens' slots.
//
// Tokens of a prompt lie side by side in a page. TT of them from an aligned
// place on are 384 bytes side by side in K and in V (whatever D is): they go
// through shared memory and leave as 16-byte stores. Tiles of tokens begin
// where the first token's slot is aligned. Other tokens store for themselves,
// V a byte at a time: 4096 tokens x 32 heads, D = 128, in runs 20 us, four prompts
// of odd lengths one behind the other 22.6 (their neighbours' bytes meet in L2),
// in random order 55.

// c of 8 codes (c + 4, 3 bits) in 24 bits, from the codes' floats (1.5 2^23 + 4 + c):
// the constant part of their bits is taken off once
__device__ __forceinline__ uint32_t pack8(const uint32_t (&b)[8]) {
  constexpr uint32_t k = 0x4B400000u * 0x249249u;  // sum of 8^i, i < 8
  uint32_t v = b[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) v = (v << 3) + b[i];
  return (v - k) & 0xFFFFFFu;
}

template <int GP>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  constexpr int D = 32 * GP, TT = 32 / GP;
  constexpr int RB = row_bytes(D);
  __shared__ __align__(16) uint8_t s_rows[8][384];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane % GP, t = lane / GP;
  pdl_wait();
  pdl_trigger();
  // (tile, K or V, head); fewer than 2^32 warps but for the very largest calls
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const int64_t tile = (w >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(w) / static_cast<uint32_t>(2 * a.H)) : w / (2 * a.H);
  const int kvh = static_cast<int>(w - tile * 2 * a.H);
  const bool is_v = kvh >= a.H;
  const int h = is_v ? kvh - static_cast<int>(a.H) : kvh;
  const int first = __ldg(a.slots);
  const int64_t tok = tile * TT - (first >= 0 ? first % TT : 0) + t;
  int slot = -1, j4 = -1;
  if (tok >= 0 && tok < a.n) {
    slot = __ldg(a.slots + tok);
    if (a.row4) j4 = __ldg(a.row4 + tok);
    if (slot >= 0 && (slot / PT >= a.n_pages || j4 >= a.C4)) {
      report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
      slot = -1;
    }
  }
  uint4 w4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w4[i] = make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0) {
    const uint16_t* src = (is_v ? a.v + tok * a.ldv : a.k + tok * a.ldk) + static_cast<int64_t>(h) * D + 32 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) w4[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
  }
  const uint32_t x[16] = {w4[0].x, w4[0].y, w4[0].z, w4[0].w, w4[1].x, w4[1].y, w4[1].z, w4[1].w,
                          w4[2].x, w4[2].y, w4[2].z, w4[2].w, w4[3].x, w4[3].y, w4[3].z, w4[3].w};
  uint32_t am = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) am = absmax_bf16x2(am, x[i]);
  uint32_t key = max(am & 0x7FFFu, (am >> 16) & 0x7FFFu);
#pragma unroll
  for (int o = GP / 2; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  const int slot0 = __shfl_sync(0xffffffffu, slot, 0);
  const bool run = __all_sync(0xffffffffu, slot0 >= 0 && slot0 % TT == 0 && slot == slot0 + t && j4 < 0);
  if (!run && slot < 0) return;
  const bool four = j4 >= 0;
  const float Q = four ? 7.f : 3.f;
  const float amax = fmaxf(__uint_as_float(key << 16), kEps);
  const float inv = __fdiv_rn(Q, amax);
  const int page = slot / PT, o = slot % PT;
  uint8_t* blk = a.pages + (static_cast<int64_t>(page) * a.H + h) * block_bytes(D);
  if (g == 0) {
    const float s = __fdiv_rn(amax, Q);
    reinterpret_cast<float*>(blk + (is_v ? off_vs(D) : off_ks(D)))[o] = four && !is_v ? -s : s;
  }
  uint32_t p[3] = {0u, 0u, 0u};
  auto value = [&](int i) { return __uint_as_float((i & 1) ? (x[i >> 1] & 0xFFFF0000u) : (x[i >> 1] << 16)); };
  if (!four) {
    // |x inv| <= 3 (1 + 2^-23): the codes need no clamp
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float lo = value(8 * e + i), hi = value(8 * e + i + 1);
        mul_then_add_rn(lo, hi, inv, 12582916.f);
        b[i] = __float_as_uint(lo);
        b[i + 1] = __float_as_uint(hi);
      }
      q[e] = pack8(b);
    }
    p[0] = q[0] | q[1] << 24;
    p[1] = q[1] >> 8 | q[2] << 16;
    p[2] = q[2] >> 16 | q[3] << 8;
  } else {
    uint32_t q[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 32; ++i) q[i >> 3] |= static_cast<uint32_t>(quant_code(value(i), inv, -8.f, 7.f) + 8) << (4 * (i & 7));
    uint8_t* r4 = a.codes4 + ((static_cast<int64_t>(page) * a.H + h) * a.C4 + j4) * D + (is_v ? D / 2 : 0);
    reinterpret_cast<uint4*>(r4)[g] = make_uint4(q[0], q[1], q[2], q[3]);
    if (!is_v && g == 0) p[0] = static_cast<uint32_t>(j4);
  }
  // where the lane's bytes go: K row o, or every fourth byte of V's group of 4 tokens
  uint8_t* dst = run ? s_rows[warp] : blk + (is_v ? off_v(D) : 0);
  const int row = run ? t : o;
  if (!is_v) {
    uint32_t* d = reinterpret_cast<uint32_t*>(dst + row * RB + 12 * g);
    d[0] = p[0]; d[1] = p[1]; d[2] = p[2];
  } else {
    uint8_t* d = dst + (row / 4) * 4 * RB + 48 * g + (row & 3);
#pragma unroll
    for (int i = 0; i < 12; ++i) d[4 * i] = static_cast<uint8_t>(p[i >> 2] >> (8 * (i & 3)));
  }
  if (run) {
    __syncwarp();
    uint8_t* out = a.pages + (static_cast<int64_t>(slot0 / PT) * a.H + h) * block_bytes(D) + (is_v ? off_v(D) : 0) + slot0 % PT * RB;
    if (lane < 24) reinterpret_cast<uint4*>(out)[lane] = reinterpret_cast<const uint4*>(s_rows[warp])[lane];
  }
}

// -------------------------------------------------------------- page copies
// Pair i copies page src[i] onto page dst[i] in every layer, the codes4 rows
// with it. A block takes 16 KB pieces of (pair, layer) in turn.
constexpr int kCopyPiece = 16384;

__global__ void __launch_bounds__(256) copy_kernel(const CopyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = a.count ? min(static_cast<int64_t>(*a.count), a.n) : a.n;
  const int64_t p3 = (a.page_bytes + kCopyPiece - 1) / kCopyPiece;
  const int64_t p4 = (a.page_bytes4 + kCopyPiece - 1) / kCopyPiece;
  const int64_t per_pair = (p3 + p4) * a.L;
  for (int64_t w = blockIdx.x; w < n * per_pair; w += gridDim.x) {
    const int64_t i = w / per_pair;
    int64_t r = w - i * per_pair;
    const int64_t l = r / (p3 + p4);
    r -= l * (p3 + p4);
    const int s = __ldg(a.src + i), d = __ldg(a.dst + i);
    if (s < 0 && d < 0) continue;  // no copy
    if (s < 0 || d < 0 || s >= a.n_pages || d >= a.n_pages) {
      if (threadIdx.x == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
      continue;
    }
    const bool four = r >= p3;
    const int64_t bytes = four ? a.page_bytes4 : a.page_bytes;
    const int64_t off = (four ? r - p3 : r) * kCopyPiece;
    uint8_t* base = (four ? a.codes4 : a.pages) + l * a.n_pages * bytes + off;
    const uint4* from = reinterpret_cast<const uint4*>(base + s * bytes);
    uint4* to = reinterpret_cast<uint4*>(base + d * bytes);
    const int m = static_cast<int>(min(static_cast<int64_t>(kCopyPiece), bytes - off) / 16);
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (threadIdx.x + 256 * k < m) v[k] = from[threadIdx.x + 256 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (threadIdx.x + 256 * k < m) to[threadIdx.x + 256 * k] = v[k];
  }
}

// --------------------------------------------------------------------- fork
// One block an entry. An entry reads its parent's row and writes its child's:
// rows that are both, and rows that are children twice, are turned down, so no
// entry reads what another one writes.
__global__ void __launch_bounds__(128) fork_kernel(const TableArgs t, const int32_t* __restrict__ parents,
                                                   const int32_t* __restrict__ children, int n) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int parent = __ldg(parents + i), child = __ldg(children + i);
  bool bad = parent < 0 || parent >= t.R || child < 0 || child >= t.R;
  for (int j = threadIdx.x; j < n; j += 128) {
    const int c = __ldg(children + j);
    bad |= c == parent || (j < i && c == child);
  }
  bad = __syncthreads_or(bad);
  int len = 0;
  if (!bad) {
    len = t.lens[parent];
    bad = len < 0 || pages_of(len) > t.W || t.lens[child] != 0;
  }
  __syncthreads();  // lens[child] has been read by all
  if (bad) {
    if (threadIdx.x == 0) report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
    return;
  }
  const int32_t* from = t.tables + static_cast<int64_t>(parent) * t.ldt;
  int32_t* to = t.tables + static_cast<int64_t>(child) * t.ldt;
  for (int j = threadIdx.x; j < pages_of(len); j += 128) {
    const int p = from[j];
    to[j] = p;
    if (p >= 0 && p < t.n_pages) atomicAdd(t.refs + p, 1);
    else report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
  }
  if (threadIdx.x == 0) t.lens[child] = len;
}

// --------------------------------------------------------------------- free
// One block a row: the pages behind the kept tokens lose a reference. A row
// named again is the first entry's alone.
__global__ void __launch_bounds__(128) free_kernel(const TableArgs t, const int32_t* __restrict__ rows,
                                                   const int32_t* __restrict__ keep, int n) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int row = __ldg(rows + i);
  bool again = false;
  for (int j = threadIdx.x; j < i; j += 128) again |= __ldg(rows + j) == row;
  if (__syncthreads_or(again)) return;
  const int k = keep ? __ldg(keep + i) : 0;
  bool bad = row < 0 || row >= t.R || k < 0;
  int len = 0;
  if (!bad) {
    len = t.lens[row];
    bad = len < 0 || pages_of(len) > t.W;
  }
  __syncthreads();  // lens[row] has been read by all
  if (bad) {
    if (threadIdx.x == 0) report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
    return;
  }
  if (k >= len) return;
  const int32_t* table = t.tables + static_cast<int64_t>(row) * t.ldt;
  for (int j = pages_of(k) + threadIdx.x; j < pages_of(len); j += 128) {
    const int p = table[j];
    if (p < 0 || p >= t.n_pages) {
      report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
    } else if (atomicSub(t.refs + p, 1) <= 0) {
      atomicAdd(t.refs + p, 1);
      report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
    }
  }
  if (threadIdx.x == 0) t.lens[row] = k;
}

// ------------------------------------------------------------- block helpers
constexpr int kBig = 1024;

// Inclusive sum over the block's threads; *total gets the sum of all.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // s_warp may still be read from the call before
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return v + (warp ? s_warp[warp - 1] : 0);
}

// --------------------------------------------------------------------- grow
// One block. Entry i wants its row to hold n_new[i] more tokens; the entries
// are served as if one after the other, in list order:
//   * a partly filled last page that others share is left (a reference less)
//     and copied to a new page: entry i does so when, after the entries
//     before it that leave the same page, more than one reference is left;
//   * new pages follow for the tokens beyond it.
// New pages are the lowest free ones, handed out in list order: entry i takes
// the free pages first[i] .. first[i] + need[i] - 1 of the pool, found by one
// walk over refs with a running count. The walk writes them into the tables
// behind the rows' ends, where entries say nothing yet; only when all needs
// are met do references, lengths and left pages change.
constexpr int kWalk = 16;  // reference counts that a thread takes at a time, at most

__global__ void __launch_bounds__(kBig) grow_kernel(const TableArgs t, const int32_t* __restrict__ rows,
                                                    const int32_t* __restrict__ n_new, int n, int max_new,
                                                    int32_t* __restrict__ slots, int32_t* __restrict__ cow_src,
                                                    int32_t* __restrict__ cow_dst) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_row[kBig], s_len[kBig], s_new[kBig], s_last[kBig], s_first[kBig + 1], s_page[kBig], s_count[kBig];
  __shared__ int s_warp[32];
  const int i = threadIdx.x;
  int row = -1, len = 0, add = 0, last = -1;
  bool bad = false;
  if (i < n) {
    row = __ldg(rows + i);
    add = __ldg(n_new + i);
    bad = row < 0 || row >= t.R || add < 0 || add > max_new;
    if (!bad) {
      len = t.lens[row];
      bad = len < 0 || (static_cast<int64_t>(len) + add + PT - 1) / PT > t.W;
    }
  }
  // an entry's earlier ones of the same row, and of the same last page below: all pairs over all threads
  auto earlier = [&](const int* of) {
    s_count[i] = 0;
    __syncthreads();
    for (int k = i; k < n * n; k += kBig) {
      const int e = k / n, j = k - e * n;
      if (j < e && of[j] == of[e]) atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    return s_count[i];
  };
  s_row[i] = row;
  bad |= earlier(s_row) > 0;
  const int have = pages_of(len);
  if (i < n && !bad && add > 0 && len % PT != 0) {
    last = t.tables[static_cast<int64_t>(row) * t.ldt + have - 1];
    if (last < 0 || last >= t.n_pages) { bad = true; last = -1; }
  }
  if (bad) { add = 0; report_status(t.status, BITLINEAR_STATUS_BAD_INDEX); }
  s_last[i] = last;
  const int shares = last >= 0 ? t.refs[last] : 0;
  const int before = earlier(s_last);
  const bool copy = shares > 1 && shares - before > 1;
  const int need = i < n && !bad ? pages_of(len + add) - have + (copy ? 1 : 0) : 0;
  int total;
  const int upto = block_scan(need, s_warp, &total);
  s_first[i] = upto - need;
  if (i == 0) s_first[kBig] = total;
  s_len[i] = len;
  s_new[i] = bad ? -1 : add;
  s_page[i] = copy ? 0 : -1;
  __syncthreads();

  // the lowest `total` free pages
  // (a small pool over all threads: a thread that finds several pages places them one after the other)
  int found = 0;
  const int walk = min(kWalk, (t.n_pages + kBig - 1) / kBig);
  for (int64_t base = 0; base < t.n_pages && found < total; base += kBig * walk) {
    const int64_t at = base + static_cast<int64_t>(i) * walk;
    uint32_t zero = 0u;
#pragma unroll
    for (int k = 0; k < kWalk; ++k)
      if (k < walk && at + k < t.n_pages && t.refs[at + k] == 0) zero |= 1u << k;
    int sum;
    int j = found + block_scan(__popc(zero), s_warp, &sum) - __popc(zero);
    while (zero && j < total) {
      const int page = static_cast<int>(at) + __ffs(zero) - 1;
      zero &= zero - 1u;
      int lo = 0, hi = n - 1;  // the last entry with first <= j (entries without need share a first)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= j) lo = mid; else hi = mid - 1;
      }
      const int e = j - s_first[lo], cp = s_page[lo] >= 0 ? 1 : 0;
      if (e < cp) s_page[lo] = page + 1;  // kept aside until the needs are met (0: wanted)
      else t.tables[static_cast<int64_t>(s_row[lo]) * t.ldt + pages_of(s_len[lo]) + e - cp] = page;
      ++j;
    }
    found += sum;
  }
  const bool met = found >= total;
  __syncthreads();
  const int to = s_page[i] - 1;  // the page that takes the copy
  if (i < n) {
    cow_src[i] = met && copy ? last : -1;
    cow_dst[i] = met && copy ? to : -1;
  }
  if (met && copy) {
    t.tables[static_cast<int64_t>(row) * t.ldt + have - 1] = to;
    t.refs[to] = 1;
    atomicSub(t.refs + last, 1);
  }
  if (met && i < n && !bad) t.lens[row] = len + add;
  if (!met && i == 0) report_status(t.status, BITLINEAR_STATUS_NO_PAGES);
  __syncthreads();
  if (met)
    for (int j = i; j < total; j += kBig) {
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= j) lo = mid; else hi = mid - 1;
      }
      const int e = j - s_first[lo], cp = s_page[lo] > 0 ? 1 : 0;
      if (e >= cp) t.refs[t.tables[static_cast<int64_t>(s_row[lo]) * t.ldt + pages_of(s_len[lo]) + e - cp]] = 1;
    }
  for (int64_t k = i; k < static_cast<int64_t>(n) * max_new; k += kBig) {
    const int e = static_cast<int>(k / max_new), u = static_cast<int>(k - static_cast<int64_t>(e) * max_new);
    int slot = -1;
    if (met && u < s_new[e]) {
      const int pos = s_len[e] + u;
      const int page = t.tables[static_cast<int64_t>(s_row[e]) * t.ldt + pos / PT];
      slot = page * PT + pos % PT;
    }
    slots[k] = slot;
  }
}

// ------------------------------------------------------------------ compact
// The live pages move into [0, n_live): hole k below n_live takes the k-th
// live page at or above it. One block counts, then lists holes and movers by
// a second walk; the copies and the tables follow in launches of their own.
__global__ void __launch_bounds__(kBig) compact_plan_kernel(int32_t* __restrict__ refs, int64_t n_pages,
                                                            int32_t* __restrict__ map, int32_t* __restrict__ src,
                                                            int32_t* __restrict__ dst, int32_t* __restrict__ count,
                                                            int32_t* __restrict__ n_live_out) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_warp[32];
  const int i = threadIdx.x;
  int mine = 0;
  for (int64_t p = i; p < n_pages; p += kBig) mine += refs[p] > 0;
  int live;
  block_scan(mine, s_warp, &live);
  int holes = 0, movers = 0;
  for (int64_t base = 0; base < n_pages; base += kBig * kWalk) {
    const int64_t at = base + static_cast<int64_t>(i) * kWalk;
    uint32_t bits = 0u;  // of holes below n_live, of live pages above
#pragma unroll
    for (int k = 0; k < kWalk; ++k)
      if (at + k < n_pages && (refs[at + k] > 0) == (at + k >= live)) bits |= 1u << k;
    // a thread's pages may lie on both sides of n_live
    const uint32_t below = at >= live ? 0u : at + kWalk <= live ? 0xFFFFu : (1u << (live - at)) - 1u;
    int sh, sm;
    uint32_t hb = bits & below, mb = bits & ~below;
    int jh = holes + block_scan(__popc(hb), s_warp, &sh) - __popc(hb);
    int jm = movers + block_scan(__popc(mb), s_warp, &sm) - __popc(mb);
    for (; hb; hb &= hb - 1u) dst[jh++] = static_cast<int>(at) + __ffs(hb) - 1;
    for (; mb; mb &= mb - 1u) src[jm++] = static_cast<int>(at) + __ffs(mb) - 1;
    holes += sh;
    movers += sm;
  }
  for (int64_t p = live + i; p < n_pages; p += kBig) map[p] = -1;
  __syncthreads();
  for (int k = i; k < movers; k += kBig) {  // as many movers as holes
    const int s = src[k], d = dst[k];
    refs[d] = refs[s];
    refs[s] = 0;
    map[s] = d;
  }
  if (i == 0) { *count = movers; *n_live_out = live; }
}

__global__ void __launch_bounds__(128) compact_tables_kernel(const TableArgs t, const int32_t* __restrict__ map,
                                                             const int32_t* __restrict__ n_live) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x;
  const int len = t.lens[row], live = *n_live;
  if (len < 0 || pages_of(len) > t.W) {
    if (threadIdx.x == 0) report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
    return;
  }
  int32_t* table = t.tables + static_cast<int64_t>(row) * t.ldt;
  for (int j = threadIdx.x; j < pages_of(len); j += 128) {
    const int p = table[j];
    int to = p;
    if (p < 0 || p >= t.n_pages) to = -1;
    else if (p >= live) to = map[p];
    if (to < 0) report_status(t.status, BITLINEAR_STATUS_BAD_INDEX);
    else if (to != p) table[j] = to;
  }
}

}  // namespace paged

cudaError_t launch_paged_append(const paged::AppendArgs& a, int64_t D, cudaStream_t s) {
  const int64_t tokens = 32 / (D / 32);  // of a tile; one tile more than fit, for the aligned beginning
  const int64_t warps = (a.n / tokens + 2) * 2 * a.H;
  const dim3 grid(static_cast<unsigned>((warps + 7) / 8));
  auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(256), 0, s, 0u, a); };
  if (D == 64) return go(paged::append_kernel<2>);
  if (D == 128) return go(paged::append_kernel<4>);
  return go(paged::append_kernel<8>);
}

static cudaError_t pages_copy(const paged::CopyArgs& a, cudaStream_t s, bool behind) {
  const int64_t pieces = (a.page_bytes + paged::kCopyPiece - 1) / paged::kCopyPiece +
                         (a.page_bytes4 + paged::kCopyPiece - 1) / paged::kCopyPiece;
  const int64_t want = a.n * a.L * pieces, cap = 8LL * num_sms();
  if (want == 0) return cudaSuccess;  // no layer, or no page to move: a kernel behind waits for the one before
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  return behind ? launch_behind(paged::copy_kernel, grid, dim3(256), 0, s, a)
                : launch_kernel(paged::copy_kernel, grid, dim3(256), 0, s, 0u, a);
}

cudaError_t launch_pages_copy(const paged::CopyArgs& a, cudaStream_t s) { return pages_copy(a, s, false); }

cudaError_t launch_pages_fork(const paged::TableArgs& t, const int32_t* parents, const int32_t* children, int64_t n,
                              cudaStream_t s) {
  return launch_kernel(paged::fork_kernel, dim3(static_cast<unsigned>(n)), dim3(128), 0, s, 0u, t, parents, children,
                       static_cast<int>(n));
}

cudaError_t launch_pages_free(const paged::TableArgs& t, const int32_t* rows, const int32_t* keep, int64_t n,
                              cudaStream_t s) {
  return launch_kernel(paged::free_kernel, dim3(static_cast<unsigned>(n)), dim3(128), 0, s, 0u, t, rows, keep,
                       static_cast<int>(n));
}

cudaError_t launch_pages_grow(const paged::TableArgs& t, const int32_t* rows, const int32_t* n_new, int64_t n,
                              int64_t max_new, int32_t* slots, int32_t* cow, const paged::CopyArgs& c,
                              cudaStream_t s) {
  cudaError_t e = launch_kernel(paged::grow_kernel, dim3(1), dim3(paged::kBig), 0, s, 0u, t, rows, n_new,
                                static_cast<int>(n), static_cast<int>(max_new), slots, cow, cow + n);
  if (e != cudaSuccess) return e;
  paged::CopyArgs a = c;
  a.src = cow;
  a.dst = cow + n;
  a.n = n;
  a.count = nullptr;
  return pages_copy(a, s, true);
}

cudaError_t launch_pages_compact(const paged::TableArgs& t, const paged::CopyArgs& c, int32_t* work,
                                 int32_t* n_live, cudaStream_t s) {
  int32_t* map = work;                       // [n_pages]
  int32_t* src = map + t.n_pages;            // at most n_pages / 2 movers
  int32_t* dst = src + (t.n_pages + 1) / 2;
  int32_t* count = dst + (t.n_pages + 1) / 2;
  cudaError_t e = launch_kernel(paged::compact_plan_kernel, dim3(1), dim3(paged::kBig), 0, s, 0u, t.refs,
                                static_cast<int64_t>(t.n_pages), map, src, dst, count, n_live);
  if (e != cudaSuccess) return e;
  paged::CopyArgs a = c;
  a.src = src;
  a.dst = dst;
  a.n = (t.n_pages + 1) / 2;
  a.count = count;
  e = pages_copy(a, s, true);
  if (e != cudaSuccess || t.R == 0) return e;
  return launch_behind(paged::compact_tables_kernel, dim3(static_cast<unsigned>(t.R)), dim3(128), 0, s, t,
                       static_cast<const int32_t*>(map), static_cast<const int32_t*>(n_live));
}

}  // namespace blt
