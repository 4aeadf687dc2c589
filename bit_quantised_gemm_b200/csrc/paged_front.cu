// Attention of many query rows over the shared pages of the paged 3-bit cache
// (layout: paged.cuh), on the 5th-generation tensor cores.
//
// The rows of all sequences that read one cache head are the rows of one
// product: 128 a tile. A CTA takes a range of the shared pages for one head and
// two "streams": two tiles on the same pages (each page taken apart once for
// both), or, where a head has an odd tile left, one tile with its even and its
// odd pages. With D = 256, tensor memory holds one stream.
//   loader      one warp, a bulk copy of a page's block into a ring (V's 16
//               groups one by one, further apart against bank conflicts, took
//               1900 clocks a page: about 100 a copy, however small)
//   unpackers   K -> [64 tokens][D], V -> [D][64 tokens] as fp16 codes - 4,
//               128-byte swizzled; a token kept at 4 bits is one of these rows
//   scaler      one warp, the scales beside them, and which tokens take part
//   issuers     a warp a stream, of which one thread issues: S = Q K^T (Q in
//               tensor memory), O += P V (P's two parts in tensor memory, where S was).
//               One warp for both streams had each wait for the other's softmax,
//               and its products queue up, which slows the softmax warps that
//               share its scheduler
//   softmax     4 warps a stream, a row a thread: s = S x (K scale),
//               p = 2^(s - m), weights p x (V scale) / 2^e as two fp16 numbers
//               each, the upper 11 bits and what is left (2^-22 of a weight is
//               lost; with one alone, 2^-11, outputs were 9e-4 from those of
//               32-bit weights, now 1e-4). The products of a page's first half
//               run while the second half's weights are made (142 us if not).
//               m bounds the scores so far and moves when one is above it. e
//               follows the largest weight, so that tokens without weight and
//               with large values do not press the others out of fp16's range,
//               and moves, and O is multiplied, when one reaches 2^15. A page's
//               largest score and V scale say whether one may: only then are
//               the weights themselves looked at. (Both in one reference, by
//               the page's largest V scale: 126 us, where this takes 128.)
// While one stream is in the softmax, the other's products run.
//
// A page of two tiles takes about 4000 clocks at D = 128 (96 sequences x 32 query
// heads on 8 cache heads behind 32768 tokens: 43 pages in 188000 clocks of a CTA,
// beginning and end included), where the tensor pipe needs 1536 and the
// exponentials 1024: a stream's chain of products, barriers, tensor-memory load,
// maximum and weights is that long, and tensor memory holds no third stream and no
// second S. While a weight was one number and a page 3500 clocks, P through shared
// memory (the next S is then there when a softmax ends) was slower, 105 us against
// 101: the products' operands, the unpackers and the scales already take more than
// half of what shared memory can move.
#include "launch.h"
#include "paged.cuh"
#include "paged_mma.cuh"
#include "paged_front.cuh"
#include "ptx.cuh"

namespace blt {
namespace paged {
namespace {

template <int D>
struct Shape {
  static constexpr int STREAMS = front_streams(D);
  static constexpr int NST = D == 256 ? 2 : 4;       // K and V tiles
  static constexpr int NRAW = D == 256 ? 3 : 4;      // blocks as they come
  static constexpr int SOFT = 4 * STREAMS, UNPACK = D == 256 ? 8 : 4;  // warps
  static constexpr int LOADER = SOFT + UNPACK, SCALER = LOADER + 1, ISSUER = SCALER + 1, THREADS = 32 * (ISSUER + STREAMS);
  static constexpr int RB = row_bytes(D);
  static constexpr int TILE = PT * D * 2;
  static constexpr int O = 0, Q = STREAMS * D, S = Q + STREAMS * (D / 2);  // tensor memory columns
  static_assert(S + STREAMS * PT <= 512);
};

template <int D>
struct Shared {
  using H = Shape<D>;
  float ks[H::NST][PT], vs[H::NST][PT];
  uint64_t dead[H::NST];  // tokens that take no part
  int v_exp[H::NST];      // the V scales are below 2^v_exp
  int page[H::NRAW];
  uint64_t raw_full[H::NRAW], raw_empty[H::NRAW], k_full[H::NST], v_full[H::NST], v_empty[H::NST];
  uint64_t q_full[2], s_full[2], p_full[2][2], pv_done[2], drain[2];
  uint32_t tmem;
  int abort;
};

// D[tmem] (+)= A[tmem] B[smem]^T, fp16 x fp16 -> fp32
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A 128-byte swizzled K-major operand's descriptor `words` 16-byte units behind
// the one whose lower half is lo (the upper half has no address in it): one
// addition an MMA, the issuing thread being the only one that can feed the tensor cores.
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t words) {
  constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | 2u << 29;
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + words), "r"(hi));
  return d;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | 1u << 16; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// two codes of a 4-bit row (in the low nibbles of the halves) as fp16 (c - 8) 2^(j - 9): exact
__device__ __forceinline__ uint32_t four_bits(uint32_t x, int jl, int jh) {
  const uint32_t scale = (jl + 6) << 10 | (jh + 6) << 26;  // 2^(j - 9)
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((x & 0x000F000Fu) | 0x64006400u), "r"(0x64086408u));  // 1024 + c - 1032
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(scale));
  return r;
}

__constant__ uint8_t kPairs[16][4] = {  // pair32's codes and their bits in the halves
#define BLT_P(I) {pair32(I).lo, pair32(I).hi, 3 * pair32(I).lo - pair32(I).n, 3 * pair32(I).hi - pair32(I).n - 16}
    BLT_P(0), BLT_P(1), BLT_P(2), BLT_P(3), BLT_P(4), BLT_P(5), BLT_P(6), BLT_P(7),
    BLT_P(8), BLT_P(9), BLT_P(10), BLT_P(11), BLT_P(12), BLT_P(13), BLT_P(14), BLT_P(15)};
#undef BLT_P

template <int D>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1) front_kernel(const __grid_constant__ FrontArgs p) {
  using H = Shape<D>;
  constexpr int STREAMS = H::STREAMS, NST = H::NST, NRAW = H::NRAW, RB = H::RB;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared<D> sm;
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  uint8_t* base = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
  uint8_t* k_tile = base;
  uint8_t* v_tile = k_tile + NST * H::TILE;
  uint8_t* raw = v_tile + NST * H::TILE;

  // ---- the item: head, tiles, pages
  const int per_head = p.plan.pairs * 2 * p.plan.k + p.plan.singles * p.plan.k;
  const int item = blockIdx.x, h = item / per_head;
  int split = item - h * per_head, parts = 2 * p.plan.k, tile0 = 0;
  const bool pair = split < p.plan.pairs * 2 * p.plan.k;
  if (pair) {
    tile0 = 2 * (split / parts);
    split %= parts;
  } else {
    split -= p.plan.pairs * 2 * p.plan.k;
    parts = p.plan.k;
    tile0 = 2 * p.plan.pairs + split / parts;
    split %= parts;
  }
  const int first = static_cast<int>(static_cast<int64_t>(a.n_shared) * split / parts);
  const int n = static_cast<int>(static_cast<int64_t>(a.n_shared) * (split + 1) / parts) - first;
  const int G = a.Hq / a.H, rows = a.B * a.Sq * G;
  const bool alternate = STREAMS == 2 && !pair;
  auto stream_pages = [&](int t) { return alternate ? (n - t + 1) >> 1 : n; };
  auto stream_rows = [&](int t) { return min(128, rows - 128 * (tile0 + (pair ? t : 0))); };

  if (tid == 0) {
    for (int i = 0; i < NRAW; ++i) { mbar_init(&sm.raw_full[i], 1); mbar_init(&sm.raw_empty[i], H::UNPACK + 1); }
    for (int i = 0; i < NST; ++i) {
      mbar_init(&sm.k_full[i], H::UNPACK + 1);
      mbar_init(&sm.v_full[i], H::UNPACK); mbar_init(&sm.v_empty[i], pair ? 2 : 1);
    }
    for (int t = 0; t < STREAMS; ++t) {
      const int live = (stream_rows(t) + 31) / 32;  // warps with rows
      mbar_init(&sm.q_full[t], live);
      mbar_init(&sm.s_full[t], 1);
      for (int i = 0; i < 2; ++i) mbar_init(&sm.p_full[t][i], live);
      mbar_init(&sm.pv_done[t], 1);
      mbar_init(&sm.drain[t], 1);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == H::ISSUER) { tmem_alloc(&sm.tmem, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tm = sm.tmem;
  volatile int* abort = &sm.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity & 1u, a.timeout_ns, abort)) return true;
    *abort = 1;
    return false;
  };

  if (warp == H::LOADER) {
    const int c4_bytes = p.c4_bytes;
    int ids = 0, put = 0;
    bool ok = true;
    for (; put < n; ++put) {
      if ((put & 31) == 0) ids = put + lane < n ? __ldg(a.shared + first + put + lane) : 0;
      const int page = __shfl_sync(0xFFFFFFFFu, ids, put & 31);
      const int st = put % NRAW;
      if (put >= NRAW) ok = wait(&sm.raw_empty[st], put / NRAW - 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const bool good = page >= 0 && page < a.n_pages;
      if (lane == 0) {
        sm.page[st] = good ? page : -1;
        if (good) mbar_arrive_expect_tx(&sm.raw_full[st], static_cast<uint32_t>(block_bytes(D) + c4_bytes));
        else { report_status(a.status, BITLINEAR_STATUS_BAD_INDEX); mbar_arrive(&sm.raw_full[st]); }
      }
      __syncwarp();
      if (good) {
        const int64_t at = static_cast<int64_t>(page) * a.H + h;
        uint8_t* dst = raw + st * p.raw_bytes;
        if (lane == 0) bulk_load(dst, a.pages + at * block_bytes(D), block_bytes(D), &sm.raw_full[st]);
        else if (lane == 1 && c4_bytes) bulk_load(dst + block_bytes(D), a.codes4 + at * c4_bytes, c4_bytes, &sm.raw_full[st]);
      }
    }
    if (*abort)  // copies in flight land before the memory is released
      for (int i = max(0, put - NRAW); i < put; ++i) mbar_wait(&sm.raw_full[i % NRAW], (i / NRAW) & 1, a.timeout_ns, nullptr);
  } else if (warp >= H::ISSUER) {
    // the warp stays together in the waits; one lane issues
    constexpr uint32_t idS = make_idesc(1, 0, 0, 128, PT), idO = make_idesc(1, 0, 0, 128, D);
    const int t = warp - H::ISSUER, np = stream_pages(t);
    const uint32_t k_lo = desc_lo(smem_u32(k_tile)), v_lo = desc_lo(smem_u32(v_tile));
    const bool lead = elect_one() != 0;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
    bool ok = np == 0 || wait_all(&sm.q_full[t], 0);
    for (int k = 0; k <= np && ok; ++k) {
      if (k > 0) {  // values of the page before
        const int pg = alternate ? 2 * (k - 1) + t : k - 1, st = pg % NST;
        const uint32_t vt = v_lo + st * (H::TILE >> 4);
        ok = wait_all(&sm.v_full[st], pg / NST);
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // the products of P's first tokens run while the others are made
          if (!(ok = ok && wait_all(&sm.p_full[t][half], k - 1))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int i = 0; i < PT / 16; ++i) {  // the weights' upper parts, then the lower ones
              const int at = PT / 32 * half + i % (PT / 32);
              mma_f16_ts(tm + H::O + t * D, tm + H::S + t * PT + 8 * at + i / (PT / 32) * (PT / 2), desc_at(vt, 2 * at), idO, k > 1 || half > 0 || i > 0);
            }
          }
        }
        if (!ok) break;
        if (lead) {
          tc_commit(&sm.pv_done[t]);
          tc_commit(&sm.v_empty[st]);
        }
        __syncwarp();
      }
      if (k < np) {  // scores of page k (in issue order behind the products that read P in their place)
        const int pg = alternate ? 2 * k + t : k, st = pg % NST;
        if (!(ok = wait_all(&sm.k_full[st], pg / NST))) break;
        tc_fence_after();
        if (lead) {
          const uint32_t kt = k_lo + st * (H::TILE >> 4);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_f16_ts(tm + H::S + t * PT, tm + H::Q + t * (D / 2) + 8 * i, desc_at(kt, (i >> 2) * (PT * 8) + (i & 3) * 2), idS, i > 0);
          tc_commit(&sm.s_full[t]);
        }
        __syncwarp();
      }
    }
    if (!ok && lead) {  // what was issued ends before the memory is released
      tc_commit(&sm.drain[t]);
      mbar_wait(&sm.drain[t], 0, a.timeout_ns, nullptr);
    }
    __syncwarp();
  } else if (warp == H::SCALER) {
    int seen = 0;  // tokens that any row sees
    for (int b = lane; b < a.B; b += 32) {
      bool bad;
      seen = max(seen, cut_len(a, b, &bad));
      if (bad && item == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
    }
    seen = __reduce_max_sync(0xFFFFFFFFu, seen);
    for (int pg = 0; pg < n; ++pg) {
      const int rs = pg % NRAW, st = pg % NST;
      bool ok = pg < NST || wait(&sm.v_empty[st], pg / NST - 1);
      ok = ok && wait(&sm.raw_full[rs], pg / NRAW);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const uint8_t* src = raw + rs * p.raw_bytes;
      const float* scales = reinterpret_cast<const float*>(src + off_ks(D));
      const int live = sm.page[rs] < 0 ? 0 : min(PT, seen - (first + pg) * PT);
      uint32_t dead[2];
      int top = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int o = lane + 32 * i;
        const float ks = scales[o], vs = scales[PT + o];
        const bool use = o < live;
        const bool bad4 = use && signbit(ks) && src[o * RB] >= a.C4;
        if (bad4) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
        dead[i] = __ballot_sync(0xFFFFFFFFu, !use || bad4);
        sm.ks[st][o] = use ? fabsf(ks) * (a.qk_scale * 1.4426950408889634f) : 0.f;
        sm.vs[st][o] = use ? vs : 0.f;
        if (use) top = max(top, __float_as_int(vs) >> 23);
      }
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (lane == 0) {
        sm.v_exp[st] = top - 126;
        sm.dead[st] = static_cast<uint64_t>(dead[1]) << 32 | dead[0];
      }
      __syncwarp();
      if (lane == 0) { mbar_arrive(&sm.k_full[st]); mbar_arrive(&sm.raw_empty[rs]); }
    }
  } else if (warp >= H::SOFT) {
    // ------------------------------------------------------------ unpackers
    const int ut = tid - 32 * H::SOFT, uw = warp - H::SOFT;
    // K: a lane a token's chunk of 32 codes; 8 (16) tokens x 4 (2) chunks a warp and step: no bank conflicts
    constexpr int CH = D / 32, CW = CH < 4 ? CH : 4, TW = 32 / CW, STEPS = PT * CH / (32 * H::UNPACK);
    const int e = lane & 7, dg = ut >> 3;  // V: a lane 8 dimensions of the tokens 4 e .. and 32 + 4 e ..
    const int p_lo = kPairs[lane & 15][0], p_hi = kPairs[lane & 15][1], p_jl = kPairs[lane & 15][2], p_jh = kPairs[lane & 15][3];
    // the words of a page, taken while the page before it is worked on
    uint32_t kw[STEPS][3], vw[2][3];
    int page = -1;
    auto take = [&](int pg) {
      const int rs = pg % NRAW;
      if (!__all_sync(0xFFFFFFFFu, wait(&sm.raw_full[rs], pg / NRAW))) return false;
      const uint8_t* src = raw + rs * p.raw_bytes;
      page = sm.page[rs];
#pragma unroll
      for (int it = 0; it < STEPS; ++it) {
        const int step = it * H::UNPACK + uw;
        const int o = step / (CH / CW) * TW + lane % TW, c = step % (CH / CW) * CW + lane / TW;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(src + o * RB + 12 * c);
#pragma unroll
        for (int i = 0; i < 3; ++i) kw[it][i] = w[i];
      }
      if (ut < D) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(src + off_v(D) + (e + 8 * q) * 4 * RB + 12 * dg);
#pragma unroll
          for (int i = 0; i < 3; ++i) vw[q][i] = w[i];
        }
      }
      return true;
    };
    bool ok = n > 0 && take(0);
    for (int pg = 0; pg < n && ok; ++pg) {
      const int rs = pg % NRAW, st = pg % NST;
      ok = pg < NST || wait(&sm.v_empty[st], pg / NST - 1);  // (the products of K end before those of V)
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const uint8_t* src = raw + rs * p.raw_bytes;
      const uint32_t kt = smem_u32(k_tile + st * H::TILE), vt = smem_u32(v_tile + st * H::TILE);
      const int now = page;
      uint64_t four = 0;  // tokens kept at 4 bits
      if (now < 0) {      // nothing there
        for (int i = ut; i < H::TILE / 16; i += 32 * H::UNPACK) st_shared_v4(kt + 16 * i, 0u, 0u, 0u, 0u);
      } else {
#pragma unroll
        for (int it = 0; it < STEPS; ++it) {
          const int step = it * H::UNPACK + uw;
          const int o = step / (CH / CW) * TW + lane % TW, c = step % (CH / CW) * CW + lane / TW;
          const uint32_t dst = kt + (c >> 1) * (PT * 128) + o * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_shared_v4(dst + ((((c & 1) * 4 + i) ^ (o & 7)) << 4), k_operand(kw[it], pair32(4 * i)), k_operand(kw[it], pair32(4 * i + 1)),
                         k_operand(kw[it], pair32(4 * i + 2)), k_operand(kw[it], pair32(4 * i + 3)));
        }
        if (a.C4 > 0) {
          const float* scales = reinterpret_cast<const float*>(src + off_ks(D));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int o = lane + 32 * i;
            four |= static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, signbit(scales[o]) && src[o * RB] < a.C4)) << (32 * i);
          }
          // their K rows, by the warp that has written what their 3-bit rows hold: lane i word i
          __syncwarp();
          for (uint64_t m = four; m; m &= m - 1) {
            const int o = __ffsll(static_cast<long long>(m)) - 1, j = src[o * RB];
            const uint8_t* r4 = p.c4_bytes ? src + block_bytes(D) + j * D : a.codes4 + ((static_cast<int64_t>(now) * a.H + h) * a.C4 + j) * D;
#pragma unroll
            for (int x = 0; x < CH / CW; ++x)
              if ((o / TW * (CH / CW) + x) % H::UNPACK == uw)
#pragma unroll
                for (int i = 0; i < CW / 2; ++i) {
                  const int c = x * CW + 2 * i + (lane >> 4);
                  const uint8_t* y = r4 + 16 * c;
                  const uint32_t v = four_bits((y[p_lo >> 1] >> (4 * (p_lo & 1)) & 15u) | (y[p_hi >> 1] >> (4 * (p_hi & 1)) & 15u) << 16, p_jl, p_jh);
                  asm volatile("st.shared.u32 [%0], %1;" ::"r"(kt + (c >> 1) * (PT * 128) + o * 128 +
                                                               ((((c & 1) * 4 + ((lane & 15) >> 2)) ^ (o & 7)) << 4) + 4 * (lane & 3)), "r"(v) : "memory");
                }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[st]);
      uint32_t x[8][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t (&X)[3] = vw[q];
        const uint32_t Y[3] = {X[0] >> 8, X[1] >> 8, X[2] >> 8};
        v_operand<0>(X, Y, x[0][2 * q], x[0][2 * q + 1]);
        v_operand<1>(X, Y, x[1][2 * q], x[1][2 * q + 1]);
        v_operand<2>(X, Y, x[2][2 * q], x[2][2 * q + 1]);
        v_operand<3>(X, Y, x[3][2 * q], x[3][2 * q + 1]);
        v_operand<4>(X, Y, x[4][2 * q], x[4][2 * q + 1]);
        v_operand<5>(X, Y, x[5][2 * q], x[5][2 * q + 1]);
        v_operand<6>(X, Y, x[6][2 * q], x[6][2 * q + 1]);
        v_operand<7>(X, Y, x[7][2 * q], x[7][2 * q + 1]);
      }
      if (pg + 1 < n) ok = take(pg + 1);
      if (now < 0) {
        for (int i = ut; i < H::TILE / 16; i += 32 * H::UNPACK) st_shared_v4(vt + 16 * i, 0u, 0u, 0u, 0u);
      } else if (ut < D) {
        const uint32_t dst = vt + dg * 1024;
#pragma unroll
        for (int d = 0; d < 8; ++d) st_shared_v4(dst + d * 128 + ((e ^ d) << 4), x[d][0], x[d][1], x[d][2], x[d][3]);
        for (uint64_t m = four; m; m &= m - 1) {  // 4-bit tokens: word 2 (o / 32) + o % 2, half o / 2 % 2
          const int o = __ffsll(static_cast<long long>(m)) - 1, j = src[o * RB];
          if (((o >> 2) & 7) != e) continue;
          const uint8_t* r4 = p.c4_bytes ? src + block_bytes(D) + j * D : a.codes4 + ((static_cast<int64_t>(now) * a.H + h) * a.C4 + j) * D;
          const uint32_t y = *reinterpret_cast<const uint32_t*>(r4 + D / 2 + 4 * dg);
          const int at = 4 * (2 * (o >> 5) + (o & 1)) + (o & 2);
#pragma unroll
          for (int d = 0; d < 8; d += 2) {
            const uint32_t v = four_bits((y >> (4 * d) & 15u) | (y >> (4 * d + 4) & 15u) << 16, v_bit(d), v_bit(d + 1));
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + d * 128 + ((e ^ d) << 4) + at), "h"(static_cast<uint16_t>(v)) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + (d + 1) * 128 + ((e ^ (d + 1)) << 4) + at), "h"(static_cast<uint16_t>(v >> 16)) : "memory");
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) { mbar_arrive(&sm.v_full[st]); mbar_arrive(&sm.raw_empty[rs]); }
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, np = stream_pages(t);
    const int r0 = 128 * (tile0 + (pair ? t : 0)) + 32 * (warp & 3), r = r0 + lane;
    const int col = 32 * (warp & 3) + lane;
    float* out = p.parts + (static_cast<int64_t>(item) * STREAMS + t) * piece_floats(D, 128);
    if (r0 < rows) {
      const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      const Segment sg{0, 0, rows, h, G, true};
      const int sees = row_sees(a, sg, r) - first * PT;  // from the item's first page on
      float kq = 0.f;
      if (np > 0) {  // the row's query: fp16, its largest value in [2^14, 2^15)
        const uint16_t* q = r < rows ? query_row(a, sg, r) : nullptr;
        uint32_t am = 0u;
        uint4 row[16];  // 128 dimensions, all of them where there are no more
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c) {
#pragma unroll
          for (int i = 0; i < (D < 128 ? D / 8 : 16); ++i) row[i] = q != nullptr ? __ldg(reinterpret_cast<const uint4*>(q) + 16 * c + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int i = 0; i < (D < 128 ? D / 8 : 16); ++i) {
            const uint4 v = row[i];
            am = max(am, max(max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu)),
                             max(max(v.z & 0x7FFFu, (v.z >> 16) & 0x7FFFu), max(v.w & 0x7FFFu, (v.w >> 16) & 0x7FFFu))));
          }
        }
        const int fb = min(268 - max(1, static_cast<int>(am >> 7)), 254);
        const float f = pow2_biased(fb);
        kq = pow2_biased(263 - fb);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // 32 dimensions
          uint32_t x[16], y[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = D <= 128 ? row[(4 * c + i) & 15] : q != nullptr ? __ldg(reinterpret_cast<const uint4*>(q) + 4 * c + i) : make_uint4(0u, 0u, 0u, 0u);
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
          }
          auto qf = [&](int d) { return __uint_as_float((d & 1) ? (x[d >> 1] & 0xFFFF0000u) : (x[d >> 1] << 16)) * f; };
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const Pair pr = pair32(i);
            y[i] = pack_f16x2(qf(pr.lo) * (1.f / (1 << (3 * pr.lo - pr.n))), qf(pr.hi) * (1.f / (1 << (3 * pr.hi - pr.n - 16))));
          }
          tmem_st16(tm + lanes + H::Q + t * (D / 2) + 16 * c, y);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[t]);
      }
      // pages before n_all are seen whole by all rows that see anything (a slot of the batch without a
      // request would send its warp through the masks on every page)
      const int n_all = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, sees <= 0 ? 0x7FFFFFFFu : static_cast<unsigned>(sees)) / PT);
      float m = -INFINITY, e = kLeastExp, l = 0.f;
      bool ok = true;
      for (int k = 0; k < np; ++k) {
        const int pg = alternate ? 2 * k + t : k, st = pg % NST;
        ok = wait(&sm.s_full[t], k);  // (the page's scales were there before S was begun)
        if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
        tc_fence_after();
        const uint64_t dead = sm.dead[st];
        const float v_top = static_cast<float>(sm.v_exp[st]);
        float2 s[PT / 2];
        {
          uint32_t x[PT];
          tmem_ld64(tm + lanes + H::S + t * PT, x);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < PT; i += 4) {
            const float4 ks = *reinterpret_cast<const float4*>(&sm.ks[st][i]);
            s[i / 2] = __fmul2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), make_float2(ks.x, ks.y));
            s[i / 2 + 1] = __fmul2_rn(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), make_float2(ks.z, ks.w));
          }
        }
        if (pg >= n_all || dead != 0) {
          const int lim = sees - pg * PT;
          const uint64_t on = ~dead & (lim >= PT ? ~0ull : lim <= 0 ? 0ull : (1ull << lim) - 1ull);
          const uint32_t w[2] = {static_cast<uint32_t>(on), static_cast<uint32_t>(on >> 32)};
#pragma unroll
          for (int i = 0; i < PT; i += 2) {
            if (!(w[i >> 5] & (1u << (i & 31)))) s[i / 2].x = -INFINITY;
            if (!(w[i >> 5] & (2u << (i & 31)))) s[i / 2].y = -INFINITY;
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < PT / 2; ++i) mx[i & 3] = max3(mx[i & 3], s[i].x, s[i].y);
        mx[0] = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        const float top = mx[0] * kq;  // (exact)
        if (__any_sync(0xFFFFFFFFu, top > m || top - m + v_top - e > 15.f)) {
          float f = 1.f;  // of the value sums
          if (top > m) {
            const float now = reference(top), d = m - now;
            l *= ex2(d);
            m = now;
            e += d;
            if (e < kLeastExp) {
              f = ex2(e - kLeastExp);
              e = kLeastExp;
            }
          }
          float w = 0.f;
          const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int i = 0; i < PT; i += 4) {
            const float4 vs = *reinterpret_cast<const float4*>(&sm.vs[st][i]);
            w = max3(w, ex2(fmaf(s[i / 2].x, kq, -mr)) * vs.x, ex2(fmaf(s[i / 2].y, kq, -mr)) * vs.y);
            w = max3(w, ex2(fmaf(s[i / 2 + 1].x, kq, -mr)) * vs.z, ex2(fmaf(s[i / 2 + 1].y, kq, -mr)) * vs.w);
          }
          if (!(w * ex2(-e) < kMostWeight)) {
            const float now = weight_exp(w);
            f *= ex2(e - now);
            e = now;
          }
          if (k > 0 && __any_sync(0xFFFFFFFFu, f != 1.f)) {
            ok = wait(&sm.pv_done[t], k - 1);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t x[32];
              tmem_ld32(tm + lanes + H::O + t * D + 32 * c, x);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
              tmem_st32(tm + lanes + H::O + t * D + 32 * c, x);
            }
            tmem_st_wait();
          }
        }
        const float mr = m == -INFINITY ? 0.f : m, wf = ex2(-e);
        const float2 kq2 = make_float2(kq, kq), mr2 = make_float2(-mr, -mr), wf2 = make_float2(wf, wf);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // the words of P in V's order: within 4 tokens 0, 2, 1, 3, and 4 tokens of each half of the page in turn
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[PT / 4], lo[PT / 4];
#pragma unroll
          for (int at = 0; at < PT / 4; at += 2) {
            const int i = PT / 4 * half + at / 4 * 4 + PT / 2 * (at / 2 % 2);
            const float4 vs = *reinterpret_cast<const float4*>(&sm.vs[st][i]);
            float2 u = __ffma2_rn(s[i / 2], kq2, mr2), v = __ffma2_rn(s[i / 2 + 1], kq2, mr2);
            u = make_float2(ex2(u.x), ex2(u.y));
            v = make_float2(ex2(v.x), ex2(v.y));
            sum[0] = __fadd2_rn(sum[0], u);
            sum[1] = __fadd2_rn(sum[1], v);
            u = __fmul2_rn(__fmul2_rn(u, make_float2(vs.x, vs.y)), wf2);
            v = __fmul2_rn(__fmul2_rn(v, make_float2(vs.z, vs.w)), wf2);
            const float2 ut = make_float2(f16_top(u.x), f16_top(u.y)), vt = make_float2(f16_top(v.x), f16_top(v.y));
            w[at] = pack_f16x2(ut.x, vt.x);
            w[at + 1] = pack_f16x2(ut.y, vt.y);
            u = __fadd2_rn(u, make_float2(-ut.x, -ut.y));
            v = __fadd2_rn(v, make_float2(-vt.x, -vt.y));
            lo[at] = pack_f16x2(u.x, v.x);
            lo[at + 1] = pack_f16x2(u.y, v.y);
          }
          tmem_st16(tm + lanes + H::S + t * PT + PT / 4 * half, w);
          tmem_st16(tm + lanes + H::S + t * PT + PT / 2 + PT / 4 * half, lo);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[t][half]);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ---- the piece
      if (ok && np > 0) {
        ok = wait(&sm.pv_done[t], np - 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
      }
      if (ok) {
        const float vf = ex2(e);
        if (np > 0)
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            tmem_ld32(tm + lanes + H::O + t * D + 32 * c, x);
            tmem_ld_wait();
            if (r < rows) {
              float4* dst = reinterpret_cast<float4*>(out + col * D + 32 * c);
              auto o = [&](int i) { return __uint_as_float(x[i]) * (512.f / static_cast<float>(1 << v_bit(i & 7))) * vf; };
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_float4(o(4 * i), o(4 * i + 1), o(4 * i + 2), o(4 * i + 3));
            }
          }
        if (r < rows) {
          out[128 * D + col] = sees > 0 ? m : -INFINITY;
          out[128 * D + 128 + col] = sees > 0 ? l : 0.f;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sm.abort) report_status(a.status, BITLINEAR_STATUS_TIMEOUT);
  if (warp == H::ISSUER) tmem_dealloc(tm, 512);
}

template <int D>
cudaError_t launch_front_t(const AttnArgs& a, const FrontPlan& plan, float* parts, cudaStream_t s) {
  using H = Shape<D>;
  FrontArgs p{};
  p.a = a;
  p.plan = plan;
  p.parts = parts;
  p.c4_bytes = a.C4 <= kStageRows4 ? a.C4 * D : 0;
  p.raw_bytes = block_bytes(D) + p.c4_bytes;
  const int smem = 1024 + 2 * H::NST * H::TILE + H::NRAW * p.raw_bytes;
  const cudaError_t e = set_smem_limit(front_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(front_kernel<D>, dim3(static_cast<unsigned>(plan.items)), dim3(H::THREADS), smem, s, 0u, p);
}

}  // namespace

cudaError_t launch_front(const AttnArgs& a, const FrontPlan& plan, float* parts, cudaStream_t s) {
  if (a.D == 64) return launch_front_t<64>(a, plan, parts, s);
  if (a.D == 128) return launch_front_t<128>(a, plan, parts, s);
  return launch_front_t<256>(a, plan, parts, s);
}

}  // namespace paged
}  // namespace blt
