// Decode attention over the paged 3-bit cache (layout: paged.cuh).
//
// Query i of sequence b (length n_b, its Sq newest tokens the queries' own)
// sees the tokens t < n_b - Sq + 1 + i: token t lies in page shared[t / 64]
// while t < 64 n_shared, in page tables[b][t / 64 - n_shared] after that.
//   s_t = (q . k_t) / sqrt(D),  p = softmax_t(s),  o = sum_t p_t v_t
#include <cmath>

#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace blt {
namespace paged {

// One block a (query, head): 8 warps take the pages in turn, a lane two tokens
// of a page for the scores and D / 32 dimensions for the values.
template <int D>
__global__ void __launch_bounds__(256) attn_kernel(const AttnArgs a) {
  constexpr int RB = row_bytes(D), DL = D / 32;
  __shared__ float s_q[D], s_w[8][PT], s_o[8][D], s_m[8], s_l[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y / a.Sq, i = blockIdx.y % a.Sq, hq = blockIdx.x;
  const int h = hq / (a.Hq / a.H);
  for (int d = tid; d < D; d += 256)
    s_q[d] = __uint_as_float(static_cast<uint32_t>(a.q[blockIdx.y * a.ldq + hq * D + d]) << 16);
  __syncthreads();
  const int64_t cap = static_cast<int64_t>(a.n_shared + a.W) * PT;
  int len = a.lens[b];
  if (len < 0 || len > cap) {
    if (tid == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
    len = len < 0 ? 0 : static_cast<int>(cap);
  }
  const int sees = max(0, len - a.Sq + 1 + i);
  const float kq = a.qk_scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f, o[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) o[k] = 0.f;
  for (int j = warp; j < pages_of(sees); j += 8) {
    const int p = j < a.n_shared ? a.shared[j] : a.tables[b * a.ldt + j - a.n_shared];
    if (p < 0 || p >= a.n_pages) {
      if (lane == 0) report_status(a.status, BITLINEAR_STATUS_BAD_INDEX);
      continue;
    }
    const uint8_t* blk = a.pages + (static_cast<int64_t>(p) * a.H + h) * block_bytes(D);
    float s[2], vs[2];
    const uint8_t* r4[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = lane + 32 * u;
      s[u] = -INFINITY;
      vs[u] = 0.f;
      r4[u] = nullptr;
      if (j * PT + t >= sees) continue;
      const uint8_t* row = blk + t * RB;
      const float ks = reinterpret_cast<const float*>(blk + off_ks(D))[t];
      float dot = 0.f;
      if (signbit(ks)) {
        if (row[0] >= a.C4) { report_status(a.status, BITLINEAR_STATUS_BAD_INDEX); continue; }
        r4[u] = a.codes4 + ((static_cast<int64_t>(p) * a.H + h) * a.C4 + row[0]) * D;
        for (int d = 0; d < D; ++d) dot = fmaf(s_q[d], static_cast<float>(((r4[u][d / 2] >> (4 * (d & 1))) & 15) - 8), dot);
      } else {
        for (int d = 0; d < D; d += 8) {
          const uint32_t c = row[3 * d / 8] | (row[3 * d / 8 + 1] << 8) | (row[3 * d / 8 + 2] << 16);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(s_q[d + e], static_cast<float>(static_cast<int>((c >> (3 * e)) & 7u) - 4), dot);
        }
      }
      s[u] = dot * (fabsf(ks) * kq);
      vs[u] = reinterpret_cast<const float*>(blk + off_vs(D))[t];
    }
    float top = fmaxf(s[0], s[1]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float m_new = fmaxf(m, top);
    if (m_new == -INFINITY) continue;
    const float corr = exp2f(m - m_new);
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float e = s[u] == -INFINITY ? 0.f : exp2f(s[u] - m_new);
      sum += e;
      s_w[warp][lane + 32 * u] = e == 0.f ? 0.f : e * vs[u];
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = fmaf(l, corr, sum);
    m = m_new;
    uint32_t four[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) four[u] = __ballot_sync(0xffffffffu, r4[u] != nullptr);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < DL; ++k) o[k] *= corr;
    for (int t = 0; t < PT; ++t) {
      const float w = s_w[warp][t];
      const uint8_t* r = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(t < 32 ? r4[0] : r4[1]), t & 31));
      if (w == 0.f) continue;
#pragma unroll
      for (int k = 0; k < DL; ++k) {
        const int d = lane + 32 * k, bit = 3 * d;
        int c;
        if ((four[t >> 5] >> (t & 31)) & 1u) {
          c = ((r[D / 2 + d / 2] >> (4 * (d & 1))) & 15) - 8;
        } else {
          const uint8_t* v = blk + off_v(D) + (t >> 2) * 4 * RB + (t & 3);
          uint32_t x = v[4 * (bit >> 3)];
          if ((bit & 7) > 5) x |= static_cast<uint32_t>(v[4 * (bit >> 3) + 4]) << 8;
          c = static_cast<int>((x >> (bit & 7)) & 7u) - 4;
        }
        o[k] = fmaf(w, static_cast<float>(c), o[k]);
      }
    }
    __syncwarp();
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int k = 0; k < DL; ++k) s_o[warp][lane + 32 * k] = o[k];
  __syncthreads();
  for (int d = tid; d < D; d += 256) {
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) M = fmaxf(M, s_m[w]);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
      L = fmaf(f, s_l[w], L);
      O = fmaf(f, s_o[w][d], O);
    }
    a.out[(static_cast<int64_t>(blockIdx.y) * a.Hq + hq) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(L > 0.f ? O / L : 0.f));
  }
}

}  // namespace paged

int64_t paged_attention_workspace(int64_t B, int64_t Sq, int64_t Hq, int64_t H, int64_t D, int64_t n_shared,
                                  int64_t W) {
  return 0;
}

cudaError_t launch_paged_attention(const paged::AttnArgs& a, cudaStream_t s, const char** why) {
  const dim3 grid(static_cast<unsigned>(a.Hq), static_cast<unsigned>(a.B * a.Sq));
  auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(256), 0, s, 0u, a); };
  if (a.D == 64) return go(paged::attn_kernel<64>);
  if (a.D == 128) return go(paged::attn_kernel<128>);
  return go(paged::attn_kernel<256>);
}

}  // namespace blt
