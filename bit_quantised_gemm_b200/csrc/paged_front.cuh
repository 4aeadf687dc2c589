// What the tensor-core kernel for the shared pages (paged_front.cu) and the
// rest of the paged attention (paged_attn.cu) have to know of each other.
#pragma once
#include "launch.h"

namespace blt {
namespace paged {

// tiles of 128 rows that a CTA has in tensor memory
__host__ __device__ constexpr int front_streams(int D) { return D == 256 ? 1 : 2; }

// A head's tiles go in pairs and a single one where their number is odd (with
// one stream, all are single); a pair's pages are split into 2 k ranges, a
// single tile's into k: each CTA has as much to do as the others. CTA
// `item` = h (2 k pairs + k singles) + ...; its stream t writes piece
// streams x item + t.
struct FrontPlan {
  int pairs, singles, k;
  int64_t items;
};

struct FrontArgs {
  AttnArgs a;
  FrontPlan plan;
  float* parts;
  int raw_bytes, c4_bytes;
};

cudaError_t launch_front(const AttnArgs& a, const FrontPlan& plan, float* parts, cudaStream_t s);

}  // namespace paged
}  // namespace blt
