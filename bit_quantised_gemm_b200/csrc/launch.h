// Internal launchers behind the C ABI (host side). Arguments are already
// validated by the entry points in api.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include "../../include/bitlinear.h"

namespace blt {

cudaError_t launch_quant_act(const uint16_t* x, const uint16_t* up, int64_t M, int64_t K,
                             int64_t ldx, int mode, void* q, float* xs, cudaStream_t s);
cudaError_t launch_topk_i8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int64_t k,
                           int8_t* q, float* xs, uint8_t* mask, cudaStream_t s);
cudaError_t launch_kv_attention(const uint16_t* q, int64_t B, int64_t H, int64_t D, int64_t T,
                                const uint8_t* k3, const uint8_t* k4, const float* ks,
                                const uint8_t* v3, const uint8_t* v4, const float* vs,
                                const int32_t* keep4, int64_t n4, uint16_t* out, int* status,
                                uint64_t timeout_ns, cudaStream_t s, const char** why);
cudaError_t launch_keep4_positions(const int32_t* ids, int64_t T, const int32_t* special, int n_special,
                                   int32_t* pos, int32_t* count, cudaStream_t s);
cudaError_t launch_kv_quant(const uint16_t* kv, int64_t T, int64_t H, int64_t D,
                            const int32_t* keep4, int64_t n4, uint8_t* codes3, uint8_t* codes4,
                            float* scale, cudaStream_t s);
cudaError_t launch_kv_quant_pair(const uint16_t* k, const uint16_t* v, int64_t T, int64_t H, int64_t D,
                                 const int32_t* keep4, int64_t n4, uint8_t* k3, uint8_t* k4, float* ks,
                                 uint8_t* v3, uint8_t* v4, float* vs, cudaStream_t s);

// The paged 3-bit cache (paged.cu, paged_attn.cu).
namespace paged {
struct AppendArgs {
  const uint16_t* k;     // bf16 [n][H][D], tokens ldk apart
  const uint16_t* v;
  int64_t ldk, ldv;
  int64_t n, H;
  const int32_t* slots;  // [n]
  const int32_t* row4;   // [n] or null
  uint8_t* pages;
  int64_t n_pages;
  uint8_t* codes4;
  int64_t C4;
  int* status;
};
struct CopyArgs {
  uint8_t* pages;        // [L][n_pages][page_bytes]
  uint8_t* codes4;       // [L][n_pages][page_bytes4]
  int64_t L, n_pages, page_bytes, page_bytes4;
  const int32_t* src;    // [n]
  const int32_t* dst;
  int64_t n;
  const int32_t* count;  // device, or null: only the first *count pairs
  int* status;
};
struct TableArgs {
  int32_t* tables;       // [R][W], rows ldt apart
  int64_t ldt;
  int R, W;
  int32_t* lens;         // [R]
  int32_t* refs;         // [n_pages]
  int n_pages;
  int* status;
};
struct AttnArgs {
  const uint16_t* q;     // bf16 [B][Sq][Hq][D], tokens (b, i) ldq apart
  int64_t ldq;
  int B, Sq, Hq, H, D;
  const uint8_t* pages;
  int n_pages;
  const uint8_t* codes4;
  int C4;
  const int32_t* shared; // [n_shared]
  int n_shared;
  const int32_t* tables; // [B][W], rows ldt apart
  int64_t ldt;
  int W;
  const int32_t* lens;   // [B]
  float qk_scale;        // 1 / sqrt(D)
  uint16_t* out;         // bf16 [B][Sq][Hq][D]
  uint8_t* work;
  int* status;
  uint64_t timeout_ns;
};
}  // namespace paged
cudaError_t launch_paged_append(const paged::AppendArgs& a, int64_t D, cudaStream_t s);
cudaError_t launch_pages_copy(const paged::CopyArgs& a, cudaStream_t s);
cudaError_t launch_pages_fork(const paged::TableArgs& t, const int32_t* parents, const int32_t* children, int64_t n,
                              cudaStream_t s);
cudaError_t launch_pages_free(const paged::TableArgs& t, const int32_t* rows, const int32_t* keep, int64_t n,
                              cudaStream_t s);
// cow: device int32 [2 n], the pages copied on write (source, destination; -1: none)
cudaError_t launch_pages_grow(const paged::TableArgs& t, const int32_t* rows, const int32_t* n_new, int64_t n,
                              int64_t max_new, int32_t* slots, int32_t* cow, const paged::CopyArgs& c,
                              cudaStream_t s);
// work: device int32 [2 n_pages + 3]
cudaError_t launch_pages_compact(const paged::TableArgs& t, const paged::CopyArgs& c, int32_t* work,
                                 int32_t* n_live, cudaStream_t s);
int64_t paged_attention_workspace(int64_t B, int64_t Sq, int64_t Hq, int64_t H, int64_t D, int64_t n_shared,
                                  int64_t W);
cudaError_t launch_paged_attention(const paged::AttnArgs& a, cudaStream_t s, const char** why);

// Epilogue of the GEMM kernels.
enum OutMode : int { kOutBf16 = 0, kOutRaw = 1 };

struct GemmArgs {
  const void* xq;        // int8 codes [M x K] or packed e2m1 [M x K/2]
  const float* xs;       // [M] (bf16 output only)
  const uint8_t* Wp;     // [N x K/4]
  const float* gamma;    // [G] (bf16 output only)
  int G;
  int group_end[8];
  int64_t M, N, K;
  void* out;             // bf16 [M x ldo] or raw int32/f32 [M x ldo]
  int64_t ldo;
  int out_mode;
  int* status;
  uint64_t timeout_ns;
};

// fp4 selects e2m1 activations (f8f6f4 kind, fp32 accumulate); otherwise int8.
// Returns a CUDA error, or cudaErrorNotSupported when the tensor-map
// encoder is unavailable (message in *why).
cudaError_t launch_gemm(const GemmArgs& a, bool fp4, cudaStream_t s, const char** why);
cudaError_t launch_gemv(const GemmArgs& a, cudaStream_t s, const char** why);
// Decode path for up to 8 tokens: warp-level MMAs (mma.sync u8 x s8) on the
// masked 2-bit codes, weights streamed by TMA before the dependency wait.
constexpr int kGemvMmaMaxTokens = 8;
bool gemv_mma_supported(int64_t M, int64_t N, int64_t K);
cudaError_t launch_gemv_mma(const GemmArgs& a, cudaStream_t s, const char** why);
// CUDA-core decode path with the activation quantiser inside (dp4a on the
// packed codes), up to 8 tokens.
constexpr int kGemvDp4aMaxTokens = 8;
bool gemv_dp4a_supported(int64_t M, int64_t K);
cudaError_t launch_gemv_dp4a(const GemmArgs& a, cudaStream_t s);
// The same with the per-token quantiser (INT8 / INT4, optional ReLU^2 gate)
// done inside the GEMV on bf16 activations x [M x ldx].
cudaError_t launch_gemv_dp4a_quant(const GemmArgs& a, const uint16_t* x, const uint16_t* up,
                                   int64_t ldx, int mode, cudaStream_t s);
cudaError_t launch_wait_probe(int* status, uint64_t timeout_ns, cudaStream_t s);
// Dense tensor-pipe rate microbenchmark (see bitlinear_tensor_peak); *units
// receives the number of ns_out entries written.
cudaError_t launch_tensor_peak(int kind, int iters, unsigned long long* ns_out, int* status,
                               uint64_t timeout_ns, int* units, cudaStream_t s);

// Driver entry point for cuTensorMapEncodeTiled, resolved once at run time.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_tiled();
int num_sms();

// Raise a kernel's dynamic shared-memory limit on the current device to at
// least `bytes` (and, with max_carveout, ask for all of the unified L1 as
// shared memory). Function attributes belong to a device's context, so this
// is kept per (device, kernel); it is thread-safe, and calls that need no
// larger limit only take a lock and a lookup.
cudaError_t set_smem_limit(const void* kern, int bytes, bool max_carveout = false);
template <typename... A>
inline cudaError_t set_smem_limit(void (*kern)(A...), int bytes, bool max_carveout = false) {
  return set_smem_limit(reinterpret_cast<const void*>(kern), bytes, max_carveout);
}

// Process-wide switch (bitlinear_set_launch_overlap): launch with
// programmatic stream serialisation so a kernel may start while the previous
// one in the stream finishes. Every kernel calls pdl_wait() before it reads
// activations or scales or writes an output.
bool launch_overlap();

// Launch with the overlap attribute (when on) and, for cluster_x > 0, a
// cluster of cluster_x CTAs along x.
template <typename... Exp, typename... Act>
inline cudaError_t launch_kernel(void (*kern)(Exp...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t s, unsigned cluster_x, Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  if (cluster_x > 0) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (launch_overlap()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Act&&>(args)...);
}

// As launch_kernel, for a later kernel of one call: it may always start before
// the kernel ahead of it has ended, and waits for that one itself (pdl_wait).
template <typename K, typename... A>
inline cudaError_t launch_behind(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
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

}  // namespace blt
