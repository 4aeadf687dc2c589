// The paged 3-bit KV cache: what its kernels share.
//
// A page holds PT = 64 tokens. One layer's cache is [n_pages][H] blocks; the
// block of a (page, head), with RB = 3 D / 8 bytes a row of codes:
//   K codes   [64 tokens][RB]            little-endian 3-bit stream per token
//   V codes   [16 groups][RB][4 tokens]  byte i of the 4 tokens of a group side by side
//   K scales  fp32 [64]                  sign bit set: the token is kept at 4 bits
//   V scales  fp32 [64]
// P V contracts over tokens: with the bytes of 4 tokens side by side, one
// masked 32-bit word is the operand register of an 8-bit MMA (4 consecutive
// values of the contracted index), with no transposition.
//
// A token at 4 bits has zero bytes for its 3-bit rows, but for byte 0 of the K
// row: the index j of its row in codes4 [n_pages][H][C4][D] (K in the first
// D / 2 bytes of the row, V in the others; code + 8, low nibble first).
#pragma once
#include "common.cuh"

namespace blt {
namespace paged {

constexpr int PT = 64;

__host__ __device__ constexpr int row_bytes(int D) { return 3 * D / 8; }
__host__ __device__ constexpr int block_bytes(int D) { return PT * (2 * row_bytes(D) + 8); }
// offsets inside a block
__host__ __device__ constexpr int off_v(int D) { return PT * row_bytes(D); }
__host__ __device__ constexpr int off_ks(int D) { return 2 * PT * row_bytes(D); }
__host__ __device__ constexpr int off_vs(int D) { return 2 * PT * row_bytes(D) + 4 * PT; }

// pages of a sequence of len >= 0 tokens
__host__ __device__ constexpr int pages_of(int len) { return len / PT + (len % PT != 0); }

}  // namespace paged
}  // namespace blt
