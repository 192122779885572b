// Matrices of 4-bit weights (sm_103a): the format and its decoding, shared by the
// kernels that read them.
//
// A weight is the bf16 number round((n - z) * s): code n in 0 .. 15, zero point z
// (8 without a zeros array) and bf16 scale s of its row and group of 32, 64 or 128
// columns.  A row's codes are 32-bit words of 8 columns: nibble p of word i is
// column 8i + 2p for p < 4 and 8i + 2(p - 4) + 1 above, so that
// (word >> 4p) & 0x000f000f holds columns 8i + 2p and 8i + 2p + 1 as the halves of
// one register: a bf16 pair after one more bit operation.
#pragma once

#include "common.cuh"

namespace qw {
namespace w4 {

constexpr int kPiece = 32;   // columns of one 16-byte load of codes; a piece lies in one group

struct Weights {
  const uint8_t* codes;    // [rows, row_bytes]
  const bf16* scales;      // [rows, groups]
  const uint8_t* zeros;    // [rows, groups] or NULL
  int64_t row_bytes;       // (columns of a row) / 2
  int groups;              // groups of a row
  int group_shift;         // log2(pieces of a group): 0, 1, 2
};

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// the pair (128 + z, 128 + z) in bf16: 128 .. 143 are one step apart
__device__ __forceinline__ uint32_t offset_pair(uint32_t z) { return 0x43004300u + z * 0x00010001u; }
__device__ __forceinline__ uint32_t scale_pair(uint32_t s_bits) { return s_bits * 0x00010001u; }

// 0x43004300 in a register that the compiler takes for unknown: (x & mask) | magic is then one instruction, with two
// constants it is two (25.9 -> 23.0 cycles a word on an SM sub-partition with the rest of decode).
__device__ __forceinline__ uint32_t code_magic() {
  uint32_t m;
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(m));
  return m;
}
// The 8 weights of a word as 4 bf16 pairs in column order: 128 + n by bit operations, less
// 128 + z (exact), times the scale (rounded once: the weight's definition).
__device__ __forceinline__ void decode(uint32_t word, uint32_t magic, uint32_t z2, uint32_t s2, uint32_t (&w)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(v) : "r"(word >> (4 * p)), "r"(magic));   // (x & mask) | magic
    w[p] = mul_bf16x2(sub_bf16x2(v, z2), s2);
  }
}

}  // namespace w4
}  // namespace qw
