// The 8-bit paged KV cache: codes, block scales and page lookup shared by the
// kernels that write it (kv8_cache.cu) and read it (attention_kv8*.cu).
//
// A cache row (one token) holds n_kv_heads x 128 one-byte codes; every aligned
// block of `scale_block` rows has one fp32 scale for each kv head, and an
// element's value is code * scale.  Codes are int8 in [-127, 127] or e4m3 (the two
// e4m3 bit patterns that stand for NaN are never written, but a recycled page may
// hold them behind a sequence's end: the attention kernels clear those V rows).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace qw {
namespace kv8 {

constexpr int HD = 128;
// Key positions of a sequence end below this, so that p - window and a tile's last key stay in 32 bits.
constexpr int kMaxPositions = 1 << 30;
// A block scale below this is stored as zero with zero codes: 1 / scale stays
// finite, and the attention kernels' logarithm of a scale stays in range.
constexpr float kTinyScale = 7.888609052210118e-31f;   // 2^-100

// KV: QW_I8 or QW_E4M3
template <int KV> __device__ constexpr float code_max() { return KV == QW_I8 ? 127.0f : 448.0f; }

// Two e4m3 codes (low 16 bits) as an f16 pair; exact for every code, subnormals included.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
  uint32_t d;
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, x;\n}" : "=r"(d) : "r"(w));
  return d;
}
template <int KV> __device__ __forceinline__ float code_f32(uint32_t b) {
  if constexpr (KV == QW_I8) return float(int(b << 24) >> 24);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3_pair(b) & 0xffffu)));
}
// four codes of a word
template <int KV> __device__ __forceinline__ void codes_f32(uint32_t w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = code_f32<KV>((w >> (8 * i)) & 0xffu);
}

// Four values already divided by their scale, none of them NaN -> codes: round to
// nearest even, clamped to the largest code.
template <int KV> __device__ __forceinline__ uint32_t quant4(const float* x) {
  if constexpr (KV == QW_I8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= (uint32_t(min(max(__float2int_rn(x[i]), -127), 127)) & 0xffu) << (8 * i);
    return w;
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
}

// The cache as the entry points get it.
struct Cache {
  const void* k;
  const void* v;
  const float* k_scale;   // [num_slots / scale_block, nkv]
  const float* v_scale;
  int64_t num_slots;
  int sb_shift;           // log2(scale_block)
  const int32_t* table;   // [n_seqs, max_blocks]
  int max_blocks;
  int block_size;
};

// Cache row of key position p of sequence s, or -1 where the block table has no
// such page or the page lies outside the cache.
__device__ __forceinline__ int64_t row_of(const int32_t* table, int max_blocks, int block_size, int64_t num_slots,
                                          int s, int p) {
  const int blk = p / block_size;
  if (blk >= max_blocks) return -1;
  const int page = table[int64_t(s) * max_blocks + blk];
  const int64_t row = int64_t(page) * block_size + (p - blk * block_size);
  return page >= 0 && row < num_slots ? row : -1;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int scale_shift(int scale_block) {
  return scale_block == 16 ? 4 : scale_block == 32 ? 5 : scale_block == 64 ? 6 : -1;
}

// Checks shared by the entry points on the cache; QW_OK or the error set.
inline int check_cache(const char* who, const void* k, const void* v, const float* ks, const float* vs,
                       int64_t num_slots, int scale_block, int kv_dtype) {
  if (kv_dtype != QW_I8 && kv_dtype != QW_E4M3)
    return set_error(QW_ERR_DTYPE, "%s: kv_dtype %d is neither QW_I8 nor QW_E4M3", who, kv_dtype);
  if (scale_shift(scale_block) < 0)
    return set_error(QW_ERR_SHAPE, "%s: scale_block %d must be 16, 32 or 64", who, scale_block);
  if (num_slots <= 0 || num_slots > INT32_MAX)
    return set_error(QW_ERR_INVALID_ARG, "%s: num_slots %lld", who, (long long)num_slots);
  if (num_slots % scale_block)
    return set_error(QW_ERR_SHAPE, "%s: num_slots %lld is not a multiple of scale_block %d", who, (long long)num_slots,
                     scale_block);
  if (!k || !v || !ks || !vs) return set_error(QW_ERR_INVALID_ARG, "%s: null cache or scale pointer", who);
  if (!aligned16(k) || !aligned16(v)) return set_error(QW_ERR_INVALID_ARG, "%s: caches must be 16-byte aligned", who);
  if ((reinterpret_cast<uintptr_t>(ks) | reinterpret_cast<uintptr_t>(vs)) & 3u)
    return set_error(QW_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", who);
  return QW_OK;
}
// (scale_block, 16, 32 or 64, divides block_size)
inline int check_table(const char* who, const int32_t* table, int max_blocks, int block_size) {
  if (!table) return set_error(QW_ERR_INVALID_ARG, "%s: null block table", who);
  if (max_blocks <= 0 || block_size <= 0 || block_size % 64)
    return set_error(QW_ERR_SHAPE, "%s: block_size %d must be a positive multiple of 64, max_blocks positive", who,
                     block_size);
  return QW_OK;
}

}  // namespace kv8
}  // namespace qw

// ---------------------------------------------------------------------------
// codes as f16 pairs for the matrix instructions: every int8 and e4m3 code is
// exact in f16
// ---------------------------------------------------------------------------
namespace qw {
namespace kv8 {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// f16 pair (1024 + u0, 1024 + u1) -> (u0 - 128, u1 - 128)
__device__ __forceinline__ uint32_t unbias(uint32_t h) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(0x64806480u));
  return d;
}
// Codes 0, 1 and 2, 3 of word w (its codes biased by 128 for int8: w ^ 0x80808080).
template <int KV> __device__ __forceinline__ void word_pairs(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if constexpr (KV == QW_I8) {
    const uint32_t u = w ^ 0x80808080u;
    p01 = unbias(prmt(u, 0x64646464u, 0x4140));   // f16 0x6400 | u = 1024 + u
    p23 = unbias(prmt(u, 0x64646464u, 0x4342));
  } else {   // (one conversion: shifts and masks that leave out the NaN patterns took three instructions)
    p01 = e4m3_pair(w);
    p23 = e4m3_pair(w >> 16);
  }
}
// Codes i of words a and b side by side, i = 0 .. 3.
template <int KV> __device__ __forceinline__ void cross_pairs(uint32_t a, uint32_t b, uint32_t (&p)[4]) {
  word_pairs<KV>(prmt(a, b, 0x5140), p[0], p[1]);
  word_pairs<KV>(prmt(a, b, 0x7362), p[2], p[3]);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Power of two that takes a row whose largest magnitude is `top` into
// [2^14, 2^15), where its bf16 values down to 2^-28 of the largest are exact in
// f16, and its inverse.
__device__ __forceinline__ void row_scale(float top, float& mul, float& inv) {
  const int e = max(int(__float_as_uint(top) >> 23), 16);     // biased exponent (bf16 rows below 2^-111: kept small)
  mul = __uint_as_float(uint32_t(min(268 - e, 254)) << 23);   // 2^(14 - (e - 127))
  inv = __uint_as_float(uint32_t(max(e - 14, 1)) << 23);      // 2^((e - 127) - 14)
}

// What a query at key position ctx - 1 sees of a sequence, as tiles of KT keys:
// tiles 0 .. ns - 1 (first tokens), then w0 .. ; nt in all.
struct Span {
  int L, lo, w0, ns, nt;
  __device__ __forceinline__ int tile(int t) const { return t < ns ? t : w0 + t - ns; }
};

}  // namespace kv8
}  // namespace qw
