// 4-bit weights: the quantiser of a bf16 matrix and the lookup of rows (embedding).
#include "w4.cuh"

namespace qw {
namespace w4 {

// ---------------------------------------------------------------------------
// Quantiser.  Symmetric: s = bf16(max|w| / 7), n = rne(w / s) within -8 .. 7, plus 8.
// Asymmetric: lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15),
// z = rne(-lo / s) within 0 .. 15, n = rne(w / s) + z within 0 .. 15.
// A thread holds 8 columns (16 bytes in, one word out) at a time, kQuant times; a group is 4, 8 or 16 lanes.
//
// rne(w / s) without a division for each weight: w and s have 8 significant bits, so w / s, at most 15.1 here, is a tie
// (some m + 1/2) or at least 2^-10 away from one.  w * (1 / s) errs by less than 2^-19, and adding 6144 = 1.5 * 2^12
// rounds it to a multiple of 2^-11: ties become exact again and nothing else becomes one.  Adding 1.5 * 2^23 less that
// then rounds to an integer, ties to even, which stands in the low bits.  In the symmetric form |w / s| < 7.1 needs no
// clamp, in the asymmetric form only the upper end does (both roundings may go up).
// Bound by its instructions, 15 a weight symmetric and 18 asymmetric: issue slots are used to 78-79% in both forms, memory
// to 65 and 54%.  151936 x 1024, group 32: 399 MB in 72 us symmetric (5.5 TB/s), 404 MB in 91 us asymmetric (4.4 TB/s).
// With a division for each weight: 170 us.
// ---------------------------------------------------------------------------
constexpr int kQuant = 4;
constexpr float kSnap = 6144.0f, kInt = 12582912.0f;   // 1.5 * 2^12, 1.5 * 2^23
constexpr uint32_t kIntBits = 0x4b400000u;              // kInt's
constexpr uint32_t int_bits_of_word() {                 // the sum of kIntBits at the eight places, modulo 2^32
  uint32_t sum = 0;
  for (int p = 0; p < 32; p += 4) sum += kIntBits << p;
  return sum;
}

// bf16(x / n) in fp32, inv = 1 / n rounded: x * inv differs from x / n by less than 4 units in its last place, so the two
// round alike unless x * inv lies within 8 of a midpoint between two bf16 numbers.
__device__ __forceinline__ float quotient_bf16(float x, float n, float inv) {
  float t = x * inv;
  if (((__float_as_uint(t) - 0x7ff8u) & 0xffffu) <= 16u) t = __fdiv_rn(x, n);
  return round_t<bf16>(t);
}

// any group: with infinities, NaN, or so small that 1 / s is no normal number
template <bool ZEROS>
__device__ __noinline__ uint32_t quantize_any(uint4 u, int lanes, uint32_t mask, float& s_out, float& z_out) {
  float x[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (isnan(x[e])) x[e] = 0.0f;
    if (!isinf(x[e])) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
    }
  }
  for (int o = 1; o < lanes; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
  }
  float top = ZEROS ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
  if (isinf(top)) top = 2.0f * __fdiv_rn(0.5f * hi - 0.5f * lo, 15.0f);   // hi - lo is past fp32
  const float s = round_t<bf16>(top);
  const float d = s == 0.0f ? 1.0f : s;
  const float z = ZEROS ? fminf(rintf(__fdiv_rn(-lo, d)), 15.0f) : 8.0f;
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(x[e], d)), -z), 15.0f - z) + z;
    word |= uint32_t(q) << (4 * ((e & 1) * 4 + e / 2));
  }
  s_out = s;
  z_out = z;
  return word;
}

template <bool ZEROS>
__global__ void __launch_bounds__(256) quantize_kernel(const uint4* __restrict__ w, int64_t n_vec, int lanes,
                                                       int lane_shift, uint32_t* __restrict__ codes,
                                                       bf16* __restrict__ scales, uint8_t* __restrict__ zeros) {
  pdl_wait();
  const int64_t v0 = int64_t(blockIdx.x) * (256 * kQuant) + threadIdx.x;
  const int lane = threadIdx.x & 31;
  const uint32_t group_mask = (lanes == 32 ? ~0u : (1u << lanes) - 1u) << (lane & ~(lanes - 1));
  uint4 u[kQuant];
#pragma unroll
  for (int i = 0; i < kQuant; ++i) {
    u[i] = make_uint4(0, 0, 0, 0);
    if (v0 + 256 * i < n_vec) u[i] = w[v0 + 256 * i];
  }
#pragma unroll
  for (int i = 0; i < kQuant; ++i) {
    const uint32_t p[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    float s, z = 8.0f;
    bool any;
    float lo = 0.0f, hi;
    if (ZEROS) {
      __nv_bfloat162 mx = __float2bfloat162_rn(0.0f), mn = mx;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&p[e]);
        mx = __hmax2_nan(mx, h);
        mn = __hmin2_nan(mn, h);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        mx = __hmax2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mn = __hmin2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      }
      const uint32_t a = *reinterpret_cast<uint32_t*>(&mx), b = *reinterpret_cast<uint32_t*>(&mn);
      hi = fmaxf(bf16_lo(a), bf16_hi(a));
      lo = fminf(bf16_lo(b), bf16_hi(b));
      // a sum of magnitudes: neither small nor a number if one of them is NaN or infinite
      any = !((bf16_lo(a) + bf16_hi(a)) - (bf16_lo(b) + bf16_hi(b)) < 0x1p120f);
      s = quotient_bf16(__fsub_rn(hi, lo), 15.0f, 1.0f / 15.0f);
    } else {
      uint32_t m = __vmaxu2(__vmaxu2(p[0] & 0x7fff7fffu, p[1] & 0x7fff7fffu), __vmaxu2(p[2] & 0x7fff7fffu, p[3] & 0x7fff7fffu));
      for (int o = 1; o < lanes; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t top = max(m >> 16, m & 0xffffu);   // |w| as bits: their order is that of the values
      any = top >= 0x7f80u;
      hi = __uint_as_float(top << 16);
      s = quotient_bf16(hi, 7.0f, 1.0f / 7.0f);
    }
    any = any || s < 0x1p-100f;   // also 0
    uint32_t word;
    if (any) {
      word = quantize_any<ZEROS>(u[i], lanes, group_mask, s, z);
    } else {
      const float r = __fdividef(1.0f, s);
      if (ZEROS) z = __fadd_rn(__fadd_rn(__fmaf_rn(-lo, r, kSnap), kInt - kSnap), -kInt);
      const float top = kSnap + 15.0f - z;
      word = (ZEROS ? uint32_t(int(z)) * 0x11111111u : 0x88888888u) - int_bits_of_word();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t = __fmaf_rn(e & 1 ? bf16_hi(p[e / 2]) : bf16_lo(p[e / 2]), r, kSnap);
        if (ZEROS) t = fminf(t, top);
        word += __float_as_uint(__fadd_rn(t, kInt - kSnap)) << (4 * ((e & 1) * 4 + e / 2));   // kIntBits + rne(w / s)
      }
    }
    const int64_t v = v0 + 256 * i;
    if (v >= n_vec) continue;
    codes[v] = word;
    if ((lane & (lanes - 1)) == 0) {
      scales[v >> lane_shift] = __float2bfloat16_rn(s);
      if (ZEROS) zeros[v >> lane_shift] = uint8_t(z);
    }
  }
}

// ---------------------------------------------------------------------------
// Rows of a 4-bit table by id.  One warp: 1024 columns of a token, a word (8 columns) in
// and 16 bytes out for each lane and step, so that loads and stores are whole lines.  Bound by memory:
// 151936 x 1024, group 32, all rows in turn 60 us (409 MB, 6.8 TB/s), 16384 random ones 7.9 us (43 MB, 5.5 TB/s).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) embed_kernel(const int64_t* __restrict__ ids, int64_t T, Weights W, int64_t V,
                                                    int H, int parts, bf16* __restrict__ out, int32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int64_t item = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t tok = item / parts;
  const int part = int(item - tok * parts);
  if (tok >= T) return;
  const int64_t id = ids[tok];
  const bool ok = id >= 0 && id < V;
  if (!ok && part == 0 && lane == 0 && err != nullptr) atomicAdd(err, 1);
  const uint32_t* row = reinterpret_cast<const uint32_t*>(W.codes + (ok ? id : 0) * W.row_bytes);
  const int64_t g0 = (ok ? id : 0) * W.groups;
  const int words = H / 8, first = part * 128 + lane;
  uint32_t c[4], s[4], z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = first + 32 * i;
    c[i] = s[i] = 0;
    z[i] = 8;
    if (ok && k < words) {
      const int g = k >> (2 + W.group_shift);
      c[i] = __ldg(row + k);
      s[i] = __ldg(reinterpret_cast<const uint16_t*>(W.scales) + g0 + g);
      if (W.zeros != nullptr) z[i] = __ldg(W.zeros + g0 + g);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = first + 32 * i;
    if (k >= words) break;
    uint32_t w[4];
    decode(c[i], code_magic(), offset_pair(z[i]), scale_pair(s[i]), w);
    if (!ok) w[0] = w[1] = w[2] = w[3] = 0;   // (0 - z) * 0 is a negative zero
    reinterpret_cast<uint4*>(out + tok * H)[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Sizes and pointers that every entry point on 4-bit weights refuses alike; K: columns of a stored row.
int check_weights(const char* who, const void* codes, const void* scales, int64_t N, int64_t K, int group) {
  if (group != 32 && group != 64 && group != 128)
    return set_error(QW_ERR_SHAPE, "%s: group %d is not 32, 64 or 128", who, group);
  if (K % group) return set_error(QW_ERR_SHAPE, "%s: %lld columns are not whole groups of %d", who, (long long)K, group);
  if (N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31)) return set_error(QW_ERR_SHAPE, "%s: dimension too large", who);
  if (!codes || !scales) return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if ((reinterpret_cast<uintptr_t>(codes) & 15) || (reinterpret_cast<uintptr_t>(scales) & 1))
    return set_error(QW_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned, scales 2-byte", who);
  return QW_OK;
}

Weights make_weights(const void* codes, const void* scales, const void* zeros, int64_t K, int group) {
  return Weights{static_cast<const uint8_t*>(codes), static_cast<const bf16*>(scales), static_cast<const uint8_t*>(zeros),
                 K / 2, int(K / group), group == 32 ? 0 : group == 64 ? 1 : 2};
}

}  // namespace w4
}  // namespace qw

using namespace qw;

static inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

extern "C" int qw_w4_quantize(const void* w, int64_t N, int64_t K, int group, void* codes, void* scales, void* zeros,
                              int dtype, void* stream) {
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "qw_w4_quantize: dtype %d", dtype);
  if (N < 0 || K <= 0) return set_error(QW_ERR_INVALID_ARG, "qw_w4_quantize: bad sizes");
  if (N == 0) return QW_OK;
  const int rc = w4::check_weights("qw_w4_quantize", codes, scales, N, K, group);
  if (rc) return rc;
  if (!w || !al16(w)) return set_error(QW_ERR_INVALID_ARG, "qw_w4_quantize: null or misaligned matrix");
  const int64_t n_vec = N * (K / 8), blocks = (n_vec + 256 * w4::kQuant - 1) / (256 * w4::kQuant);
  if (blocks >= (int64_t(1) << 31)) return set_error(QW_ERR_SHAPE, "qw_w4_quantize: more than 2^42 weights");
  const int lanes = group / 8, shift = group == 32 ? 2 : group == 64 ? 3 : 4;
  launch_pdl(zeros ? w4::quantize_kernel<true> : w4::quantize_kernel<false>, unsigned(blocks), 256, 0,
             static_cast<cudaStream_t>(stream), static_cast<const uint4*>(w), n_vec, lanes, shift,
             static_cast<uint32_t*>(codes), static_cast<bf16*>(scales), static_cast<uint8_t*>(zeros));
  return check_launch("qw_w4_quantize");
}

extern "C" int qw_w4_embed_vocab(const int64_t* ids, int64_t T, const void* codes, const void* scales, const void* zeros,
                                 int64_t V, int64_t H, int group, int tp, void* out, int32_t* err_count, int dtype,
                                 void* stream) {
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "qw_w4_embed_vocab: dtype %d", dtype);
  if (T < 0 || V <= 0 || H <= 0 || tp <= 0) return set_error(QW_ERR_INVALID_ARG, "qw_w4_embed_vocab: bad sizes");
  if (V % tp) return set_error(QW_ERR_SHAPE, "qw_w4_embed_vocab: V=%lld not divisible by tp=%d", (long long)V, tp);
  if (T == 0) return QW_OK;
  const int rc = w4::check_weights("qw_w4_embed_vocab", codes, scales, V, H, group);
  if (rc) return rc;
  if (!ids || !out || !al16(out)) return set_error(QW_ERR_INVALID_ARG, "qw_w4_embed_vocab: null or misaligned pointer");
  const int64_t parts = (H / 8 + 127) / 128;
  if (T > (int64_t(1) << 33) / parts) return set_error(QW_ERR_SHAPE, "qw_w4_embed_vocab: too many tokens");
  launch_pdl(w4::embed_kernel, unsigned((T * parts + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream), ids, T,
             w4::make_weights(codes, scales, zeros, H, group), V, int(H), int(parts), static_cast<bf16*>(out), err_count);
  return check_launch("qw_w4_embed_vocab");
}
