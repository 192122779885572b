// Writing and reading the 8-bit paged KV cache: QK-RMSNorm + RoPE + quantised
// append (qw_kv8_append) and rows back as values (qw_kv8_read).
#include <algorithm>

#include "kv8.cuh"

namespace qw {
namespace kv8 {

struct AppendArgs {
  const bf16* qkv;            // [T, tp * (nh/tp + 2 nkv/tp) * 128]
  int64_t T;
  int nh, nkv, tp;
  const int64_t* positions;   // [T]
  const float* cos_sin;       // [max_pos, 128]
  int64_t max_pos;
  const bf16* q_gamma;
  const bf16* k_gamma;
  float eps;
  const int32_t* cu_q;        // [n_seqs + 1], or null: one token per sequence
  const int32_t* ctx;         // [n_seqs]
  const int32_t* table;
  int max_blocks, block_size, n_seqs;
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t num_slots;
  bf16* q_out;
  int32_t* err;
  int64_t kv_ctas;            // CTAs with k and v, ahead of those with q
};

__device__ __forceinline__ int seq_begin(const AppendArgs& a, int s) { return a.cu_q != nullptr ? a.cu_q[s] : s; }

// The sequence and the scale block of block task `t`: sequences in order, each
// with the blocks that its new tokens touch.  One warp scans the sequences 32
// at a time, a memory round trip each: nothing for tens of sequences, but every
// task does it, so that its cost grows with the square of a large batch.  s = -1
// when there are fewer tasks.
__device__ __forceinline__ void find_block(const AppendArgs& a, int64_t t, int sb, int& s_out, int& blk_out) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  s_out = -1;
  blk_out = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int cnt = 0, b0 = 0;
    if (s < a.n_seqs) {
      const int lq = seq_begin(a, s + 1) - seq_begin(a, s), ctx = a.ctx[s];
      const int first = max(ctx - lq, 0);
      b0 = first / sb;
      cnt = lq > 0 && ctx > 0 ? (ctx - 1) / sb - b0 + 1 : 0;
    }
    int64_t upto = cnt;   // inclusive prefix sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const bool here = t >= before + upto - cnt && t < before + upto;
    const unsigned m = __ballot_sync(0xffffffffu, here);
    if (m) {
      const int src = __ffs(m) - 1;
      s_out = s0 + src;
      blk_out = __shfl_sync(0xffffffffu, b0 + int(t - (before + upto - cnt)), src);
      return;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// Two fp32 products an instruction, each rounded by itself: half the issue slots of
// the scalar form.  Sums stay scalar: a packed sum of packed products was fused into
// one rounding, which moved q by a bf16 step in one element of 10^5.
__device__ __forceinline__ void mul2(float a0, float a1, float b0, float b1, float& d0, float& d1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// The RoPE row of one token's eight lanes: lane `sub` owns elements 8 sub .. + 7
// and 64 + 8 sub .. + 7 of a head, so RoPE pairs meet in one lane.
struct Rope {
  float c[8], sn[8];
  bool ok;
};
__device__ __forceinline__ Rope rope_row(const AppendArgs& a, int64_t pos, int i0) {
  Rope r;
  r.ok = pos >= 0 && pos < a.max_pos;
  const float* cs = a.cos_sin + (r.ok ? pos : 0) * HD;
  *reinterpret_cast<float4*>(r.c) = *reinterpret_cast<const float4*>(cs + i0);
  *reinterpret_cast<float4*>(r.c + 4) = *reinterpret_cast<const float4*>(cs + i0 + 4);
  *reinterpret_cast<float4*>(r.sn) = *reinterpret_cast<const float4*>(cs + 64 + i0);
  *reinterpret_cast<float4*>(r.sn + 4) = *reinterpret_cast<const float4*>(cs + 64 + i0 + 4);
  return r;
}
// x: eight + eight elements of a head (in), normed and roped (out), by the steps and
// roundings of qk_ss8 .. qk_rope_pair; ROUND: the norm's output rounded to bf16.
template <bool ROUND>
__device__ __forceinline__ void norm_rope(float (&x1)[8], float (&x2)[8], const float (&g1)[8], const float (&g2)[8],
                                          const Rope& r, float eps) {
  const unsigned lanes = 0xffu << (threadIdx.x & 24);   // this token's eight lanes
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float a0, a1, b0, b1;
    mul2(x1[e], x1[e + 1], x1[e], x1[e + 1], a0, a1);
    mul2(x2[e], x2[e + 1], x2[e], x2[e + 1], b0, b1);
    ss = __fadd_rn(__fadd_rn(ss, __fadd_rn(a0, b0)), __fadd_rn(a1, b1));
  }
  ss = __fadd_rn(ss, __shfl_xor_sync(lanes, ss, 1));
  ss = __fadd_rn(ss, __shfl_xor_sync(lanes, ss, 2));
  ss = __fadd_rn(ss, __shfl_xor_sync(lanes, ss, 4));
  const float inv = qk_inv_rms(ss, eps);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float n1[2], n2[2], p[2], q[2];
    mul2(x1[e], x1[e + 1], inv, inv, n1[0], n1[1]);
    mul2(n1[0], n1[1], g1[e], g1[e + 1], n1[0], n1[1]);
    mul2(x2[e], x2[e + 1], inv, inv, n2[0], n2[1]);
    mul2(n2[0], n2[1], g2[e], g2[e + 1], n2[0], n2[1]);
    if constexpr (ROUND) {
      const uint32_t h1 = pack_bf16(n1[0], n1[1]), h2 = pack_bf16(n2[0], n2[1]);
      n1[0] = bf16_lo(h1);
      n1[1] = bf16_hi(h1);
      n2[0] = bf16_lo(h2);
      n2[1] = bf16_hi(h2);
    }
    mul2(n1[0], n1[1], r.c[e], r.c[e + 1], p[0], p[1]);
    mul2(n2[0], n2[1], r.sn[e], r.sn[e + 1], q[0], q[1]);
    x1[e] = __fsub_rn(p[0], q[0]);
    x1[e + 1] = __fsub_rn(p[1], q[1]);
    mul2(n2[0], n2[1], r.c[e], r.c[e + 1], p[0], p[1]);
    mul2(n1[0], n1[1], r.sn[e], r.sn[e + 1], q[0], q[1]);
    x2[e] = __fadd_rn(p[0], q[0]);
    x2[e + 1] = __fadd_rn(p[1], q[1]);
  }
  if (!r.ok)
#pragma unroll
    for (int e = 0; e < 8; ++e) x1[e] = x2[e] = 0.0f;
}
// The largest finite magnitude; `odd`: there are values that are not finite.
__device__ __forceinline__ float finite_top(const float (&x1)[8], const float (&x2)[8], bool& odd) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {   // NaN stays
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x1[e])));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x2[e])));
  }
  odd = !(top < INFINITY);
  if (odd) {
    top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = fabsf(x1[e]), w = fabsf(x2[e]);
      top = fmaxf(top, fmaxf(u < INFINITY ? u : 0.0f, w < INFINITY ? w : 0.0f));
    }
  }
  return top;
}
// Element offset of kv head g's k (v: nkv / tp heads further) in a token's merged QKV row.
__device__ __forceinline__ int64_t k_offset(const AppendArgs& a, int g) {
  const int nh_l = a.nh / a.tp, nkv_l = a.nkv / a.tp;
  return (int64_t(g / nkv_l) * (nh_l + 2 * nkv_l) + nh_l + g % nkv_l) * HD;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
}

// Q heads [h0, h0 + QH) of one token by eight lanes.
template <int QH>
__device__ __forceinline__ void append_q(const AppendArgs& a, int64_t tok, int h0, int sub) {
  const int i0 = 8 * sub, nh_l = a.nh / a.tp, nkv_l = a.nkv / a.tp;
  const int64_t width_r = int64_t(nh_l + 2 * nkv_l) * HD;
  const bf16* row = a.qkv + tok * width_r * a.tp;
  const int64_t pos = a.positions[tok];
  uint4 xa[QH], xb[QH];
  float g1[8], g2[8];
  int hl = h0 % nh_l;
  const bf16* src = row + (h0 / nh_l) * width_r + int64_t(hl) * HD + i0;
#pragma unroll
  for (int i = 0; i < QH; ++i) {   // every load in flight at once
    xa[i] = *reinterpret_cast<const uint4*>(src);
    xb[i] = *reinterpret_cast<const uint4*>(src + 64);
    if (h0 + i + 1 < a.nh) {
      src += HD;
      if (++hl == nh_l) {   // the next shard's q heads
        hl = 0;
        src += 2 * int64_t(nkv_l) * HD;
      }
    }
  }
  load16(a.q_gamma + i0, g1);
  load16(a.q_gamma + 64 + i0, g2);
  const Rope r = rope_row(a, pos, i0);
#pragma unroll
  for (int i = 0; i < QH; ++i) {
    float x1[8], x2[8];
    unpack8(xa[i], x1);
    unpack8(xb[i], x2);
    norm_rope<true>(x1, x2, g1, g2, r, a.eps);
    if (h0 + i >= a.nh) continue;   // (uniform over the eight lanes)
    bf16* o = a.q_out + (tok * a.nh + h0 + i) * int64_t(HD);
    store16(o + i0, x1);
    store16(o + 64 + i0, x2);
  }
  if (!r.ok && sub == 0 && h0 == 0 && a.err != nullptr) atomicAdd(a.err, 1);
}
__device__ __forceinline__ bool in_sequence(const AppendArgs& a, int64_t tok) {
  return tok < a.T && tok >= seq_begin(a, 0) && tok < seq_begin(a, a.n_seqs);
}
// A block without a page: its tokens are counted once (one with a bad position is counted with its q).
__device__ __forceinline__ void count_missing(const AppendArgs& a, int64_t tok) {
  const int64_t pos = a.positions[tok];
  if (a.err != nullptr && pos >= 0 && pos < a.max_pos) atomicAdd(a.err, 1);
}
// The block's new scale and its inverse from its old scale and the new tokens' top.
template <int KV> __device__ __forceinline__ float new_scale(float was, float top, float& inv) {
  float cand = top / code_max<KV>();
  if (cand < kTinyScale) cand = 0.0f;
  const float now = fmaxf(was, cand);
  inv = now > 0.0f ? 1.0f / now : 0.0f;
  return now;
}
template <int KV>
__device__ __forceinline__ void put_codes(uint8_t* dst, int i0, float (&x1)[8], float (&x2)[8], float inv, bool odd) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x1[e] = __fmul_rn(x1[e], inv);
    x2[e] = __fmul_rn(x2[e], inv);
  }
  if (odd)   // NaN becomes 0
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x1[e] = x1[e] == x1[e] ? x1[e] : 0.0f;
      x2[e] = x2[e] == x2[e] ? x2[e] : 0.0f;
    }
  *reinterpret_cast<uint2*>(dst + i0) = make_uint2(quant4<KV>(x1), quant4<KV>(x1 + 4));
  *reinterpret_cast<uint2*>(dst + 64 + i0) = make_uint2(quant4<KV>(x2), quant4<KV>(x2 + 4));
}
// An older token's codes (16 bytes of a lane) in units of the new scale.
template <int KV> __device__ __forceinline__ uint4 requant(const uint4& c, float ratio) {
  float f[16];
  codes_f32<KV>(c.x, f);
  codes_f32<KV>(c.y, f + 4);
  codes_f32<KV>(c.z, f + 8);
  codes_f32<KV>(c.w, f + 12);
#pragma unroll
  for (int e = 0; e < 16; ++e) f[e] = __fmul_rn(f[e], ratio);
  return make_uint4(quant4<KV>(f), quant4<KV>(f + 4), quant4<KV>(f + 8), quant4<KV>(f + 12));
}

// Many tokens a sequence.  One CTA per (scale block touched, kv head) with eight
// lanes per token of the block, then CTAs of eight lanes per (token, QH q heads).
// A block's tokens meet in one CTA because they share a scale: the block maxima of
// k and of v are formed in shared memory and every value is quantised from the
// registers that it was computed in, so each input is read once.  k and v
// together, and two q heads on one RoPE row, put more loads in flight: 8 x 2048
// tokens of 16 q and 8 kv heads take 55.7 us, 4.2 TB/s (83 us with one of them at a
// time; four q heads 65 us, one 61 us, 1024 threads an SM in each).  Neither issue
// (65% of the slots, about 20 instructions an element) nor memory (DRAM at 51% of
// the copy rate) is full: the largest stall is the wait for loads, which 1024 threads
// of 64 registers cover in part.  The 64 are not enough for k, v and the gammas: 68 to
// 76 bytes a thread are spilled and 92 read back, in every instantiation.
constexpr int QH = 2;
template <int KV, int SB>
__global__ void __launch_bounds__(SB * 8, 1024 / (SB * 8)) kv8_append_kernel(const AppendArgs a) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  constexpr int THREADS = SB * 8;
  const int sub = threadIdx.x & 7, grp = threadIdx.x >> 3, i0 = 8 * sub;
  if (blockIdx.x >= a.kv_ctas) {   // ---- q heads
    const int chunks = (a.nh + QH - 1) / QH;
    const unsigned unit = (blockIdx.x - unsigned(a.kv_ctas)) * SB + grp, tok = unit / unsigned(chunks);
    if (in_sequence(a, tok)) append_q<QH>(a, tok, int(unit - tok * chunks) * QH, sub);   // (rows of no sequence stay)
    return;
  }
  // ---- k and v of one kv head in one scale block
  const int g = int(blockIdx.x % unsigned(a.nkv));
  int s, blk;
  find_block(a, blockIdx.x / unsigned(a.nkv), SB, s, blk);   // every warp, the same answer
  if (s < 0) return;
  const int tok0 = seq_begin(a, s), lq = seq_begin(a, s + 1) - tok0, ctx = a.ctx[s];
  const int start = ctx - lq;                     // key position of the sequence's first new token (may be negative)
  const int p = blk * SB + grp;                   // this group's key position
  const int64_t tok = int64_t(tok0) + (p - start);
  const bool fresh = p >= start && p < ctx && tok >= 0 && tok < a.T;
  float k1[8], k2[8], v1[8], v2[8], top_k = 0.0f, top_v = 0.0f;
  bool odd_k = false, odd_v = false;
  if (fresh) {
    const int64_t pos = a.positions[tok];
    const int nkv_l = a.nkv / a.tp;
    const bf16* src = a.qkv + tok * (int64_t(a.nh + 2 * a.nkv) * HD) + k_offset(a, g);
    float g1[8], g2[8];
    load16(src + i0, k1);
    load16(src + 64 + i0, k2);
    load16(src + int64_t(nkv_l) * HD + i0, v1);
    load16(src + int64_t(nkv_l) * HD + 64 + i0, v2);
    load16(a.k_gamma + i0, g1);
    load16(a.k_gamma + 64 + i0, g2);
    const Rope r = rope_row(a, pos, i0);
    norm_rope<false>(k1, k2, g1, g2, r, a.eps);
    if (!r.ok)
#pragma unroll
      for (int e = 0; e < 8; ++e) v1[e] = v2[e] = 0.0f;
    top_k = finite_top(k1, k2, odd_k);
    top_v = finite_top(v1, v2, odd_v);
  }
  const int64_t row0 = row_of(a.table, a.max_blocks, a.block_size, a.num_slots, s, blk * SB);
  if (row0 < 0) {   // no page: nothing is stored (uniform over the CTA)
    if (fresh && g == 0 && sub == 0) count_missing(a, tok);
    return;
  }
  __shared__ float s_top[2][THREADS / 32];
  top_k = warp_max(top_k);
  top_v = warp_max(top_v);
  if ((threadIdx.x & 31) == 0) {
    s_top[0][threadIdx.x >> 5] = top_k;
    s_top[1][threadIdx.x >> 5] = top_v;
  }
  const int64_t sc = (row0 / SB) * a.nkv + g;
  const bool held = start > blk * SB;             // tokens before the first new one
  const float was_k = held ? a.k_scale[sc] : 0.0f, was_v = held ? a.v_scale[sc] : 0.0f;
  __syncthreads();                                // (every thread has read the old scales)
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    top_k = fmaxf(top_k, s_top[0][w]);
    top_v = fmaxf(top_v, s_top[1][w]);
  }
  float inv_k, inv_v;
  const float now_k = new_scale<KV>(was_k, top_k, inv_k), now_v = new_scale<KV>(was_v, top_v, inv_v);
  const int64_t at = ((row0 + grp) * a.nkv + g) * int64_t(HD);
  if (fresh) {
    put_codes<KV>(a.k + at, i0, k1, k2, inv_k, odd_k);
    put_codes<KV>(a.v + at, i0, v1, v2, inv_v, odd_v);
  } else if (p < start) {                         // an older token, where the scale grew
    if (now_k > was_k) {
      uint4* w = reinterpret_cast<uint4*>(a.k + at + 16 * sub);
      *w = requant<KV>(*w, __fmul_rn(was_k, inv_k));
    }
    if (now_v > was_v) {
      uint4* w = reinterpret_cast<uint4*>(a.v + at + 16 * sub);
      *w = requant<KV>(*w, __fmul_rn(was_v, inv_v));
    }
  }
  if (threadIdx.x == 0) {
    a.k_scale[sc] = now_k;
    a.v_scale[sc] = now_v;
  }
}

// Few tokens a sequence (decode): one warp per (scale block touched, kv head, K or
// V), its new tokens four at a time (a block with more of them computes them again
// to quantise them), then eight lanes per (token, q head).  The kernel above
// would keep eight lanes of 512 busy.
template <int KV, int SB>
__global__ void __launch_bounds__(128) kv8_append_few_kernel(const AppendArgs a) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  const int lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3, i0 = 8 * sub;
  unsigned unit = blockIdx.x * 4 + (threadIdx.x >> 5);   // warp
  const unsigned kv_units = unsigned(a.kv_ctas) * 4;
  if (unit >= kv_units) {   // ---- q heads
    unit = (unit - kv_units) * 4 + grp;
    const unsigned tok = unit / unsigned(a.nh);
    if (in_sequence(a, tok)) append_q<1>(a, tok, int(unit - tok * a.nh), sub);   // (rows of no sequence stay)
    return;
  }
  const bool is_v = unit & 1;
  const int g = int((unit >> 1) % unsigned(a.nkv));
  int s, blk;
  find_block(a, (unit >> 1) / unsigned(a.nkv), SB, s, blk);
  if (s < 0) return;
  const int tok0 = seq_begin(a, s), lq = seq_begin(a, s + 1) - tok0, ctx = a.ctx[s];
  const int start = ctx - lq;                                    // key position of the first new token (may be negative)
  const int p_new = max(start, blk * SB), p_end = min(ctx, (blk + 1) * SB);   // new tokens of the block: at least one
  const bf16* head = a.qkv + k_offset(a, g) + (is_v ? int64_t(a.nkv / a.tp) * HD : 0);
  const int64_t row_w = int64_t(a.nh + 2 * a.nkv) * HD;
  float x1[8], x2[8];
  // the token at key position p (or nothing) in this group's registers
  auto take = [&](int p) -> bool {
    const int64_t tok = int64_t(tok0) + (p - start);
    const bool fresh = p < p_end && tok >= 0 && tok < a.T;
#pragma unroll
    for (int e = 0; e < 8; ++e) x1[e] = x2[e] = 0.0f;
    if (fresh) {
      const int64_t pos = a.positions[tok];
      load16(head + tok * row_w + i0, x1);
      load16(head + tok * row_w + 64 + i0, x2);
      if (is_v) {
        if (pos < 0 || pos >= a.max_pos)
#pragma unroll
          for (int e = 0; e < 8; ++e) x1[e] = x2[e] = 0.0f;
      } else {
        float g1[8], g2[8];
        load16(a.k_gamma + i0, g1);
        load16(a.k_gamma + 64 + i0, g2);
        norm_rope<false>(x1, x2, g1, g2, rope_row(a, pos, i0), a.eps);
      }
    }
    return fresh;
  };
  const int64_t row0 = row_of(a.table, a.max_blocks, a.block_size, a.num_slots, s, blk * SB);
  const int64_t sc = row0 >= 0 ? (row0 / SB) * a.nkv + g : 0;
  float* scale = is_v ? a.v_scale : a.k_scale;
  const float was = row0 >= 0 && start > blk * SB ? scale[sc] : 0.0f;   // tokens before the first new one
  if (row0 < 0) {   // no page: nothing is stored
    if (!is_v && g == 0 && sub == 0)
      for (int p = p_new + grp; p < p_end; p += 4)
        if (tok0 >= 0 && int64_t(tok0) + (p - start) < a.T) count_missing(a, int64_t(tok0) + (p - start));
    return;
  }
  bool fresh = take(p_new + grp), odd;
  float top = finite_top(x1, x2, odd);
  for (int p = p_new + 4; p < p_end; p += 4) {
    bool more;
    take(p + grp);
    top = fmaxf(top, finite_top(x1, x2, more));
    odd |= more;
  }
  top = warp_max(top);
  float inv;
  const float now = new_scale<KV>(was, top, inv);
  uint8_t* rows = (is_v ? a.v : a.k) + (row0 * a.nkv + g) * int64_t(HD);
  const int64_t step = int64_t(a.nkv) * HD;
  if (now > was) {   // older tokens in units of the new scale
    const float ratio = __fmul_rn(was, inv);
    const int n_old = start - blk * SB;
#pragma unroll 4
    for (int i = grp; i < n_old; i += 4) {
      uint4* w = reinterpret_cast<uint4*>(rows + i * step + 16 * sub);
      *w = requant<KV>(*w, ratio);
    }
  }
  for (int p = p_new; p < p_end; p += 4) {
    if (p_end - p_new > 4) fresh = take(p + grp);
    if (fresh) put_codes<KV>(rows + (p + grp - blk * SB) * step, i0, x1, x2, inv, odd);
  }
  if (lane == 0) scale[sc] = now;
}

// Sixteen codes of K and of V per thread.  Bound by memory: 60000 rows of 8 heads, 369 MB,
// in 56.9 us, 6.5 TB/s.
template <typename T, int KV>
__global__ void __launch_bounds__(256) kv8_read_kernel(const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                                                       const float* __restrict__ ks, const float* __restrict__ vs,
                                                       int64_t num_slots, int sb_shift, int nkv,
                                                       const int64_t* __restrict__ rows, int64_t n,
                                                       T* __restrict__ k_out, T* __restrict__ v_out, int32_t* err) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  const int64_t idx = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int per_row = nkv * (HD / 16);
  if (idx >= n * per_row) return;
  const int64_t i = idx / per_row;
  const int c = int(idx % per_row), g = c / (HD / 16);
  const int64_t row = rows[i];
  const bool ok = row >= 0 && row < num_slots;
  if (!ok && row != -1 && c == 0 && err != nullptr) atomicAdd(err, 1);
  const int64_t at = (ok ? row : 0) * nkv * HD + 16 * c;
  const int64_t sc = ((ok ? row : 0) >> sb_shift) * nkv + g;
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  float sk = 0.0f, sv = 0.0f;
  if (ok && k_out != nullptr) {
    a = *reinterpret_cast<const uint4*>(k + at);
    sk = ks[sc];
  }
  if (ok && v_out != nullptr) {
    b = *reinterpret_cast<const uint4*>(v + at);
    sv = vs[sc];
  }
  auto put = [&](T* out, const uint4& w, float s) {
    float f[16];
    codes_f32<KV>(w.x, f);
    codes_f32<KV>(w.y, f + 4);
    codes_f32<KV>(w.z, f + 8);
    codes_f32<KV>(w.w, f + 12);
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] *= s;
    T* o = out + idx * 16;
#pragma unroll
    for (int e = 0; e < 16; e += V16<T>::N) store16(o + e, f + e);
  };
  if (k_out != nullptr) put(k_out, a, sk);
  if (v_out != nullptr) put(v_out, b, sv);
}

template <int KV, int SB>
int launch_append(const AppendArgs& a0, cudaStream_t st) {
  AppendArgs a = a0;
  // every touched block holds at least one new token, and a sequence with Lq of
  // them touches at most (Lq + sb - 2) / sb + 1 blocks
  const int64_t blocks = std::min(a.T, a.T / SB + 2 * int64_t(a.n_seqs));
  // Up to eight tokens a sequence on average: warps instead of CTAs.  16 q and 8 kv
  // heads, scale_block 64: 64 sequences of one token 3.4 us against 7.4, of eight 5.8
  // against 11.3, 16 sequences of eight 4.2 against 4.1, of sixteen 6.4 against 5.0.
  // (Only the average is known here: a long chunk among single tokens goes this way too,
  // where its k and v are computed twice.)
  const bool few = a.T <= 8 * int64_t(a.n_seqs);
  a.kv_ctas = few ? (blocks * a.nkv * 2 + 3) / 4 : blocks * a.nkv;
  const int64_t q_ctas = few ? (a.T * a.nh + 15) / 16 : (a.T * ((a.nh + QH - 1) / QH) + SB - 1) / SB;
  if (a.T * (a.nh + 2 * int64_t(a.nkv)) > (int64_t(1) << 30) || blocks * a.nkv > (int64_t(1) << 28))
    return set_error(QW_ERR_SHAPE, "qw_kv8_append: %lld tokens are too many for one call", (long long)a.T);
  const unsigned ctas = unsigned(a.kv_ctas + q_ctas);
  if (few) launch_pdl(kv8_append_few_kernel<KV, SB>, ctas, 128, 0, st, a);
  else launch_pdl(kv8_append_kernel<KV, SB>, ctas, SB * 8, 0, st, a);
  return check_launch("kv8_append");
}
template <int KV>
int launch_append_sb(const AppendArgs& a, int scale_block, cudaStream_t st) {
  switch (scale_block) {
    case 16: return launch_append<KV, 16>(a, st);
    case 32: return launch_append<KV, 32>(a, st);
    default: return launch_append<KV, 64>(a, st);
  }
}

template <typename T, int KV>
int launch_read(const void* k, const void* v, const float* ks, const float* vs, int64_t num_slots, int scale_block,
                int nkv, const int64_t* rows, int64_t n, void* k_out, void* v_out, int32_t* err, cudaStream_t st) {
  const int64_t ctas = (n * nkv * (HD / 16) + 255) / 256;
  if (ctas > INT32_MAX) return set_error(QW_ERR_SHAPE, "qw_kv8_read: too many rows");
  launch_pdl(kv8_read_kernel<T, KV>, unsigned(ctas), 256, 0, st, static_cast<const uint8_t*>(k),
             static_cast<const uint8_t*>(v), ks, vs, num_slots, scale_shift(scale_block), nkv, rows, n,
             static_cast<T*>(k_out), static_cast<T*>(v_out), err);
  return check_launch("kv8_read_kernel");
}

}  // namespace kv8
}  // namespace qw

using namespace qw;

extern "C" int qw_kv8_append(const void* qkv, int64_t T, int n_heads, int n_kv_heads, int head_dim, int tp,
                             const int64_t* positions, const float* cos_sin, int64_t max_position, const void* q_gamma,
                             const void* k_gamma, float eps, const int32_t* cu_seqlens_q, const int32_t* context_lens,
                             const int32_t* block_table, int max_blocks, int block_size, int n_seqs, void* k_cache,
                             void* v_cache, float* k_scale, float* v_scale, int64_t num_slots, int scale_block,
                             void* q_out, int32_t* err_count, int dtype, int kv_dtype, void* stream) {
  const char* who = "qw_kv8_append";
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "%s: bf16 only", who);
  if (T < 0 || n_seqs < 0 || n_heads <= 0 || n_kv_heads <= 0 || tp <= 0 || max_position <= 0)
    return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != kv8::HD || n_heads % tp || n_kv_heads % tp)
    return set_error(QW_ERR_SHAPE, "%s: needs head_dim 128 and tp | nh, nkv", who);
  if (!cu_seqlens_q && T < n_seqs)
    return set_error(QW_ERR_SHAPE, "%s: %lld tokens for %d sequences of one token", who, (long long)T, n_seqs);
  int rc = kv8::check_cache(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, kv_dtype);
  if (rc) return rc;
  rc = kv8::check_table(who, block_table, max_blocks, block_size);
  if (rc) return rc;
  if (T == 0 || n_seqs == 0) return QW_OK;
  if (!qkv || !positions || !cos_sin || !q_gamma || !k_gamma || !context_lens || !q_out)
    return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!kv8::aligned16(qkv) || !kv8::aligned16(cos_sin) || !kv8::aligned16(q_gamma) || !kv8::aligned16(k_gamma) ||
      !kv8::aligned16(q_out))
    return set_error(QW_ERR_INVALID_ARG, "%s: qkv, cos_sin, gammas and q_out must be 16-byte aligned", who);
  kv8::AppendArgs a;
  a.qkv = static_cast<const bf16*>(qkv);
  a.T = T;
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.tp = tp;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.max_pos = max_position;
  a.q_gamma = static_cast<const bf16*>(q_gamma);
  a.k_gamma = static_cast<const bf16*>(k_gamma);
  a.eps = eps;
  a.cu_q = cu_seqlens_q;
  a.ctx = context_lens;
  a.table = block_table;
  a.max_blocks = max_blocks;
  a.block_size = block_size;
  a.n_seqs = n_seqs;
  a.k = static_cast<uint8_t*>(k_cache);
  a.v = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.num_slots = num_slots;
  a.q_out = static_cast<bf16*>(q_out);
  a.err = err_count;
  a.kv_ctas = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_dtype == QW_I8 ? kv8::launch_append_sb<QW_I8>(a, scale_block, st)
                           : kv8::launch_append_sb<QW_E4M3>(a, scale_block, st);
}

extern "C" int qw_kv8_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                           int64_t num_slots, int scale_block, int n_kv_heads, int head_dim, const int64_t* rows,
                           int64_t n_rows, void* k_out, void* v_out, int32_t* err_count, int dtype, int kv_dtype,
                           void* stream) {
  const char* who = "qw_kv8_read";
  if (dtype != QW_BF16 && dtype != QW_F32) return set_error(QW_ERR_DTYPE, "%s: dtype %d", who, dtype);
  if (n_rows < 0 || n_kv_heads <= 0) return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != kv8::HD) return set_error(QW_ERR_SHAPE, "%s: needs head_dim 128", who);
  const int rc = kv8::check_cache(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, kv_dtype);
  if (rc) return rc;
  if (n_rows == 0 || (!k_out && !v_out)) return QW_OK;
  if (!rows) return set_error(QW_ERR_INVALID_ARG, "%s: null rows", who);
  if (!kv8::aligned16(k_out) || !kv8::aligned16(v_out))
    return set_error(QW_ERR_INVALID_ARG, "%s: outputs must be 16-byte aligned", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define QW_READ(TT, KV)                                                                                             \
  kv8::launch_read<TT, KV>(k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, n_kv_heads, rows, n_rows, k_out, \
                           v_out, err_count, st)
  if (dtype == QW_BF16) return kv_dtype == QW_I8 ? QW_READ(bf16, QW_I8) : QW_READ(bf16, QW_E4M3);
  return kv_dtype == QW_I8 ? QW_READ(float, QW_I8) : QW_READ(float, QW_E4M3);
#undef QW_READ
}
