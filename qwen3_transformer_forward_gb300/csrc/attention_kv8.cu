// Decode attention over the 8-bit paged KV cache, with a sliding window and
// first tokens that stay visible (prefill: attention_kv8_prefill.cu).
#include <math.h>

#include <algorithm>

#include "kv8.cuh"
#include "tc_common.cuh"

namespace qw {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f;

// Error word of this file's kernels: kErrContextOverflow (common.cuh), else a bounded wait that gave up.
__device__ unsigned int g_kv8_error = 0;

// ---------------------------------------------------------------------------
// decode
//
// A tile is KT = 128 / HG tokens of HG kv heads (HG = 8, 4, 2 or 1, the group of
// kv heads that a CTA reads together): 16 KB of K and 16 KB of V, which sit side
// by side in memory, so that the copies of one tile cover whole DRAM rows however
// the tiles are dealt out.  One CTA per SM.  Every CTA sums the sequences' visible
// tiles (their lengths are on the device) and takes an equal, contiguous share:
// ragged batches and windows stay balanced.  A producer warp streams the share
// through a ring of stages (TMA boxes of 16 tokens x HG heads, which lie in one
// page and one scale block; 128-byte swizzle; the block scales by 4-byte
// asynchronous copies on the same barrier).  Eight consumer warps each take the
// 16 keys x 128 dims of one kv head:
//   S^T [16 keys, 8 heads] = K Q^T   8 mma.m16n8k16: keys are the rows, so that a
//   O^T [128 dims, 8 heads] += V^T P  group of up to 8 q heads fills the columns
// Operands are f16: codes are exact in it, q is moved by a power of two per row
// (exact, see row_scale), weights keep 11 bits.  The order of the dims inside a
// k-step is free as long as Q and K share it, so a lane loads 16 codes at a time
// and converts them in registers, without ldmatrix.  A step's 16 keys share one
// scale: with x = score * log2 e * k_scale + log2(v_scale), the running maximum m
// is over x, the weights are 2^(x - m + 15) <= 2^15 (f16 keeps 11 bits down to
// 2^-29 of the largest), O takes the codes of V alone, and the denominator is
// sum 2^(x - m) / v_scale, in fp32, of the weights before they are rounded.  One f16 is
// enough: at most 2^-11 of a weight, independent for each key, against the 2^-8 that
// the bf16 output is rounded by, and a second f16 for the rest would double the PV
// products.  The exponentials and logarithms are the hardware's approximations (2^-22).
// A (sequence, kv head) that ends inside one CTA is written out; otherwise every
// CTA of it leaves (m, l, O) in the workspace slot (CTA + pair), distinct for each
// that occurs, and the last to finish, by the pair's counter, adds them in CTA
// order.
// Bound by the copies, and next to them by the latency of a consumer step (two warps
// on an SM sub-partition): 64 sequences of 256 - 2048 tokens, 16 / 8 heads, int8,
// 39.1 us, 4.0 TB/s (34.5 us without the arithmetic); 7 of 9000 - 32768, 32 / 8 heads,
// e4m3, 62.9 us, 4.9 TB/s.  Eight kv heads side by side against one: 39.4 and 61.6 us
// for the 64 sequences.
// ---------------------------------------------------------------------------
constexpr int DK_WARPS = 8, DK_THREADS = 32 * (DK_WARPS + 1);
constexpr int DK_CTAS = 152;                       // at most one CTA per SM
constexpr uint32_t DK_SUB = 2048;                  // 16 keys x 128 codes of one kv head
constexpr uint32_t DK_STAGE = 2 * DK_WARPS * DK_SUB;
constexpr int DK_MIN_TILES = 8;                    // tiles that a CTA gets at least
constexpr float kShift = 15.0f;                    // weights are held times 2^15
constexpr float kUnshift = 1.0f / 32768.0f;

template <int HG, int NT> __host__ __device__ constexpr int dk_stages() { return HG == DK_WARPS ? 6 : NT == 1 ? 5 : 4; }
// ring | merge [8 warps][36 NT words][32 lanes], with several warps per kv head | scales | barriers
template <int HG, int NT> __host__ __device__ constexpr uint32_t dk_merge_bytes() {
  return HG == DK_WARPS ? 0u : uint32_t(DK_WARPS) * 36u * NT * 128u;
}
template <int HG, int NT> __host__ __device__ constexpr size_t dk_smem() {
  static_assert(1024 + dk_stages<HG, NT>() * (DK_STAGE + 2 * DK_WARPS * 4 + 16) + dk_merge_bytes<HG, NT>() + 512 <= 232448,
                "shared memory of one CTA");
  return 1024 + size_t(dk_stages<HG, NT>()) * (DK_STAGE + 2 * DK_WARPS * 4 + 16) + dk_merge_bytes<HG, NT>() + 256;
}

struct DecodeArgs {
  const bf16* q;
  const int32_t* ctx;
  Cache c;
  int B, nh, nkv, G, nhg;   // G: q heads of a kv head; nhg: groups of HG kv heads
  int max_ctx, window, n_sink;
  float scale_log2;
  float* ws_o;              // [slots][HG][G][128]
  float* ws_ml;             // [slots][HG][G][2]
  unsigned int* counters;   // [B * nkv]
  bf16* out;
};

__device__ __forceinline__ Span decode_span(int ctx, int max_ctx, int window, int n_sink, int kt) {
  Span s;
  s.L = max(min(ctx, max_ctx), 0);
  s.lo = window > 0 ? max(ctx - window, 0) : 0;
  const int tb = (s.L + kt - 1) / kt;
  s.w0 = s.lo / kt;
  s.ns = min(min((min(n_sink, s.lo) + kt - 1) / kt, s.w0), tb);
  s.nt = s.ns + max(tb - s.w0, 0);
  return s;
}
__device__ __forceinline__ bool any_visible(const Span& s, int n_sink, int key0) {   // of 16 keys from key0
  return max(key0, s.lo) < min(key0 + 16, s.L) || key0 < min(n_sink, s.L);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ unsigned int atom_add_acq_rel(unsigned int* p, unsigned int v) {
  unsigned int old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {   // when this thread's copies so far have landed
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Writes 16 outputs of one head: dims 16 gq .. + 15.
__device__ __forceinline__ void store_out16(bf16* o, const float (&f)[16]) {
  store16(o, f);
  store16(o + 8, f + 8);
}

template <int KV, int HG, int NT>
__global__ void __launch_bounds__(DK_THREADS, 1) attn_decode_kv8_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                       const __grid_constant__ CUtensorMap tmV,
                                                                       const DecodeArgs a) {
  constexpr int KS = DK_WARPS / HG, KT = 16 * KS, ST = dk_stages<HG, NT>();
  // tiles of a consumer step (two n-tiles: one, and even so 84 to 108 bytes a thread are spilled; of one, none)
  constexpr int UN = NT == 1 ? 2 : 1;
  constexpr uint32_t kBox = 16 * HG * HD;            // bytes of one TMA box
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(sm);
  float* merge = reinterpret_cast<float*>(sm + ST * DK_STAGE);
  float* scales = reinterpret_cast<float*>(sm + ST * DK_STAGE + dk_merge_bytes<HG, NT>());   // [ST][K, V][8]
  const uint32_t bars = smem_u32(scales + ST * 2 * DK_WARPS);
  auto full = [&](int s) { return bars + 8u * uint32_t(s); };
  auto empty = [&](int s) { return bars + 8u * uint32_t(ST + s); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      tcx::mbar_init(full(s), 33);
      tcx::mbar_init(empty(s), DK_WARPS);
    }
    tcx::fence_mbar_init();
    tcx::prefetch_map(&tmK);
    tcx::prefetch_map(&tmV);
  }
  __syncthreads();
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue

  // ---- this CTA's share: an equal part of all sequences' visible tiles.  Every warp finds it by
  // itself: a lane takes `chunk` sequences in a row, a scan over the lanes gives the total and
  // the lane with tile `lo`, which walks through its sequences.
  auto span_of = [&](int b) { return decode_span(a.ctx[b], a.max_ctx, a.window, a.n_sink, KT); };
  const int chunk = (a.B + 31) / 32;
  int mine = 0;
  for (int i = 0; i < chunk; ++i) {
    const int b = lane * chunk + i, ctx = b < a.B ? a.ctx[b] : 1;
    const int nt = b < a.B ? decode_span(ctx, a.max_ctx, a.window, a.n_sink, KT).nt : 0;
    mine += nt * a.nhg;
    // of the sequences dealt to this CTA: note a context that is too long, zero the rows of one that sees nothing
    const bool dealt = warp == 1 && b < a.B && b % gridDim.x == blockIdx.x;
    if (dealt && ctx > a.max_ctx) atomicOr(&g_kv8_error, kErrContextOverflow);
    for (unsigned m = __ballot_sync(0xffffffffu, dealt && nt == 0); m; m &= m - 1) {
      const int64_t zb = int64_t(__ffs(m) - 1) * chunk + i;
      for (int c = lane; c < a.nh * HD / 8; c += 32)
        *reinterpret_cast<uint4*>(a.out + zb * a.nh * HD + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31);
  const int per = max(DK_MIN_TILES, (total + int(gridDim.x) - 1) / int(gridDim.x));
  const int lo = int(blockIdx.x) * per, hi = min(total, lo + per);
  if (lo >= hi) return;   // uniform over the CTA
  // position in the share: tile t of kv head group hg of sequence b; `start` is the
  // first tile of that (sequence, group) in the common order
  int b = 0, before = upto - mine;
  {
    const bool here = lo >= before && lo < upto;
    if (here)
      for (b = lane * chunk;; ++b) {
        const int n = span_of(b).nt * a.nhg;
        if (lo < before + n) break;
        before += n;
      }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    b = __shfl_sync(0xffffffffu, b, src);
    before = __shfl_sync(0xffffffffu, before, src);
  }
  Span sp = span_of(b);
  int hg = (lo - before) / sp.nt, t = (lo - before) % sp.nt;
  const int count = hi - lo;
  auto next_pair = [&]() {   // only while a tile is left
    t = 0;
    if (++hg == a.nhg) {
      hg = 0;
      do sp = span_of(++b);
      while (sp.nt == 0);
    }
  };
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity, unsigned int code) {
    if (ok && !tcx::mbar_wait(bar, parity, &g_kv8_error, code)) ok = false;
  };

  if (warp == DK_WARPS) {
    // ---------------- producer warp
    int j = 0;
    for (; j < count; ++j, ++t) {
      if (t == sp.nt) next_pair();
      const int s = j % ST;
      if (j >= ST) wait(empty(s), uint32_t(j / ST - 1) & 1u, 0x1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // the consumers read this stage through the generic proxy, the copies write through the async proxy
      tcx::fence_proxy_async();
      const int key0 = (sp.tile(t) * KS + (lane & (KS - 1))) * 16;   // lane ks < KS: 16 tokens of every head
      const bool act = any_visible(sp, a.n_sink, key0);
      const int64_t row = act ? row_of(a.c.table, a.c.max_blocks, a.c.block_size, a.c.num_slots, b, key0) : -1;
      const unsigned boxes = __popc(__ballot_sync(0xffffffffu, act && lane < KS));
      if (lane == 0) tcx::mbar_expect_tx(full(s), boxes * 2 * kBox);
      __syncwarp();
      if (act && lane < KS) {
        const int y = row >= 0 ? int(row) : int(a.c.num_slots);      // outside: zeros
        const uint32_t dst = ring + uint32_t(s) * DK_STAGE + uint32_t(lane) * kBox;
        tcx::tma_load_3d(dst, &tmK, full(s), 0, y, hg * HG);
        tcx::tma_load_3d(dst + DK_STAGE / 2, &tmV, full(s), 0, y, hg * HG);
      }
      // scales of consumer warp `lane`: its 16 keys are lane / HG, its kv head lane % HG
      const int64_t wrow = __shfl_sync(0xffffffffu, row, (lane & 7) / HG);
      const int g = hg * HG + lane % HG;
      if (lane < DK_WARPS) {
        const bool has = wrow >= 0 && g < a.nkv;
        const int64_t at = has ? (wrow >> a.c.sb_shift) * a.nkv + g : 0;
        const uint32_t dst = smem_u32(scales + s * 2 * DK_WARPS + lane);
        cp_async4_zfill(dst, a.c.k_scale + at, has);
        cp_async4_zfill(dst + 4 * DK_WARPS, a.c.v_scale + at, has);
      }
      cp_async_arrive(full(s));
    }
    // the last copy of each stage has landed before this CTA may end
    for (int i = max(0, j - ST); i < j; ++i)
      tcx::mbar_wait(full(i % ST), uint32_t(i / ST) & 1u, &g_kv8_error, 0x4u);
    return;
  }

  // ---------------- consumer warps
  const int gq = lane >> 2, tq = lane & 3;
  const int h = warp % HG, ks = warp / HG;
  int start = lo - t;
  // split pairs whose part this warp has written: the first of the share, counted during the
  // next pair's tiles (so that neither the fence nor the atomic holds up the ring), and the last
  int pend = 0, p0_b = 0, p0_hg = 0, p0_first = 0, p0_last = 0, p1_b = 0, p1_hg = 0, p1_first = 0, p1_last = 0;
  bool counted = false;
  unsigned int done = 0;
  int j = 0;
  while (j < count) {
    if (t == sp.nt) {
      start += sp.nt;
      next_pair();
    }
    const int g = hg * HG + h;
    const bool head_ok = g < a.nkv;
    const int n_seg = min(sp.nt - t, count - j);
    // q: head column 8 nt + gq, dims 32 tq .. + 31, moved into f16's range
    uint32_t qb[NT][8][2];
    float qa[NT][2];   // score factor of heads 8 nt + 2 tq, + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int hd = 8 * n + gq;
      const bool has = head_ok && hd < a.G;
      const bf16* src = a.q + (int64_t(b) * a.nh + (has ? g * a.G + hd : 0)) * HD + 32 * tq;
      float f[32], top = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) load16(src + 8 * e, f + 8 * e);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        f[e] = has ? f[e] : 0.0f;
        top = fmaxf(top, fabsf(f[e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float mul, inv;
      row_scale(top, mul, inv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        qb[n][e][0] = pack_f16(f[4 * e] * mul, f[4 * e + 1] * mul);
        qb[n][e][1] = pack_f16(f[4 * e + 2] * mul, f[4 * e + 3] * mul);
      }
      inv *= a.scale_log2;
      qa[n][0] = __shfl_sync(0xffffffffu, inv, 8 * tq);
      qa[n][1] = __shfl_sync(0xffffffffu, inv, 8 * tq + 4);
    }
    float o[NT][8][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }
    // UN tiles at a time: their chains of loads, conversions and matrix instructions overlap
    for (int i = 0; i < n_seg; i += UN, j += UN, t += UN) {
      const bool two = UN > 1 && i + 1 < n_seg;
      int st[UN], key0[UN];
      bool act[UN], any = false;
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        st[u] = (j + u) % ST;
        key0[u] = (sp.tile(t + u) * KS + ks) * 16;
        act[u] = head_ok && (u == 0 || two) && any_visible(sp, a.n_sink, key0[u]);
        any |= act[u];
      }
      wait(full(st[0]), uint32_t(j / ST) & 1u, 0x2u);
      if (two) wait(full(st[UN - 1]), uint32_t((j + 1) / ST) & 1u, 0x2u);
      if (any) {
        float c[UN][NT][4], sk[UN], lsv[UN], isv[UN];
        bool v_none[UN], vis[UN][2];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const uint32_t sK = ring + uint32_t(st[u]) * DK_STAGE + uint32_t(warp) * DK_SUB;
          // a tile that is not there has no visible key, whatever codes are read
          const float* sc = scales + st[u] * 2 * DK_WARPS + warp;
          sk[u] = act[u] ? sc[0] : 0.0f;
          const float sv = act[u] ? sc[DK_WARPS] : 1.0f;
          v_none[u] = sv < kTinyScale;
          const float svc = v_none[u] ? kTinyScale : sv;
          lsv[u] = lg2(svc);
          isv[u] = __fdividef(kUnshift, svc);
          const bool all = key0[u] + 16 <= sp.L && (key0[u] >= sp.lo || key0[u] + 16 <= a.n_sink);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int kp = key0[u] + gq + 8 * r;
            vis[u][r] = act[u] && (all || (kp < sp.L && (kp >= sp.lo || kp < a.n_sink)));
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) c[u][n][0] = c[u][n][1] = c[u][n][2] = c[u][n][3] = 0.0f;
          // keys gq and gq + 8, dims 32 tq .. + 31 (16-byte chunks 2 tq, 2 tq + 1)
          uint32_t k0[8], k1[8];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t at = sK + uint32_t(gq) * 128u + (uint32_t((2 * tq + w) ^ gq) << 4);
            const uint4 x = lds128(at), y = lds128(at + 1024u);
            k0[4 * w] = x.x; k0[4 * w + 1] = x.y; k0[4 * w + 2] = x.z; k0[4 * w + 3] = x.w;
            k1[4 * w] = y.x; k1[4 * w + 1] = y.y; k1[4 * w + 2] = y.z; k1[4 * w + 3] = y.w;
          }
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t a0, a1, a2, a3;
            word_pairs<KV>(k0[kk], a0, a2);
            word_pairs<KV>(k1[kk], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(c[u][n], a0, a1, a2, a3, qb[n][kk][0], qb[n][kk][1]);
          }
        }
        uint32_t pb[UN][NT][2];
        bool grew = false;
        float al[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[UN][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x[UN][2], mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < UN; ++u) {
              const float f = qa[n][e] * sk[u];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                x[u][r] = vis[u][r] ? fmaf(c[u][n][e + 2 * r], f, lsv[u]) : -INFINITY;
                mx = fmaxf(mx, x[u][r]);
              }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(m[n][e], mx);   // finite: a key of these tiles is visible
            grew |= m_new > m[n][e];
            al[n][e] = ex2(m[n][e] - m_new);
            m[n][e] = m_new;
            l[n][e] *= al[n][e];
#pragma unroll
            for (int u = 0; u < UN; ++u) {   // (x - m first: both may be huge, the difference of the largest is exactly zero)
              p[u][e] = ex2(x[u][0] - m_new + kShift);
              p[u][e + 2] = ex2(x[u][1] - m_new + kShift);
              l[n][e] = fmaf(p[u][e] + p[u][e + 2], isv[u], l[n][e]);
            }
          }
#pragma unroll
          for (int u = 0; u < UN; ++u) {
            pb[u][n][0] = transpose8(v_none[u] ? 0u : pack_f16(p[u][0], p[u][1]));   // keys 2 tq, + 1 of head gq
            pb[u][n][1] = transpose8(v_none[u] ? 0u : pack_f16(p[u][2], p[u][3]));   // keys 8 + 2 tq, + 1
          }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              o[n][d][0] *= al[n][0];
              o[n][d][1] *= al[n][1];
              o[n][d][2] *= al[n][0];
              o[n][d][3] *= al[n][1];
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          // V: keys 2 tq, 2 tq + 1 and the same + 8, dims 16 gq .. + 15
          const uint32_t sV = ring + uint32_t(st[u]) * DK_STAGE + DK_STAGE / 2 + uint32_t(warp) * DK_SUB;
          uint32_t v[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * tq + (r & 1) + 8 * (r >> 1);
            const uint4 x = lds128(sV + uint32_t(row) * 128u + (uint32_t(gq ^ (row & 7)) << 4));
            // (a row that is not there may hold any code, NaN too: 0 * V has to stay 0)
            const bool there = act[u] && key0[u] + row < sp.L;
            v[r][0] = there ? x.x : 0u;
            v[r][1] = there ? x.y : 0u;
            v[r][2] = there ? x.z : 0u;
            v[r][3] = there ? x.w : 0u;
          }
          // O^T rows: tile d holds dims 16 gq + 2 d (row gq) and 16 gq + 2 d + 1 (row gq + 8)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t lo4[4], hi4[4];
            cross_pairs<KV>(v[0][w], v[1][w], lo4);
            cross_pairs<KV>(v[2][w], v[3][w], hi4);
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(o[n][2 * w + d], lo4[2 * d], lo4[2 * d + 1], hi4[2 * d], hi4[2 * d + 1], pb[u][n][0],
                        pb[u][n][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        tcx::mbar_arrive(empty(st[0]));
        if (two) tcx::mbar_arrive(empty(st[UN - 1]));
      }
      if (pend == 1 && !counted && i >= UN) {   // (the part's stores are a step old: the fence is short)
        __threadfence();
        __syncwarp();
        if (lane == 0) done = atom_add_acq_rel(a.counters + p0_b * a.nkv + p0_hg * HG + h, 1u);
        counted = true;
      }
      if (UN > 1 && !two) {   // the part's last tile stood alone
        --j;
        --t;
      }
    }
    // ---- end of this CTA's part of the pair: sums over the lanes of a head, then over the head's warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
      }
    if constexpr (KS > 1) {
      float* mw = merge + warp * 36 * NT * 32 + lane;
      if (ks > 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) mw[((n * 8 + i) * 4 + e) * 32] = o[n][i][e];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mw[(32 * NT + 4 * n + e) * 32] = m[n][e];
            mw[(32 * NT + 4 * n + 2 + e) * 32] = l[n][e];
          }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * DK_WARPS) : "memory");
      if (ks == 0) {
#pragma unroll 1
        for (int w = h + HG; w < DK_WARPS; w += HG) {
          const float* ow = merge + w * 36 * NT * 32 + lane;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float mine_[2], theirs[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float mo = ow[(32 * NT + 4 * n + e) * 32], lo_ = ow[(32 * NT + 4 * n + 2 + e) * 32];
              const float mx = fmaxf(m[n][e], mo), mu = mx == -INFINITY ? 0.0f : mx;
              mine_[e] = ex2(m[n][e] - mu);
              theirs[e] = ex2(mo - mu);
              m[n][e] = mx;
              l[n][e] = l[n][e] * mine_[e] + lo_ * theirs[e];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[n][i][e] = o[n][i][e] * mine_[e & 1] + ow[((n * 8 + i) * 4 + e) * 32] * theirs[e & 1];
          }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * DK_WARPS) : "memory");   // the area is free again
    }
    if (ks == 0 && head_ok) {
      const int c_first = start / per, c_last = (start + sp.nt - 1) / per;
      const bool split = c_first != c_last;
      const int pair = b * a.nhg + hg;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int hd = 8 * n + 2 * tq + e;
          if (hd >= a.G) continue;
          float f[16];
          // no visible key: l = 0, a zero row; a query with NaN: l NaN, and so is the row
          const float fac = split ? 1.0f : (l[n][e] == 0.0f ? 0.0f : kUnshift / l[n][e]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[2 * i] = o[n][i][e] * fac;
            f[2 * i + 1] = o[n][i][e + 2] * fac;
          }
          if (!split) {
            store_out16(a.out + (int64_t(b) * a.nh + g * a.G + hd) * HD + 16 * gq, f);
          } else {
            const int64_t idx = ((int64_t(blockIdx.x) + pair) * HG + h) * a.G + hd;
#pragma unroll
            for (int i = 0; i < 4; ++i) store16(a.ws_o + idx * HD + 16 * gq + 4 * i, f + 4 * i);
            if (gq == 0) {
              a.ws_ml[2 * idx] = m[n][e];
              a.ws_ml[2 * idx + 1] = l[n][e];
            }
          }
        }
      if (split) {   // the first and the last pair of a share at most
        if (pend == 0) {
          p0_b = b; p0_hg = hg; p0_first = c_first; p0_last = c_last;
        } else {
          p1_b = b; p1_hg = hg; p1_first = c_first; p1_last = c_last;
        }
        ++pend;
      }
    }
  }
  // ---- pairs that other CTAs work on too: this CTA's part counts as done, and the last to be
  // done adds the parts
#pragma unroll 1
  for (int k = 0; k < pend; ++k) {
    const int pb = k ? p1_b : p0_b, phg = k ? p1_hg : p0_hg, c_first = k ? p1_first : p0_first, c_last = k ? p1_last : p0_last;
    const int g = phg * HG + h, pair = pb * a.nhg + phg;
    if (k || !counted) {
      __threadfence();
      __syncwarp();
      if (lane == 0) done = atom_add_acq_rel(a.counters + pb * a.nkv + g, 1u);
    }
    if (__shfl_sync(0xffffffffu, done, 0) != unsigned(c_last - c_first)) continue;
    __threadfence();
    // four heads at a time, four CTAs' parts each: 32 loads in flight for a lane
    for (int h0 = 0; h0 < a.G; h0 += 4) {
      auto index = [&](int c, int u) { return ((int64_t(c) + pair) * HG + h) * a.G + min(h0 + u, a.G - 1); };
      float M[4], lsum[4];
      float4 acc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        M[u] = -INFINITY;
        lsum[u] = 0.0f;
        acc[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      for (int c = c_first + lane; c <= c_last; c += 32)
#pragma unroll
        for (int u = 0; u < 4; ++u) M[u] = fmaxf(M[u], __ldcg(a.ws_ml + 2 * index(c, u)));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        M[u] = warp_max(M[u]);
        if (M[u] == -INFINITY) M[u] = 0.0f;
      }
      for (int c0 = c_first; c0 <= c_last; c0 += 4) {
        float2 ml[4][4];
        float4 x[4][4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int64_t idx = index(min(c0 + v, c_last), u);
            ml[v][u] = __ldcg(reinterpret_cast<const float2*>(a.ws_ml) + idx);
            x[v][u] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + idx * HD) + lane);
          }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float w = c0 + v <= c_last ? ex2(ml[v][u].x - M[u]) : 0.0f;
            lsum[u] = fmaf(ml[v][u].y, w, lsum[u]);
            acc[u].x = fmaf(x[v][u].x, w, acc[u].x);
            acc[u].y = fmaf(x[v][u].y, w, acc[u].y);
            acc[u].z = fmaf(x[v][u].z, w, acc[u].z);
            acc[u].w = fmaf(x[v][u].w, w, acc[u].w);
          }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (h0 + u >= a.G) continue;
        const float fac = lsum[u] == 0.0f ? 0.0f : kUnshift / lsum[u];   // (NaN stays)
        *reinterpret_cast<uint2*>(a.out + (int64_t(pb) * a.nh + g * a.G + h0 + u) * HD + 4 * lane) =
            make_uint2(pack_bf16(acc[u].x * fac, acc[u].y * fac), pack_bf16(acc[u].z * fac, acc[u].w * fac));
      }
    }
    if (lane == 0) a.counters[pb * a.nkv + g] = 0u;
  }
}

int head_group(int nkv) { return nkv > 4 ? 8 : nkv > 2 ? 4 : nkv; }

// Room for the partial results: one (m, l, O) per (CTA, pair) that can occur.
size_t decode_slots(int B, int nkv) {
  const int hg = head_group(nkv);
  return size_t(DK_CTAS) + size_t(B) * ((nkv + hg - 1) / hg);
}
size_t decode_workspace(int B, int nh, int nkv) {
  return kCounterBytes + decode_slots(B, nkv) * head_group(nkv) * (nh / nkv) * (HD + 2) * sizeof(float);
}

template <int KV, int HG, int NT>
int launch_decode(const DecodeArgs& a, int64_t num_slots, cudaStream_t st) {
  // tiles of the longest sequences that the call allows
  constexpr int KT = 16 * (DK_WARPS / HG);
  int64_t tiles = (int64_t(a.max_ctx) + KT - 1) / KT;
  if (a.window > 0)
    tiles = std::min(tiles, (int64_t(a.window) + KT - 1) / KT + 1 + (int64_t(a.n_sink) + KT - 1) / KT);
  if (tiles * a.B * a.nhg > INT32_MAX / 2)
    return set_error(QW_ERR_SHAPE, "qw_attention_decode_kv8: %d sequences of up to %d keys are too many", a.B, a.max_ctx);
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(attn_decode_kv8_kernel<KV, HG, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(dk_smem<HG, NT>()));
    if (e != cudaSuccess) return set_error(QW_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    configured = true;
  }
  // K and V as [kv head][slot][128 bytes] (64 two-byte elements: the copies move bits)
  CUtensorMap mk, mv;
  const uint64_t dims[3] = {64, uint64_t(num_slots), uint64_t(a.nkv)};
  const uint64_t strides[2] = {uint64_t(a.nkv) * HD, HD};
  const uint32_t box[3] = {64, 16, HG};
  int rc = make_tensor_map(&mk, a.c.k, 3, dims, strides, box);
  if (rc) return rc;
  rc = make_tensor_map(&mv, a.c.v, 3, dims, strides, box);
  if (rc) return rc;
  // no more CTAs than get tiles
  const int64_t ctas = (std::max<int64_t>(tiles, 1) * a.B * a.nhg + DK_MIN_TILES - 1) / DK_MIN_TILES;
  launch_pdl(attn_decode_kv8_kernel<KV, HG, NT>, unsigned(std::min<int64_t>(ctas, DK_CTAS)), DK_THREADS,
             dk_smem<HG, NT>(), st, mk, mv, a);
  return check_launch("attn_decode_kv8_kernel");
}
template <int KV, int HG>
int launch_decode_nt(const DecodeArgs& a, int64_t num_slots, cudaStream_t st) {
  return a.G <= 8 ? launch_decode<KV, HG, 1>(a, num_slots, st) : launch_decode<KV, HG, 2>(a, num_slots, st);
}
template <int KV>
int launch_decode_hg(const DecodeArgs& a, int64_t num_slots, cudaStream_t st) {
  switch (head_group(a.nkv)) {
    case 1: return launch_decode_nt<KV, 1>(a, num_slots, st);
    case 2: return launch_decode_nt<KV, 2>(a, num_slots, st);
    case 4: return launch_decode_nt<KV, 4>(a, num_slots, st);
    default: return launch_decode_nt<KV, 8>(a, num_slots, st);
  }
}

// Checks shared by the two attention entry points.
int check_attention(const char* who, const void* k, const void* v, const float* ks, const float* vs, int64_t num_slots,
                    int scale_block, const int32_t* table, int max_blocks, int block_size, int n_seqs, int max_context,
                    int nh, int nkv, int head_dim, int window, int n_sink, int dtype, int kv_dtype) {
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "%s: bf16 only", who);
  if (n_seqs < 0 || max_context < 0 || nh <= 0 || nkv <= 0 || window < 0 || n_sink < 0)
    return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != HD || nh % nkv || nh / nkv > 16)
    return set_error(QW_ERR_SHAPE, "%s: needs head_dim 128 and nh a multiple of nkv, at most 16 times it", who);
  int rc = check_cache(who, k, v, ks, vs, num_slots, scale_block, kv_dtype);
  if (rc) return rc;
  rc = check_table(who, table, max_blocks, block_size);
  if (rc) return rc;
  if (int64_t(max_context) > int64_t(max_blocks) * block_size || max_context > kMaxPositions)
    return set_error(QW_ERR_SHAPE, "%s: max_context %d > max_blocks x block_size or 2^30", who, max_context);
  return QW_OK;
}

}  // namespace kv8
}  // namespace qw

using namespace qw;

extern "C" size_t qw_attention_decode_kv8_workspace_size(int B, int max_context, int n_heads, int n_kv_heads) {
  if (B < 0 || max_context < 0 || n_heads <= 0 || n_kv_heads <= 0) return 0;
  return kv8::decode_workspace(B, n_heads, n_kv_heads);
}

extern "C" int qw_attention_decode_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                       const float* v_scale, int64_t num_slots, int scale_block,
                                       const int32_t* context_lens, const int32_t* block_table, int max_blocks,
                                       int block_size, int B, int max_context, int n_heads, int n_kv_heads,
                                       int head_dim, float scale, int window, int n_sink, void* out, void* workspace,
                                       size_t workspace_bytes, int dtype, int kv_dtype, void* stream) {
  const char* who = "qw_attention_decode_kv8";
  const int rc = kv8::check_attention(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, block_table,
                                      max_blocks, block_size, B, max_context, n_heads, n_kv_heads, head_dim, window,
                                      n_sink, dtype, kv_dtype);
  if (rc) return rc;
  if (B == 0) return QW_OK;
  if (!q || !context_lens || !out) return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!kv8::aligned16(q) || !kv8::aligned16(out))
    return set_error(QW_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  if (int64_t(B) * n_kv_heads > int64_t(kCounterBytes / sizeof(unsigned int)))
    return set_error(QW_ERR_SHAPE, "%s: %d sequences x %d kv heads exceed the counter area", who, B, n_kv_heads);
  const size_t need = qw_attention_decode_kv8_workspace_size(B, max_context, n_heads, n_kv_heads);
  if (!workspace || workspace_bytes < need)
    return set_error(QW_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  if (!kv8::aligned16(workspace)) return set_error(QW_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
  kv8::DecodeArgs a;
  a.q = static_cast<const bf16*>(q);
  a.ctx = context_lens;
  a.c = kv8::Cache{k_cache, v_cache, k_scale, v_scale, num_slots, kv8::scale_shift(scale_block), block_table, max_blocks,
                   block_size};
  const int hg = kv8::head_group(n_kv_heads);
  a.B = B;
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.G = n_heads / n_kv_heads;
  a.nhg = (n_kv_heads + hg - 1) / hg;
  a.max_ctx = max_context;
  a.window = std::min(window, kv8::kMaxPositions);
  a.n_sink = std::min(n_sink, max_context);
  a.scale_log2 = scale * kv8::kLog2e;
  a.counters = static_cast<unsigned int*>(workspace);
  a.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  a.ws_ml = a.ws_o + kv8::decode_slots(B, n_kv_heads) * hg * a.G * kv8::HD;
  a.out = static_cast<bf16*>(out);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_dtype == QW_I8 ? kv8::launch_decode_hg<QW_I8>(a, num_slots, st)
                           : kv8::launch_decode_hg<QW_E4M3>(a, num_slots, st);
}

namespace qw {
unsigned int take_kv8_prefill_errors();   // attention_kv8_prefill.cu
unsigned int take_kv8_errors() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, kv8::g_kv8_error, sizeof(v));
  if (v) cudaMemcpyToSymbol(kv8::g_kv8_error, &z, sizeof(z));
  return v | take_kv8_prefill_errors();
}
}  // namespace qw
