// Causal varlen prefill attention over the 8-bit paged KV cache on tcgen05
// tensor cores, with a sliding window and first tokens that stay visible.
//
// The query rows of one kv head are packed: row R of a sequence is token R / G,
// q head R % G of its group of G, so that any group size fills the 128-row units
// and a short prompt wastes few rows.  One CTA owns two units (256 rows) and
// walks the key tiles (128 keys) that any of its rows sees.  Per CTA (16 warps):
//   warp 0        allocates 512 TMEM columns and issues every MMA from one lane, in
//                 steps of 64 keys (two a tile), S double-buffered in each unit:
//                   S_u(t)  = Q_u K^T   A = Q_u (smem), B = K (smem), both K-major
//                   O_u    += P_u(t) V  A = P_u (TMEM), B = V (smem, MN-major)
//                 in the order PV_0(t), PV_1(t), S_0(t+2), S_1(t+2): a unit's softmax
//                 works on step t + 1 while the tensor pipe serves both
//   warps 4-7     read the codes of K_j and V_j from the cache into registers one
//                 tile ahead, convert them to f16 (exact) and store them as
//                 128-byte-swizzled operand tiles, two slots each: once for the 256
//                 rows of both units
//   warps 8-11    softmax of unit 0, warps 12-15 of unit 1: one row per thread
// Block scales never touch the operands.  A block of 16 keys shares one scale,
// so with x = score * log2 e * k_scale + log2(v_scale) the running maximum m is
// over x, P = 2^(x - m + 7) is rounded to f16 (m is raised lazily, when a row's
// maximum grows by more than 2^8, so that P <= 2^15), O takes the codes of V alone
// and the denominator is sum 2^(x - m) / v_scale in fp32, of the weights before they
// are rounded.  P keeps 11 bits down to 2^-21 of the largest weight and 2^-32 of it
// below: far under the 2^-8 of the bf16 output, and the A operand in TMEM holds f16.
// The exponentials and logarithms are the hardware's approximations (2^-22).  q is moved by a
// power of two per row (row_scale), exact in f16.  k_scale >= 0 and the softmax
// scale's sign sits in q, so a block's largest x belongs to its largest score:
// the maximum is taken over the raw scores.
// TMEM columns: S of unit u at 128 u + 64 (t & 1), P over the first half of its S;
// O_0 [256,384), O_1 [384,512).
// Few rows over many keys: the tiles are cut into `splits` shares (host rule in
// prefill_splits), each CTA leaves (m, l, O) in fp32 and a second kernel adds them
// in order.
// Bound: a tile of 128 keys takes about 4600 cycles a CTA against 2560 of tensor
// pipe; the softmax's dependent steps (two warps on an SM sub-partition) and the
// operand traffic through shared memory (Q is read again for each step, K and V are
// written by the converters: about 2600 cycles of its bandwidth) hold it there.
// 8 x 2048 tokens, 16 q / 8 kv heads, int8: 213.5 us, 644 TFLOP/s; 2 x 2500 new tokens
// over 24000, 32 / 8 heads, e4m3, window 8192: 643 us, 955 TFLOP/s.
// Every mbarrier wait is bounded (2 s); on timeout the kernel records an error
// word and runs to its end without waiting further, except for its own MMAs in flight.
#include <math.h>

#include <algorithm>

#include "kv8.cuh"
#include "tc_common.cuh"

namespace qw {
namespace kv8p {

using namespace kv8;

__device__ unsigned int g_kv8_prefill_error = 0;
// A wait that gives up sets bit `code` of the word, 0 .. 15: none is the bit of an overlong context.
constexpr uint32_t kWaitCodeMask = 15u;
static_assert((kErrContextOverflow & 0xffffu) == 0u, "the low 16 bits are the waits'");

constexpr int BM = 128, BN = 128, HALF = 64, ROWS = 2 * BM, THREADS = 512;
constexpr uint32_t BOX = 16384;                    // 128 rows x 64 f16
constexpr uint32_t TILE = 2 * BOX;                 // 128 rows x 128 f16
constexpr uint32_t OFF_Q = 0;                      // Q_0, Q_1 (then the output staging)
constexpr uint32_t OFF_K = 2 * TILE;               // K_j in slot j % 2
constexpr uint32_t OFF_V = 4 * TILE;
constexpr uint32_t OFF_SCL = 6 * TILE;             // [4 tiles][8 blocks] {k_scale, log2 v_scale, 2^-7 / v_scale, -}
constexpr uint32_t OFF_BAR = OFF_SCL + 4 * 8 * 16;
constexpr size_t SMEM = 1024 + OFF_BAR + 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f, kShift = 7.0f, kUnshift = 1.0f / 128.0f;
// Past this |m| the exponent is formed as (x - m) + 7 instead of one fused step,
// whose constant log2(v_scale) - m + 7 would be rounded too coarsely.
constexpr float kBigScore = 512.0f;
constexpr float kTinyFactor = 1e-30f;   // score factors are never zero, so that a masked -inf stays one

// B_S_FULL and B_P_FULL + 2 u + buffer.  (P needs one for each buffer: a softmax warp may
// finish step t + 1 before the MMA warp has seen step t.  The last PV has one of its own:
// after P(last) up to two phases of B_O_DONE are open, which a parity cannot tell apart.)
constexpr int B_K_FULL = 0, B_K_EMPTY = 2, B_V_FULL = 4, B_V_EMPTY = 6, B_Q = 8, B_S_FULL = 10, B_P_FULL = 14,
              B_O_DONE = 18, B_O_LAST = 20, B_DONE = 22, N_BARS = 23;
static_assert(N_BARS * 8 + 4 <= 256, "barrier area");

// kind::f16 instruction descriptor with f16 A and B, fp32 D
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24); }
constexpr uint32_t IDESC_S = idesc_f16(BM, HALF);
constexpr uint32_t IDESC_PV = idesc_f16(BM, HD) | tcx::kIdescBMajorMN;

__device__ __forceinline__ uint32_t tile_off(int r, int c) {   // row r, 16-byte chunk c of 16
  return uint32_t(c >> 3) * BOX + uint32_t(r) * 128u + (uint32_t((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// One MMA step, issued by the lane with `lead`.  Descriptors come as their low
// words (the start address moves, the rest is one constant for each layout), and
// the lead is a predicate, not a branch: the issuing warp stays convergent and its
// operands in uniform registers (8 x 2048 tokens: 313 -> 298 us against building each
// 64-bit descriptor inside an `if (lane == 0)`).
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                        uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n setp.ne.b32 q, %0, 0;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 x, {%2, %4};\n mov.b64 y, {%3, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], x, y, %5, p;\n}\n" ::"r"(lead),
      "r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi,
                                        uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n setp.ne.b32 q, %0, 0;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 y, {%3, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], y, %5, p;\n}\n" ::"r"(lead),
      "r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}\n" ::"r"(lead),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// 64 columns of TMEM, arrived (load and wait in one statement: no use can come between)
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {   // arrived
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair64(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpair64(uint64_t p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

struct PrefillArgs {
  const bf16* q;
  Cache c;
  const int32_t* cu_q;
  const int32_t* ctx;
  int64_t total_q;
  int max_q, max_ctx, nh, nkv, G, window, n_sink, splits;
  float scale_log2;     // |scale| log2 e
  float q_sign;         // sign of the scale
  bf16* out;
  int64_t part_rows;    // n_seqs * max_q * nh
  float* ws_o;          // [splits][part_rows][128]
  float* ws_ml;         // [splits][part_rows][2]
};

// Rows of one CTA (or one row of the merge): the sequence's packed rows from R0.
struct Rows {
  int qs, lq, start, n;   // first token, new tokens, key position of token 0, packed rows that exist
  __device__ __forceinline__ int64_t id(const PrefillArgs& a, int R, int g) const {   // row of q and out
    const int tok = R / a.G;
    return (int64_t(qs) + tok) * a.nh + g * a.G + (R - tok * a.G);
  }
  // What takes a row of q and out of sequence s to its row in a part: parts have room for max_q
  // tokens a sequence, so that rows of q that belong to none ask for none.
  __device__ __forceinline__ int64_t to_part(const PrefillArgs& a, int s) const {
    return (int64_t(s) * a.max_q - qs) * a.nh;
  }
};
__device__ __forceinline__ Rows rows_of(const PrefillArgs& a, int s) {
  Rows r;
  r.qs = a.cu_q[s];
  r.lq = a.cu_q[s + 1] - r.qs;
  r.start = a.ctx[s] - r.lq;
  int tok = min(r.lq, a.max_q);
  if (r.qs < 0 || int64_t(r.qs) + tok > a.total_q) tok = 0;
  r.n = max(tok, 0) * a.G;
  return r;
}

template <int KV>
__global__ void __launch_bounds__(THREADS, 1) attn_prefill_kv8_kernel(const PrefillArgs a) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(sm);
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * uint32_t(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_BAR + N_BARS * 8);
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;

  const int s = blockIdx.z, g = blockIdx.y;
  const int n_x = int(gridDim.x) / a.splits;
  const int split = int(blockIdx.x) % a.splits;
  const int R0 = (n_x - 1 - int(blockIdx.x) / a.splits) * ROWS;   // longest (causal) rows first
  const Rows rw = rows_of(a, s);
  if (R0 >= rw.n) return;   // uniform over the CTA, before any barrier or TMEM use
  if (a.ctx[s] > a.max_ctx && threadIdx.x == 0) atomicOr(&g_kv8_prefill_error, kErrContextOverflow);
  // key tiles that any row sees: 0 .. ns - 1 (first tokens), then w0 .. ; unit u needs the first n_u of the list
  const int cap = min(a.ctx[s], a.max_ctx);                       // keys past it are not read
  const int p_lo = rw.start + R0 / a.G;                           // key position of the CTA's first row
  const int lo_cta = a.window > 0 ? max(p_lo + 1 - a.window, 0) : 0;
  const int w0 = lo_cta / BN;
  const int ns = min((min(a.n_sink, lo_cta) + BN - 1) / BN, w0);
  int n_u[2], hi_u[2], hi_cta = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int last = min(R0 + BM * u + BM, rw.n) - 1;             // the unit's last row
    const int hi = last >= R0 + BM * u ? min(rw.start + last / a.G + 1, cap) : 0;   // keys its rows see end here
    hi_cta = max(hi_cta, hi);
    hi_u[u] = hi;
    const int tb = hi > 0 ? (hi + BN - 1) / BN : 0;
    n_u[u] = tb > w0 ? ns + tb - w0 : min(ns, tb);
  }
  const int n_all = max(n_u[0], n_u[1]);
  const int t0 = int(int64_t(n_all) * split / a.splits), t1 = int(int64_t(n_all) * (split + 1) / a.splits);
#pragma unroll
  for (int u = 0; u < 2; ++u) n_u[u] = max(min(n_u[u], t1) - t0, 0);
  const int n_kv = max(n_u[0], n_u[1]);                           // tiles of this CTA
  auto tile_key = [&](int j) { return (t0 + j < ns ? t0 + j : w0 + t0 + j - ns) * BN; };   // first key of tile j
  int s_u[2];   // steps of 64 keys: two a tile, without a last one that the unit does not see
#pragma unroll
  for (int u = 0; u < 2; ++u) s_u[u] = 2 * n_u[u] - (n_u[u] > 0 && tile_key(n_u[u] - 1) + HALF >= hi_u[u] ? 1 : 0);

  // row of this CTA's part for a row of q and out
  auto part_row = [&](int64_t id) { return split * a.part_rows + id + rw.to_part(a, s); };
  // rows without a tile: zero output, or an empty part
  auto no_tiles = [&](int R, int n, int t, int step) {
    for (int i = t; i < n * 16; i += step) {
      const int row = R + i / 16, c = i % 16;
      if (row >= rw.n) break;
      const int64_t id = rw.id(a, row, g);
      if (a.splits == 1) {
        *reinterpret_cast<uint4*>(a.out + id * HD + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
      } else if (c == 0) {
        const int64_t at = part_row(id);
        a.ws_ml[2 * at] = -INFINITY;
        a.ws_ml[2 * at + 1] = 0.0f;
      }
    }
  };
  if (n_kv == 0) {
    no_tiles(R0, ROWS, threadIdx.x, THREADS);
    return;   // uniform over the CTA
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tcx::mbar_init(bar(B_K_FULL + i), 4);
      tcx::mbar_init(bar(B_K_EMPTY + i), 1);
      tcx::mbar_init(bar(B_V_FULL + i), 4);
      tcx::mbar_init(bar(B_V_EMPTY + i), 1);
      tcx::mbar_init(bar(B_Q + i), BM);
      tcx::mbar_init(bar(B_S_FULL + i), 1);
      tcx::mbar_init(bar(B_S_FULL + 2 + i), 1);
      tcx::mbar_init(bar(B_P_FULL + i), 4);
      tcx::mbar_init(bar(B_P_FULL + 2 + i), 4);
      tcx::mbar_init(bar(B_O_DONE + i), 1);
      tcx::mbar_init(bar(B_O_LAST + i), 1);
    }
    tcx::mbar_init(bar(B_DONE), 1);
    tcx::fence_mbar_init();
  }
  if (warp == 0) {
    tcx::tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tcx::tmem_relinquish();
  }
  // ---- every role's first reads, before the barrier that the set-up ends with
  // converters: warp w holds keys 32 w .. + 31 of every tile
  const int w = warp - 4, rsub = lane >> 2, c4 = lane & 3;
  const int64_t row_bytes = int64_t(a.nkv) * HD;
  uint4 kr[8], vr[8];
  float sk = 0.0f, sv = 0.0f;            // lanes 0, 1: scales of the warp's two blocks
  int64_t row0 = -1;                     // cache row of the warp's first key
  bool has[2] = {false, false};          // its two blocks are seen by some row and have a page
  int page = -1;                         // block table entry of the tile after the one in row0
  auto fetch_page = [&](int j) {         // its load is in flight until the next find()
    const int blk = (tile_key(j) + 32 * w) / a.c.block_size;
    page = j < n_kv && blk < a.c.max_blocks ? a.c.table[int64_t(s) * a.c.max_blocks + blk] : -1;
  };
  auto find = [&](int j) {
    const int key0 = tile_key(j) + 32 * w;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int k = key0 + 16 * b;
      has[b] = max(k, lo_cta) < min(k + 16, hi_cta) || k < min(a.n_sink, hi_cta);
    }
    row0 = int64_t(page) * a.c.block_size + key0 % a.c.block_size;
    // (the cache may end inside a page, after a whole block)
    has[0] = has[0] && page >= 0 && row0 < a.c.num_slots;
    has[1] = has[1] && page >= 0 && row0 + 16 < a.c.num_slots;
  };
  auto load = [&](uint4 (&x)[8], const void* cache) {
    const uint8_t* base = static_cast<const uint8_t*>(cache) + (row0 + rsub) * row_bytes + int64_t(g) * HD + 16 * c4;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        x[2 * k + b] = has[k >> 1] ? __ldg(reinterpret_cast<const uint4*>(base + 8 * k * row_bytes + 64 * b))
                                   : make_uint4(0u, 0u, 0u, 0u);
  };
  auto load_scales = [&]() {
    sk = sv = 0.0f;
    if (lane < 2 && (lane ? has[1] : has[0])) {
      const int64_t at = ((row0 + 16 * lane) >> a.c.sb_shift) * a.nkv + g;
      sk = a.c.k_scale[at];
      sv = a.c.v_scale[at];
    }
  };
  // softmax warps: one query row per thread, TMEM lane = row
  const int u = (warp >> 2) & 1, quarter = warp & 3, r = quarter * 32 + lane;
  const int Ru = R0 + BM * u;
  uint8_t* sQ = sm + OFF_Q + u * TILE;
  const bool valid = Ru + r < rw.n;
  const int64_t id = rw.id(a, valid ? Ru + r : Ru, g);
  float rowf = 0.0f;
  if (warp >= 8) {
    uint4 x[16];
#pragma unroll
    for (int c = 0; c < 16; ++c)
      x[c] = valid ? *reinterpret_cast<const uint4*>(a.q + id * HD + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    // largest magnitude, two bf16 at a time (bit patterns without the sign order like the values)
    uint32_t t2[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      t2[0] = __vmaxu2(t2[0], x[c].x & 0x7fff7fffu);
      t2[1] = __vmaxu2(t2[1], x[c].y & 0x7fff7fffu);
      t2[2] = __vmaxu2(t2[2], x[c].z & 0x7fff7fffu);
      t2[3] = __vmaxu2(t2[3], x[c].w & 0x7fff7fffu);
    }
    const uint32_t tm = __vmaxu2(__vmaxu2(t2[0], t2[1]), __vmaxu2(t2[2], t2[3]));
    const float top = __uint_as_float(max(tm << 16, tm & 0xffff0000u));
    float mul, inv;
    row_scale(top, mul, inv);
    mul *= a.q_sign;
    rowf = inv * a.scale_log2;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      auto cv = [&](uint32_t v) { return pack_f16(bf16_lo(v) * mul, bf16_hi(v) * mul); };
      *reinterpret_cast<uint4*>(sQ + tile_off(r, c)) = make_uint4(cv(x[c].x), cv(x[c].y), cv(x[c].z), cv(x[c].w));
    }
    tcx::fence_proxy_async();
  } else if (warp >= 4) {
    fetch_page(0);
    find(0);
    fetch_page(1);
    load_scales();
    load(kr, a.c.k);
    load(vr, a.c.v);
  }
  tcx::tc_fence_before();
  __syncthreads();
  tcx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  auto wait = [&](int b, uint32_t parity, uint32_t code) {
    if (ok && !tcx::mbar_wait(bar(b), parity, &g_kv8_prefill_error, 1u << (code & kWaitCodeMask))) ok = false;
  };

  if (warp < 4) {
    // ---------------- MMA issuer (warp 0, one elected lane) ----------------
    if (warp == 0) {
      const uint32_t lead = elect_one();
      const uint64_t dk = tcx::sw128_desc(sbase), dv = tcx::sw128_desc_mn(sbase, BOX);   // + (offset >> 4)
      const uint32_t k_lo = uint32_t(dk), k_hi = uint32_t(dk >> 32), v_lo = uint32_t(dv), v_hi = uint32_t(dv >> 32);
      auto issue_s = [&](int u, int t) {   // S_u(t) = Q_u K^T: keys 64 (t & 1) .. + 63 of tile t / 2
        const uint32_t qd = k_lo + ((OFF_Q + uint32_t(u) * TILE) >> 4);
        const uint32_t kd = k_lo + ((OFF_K + uint32_t((t >> 1) & 1) * TILE + uint32_t(t & 1) * (BOX / 2)) >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = (uint32_t(kk >> 2) * BOX + uint32_t(kk & 3) * 32u) >> 4;
          umma_ss(lead, tmem + uint32_t(u) * 128u + uint32_t(t & 1) * 64u, qd + off, kd + off, k_hi, IDESC_S,
                  kk > 0 ? 1u : 0u);
        }
        commit(lead, bar(B_S_FULL + 2 * u + (t & 1)));
      };
      auto issue_pv = [&](int u, int t) {   // O_u += P_u(t) V
        const uint32_t vd = v_lo + ((OFF_V + uint32_t((t >> 1) & 1) * TILE + uint32_t(t & 1) * (BOX / 2)) >> 4);
        const uint32_t tP = tmem + uint32_t(u) * 128u + uint32_t(t & 1) * 64u;
#pragma unroll
        for (int kk = 0; kk < HALF / 16; ++kk)
          umma_ts(lead, tmem + 256u + uint32_t(u) * 128u, tP + uint32_t(kk) * 8u, vd + uint32_t(kk) * (2048u >> 4), v_hi,
                  IDESC_PV, (t > 0 || kk > 0) ? 1u : 0u);
        commit(lead, bar(B_O_DONE + u));
        if (t + 1 == s_u[u]) commit(lead, bar(B_O_LAST + u));
      };
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (s_u[u] > 0) wait(B_Q + u, 0u, 5u);
      wait(B_K_FULL, 0u, 6u);
      tcx::tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (t < s_u[u]) issue_s(u, t);
      commit(lead, bar(B_K_EMPTY));   // K_0 is free once these complete
      const int steps = max(s_u[0], s_u[1]);
      for (int t = 0; t < steps; ++t) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (t < s_u[u]) {
            // P_u(t) written; its softmax also saw V of this tile (and, t even, K of the next) land
            wait(B_P_FULL + 2 * u + (t & 1), uint32_t(t >> 1) & 1u, 8u);
            tcx::tc_fence_after();
            issue_pv(u, t);
          }
        if (t & 1) commit(lead, bar(B_V_EMPTY + ((t >> 1) & 1)));
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (t + 2 < s_u[u]) {
            // S_u(t+2) overwrites the P_u(t) that PV_u(t) reads
            wait(B_O_DONE + u, uint32_t(t) & 1u, 10u);
            tcx::tc_fence_after();
            issue_s(u, t + 2);
          }
        if (t & 1) commit(lead, bar(B_K_EMPTY + (((t + 2) >> 1) & 1)));
      }
      // every MMA of this CTA has completed before TMEM and shared memory are released: waited for
      // (as long as any wait) after a wait that gave up, too
      commit(lead, bar(B_DONE));
      ok = true;
      wait(B_DONE, 0u, 11u);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------- converters: warp w holds keys 32 w .. + 31 of every tile ----------------
    auto store = [&](const uint4 (&x)[8], uint32_t off) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint8_t* dst = sm + off + uint32_t(b) * BOX + uint32_t(32 * w + 8 * k + rsub) * 128u;
          const uint4 y = x[2 * k + b];
          uint4 lo, hi;
          word_pairs<KV>(y.x, lo.x, lo.y);
          word_pairs<KV>(y.y, lo.z, lo.w);
          word_pairs<KV>(y.z, hi.x, hi.y);
          word_pairs<KV>(y.w, hi.z, hi.w);
          *reinterpret_cast<uint4*>(dst + (((2 * c4) ^ rsub) << 4)) = lo;
          *reinterpret_cast<uint4*>(dst + (((2 * c4 + 1) ^ rsub) << 4)) = hi;
        }
    };
    auto publish = [&](int b) {
      tcx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tcx::mbar_arrive(bar(b));
    };
    for (int j = 0; j < n_kv; ++j) {
      const int slot = j & 1;
      bool zero_v[2];   // blocks whose v_scale counts as zero
#pragma unroll
      for (int b = 0; b < 2; ++b) zero_v[b] = !(__shfl_sync(0xffffffffu, sv, b) >= kTinyScale);
      const int tail_key = tile_key(j) + 32 * w + rsub;
      const bool past_end = tile_key(j) + 32 * w + 32 > hi_cta;
      const bool seen = lane ? has[1] : has[0];
      const int key0 = tile_key(j) + 32 * w + 16 * (lane & 1);
      // a block without a page counts as zero keys; one that no row sees is left out
      const bool act = max(key0, lo_cta) < min(key0 + 16, hi_cta) || key0 < min(a.n_sink, hi_cta);
      if (j >= 2) wait(B_K_EMPTY + slot, uint32_t((j >> 1) - 1) & 1u, 1u);
      if (lane < 2) {
        const float svc = fmaxf(seen ? sv : 0.0f, kTinyScale);
        *reinterpret_cast<float4*>(sm + OFF_SCL + ((j & 3) * 8 + 2 * w + lane) * 16) =
            act ? make_float4(seen ? sk : 0.0f, lg2(svc), __fdividef(kUnshift, svc), 0.0f)
                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      store(kr, OFF_K + uint32_t(slot) * TILE);
      publish(B_K_FULL + slot);
      if (j + 1 < n_kv) {
        find(j + 1);
        fetch_page(j + 2);
        load_scales();
        load(kr, a.c.k);
      }
      if (j >= 2) wait(B_V_EMPTY + slot, uint32_t((j >> 1) - 1) & 1u, 2u);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (zero_v[i >> 2]) vr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (past_end) {   // rows that no query sees may hold any code, NaN too: 0 * V has to stay 0
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (tail_key + 8 * (i >> 1) >= hi_cta) vr[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      store(vr, OFF_V + uint32_t(slot) * TILE);
      publish(B_V_FULL + slot);
      if (j + 1 < n_kv) load(vr, a.c.v);
    }
  } else {
    // ---------------- softmax (one query row per thread) ----------------
    const int steps = u ? s_u[1] : s_u[0];
    if (steps == 0) {
      no_tiles(Ru, BM, r, BM);
    } else {
      // The first tile's scales.  Waited for before this thread lets S(0) start: the slot is
      // filled again only after S(0), so this phase cannot be missed.
      wait(B_K_FULL, 0u, 14u);
      tcx::mbar_arrive(bar(B_Q + u));

      const int p = rw.start + (Ru + r) / a.G;              // key position of this row
      const int hi = valid ? min(p + 1, cap) : 0;           // it sees keys lo_row .. hi - 1 and 0 .. n_sink - 1 below hi
      const int lo_row = a.window > 0 ? max(p + 1 - a.window, 0) : 0;
      const uint32_t tS = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(u) * 128u;
      const uint32_t tO = tS + 256u;
      float m = -INFINITY, l = 0.0f;
      for (int t = 0; t < steps; ++t) {
        const int j = t >> 1;
        const uint32_t tX = tS + uint32_t(t & 1) * 64u;   // S_u(t), then P_u(t) over its first 32 columns
        wait(B_S_FULL + 2 * u + (t & 1), uint32_t(t >> 1) & 1u, 12u);
        tcx::tc_fence_after();
        const int k0 = tile_key(j) + HALF * (t & 1);
        const int end = hi - k0, beg = lo_row - k0, snk = a.n_sink - k0;   // columns [beg, end) and [0, min(snk, end))
        // A masked step writes -inf into S first.  Rare paths are short loops over TMEM, not
        // unrolled over the registers of S: they would sit in the middle of the loop's code
        // (222 -> 215 us for 8 x 2048 tokens).
        if (__any_sync(0xffffffffu, !(HALF <= end && (0 >= beg || HALF <= snk)))) {
#pragma unroll 1
          for (int c = 0; c < HALF; c += 16) {
            uint32_t y[16];
            tmem_ld16(tX + c, y);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!(c + e < end && (c + e >= beg || c + e < snk))) y[e] = __float_as_uint(-INFINITY);
            tmem_st16(tX + c, y);
          }
          tcx::tmem_st_wait();
        }
        uint32_t x[64];
        tmem_ld64(tX, x);
        const float4* scl = reinterpret_cast<const float4*>(sm + OFF_SCL) + (j & 3) * 8 + 4 * (t & 1);
        float fb[4], m_step = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t* y = x + 16 * b;
          auto f = [&](int e) { return __uint_as_float(y[e]); };
          const float mx = max3(max3(max3(f(0), f(1), f(2)), max3(f(3), f(4), f(5)), max3(f(6), f(7), f(8))),
                                max3(max3(f(9), f(10), f(11)), max3(f(12), f(13), f(14)), f(15)), -INFINITY);
          const float4 sc = scl[b];
          fb[b] = fmaxf(rowf * sc.x, kTinyFactor);
          m_step = fmaxf(m_step, fmaf(mx, fb[b], sc.y));
        }
        float alpha = 1.0f;
        bool rescale = false;
        if (m_step > m + kRescaleLog2) {
          alpha = ex2(m - m_step);
          m = m_step;
          rescale = true;
        }
        const float m_use = m == -INFINITY ? 0.0f : m;
        l *= alpha;
        const bool big = __any_sync(0xffffffffu, fabsf(m_use) > kBigScore);
        float unit = 1.0f;   // 0: x holds the exponents already
        if (big) {
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t y[16];
            tmem_ld16(tX + 16u * b, y);
            const float4 sc = scl[b];
            const float f = fmaxf(rowf * sc.x, kTinyFactor);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              y[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), f, sc.y) - m_use + kShift);
            tmem_st16(tX + 16u * b, y);
          }
          tcx::tmem_st_wait();
          tmem_ld64(tX, x);
          unit = 0.0f;
        }
        uint32_t pk[32];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float4 sc = scl[b];
          const float f = big ? 1.0f : fb[b], cb = unit * (sc.y - m_use + kShift);
          const uint64_t f2 = pair64(f, f), c2 = pair64(cb, cb);
          uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float y0, y1;
            unpair64(fma2(pair64(__uint_as_float(x[16 * b + e]), __uint_as_float(x[16 * b + e + 1])), f2, c2), y0, y1);
            const float p0 = ex2(y0), p1 = ex2(y1);
            uint64_t& sum = e & 2 ? sum1 : sum0;
            sum = add2(sum, pair64(p0, p1));
            pk[8 * b + e / 2] = pack_f16(p0, p1);
          }
          float s0, s1;
          unpair64(add2(sum0, sum1), s0, s1);
          l = fmaf(s0 + s1, sc.z, l);
        }
        tcx::tmem_st32(tX, pk);
        if (t >= 1 && __any_sync(0xffffffffu, rescale)) {
          // PV_u(t-1) is the last MMA on O_u before this thread's P_u(t) lets the next one start
          wait(B_O_DONE + u, uint32_t(t - 1) & 1u, 15u);
          tcx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tcx::tmem_ld32(tO + 32u * c, o);
            tcx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tcx::tmem_st32(tO + 32u * c, o);
          }
        }
        tcx::tmem_st_wait();
        // the MMA warp issues PV_u(t), and after it S_u(t+2), on this signal alone
        if (!(t & 1)) {
          wait(B_V_FULL + (j & 1), uint32_t(j >> 1) & 1u, 14u);
          if (t + 2 < steps) wait(B_K_FULL + ((j + 1) & 1), uint32_t((j + 1) >> 1) & 1u, 14u);
        }
        tcx::tc_fence_before();
        __syncwarp();
        if (lane == 0) tcx::mbar_arrive(bar(B_P_FULL + 2 * u + (t & 1)));
      }
      wait(B_O_LAST + u, 0u, 13u);
      tcx::tc_fence_after();
      if (a.splits == 1) {
        // O / l -> bf16, staged in Q_u (every S_u MMA completed before the last PV_u), stored coalesced
        const float inv = l == 0.0f ? 0.0f : kUnshift / l;   // no visible key: a zero row; l NaN stays
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tcx::tmem_ld32(tO + 32u * c, o);
          tcx::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(sQ + tile_off(r, 4 * c + k)) =
                make_uint4(pack_bf16(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                           pack_bf16(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                           pack_bf16(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                           pack_bf16(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
        }
        tcx::tc_fence_before();
        named_sync(1 + u, BM);
        const int cc = r & 15, tok0 = Ru / a.G, rem = Ru - tok0 * a.G;
        const uint32_t rcp = 65536u / uint32_t(a.G) + 1u;   // x / G = x * rcp >> 16 for x < 144, G <= 16
        bf16* base = a.out + ((int64_t(rw.qs) + tok0) * a.nh + g * a.G) * HD + 8 * cc;
#pragma unroll 4
        for (int it = 0; it < BM / 8; ++it) {
          const int rr = it * 8 + (r >> 4);
          const int dt = int((uint32_t(rem + rr) * rcp) >> 16);
          if (Ru + rr < rw.n)
            *reinterpret_cast<uint4*>(base + (int64_t(dt) * a.nh + (rem + rr - dt * a.G)) * HD) =
                *reinterpret_cast<const uint4*>(sQ + tile_off(rr, cc));
        }
      } else {
        const int64_t at = part_row(id);
        const float fac = kUnshift;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tcx::tmem_ld32(tO + 32u * c, o);
          tcx::tmem_ld_wait();
          if (valid)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(a.ws_o + at * HD + 32 * c + 4 * k) =
                  make_float4(__uint_as_float(o[4 * k]) * fac, __uint_as_float(o[4 * k + 1]) * fac,
                              __uint_as_float(o[4 * k + 2]) * fac, __uint_as_float(o[4 * k + 3]) * fac);
        }
        if (valid) {
          a.ws_ml[2 * at] = m;
          a.ws_ml[2 * at + 1] = l;
        }
        tcx::tc_fence_before();
      }
    }
  }
  tcx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tcx::tc_fence_after();
    tcx::tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Adds the splits' parts in order: one warp per packed row, lane owns dims 4 lane .. + 3.
// At most 152 x 256 rows of parts, 20 MB, which L2 still holds: bound by latency.
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillArgs a) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  const int lane = threadIdx.x & 31, R = int(blockIdx.x) * 8 + int(threadIdx.x >> 5), g = blockIdx.y;
  const Rows rw = rows_of(a, blockIdx.z);
  if (R >= rw.n) return;
  const int64_t id = rw.id(a, R, g), part = id + rw.to_part(a, blockIdx.z), n = a.part_rows;
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml);
  float2 mine = make_float2(-INFINITY, 0.0f);   // part `lane` (at most 32)
  if (lane < a.splits) mine = ml[lane * n + part];
  const float M = warp_max(mine.x);
  // A part without a visible key has (-inf, 0).  One of a query with NaN may have (-inf, NaN): its
  // weight is 0 too, but the NaN reaches l, and through l the row.
  const float w = mine.x == -INFINITY ? 0.0f : ex2(mine.x - M);
  const float l = warp_sum(mine.y * w);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = 0; i < a.splits; ++i) {
    const float wi = __shfl_sync(0xffffffffu, w, i);
    if (wi == 0.0f) continue;   // (an empty part has no O)
    const float4 x = *(reinterpret_cast<const float4*>(a.ws_o + (i * n + part) * HD) + lane);
    acc.x = fmaf(x.x, wi, acc.x);
    acc.y = fmaf(x.y, wi, acc.y);
    acc.z = fmaf(x.z, wi, acc.z);
    acc.w = fmaf(x.w, wi, acc.w);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + id * HD + 4 * lane) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// Shares that the key tiles are cut into: as many as still fit the GPU's SMs at
// once, with four tiles of max_context each at least.  The host knows neither the
// lengths nor, here, the window: shares of a shorter or windowed sequence have fewer
// tiles, down to none.  More CTAs than half the SMs are not split, and nor are rows that
// fill the SMs by themselves.
int prefill_splits(int n_seqs, int max_q, int max_ctx, int nh, int nkv) {
  constexpr int kSms = 152;
  const int64_t ctas = (int64_t(max_q) * (nh / nkv) + ROWS - 1) / ROWS * nkv * n_seqs;
  const int64_t tiles = (int64_t(max_ctx) + BN - 1) / BN;
  return int(std::max<int64_t>(1, std::min({kSms / std::max<int64_t>(ctas, 1), tiles / 4, int64_t(32)})));
}

template <int KV>
int launch(const PrefillArgs& a, int n_seqs, cudaStream_t st) {
  static bool configured = false;
  if (!configured) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_prefill_kv8_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
    if (e != cudaSuccess) return set_error(QW_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    configured = true;
  }
  const int64_t rows = int64_t(a.max_q) * a.G;
  const dim3 grid(unsigned((rows + ROWS - 1) / ROWS * a.splits), unsigned(a.nkv), unsigned(n_seqs));
  launch_pdl(attn_prefill_kv8_kernel<KV>, grid, THREADS, SMEM, st, a);
  int rc = check_launch("attn_prefill_kv8_kernel");
  if (rc || a.splits == 1) return rc;
  launch_pdl(prefill_merge_kernel, dim3(unsigned((rows + 7) / 8), unsigned(a.nkv), unsigned(n_seqs)), 256, 0, st, a);
  return check_launch("prefill_merge_kernel");
}

}  // namespace kv8p

namespace kv8 {
int check_attention(const char* who, const void* k, const void* v, const float* ks, const float* vs, int64_t num_slots,
                    int scale_block, const int32_t* table, int max_blocks, int block_size, int n_seqs, int max_context,
                    int nh, int nkv, int head_dim, int window, int n_sink, int dtype, int kv_dtype);
}

unsigned int take_kv8_prefill_errors() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, kv8p::g_kv8_prefill_error, sizeof(v));
  if (v) cudaMemcpyToSymbol(kv8p::g_kv8_prefill_error, &z, sizeof(z));
  return v;
}
}  // namespace qw

using namespace qw;

extern "C" size_t qw_attention_prefill_kv8_workspace_size(int n_seqs, int64_t total_q, int max_seqlen_q,
                                                          int max_context, int n_heads, int n_kv_heads) {
  if (n_seqs <= 0 || total_q <= 0 || max_seqlen_q <= 0 || max_context < 0 || n_heads <= 0 || n_kv_heads <= 0) return 0;
  const int s = kv8p::prefill_splits(n_seqs, max_seqlen_q, max_context, n_heads, n_kv_heads);
  return s == 1 ? 0 : kCounterBytes + size_t(s) * n_seqs * max_seqlen_q * n_heads * (kv8::HD + 2) * sizeof(float);
}

extern "C" int qw_attention_prefill_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                        const float* v_scale, int64_t num_slots, int scale_block,
                                        const int32_t* cu_seqlens_q, const int32_t* context_lens,
                                        const int32_t* block_table, int max_blocks, int block_size, int n_seqs,
                                        int64_t total_q, int max_seqlen_q, int max_context, int n_heads,
                                        int n_kv_heads, int head_dim, float scale, int window, int n_sink, void* out,
                                        void* workspace, size_t workspace_bytes, int dtype, int kv_dtype,
                                        void* stream) {
  const char* who = "qw_attention_prefill_kv8";
  if (total_q < 0 || max_seqlen_q < 0) return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  const int rc = kv8::check_attention(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, block_table,
                                      max_blocks, block_size, n_seqs, max_context, n_heads, n_kv_heads, head_dim,
                                      window, n_sink, dtype, kv_dtype);
  if (rc) return rc;
  if (n_seqs > 65535 || n_kv_heads > 65535 || int64_t(max_seqlen_q) * (n_heads / n_kv_heads) > INT32_MAX)
    return set_error(QW_ERR_SHAPE, "%s: more than 65535 sequences or kv heads, or 2^31 rows of a sequence", who);
  if (n_seqs == 0 || max_seqlen_q == 0 || total_q == 0) return QW_OK;
  if (!q || !cu_seqlens_q || !context_lens || !out) return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!kv8::aligned16(q) || !kv8::aligned16(out))
    return set_error(QW_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  const size_t need =
      qw_attention_prefill_kv8_workspace_size(n_seqs, total_q, max_seqlen_q, max_context, n_heads, n_kv_heads);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return set_error(QW_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  if (need > 0 && !kv8::aligned16(workspace))
    return set_error(QW_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
  kv8p::PrefillArgs a;
  a.q = static_cast<const bf16*>(q);
  a.c = kv8::Cache{k_cache, v_cache, k_scale, v_scale, num_slots, kv8::scale_shift(scale_block), block_table, max_blocks,
                   block_size};
  a.cu_q = cu_seqlens_q;
  a.ctx = context_lens;
  a.total_q = total_q;
  a.max_q = max_seqlen_q;
  a.max_ctx = max_context;
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.G = n_heads / n_kv_heads;
  a.window = std::min(window, kv8::kMaxPositions);
  a.n_sink = std::min(n_sink, max_context);
  a.part_rows = int64_t(n_seqs) * max_seqlen_q * n_heads;
  a.splits = kv8p::prefill_splits(n_seqs, max_seqlen_q, max_context, n_heads, n_kv_heads);
  a.scale_log2 = fabsf(scale) * kv8p::kLog2e;
  a.q_sign = scale < 0.0f ? -1.0f : 1.0f;
  a.out = static_cast<bf16*>(out);
  a.ws_o = need > 0 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes) : nullptr;   // (no counters here)
  a.ws_ml = need > 0 ? a.ws_o + a.splits * a.part_rows * kv8::HD : nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_dtype == QW_I8 ? kv8p::launch<QW_I8>(a, n_seqs, st) : kv8p::launch<QW_E4M3>(a, n_seqs, st);
}
