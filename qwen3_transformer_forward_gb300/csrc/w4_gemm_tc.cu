// Linear layers with 4-bit weights for many tokens, on tcgen05 tensor cores (sm_103a).
//
// D[weight row, token] = W X^T: the weights are the MMA's A operand and lie in TMEM,
// where the threads that decode them put them straight from registers; the tokens are B,
// copied by TMA.  Two CTAs (cta_group::2) share a tile of 256 weight rows: each decodes
// 128 of them and holds half of the tokens, so that the tokens cross L2 and each shared
// memory once for 256 rows.
//
// Warps of a CTA: 0 copies tokens, 2 codes, 1 (of the pair's rank 0) issues the MMAs, from 4 on sets of four decode (a
// thread a weight row), the last four store.  TMEM: two accumulators of up to 192 tokens (128 in the narrow form) and a
// ring of decoded weights, two steps of 128 columns (four).  What a step of 192 tokens costs, in cycles: its MMAs 770,
// decoding about 400 of the sub-partition's pipes, the MMA warp's waits and issue about 450; so the tensor pipe leads
// (N of 192 rather than 256 leaves TMEM for the second accumulator: stores overlap the next tile's MMAs).
// 16384 x 12288 x 2048 with SiluAndMul: 480-496 us, 1.66-1.72 PFLOP/s, the rate that a large library product sustains
// under the power limit; 4096 x 12288 x 2048: 112-121 us, 1.70-1.85 PFLOP/s; 16384 x 2048 x 6144 in two row shards 225 us,
// 1.83.  With few tokens the decoding sets' latency leads: about 365 cycles for 128 rows x 64 columns, of which the decoding's
// instructions need 184, against 190 of memory (128 x 28672 x 8192 58 us; 65 x 151936 x 1024 34 us).
// One CTA for itself with 192 tokens ran at 793 us (tokens' traffic twice), the MMAs issued by one lane in a branch at
// 1162, arrivals at the other CTA's barriers that release all memory at 887 against 637.
#include <algorithm>
#include <type_traits>

#include "tc_common.cuh"
#include "w4.cuh"

namespace qw {
namespace w4 {

__device__ unsigned int g_w4_error = 0;

constexpr int kRows = 128;          // weight rows of a CTA (SiluAndMul: 64 gate rows and their up rows), two CTAs a tile
// K advances in steps of 128 columns.  Stages: tokens (a step), codes (two), decoded weights (a step).  TMEM holds two
// accumulators and the decoded weights.
template <bool NARROW> struct Tile {
  static constexpr int TOKENS = NARROW ? 128 : 192, XS = NARROW ? 5 : 4, CS = NARROW ? 8 : 4, AS = NARROW ? 4 : 2;
  static constexpr int SETS = NARROW ? 3 : 2;   // sets of four decoding warps, which take the steps in turn
  // A set's next step lies SETS on and waits for the MMAs of the step AS before that one.  With SETS <= AS it is among
  // those that the set's last step waited for, or that step itself, so a parity is never two phases old.
  static_assert(SETS <= AS, "");
  // The same for codes: that wait showed that all steps up to SETS + AS before the set's next one had their codes, and
  // the stage CS before the next one's ends at least CS steps before it (a shard of one step is a stage of its own).
  static_assert(CS >= SETS + AS, "");
  static constexpr int EPILOGUE0 = 4 + 4 * SETS, THREADS = 32 * (EPILOGUE0 + 4);
  static constexpr uint32_t X_HALF = TOKENS / 2 * 128, X_BYTES = 2 * X_HALF, C_BYTES = kRows * 128;
  static constexpr uint32_t OFF_X = 0, OFF_C = XS * X_BYTES, OFF_BAR = OFF_C + CS * C_BYTES;
  // More than the stages need: an SM then has no room for a CTA of another kernel that takes TMEM, so that the pairs of
  // two kernels on two streams cannot each hold the columns that the other's second CTA waits for.
  static constexpr size_t SMEM = (NARROW ? 212 : 200) * 1024;
  static_assert(SMEM >= 1024 + OFF_BAR + 512, "");
  static constexpr uint32_t A = 2 * TOKENS;   // TMEM column of the decoded weights
  static_assert(A + 64 * AS <= 512, "");
  static constexpr int B_X_FULL = 0, B_X_EMPTY = B_X_FULL + XS, B_C_FULL = B_X_EMPTY + XS, B_C_EMPTY = B_C_FULL + CS,
                       B_A_FULL = B_C_EMPTY + CS, B_A_EMPTY = B_A_FULL + AS, B_ACC_FULL = B_A_EMPTY + AS,
                       B_ACC_EMPTY = B_ACC_FULL + 2, B_DRAIN = B_ACC_EMPTY + 2, N_BARS = B_DRAIN + 1;
  static_assert(N_BARS * 8 + 8 <= 512, "barrier area");
};
constexpr uint32_t kTmemCols = 512;
constexpr int kPairs = 76;          // of 152 SMs

struct TcArgs {
  bf16* out;
  Weights w;
  int64_t rows, ldc, i_l;
  int M, bn;              // tokens, tokens of a tile
  int p_tiles, q_tiles;   // weight row tiles, token tiles
  int shard_tiles;        // SiluAndMul: row tiles of a shard
  int shards, steps_l;    // shards of K, steps of 128 columns of a shard (the last may end in zeros)
  int early;              // the weights may be read ahead of the programmatic wait
  int splits;             // pairs that share a tile's K (a cluster, one tile each); 1: every pair walks over tiles
};

// The two CTAs of a pair: rank 0 issues the MMAs and holds the barriers that both feed.
// Issued by the lane with `lead`, as a predicate: the warp stays converged and its operands in uniform registers (61 ->
// 20 cycles an MMA, 110 -> 22 a commit, against one lane in a branch).
__device__ __forceinline__ void umma_commit_pair(uint32_t lead, uint32_t bar, uint32_t mask) {   // at this offset in the CTAs of mask
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%1], %2;\n}\n" ::"r"(lead),
      "r"(bar), "h"(uint16_t(mask))
      : "memory");
}
// B descriptors come as their low word and a constant high word
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n setp.ne.b32 q, %0, 0;\n setp.ne.b32 p, %6, 0;\n mov.b64 y, {%3, %4};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%1], [%2], y, %5, p;\n}\n" ::"r"(lead),
      "r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// A barrier of either CTA, by its cluster address.  What these arrivals hand over is TMEM, which the tcgen05 waits and
// fences order: a release of all other memory to the cluster would cost about 800 cycles.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// copies into this CTA's shared memory: completing on its own barrier, and on rank 0's
__device__ __forceinline__ void tma_load(uint32_t lead, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
      " @q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2, {%4, %5, %6}], [%3];\n}\n" ::"r"(lead),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair(uint32_t lead, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                              int z) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
      " @q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2, {%4, %5, %6}], "
      "[%3];\n}\n" ::"r"(lead),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t lead, uint32_t bar, uint32_t bytes) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], %2;\n}\n" ::"r"(lead),
               "r"(bar), "r"(bytes)
               : "memory");
}

// 32 columns of TMEM, arrived (load and wait in one statement: no use can come between)
__device__ __forceinline__ void tmem_ld32_arrived(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

template <bool SILU, int GS, bool NARROW>   // GS: log2 of a group's pieces of 32 columns
__global__ void __launch_bounds__(Tile<NARROW>::THREADS, 1)
    gemm_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_c, TcArgs a) {
  using T = Tile<NARROW>;
  constexpr int XS = T::XS, CS = T::CS, AS = T::AS;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sx = smem_u32(sm + T::OFF_X), sc = smem_u32(sm + T::OFF_C), bars = smem_u32(sm + T::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + T::OFF_BAR + T::N_BARS * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  auto bar = [&](int b) { return bars + uint32_t(b) * 8u; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // rank 0 of the pair leads it; the pairs of a cluster share one tile's K
  const uint32_t crank = cluster_rank(), lead_rank = crank & ~1u, both = 3u << lead_rank;
  const int rank = int(crank & 1), split = int(crank >> 1);
  const int pair = blockIdx.x / (2 * a.splits), pairs = gridDim.x / (2 * a.splits);
  auto lead_bar = [&](int b) { return map_to_rank(bar(b), lead_rank); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < XS; ++i) tcx::mbar_init(bar(T::B_X_FULL + i), 1), tcx::mbar_init(bar(T::B_X_EMPTY + i), 1);
    for (int i = 0; i < CS; ++i) tcx::mbar_init(bar(T::B_C_FULL + i), 1), tcx::mbar_init(bar(T::B_C_EMPTY + i), 8);
    for (int i = 0; i < AS; ++i) tcx::mbar_init(bar(T::B_A_FULL + i), 8), tcx::mbar_init(bar(T::B_A_EMPTY + i), 1);
    for (int i = 0; i < 2; ++i) tcx::mbar_init(bar(T::B_ACC_FULL + i), 1), tcx::mbar_init(bar(T::B_ACC_EMPTY + i), 8);
    tcx::mbar_init(bar(T::B_DRAIN), 1);
    *abort_flag = 0;
    tcx::fence_mbar_init();
    tcx::prefetch_map(&tm_x);
    tcx::prefetch_map(&tm_c);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tcx::tc_fence_before();
  __syncwarp();
  cluster_sync_all();   // both CTAs' barriers and TMEM are there
  tcx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // every wait is bounded; the first that gives up, or another role's, ends the loops
  auto wait = [&](int b, uint32_t parity, uint32_t code) -> bool {
    if (tcx::mbar_try_wait(bar(b), parity)) return true;
    const uint64_t t0 = tcx::globaltimer();
    while (!tcx::mbar_try_wait(bar(b), parity)) {
      if (*abort_flag) return false;
      if (tcx::globaltimer() - t0 > tcx::kTimeoutNs) {
        atomicOr(&g_w4_error, code);
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  };
  const int tiles = a.p_tiles * a.q_tiles, ncs_l = (a.steps_l + 1) / 2;
  // this pair's part of K: the code stages c0 .. c1 - 1 of shards * ncs_l, at two steps each (a shard's last may have one)
  const int c0 = int(int64_t(a.shards) * ncs_l * split / a.splits), c1 = int(int64_t(a.shards) * ncs_l * (split + 1) / a.splits);
  const int r0 = c0 / ncs_l, r1 = (c1 - 1) / ncs_l;
  const int first0 = 2 * (c0 % ncs_l), end1 = min(2 * ((c1 - 1) % ncs_l) + 2, a.steps_l);
  auto first_step = [&](int r) { return r == r0 ? first0 : 0; };      // steps of shard r: from first_step to end_step - 1
  auto end_step = [&](int r) { return r == r1 ? end1 : a.steps_l; };
  // first weight row (gate row) of a row tile; the stored rows of shard r of K begin at r * rows
  auto tile_row = [&](int p) -> int64_t {
    if (!SILU) return (int64_t(p) * 2 + rank) * kRows;
    const int r = p / a.shard_tiles;
    return int64_t(r) * 2 * a.i_l + (int64_t(p % a.shard_tiles) * 2 + rank) * (kRows / 2);
  };

  if (!a.early) pdl_wait();   // weights that the kernel before may have written
  if (warp == 0) {
    // ---- tokens: this CTA's half of each block ----
    const uint32_t lead = elect_one();
    uint32_t n = 0;
    bool ok = true;
    pdl_wait();   // the tokens may come from the kernel before
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      const int m0 = tile / a.p_tiles * a.bn + rank * (a.bn / 2);
      for (int r = r0; r <= r1 && ok; ++r)
        for (int k = first_step(r); k < end_step(r); ++k, ++n) {
          const uint32_t s = n % XS, dst = sx + s * T::X_BYTES;
          ok = wait(T::B_X_EMPTY + s, ((n / XS) & 1) ^ 1, 2u);
          if (!ok) break;
          if (rank == 0) expect_tx(lead, bar(T::B_X_FULL + s), uint32_t(a.bn) * 256u);   // both CTAs' halves
          tma_load_pair(lead, dst, &tm_x, lead_bar(T::B_X_FULL + s), k * 128, r, m0);
          tma_load_pair(lead, dst + T::X_HALF, &tm_x, lead_bar(T::B_X_FULL + s), k * 128 + 64, r, m0);
        }
    }
    if (!ok && rank == 0)   // the copies in flight land before the block ends
      for (uint32_t i = n > XS ? n - XS : 0; i < n; ++i) tcx::mbar_wait(bar(T::B_X_FULL + i % XS), (i / XS) & 1, &g_w4_error, 2u);
  } else if (warp == 2) {
    // ---- codes: 256 columns of this CTA's rows at a time ----
    const uint32_t lead = elect_one();
    uint32_t n = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      const int row = int(tile_row(tile % a.p_tiles));
      for (int r = r0; r <= r1 && ok; ++r)
        for (int c = first_step(r) / 2; 2 * c < end_step(r); ++c, ++n) {
          const uint32_t s = n % CS, dst = sc + s * T::C_BYTES;
          ok = wait(T::B_C_EMPTY + s, ((n / CS) & 1) ^ 1, 1u);
          if (!ok) break;
          expect_tx(lead, bar(T::B_C_FULL + s), T::C_BYTES);
          tma_load(lead, dst, &tm_c, bar(T::B_C_FULL + s), c * 64, row, r);
          if (SILU) tma_load(lead, dst + T::C_BYTES / 2, &tm_c, bar(T::B_C_FULL + s), c * 64, row + int(a.i_l), r);
        }
    }
    if (!ok)
      for (uint32_t i = n > CS ? n - CS : 0; i < n; ++i) tcx::mbar_wait(bar(T::B_C_FULL + i % CS), (i / CS) & 1, &g_w4_error, 1u);
  } else if (warp == 1) {
    if (rank == 0) {
      // ---- MMA, for both CTAs ----
      const uint32_t lead = elect_one();
      const uint32_t idesc = tcx::idesc_bf16(2 * kRows, a.bn);
      const uint64_t desc = tcx::sw128_desc(sx);
      const uint32_t b_lo = uint32_t(desc), b_hi = uint32_t(desc >> 32);
      uint32_t n = 0, u = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs, ++u) {
        const uint32_t d = tmem + (u & 1) * T::TOKENS;
        uint32_t add = 0;
        ok = wait(T::B_ACC_EMPTY + (u & 1), ((u >> 1) & 1) ^ 1, 4u);
        for (int r = r0; r <= r1 && ok; ++r)
          for (int i = first_step(r); i < end_step(r); ++i, ++n) {
            const uint32_t s = n % XS, h = n % AS;
            ok = wait(T::B_X_FULL + s, (n / XS) & 1, 8u) && wait(T::B_A_FULL + h, (n / AS) & 1, 16u);
            if (!ok) break;
            tcx::tc_fence_after();
            const uint32_t b = b_lo + s * (T::X_BYTES >> 4), at = tmem + T::A + h * 64;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              umma_ts(lead, d, at + k * 8, b + (k >> 2) * (T::X_HALF >> 4) + 2 * (k & 3), b_hi, idesc, add);
              add = 1;
            }
            umma_commit_pair(lead, bar(T::B_A_EMPTY + h), both);
            umma_commit_pair(lead, bar(T::B_X_EMPTY + s), both);
          }
        if (ok) umma_commit_pair(lead, bar(T::B_ACC_FULL + (u & 1)), both);
      }
      umma_commit_pair(lead, bar(T::B_DRAIN), both);
      tcx::mbar_wait(bar(T::B_DRAIN), 0, &g_w4_error, 32u);
    }
  } else if (warp >= 4 && warp < T::EPILOGUE0) {
    // ---- decode: one weight row a thread, four warps the rows of a step ----
    const int q = warp & 3, set = (warp - 4) >> 2;
    const uint32_t magic = code_magic();
    const int srow = SILU ? (lane >> 4) * 64 + 16 * q + (lane & 15) : 32 * q + lane;   // row in the code stage
    const int64_t row_off = SILU ? (lane >> 4) * a.i_l + 16 * q + (lane & 15) : srow;
    const uint32_t code_row = sc + uint32_t(srow) * 128u, tmem_row = tmem + (uint32_t(32 * q) << 16) + T::A;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(a.w.scales);
    // the step: number n, its tile, shard r of K, place k in the shard, which ends at k_end; cs0: code stages before the
    // shard's first (less those of the shard that are not this pair's)
    int tile = pair, r = r0, k = first0 + set, k_end = end_step(r0);
    uint32_t n = set, cs0 = uint32_t(-(first0 / 2));
    const uint16_t* sp = nullptr;   // scales and zeros of this thread's row in the step's shard
    const uint8_t* zp = nullptr;
    bool have = false;
    auto settle = [&]() {   // k may lie past its shard
      while (k >= k_end) {
        cs0 += (k_end + 1) / 2;
        k -= k_end;
        if (++r > r1) {
          r = r0;
          tile += pairs;
          k += first0;
          cs0 -= first0 / 2;
        }
        k_end = end_step(r);
      }
      if (tile >= tiles) return;
      const int64_t row = tile_row(tile % a.p_tiles) + row_off, at = (int64_t(r) * a.rows + row) * a.w.groups;
      have = row < a.rows;
      sp = scales + at;
      zp = a.w.zeros != nullptr ? a.w.zeros + at : nullptr;
    };
    // scales and zero points of the step's groups, the scale 0 where there is none
    constexpr int NG = 4 >> GS;
    uint32_t s[NG], z[NG];
    auto load_scales = [&]() {
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        const int g = k * NG + e;
        const bool in = have && g < a.w.groups;
        s[e] = in ? __ldg(sp + g) : 0u;
        z[e] = in && zp != nullptr ? __ldg(zp + g) : 8u;
      }
    };
    settle();
    if (tile < tiles) load_scales();
    while (tile < tiles) {
      const uint32_t cs = cs0 + uint32_t(k >> 1), st = cs % CS, in_stage = uint32_t(k & 1);
      const uint32_t h = n % AS, a_parity = ((n / AS) & 1) ^ 1;
      const uint32_t arrivals = k == k_end - 1 && !in_stage ? 2u : 1u;   // for the step that its code stage lacks, too
      uint32_t s2[NG], z2[NG];
#pragma unroll
      for (int e = 0; e < NG; ++e) s2[e] = scale_pair(s[e]), z2[e] = offset_pair(z[e]);
      n += T::SETS;
      k += T::SETS;
      if (k >= k_end) settle();
      if (tile < tiles) load_scales();   // of this warp's next step, in flight meanwhile
      if (!__all_sync(0xffffffffu, wait(T::B_C_FULL + st, (cs / CS) & 1, 64u))) break;   // the warp goes on as one
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[e].x), "=r"(v[e].y), "=r"(v[e].z), "=r"(v[e].w)
                     : "r"(code_row + st * T::C_BYTES + (((4 * in_stage + e) ^ uint32_t(srow & 7)) << 4)));
      uint32_t w[2][32];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t word[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
          decode(word[i], magic, z2[e >> GS], s2[e >> GS], o);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[e >> 1][16 * (e & 1) + 4 * i + j] = o[j];
        }
      }
      __syncwarp();
      if (lane == 0)   // a stage is free after 8 arrivals: of the four warps of each of its two steps
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar(T::B_C_EMPTY + st)), "r"(arrivals) : "memory");
      if (!__all_sync(0xffffffffu, wait(T::B_A_EMPTY + h, a_parity, 128u))) break;
      tcx::tc_fence_after();
      tcx::tmem_st32(tmem_row + h * 64, w[0]);
      tcx::tmem_st32(tmem_row + h * 64 + 32, w[1]);
      tcx::tmem_st_wait();
      tcx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(lead_bar(T::B_A_FULL + h));
    }
  } else if (warp >= T::EPILOGUE0) {
    // ---- epilogue ----
    const int q = warp & 3;
    const bool even = (a.ldc & 1) == 0;   // two outputs of a token make an aligned word
    uint32_t u = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++u) {
      if (!__all_sync(0xffffffffu, wait(T::B_ACC_FULL + (u & 1), (u >> 1) & 1, 256u))) break;
      tcx::tc_fence_after();
      const int p = tile % a.p_tiles, m0 = tile / a.p_tiles * a.bn, m1 = min(m0 + a.bn, a.M);
      const uint32_t d = tmem + (uint32_t(32 * q) << 16) + (u & 1) * T::TOKENS;
      int64_t o;       // output column of this thread
      bool have;
      if (SILU) {
        const int64_t j = (int64_t(p % a.shard_tiles) * 2 + rank) * (kRows / 2) + 16 * q + (lane & 15);
        o = int64_t(p / a.shard_tiles) * a.i_l + j;
        have = j < a.i_l;
      } else {
        o = (int64_t(p) * 2 + rank) * kRows + 32 * q + lane;
        have = o < a.rows;
      }
      if (a.splits > 1) {   // to the cluster: the sum of this part of K, [token][row] over the token stages, which are done
        for (int c = 0; c < a.bn; c += 32) {
          uint32_t v[32];
          tmem_ld32_arrived(d + c, v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sx + uint32_t((c + i) * kRows + 32 * q + lane) * 4u), "r"(v[i]) : "memory");
        }
        break;
      }
      const bool pairs_of = !SILU && even && (int64_t(p) * 2 + rank) * kRows + 32 * q + 32 <= a.rows;
      for (int c = 0; c < a.bn; c += 32) {
        uint32_t v[32];
        tmem_ld32_arrived(d + c, v);
        if (c + 32 >= a.bn) {   // the accumulator is read out
          tcx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(lead_bar(T::B_ACC_EMPTY + (u & 1)));
        }
        const int left = m1 - m0 - c;   // tokens of these columns
        if (SILU) {
          // lanes 0-15 hold the gate, 16-31 the up of output (lane & 15); the halves take tokens in turn
          bf16* to = a.out + int64_t(m0 + c + (lane >> 4)) * a.ldc + o;
          bf16 y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {   // all before the stores, whose conditions would keep them apart
            const float give = __uint_as_float(lane < 16 ? v[2 * i + 1] : v[2 * i]);
            const float got = __shfl_xor_sync(0xffffffffu, give, 16);
            const float gate = lane < 16 ? __uint_as_float(v[2 * i]) : got;
            const float up = lane < 16 ? got : __uint_as_float(v[2 * i + 1]);
            y[i] = __float2bfloat16_rn(__fdividef(gate, 1.0f + __expf(-gate)) * up);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i, to += 2 * a.ldc)
            if (have && 2 * i + (lane >> 4) < left) *to = y[i];
        } else if (pairs_of) {
          // lanes in twos exchange halves: the even one stores both columns of token i, the odd one of token i + 1
          const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
          bf16* to = a.out + int64_t(m0 + c + (lane & 1)) * a.ldc + (o & ~int64_t(1));
#pragma unroll
          for (int i = 0; i < 32; i += 2, to += 2 * a.ldc) {
            const uint32_t mine = pack_bf16(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
            if (i + (lane & 1) < left) *reinterpret_cast<uint32_t*>(to) = __byte_perm(mine, other, sel);
          }
        } else {
          bf16* to = a.out + int64_t(m0 + c) * a.ldc + o;
#pragma unroll
          for (int i = 0; i < 32; ++i, to += a.ldc)
            if (have && i < left) *to = __float2bfloat16_rn(__uint_as_float(v[i]));
        }
      }
    }
  }
  __syncwarp();
  tcx::tc_fence_before();
  cluster_sync_all();   // neither CTA leaves while the other may arrive at its barriers or use its TMEM
  if (a.splits > 1) {
    // the parts' sums in their order; the pairs take the tokens in shares, two at a time
    const int row = threadIdx.x & 127, q = row >> 5, tile = pair, p = tile % a.p_tiles, m0 = tile / a.p_tiles * a.bn;
    const int64_t j = SILU ? (int64_t(p % a.shard_tiles) * 2 + rank) * (kRows / 2) + 16 * q + (lane & 15) : 0;
    const int64_t o = SILU ? int64_t(p / a.shard_tiles) * a.i_l + j : (int64_t(p) * 2 + rank) * kRows + row;
    const bool have = SILU ? j < a.i_l : o < a.rows;
    const int end = a.bn / 2 * (split + 1) / a.splits;
    for (int t = a.bn / 2 * split / a.splits + (threadIdx.x >> 7); t < end; t += T::THREADS / 128) {
      float v0 = 0.0f, v1 = 0.0f;
      for (int s = 0; s < a.splits; ++s) {
        const uint32_t at = map_to_rank(sx + uint32_t(2 * t * kRows + row) * 4u, uint32_t(2 * s + rank));
        v0 += ld_cluster_f32(at);
        v1 += ld_cluster_f32(at + kRows * 4);
      }
      const int m = m0 + 2 * t;
      if (SILU) {
        const float got = __shfl_xor_sync(0xffffffffu, lane < 16 ? v1 : v0, 16);
        const float gate = lane < 16 ? v0 : got, up = lane < 16 ? got : v1;
        const int mine = m + (lane >> 4);
        if (have && mine < a.M) a.out[int64_t(mine) * a.ldc + o] = __float2bfloat16_rn(__fdividef(gate, 1.0f + __expf(-gate)) * up);
      } else if (have) {
        if (m < a.M) a.out[int64_t(m) * a.ldc + o] = __float2bfloat16_rn(v0);
        if (m + 1 < a.M) a.out[int64_t(m + 1) * a.ldc + o] = __float2bfloat16_rn(v1);
      }
    }
    cluster_sync_all();   // the others have read this CTA's sums
  }
  if (warp == 1) {
    tcx::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <bool SILU, int GS, bool NARROW>
static int launch(const CUtensorMap& mx, const CUtensorMap& mc, const TcArgs& a, cudaStream_t st) {
  auto kern = gemm_tc_kernel<SILU, GS, NARROW>;
  static const cudaError_t set =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Tile<NARROW>::SMEM));
  if (set != cudaSuccess) return set_error(QW_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(set));
  const int tiles = a.p_tiles * a.q_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.splits > 1 ? 2 * a.splits * tiles : 2 * std::min(tiles, kPairs)));
  cfg.blockDim = dim3(Tile<NARROW>::THREADS);
  cfg.dynamicSmemBytes = Tile<NARROW>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(2 * a.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mx, mc, a);
  if (e != cudaSuccess) return set_error(QW_ERR_CUDA, "w4 gemm_tc_kernel launch: %s", cudaGetErrorString(e));
  return check_launch("w4 gemm_tc_kernel");
}

// Few tiles: their K in parts, as many as run at once (15 clusters of 8 CTAs, 23 of 6, 36 of 4, 76 pairs).  16 tokens,
// K 8192, us in 4 / 3 / 2 / 1 parts: 15 tiles 13.5 / 15.5 / 18.5 / 28.6, 16 tiles 23.9 / 15.5 / 18.5 / 28.7,
// 22 tiles 24.7 / 15.9 / 18.9 / 29.0, 36 tiles 36.6 / 29.7 / 19.7 / 29.6.
static int parts_of_k(int64_t tiles, int64_t stages) {
  return int(std::min<int64_t>(tiles <= 15 ? 4 : tiles <= 23 ? 3 : tiles <= 36 ? 2 : 1, stages));
}
static int64_t row_tiles(int64_t N, int silu_shards) {   // silu_shards: shards of a SiluAndMul, else 0
  return silu_shards ? silu_shards * ((N / 2 / silu_shards + kRows - 1) / kRows) : (N + 2 * kRows - 1) / (2 * kRows);
}
// steps of 128 columns that the busiest pair walks through with one tile of tokens
int64_t tc_steps(int64_t N, int64_t K_l, int silu_shards, int shards) {
  const int64_t tiles = row_tiles(N, silu_shards), stages = shards * ((K_l + 255) / 256), parts = parts_of_k(tiles, stages);
  return (tiles * parts + kPairs - 1) / kPairs * 2 * ((stages + parts - 1) / parts);
}

int gemm_tc(const bf16* x, const Weights& w, bf16* out, int64_t M, int64_t N, int64_t K, int shards, int tp, bool silu,
            int early, cudaStream_t st) {
  const int64_t K_l = K / shards;
  TcArgs a{};
  a.out = out;
  a.w = w;
  a.rows = N;
  a.ldc = silu ? N / 2 : N;
  a.i_l = silu ? N / 2 / tp : 0;
  a.M = int(M);
  a.early = early;
  a.q_tiles = int((M + Tile<false>::TOKENS - 1) / Tile<false>::TOKENS);
  a.bn = int((M + a.q_tiles - 1) / a.q_tiles + 15) / 16 * 16;
  a.q_tiles = int((M + a.bn - 1) / a.bn);
  a.shard_tiles = silu ? int((a.i_l + kRows - 1) / kRows) : 0;
  const int64_t p_tiles = row_tiles(N, silu ? tp : 0);
  if (p_tiles * a.q_tiles >= (int64_t(1) << 30)) return set_error(QW_ERR_SHAPE, "qw_w4_gemm: too many output tiles");
  a.p_tiles = int(p_tiles);
  a.shards = shards;
  a.steps_l = int((K_l + 127) / 128);
  a.splits = parts_of_k(p_tiles * a.q_tiles, int64_t(shards) * ((a.steps_l + 1) / 2));
  CUtensorMap mx, mc;
  const uint64_t xd[3] = {uint64_t(K_l), uint64_t(shards), uint64_t(M)}, xst[2] = {uint64_t(K_l) * 2, uint64_t(K) * 2};
  const uint32_t xb[3] = {64, 1, uint32_t(a.bn / 2)};
  int rc = make_tensor_map(&mx, x, 3, xd, xst, xb);
  if (rc) return rc;
  // codes as 2-byte elements: 64 of them are 256 columns
  const uint64_t cd[3] = {uint64_t(K_l) / 4, uint64_t(N), uint64_t(shards)},
                 cst[2] = {uint64_t(K_l) / 2, uint64_t(K_l) / 2 * uint64_t(N)};
  const uint32_t cb[3] = {64, silu ? 64u : 128u, 1};
  rc = make_tensor_map(&mc, w.codes, 3, cd, cst, cb);
  if (rc) return rc;
  const int gs = w.group_shift;
  auto go = [&](auto narrow) {
    constexpr bool NA = decltype(narrow)::value;
    if (silu) return gs == 0 ? launch<true, 0, NA>(mx, mc, a, st) : gs == 1 ? launch<true, 1, NA>(mx, mc, a, st) : launch<true, 2, NA>(mx, mc, a, st);
    return gs == 0 ? launch<false, 0, NA>(mx, mc, a, st) : gs == 1 ? launch<false, 1, NA>(mx, mc, a, st) : launch<false, 2, NA>(mx, mc, a, st);
  };
  return a.bn <= Tile<true>::TOKENS ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace w4

unsigned int take_w4_errors() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, w4::g_w4_error, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(w4::g_w4_error, &zero, sizeof(zero));
  return v;
}

}  // namespace qw
