// Linear layers with 4-bit weights for many tokens, on tcgen05 tensor cores (sm_103a).
//
// D[weight row, token] = W X^T: the weights are the MMA's A operand and lie in TMEM,
// where the threads that decode them put them straight from registers; the tokens are B,
// copied by TMA.  Two CTAs (cta_group::2) share a tile of 256 weight rows: each decodes
// 128 of them and holds half of the tokens, so that the tokens cross L2 and each shared
// memory once for 256 rows.
#include <algorithm>

#include "tc_common.cuh"
#include "w4.cuh"

namespace qw {
namespace w4 {

__device__ unsigned int g_w4_error = 0;

constexpr int kRows = 128;          // weight rows of a CTA (SiluAndMul: 64 gate rows and their up rows), two CTAs a tile
constexpr int kMaxTokens = 192;     // tokens of a tile: two accumulators and four stages of A fill TMEM
constexpr int kThreads = 512;
constexpr int XS = 8, CS = 4, AS = 4;                    // stages: tokens (64 columns), codes (256), decoded weights (64)
constexpr uint32_t X_BYTES = kMaxTokens / 2 * 128, C_BYTES = kRows * 128;
constexpr uint32_t OFF_X = 0, OFF_C = XS * X_BYTES, OFF_BAR = OFF_C + CS * C_BYTES;
constexpr size_t kTcSmem = 1024 + OFF_BAR + 512;
constexpr uint32_t kTmemCols = 512, kTmemA = 2 * kMaxTokens;
constexpr int B_X_FULL = 0, B_X_EMPTY = B_X_FULL + XS, B_C_FULL = B_X_EMPTY + XS, B_C_EMPTY = B_C_FULL + CS,
              B_A_FULL = B_C_EMPTY + CS, B_A_EMPTY = B_A_FULL + AS, B_ACC_FULL = B_A_EMPTY + AS, B_ACC_EMPTY = B_ACC_FULL + 2,
              B_DRAIN = B_ACC_EMPTY + 2, N_BARS = B_DRAIN + 1;
static_assert(N_BARS * 8 + 8 <= 512, "barrier area");

struct TcArgs {
  bf16* out;
  Weights w;
  int64_t rows, ldc, i_l;
  int M, bn;              // tokens, tokens of a tile
  int p_tiles, q_tiles;   // weight row tiles, token tiles
  int shard_tiles;        // SiluAndMul: row tiles of a shard
  int shards, nk_l;       // shards of K, 64-column blocks of a shard
};

// The two CTAs of a pair: rank 0 issues the MMAs and holds the barriers that both feed.
// Issued by the lane with `lead`, as a predicate: the warp stays converged and its operands in uniform registers (61 ->
// 20 cycles an MMA, 110 -> 22 a commit, against one lane in a branch).
__device__ __forceinline__ void umma_commit_pair(uint32_t lead, uint32_t bar) {   // arrives at this offset in both CTAs
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%1], %2;\n}\n" ::"r"(lead),
      "r"(bar), "h"(uint16_t(3))
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
// into this CTA's shared memory, completing on rank 0's barrier
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
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

template <bool SILU>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_c, TcArgs a) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sx = smem_u32(sm + OFF_X), sc = smem_u32(sm + OFF_C), bars = smem_u32(sm + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_BAR + N_BARS * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  auto bar = [&](int b) { return bars + uint32_t(b) * 8u; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank()), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto lead_bar = [&](int b) { return map_to_rank(bar(b), 0); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < XS; ++i) tcx::mbar_init(bar(B_X_FULL + i), 1), tcx::mbar_init(bar(B_X_EMPTY + i), 1);
    for (int i = 0; i < CS; ++i) tcx::mbar_init(bar(B_C_FULL + i), 1), tcx::mbar_init(bar(B_C_EMPTY + i), 8);
    for (int i = 0; i < AS; ++i) tcx::mbar_init(bar(B_A_FULL + i), 8), tcx::mbar_init(bar(B_A_EMPTY + i), 1);
    for (int i = 0; i < 2; ++i) tcx::mbar_init(bar(B_ACC_FULL + i), 1), tcx::mbar_init(bar(B_ACC_EMPTY + i), 8);
    tcx::mbar_init(bar(B_DRAIN), 1);
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
  const int tiles = a.p_tiles * a.q_tiles, ncs_l = (a.nk_l + 3) / 4;
  // first weight row (gate row) of a row tile; the stored rows of shard r of K begin at r * rows
  auto tile_row = [&](int p) -> int64_t {
    if (!SILU) return (int64_t(p) * 2 + rank) * kRows;
    const int r = p / a.shard_tiles;
    return int64_t(r) * 2 * a.i_l + (int64_t(p % a.shard_tiles) * 2 + rank) * (kRows / 2);
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA: code stages ahead of the token stages that they go with ----
      uint32_t cs = 0, xs = 0;
      bool ok = true;
      auto load_codes = [&](int64_t row, int r, int c) {
        const uint32_t s = cs % CS;
        ok = wait(B_C_EMPTY + s, ((cs / CS) & 1) ^ 1, 1u);
        if (!ok) return;
        tcx::mbar_expect_tx(bar(B_C_FULL + s), C_BYTES);
        const uint32_t dst = sc + s * C_BYTES;
        tcx::tma_load_3d(dst, &tm_c, bar(B_C_FULL + s), c * 64, int(row), r);
        if (SILU) tcx::tma_load_3d(dst + C_BYTES / 2, &tm_c, bar(B_C_FULL + s), c * 64, int(row + a.i_l), r);
        ++cs;
      };
      bool waited = false;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        const int64_t row = tile_row(tile % a.p_tiles);
        const int m0 = tile / a.p_tiles * a.bn + rank * (a.bn / 2);
        for (int r = 0; r < a.shards && ok; ++r)
          for (int c = 0; c < ncs_l && ok; ++c) {
            load_codes(row, r, c);
            if (!waited) {
              pdl_wait();   // the tokens may come from the kernel before; the weights are constants
              waited = true;
            }
            for (int kb = 4 * c; kb < min(4 * c + 4, a.nk_l) && ok; ++kb) {
              const uint32_t s = xs % XS;
              ok = wait(B_X_EMPTY + s, ((xs / XS) & 1) ^ 1, 2u);
              if (!ok) break;
              if (rank == 0) tcx::mbar_expect_tx(bar(B_X_FULL + s), uint32_t(a.bn) * 128u);   // both halves
              tma_load_3d_pair(sx + s * X_BYTES, &tm_x, lead_bar(B_X_FULL + s), kb * 64, r, m0);
              ++xs;
            }
          }
      }
      if (!ok) {   // the copies in flight land before the block ends
        for (uint32_t i = cs > CS ? cs - CS : 0; i < cs; ++i) tcx::mbar_wait(bar(B_C_FULL + i % CS), (i / CS) & 1, &g_w4_error, 1u);
        for (uint32_t i = xs > XS ? xs - XS : 0; i < xs && rank == 0; ++i) tcx::mbar_wait(bar(B_X_FULL + i % XS), (i / XS) & 1, &g_w4_error, 2u);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---- MMA, for both CTAs ----
      const uint32_t lead = elect_one();
      const uint32_t idesc = tcx::idesc_bf16(2 * kRows, a.bn);
      const uint64_t desc = tcx::sw128_desc(sx);
      const uint32_t b_lo = uint32_t(desc), b_hi = uint32_t(desc >> 32);
      const int nk = a.shards * a.nk_l;
      uint32_t it = 0, u = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs, ++u) {
        const uint32_t d = tmem + (u & 1) * kMaxTokens;
        ok = __all_sync(0xffffffffu, wait(B_ACC_EMPTY + (u & 1), ((u >> 1) & 1) ^ 1, 4u));
        for (int kb = 0; kb < nk && ok; ++kb, ++it) {
          const uint32_t s = it % XS, as = it % AS;
          ok = __all_sync(0xffffffffu, wait(B_X_FULL + s, (it / XS) & 1, 8u) && wait(B_A_FULL + as, (it / AS) & 1, 16u));
          if (!ok) break;
          tcx::tc_fence_after();
          const uint32_t b = b_lo + s * (X_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ts(lead, d, tmem + kTmemA + as * 32 + k * 8, b + 2 * k, b_hi, idesc, (kb > 0 || k > 0) ? 1u : 0u);
          umma_commit_pair(lead, bar(B_X_EMPTY + s));
          umma_commit_pair(lead, bar(B_A_EMPTY + as));
        }
        if (ok) umma_commit_pair(lead, bar(B_ACC_FULL + (u & 1)));
      }
      umma_commit_pair(lead, bar(B_DRAIN));
      tcx::mbar_wait(bar(B_DRAIN), 0, &g_w4_error, 32u);
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- decode: one weight row a thread; four warps cover the rows, two such sets take the 64-column blocks in turn ----
    const int q = warp & 3, h = (warp - 4) >> 2;
    const int srow = SILU ? (lane >> 4) * 64 + 16 * q + (lane & 15) : 32 * q + lane;   // row in the code stage
    const uint32_t lane_base = uint32_t(32 * q) << 16;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(a.w.scales);
    uint32_t cs = 0, it0 = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      const int p = tile % a.p_tiles;
      int64_t row = tile_row(p);
      row += SILU ? (lane >> 4) * a.i_l + 16 * q + (lane & 15) : srow;
      const bool have = row < a.rows;
      for (int r = 0; r < a.shards && ok; ++r) {
        const int64_t g0 = (int64_t(r) * a.rows + row) * a.w.groups;
        for (int c = 0; c < ncs_l && ok; ++c, ++cs) {
          const int kend = min(4 * c + 4, a.nk_l);
          // scales of this warp's two blocks: two pieces of 32 columns in each
          uint32_t s[2][2], z[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int g = ((4 * c + 2 * j + h) * 2 + e) >> a.w.group_shift;
              const bool in = have && g < a.w.groups;
              s[j][e] = in ? __ldg(scales + g0 + g) : 0u;
              z[j][e] = in && a.w.zeros != nullptr ? __ldg(a.w.zeros + g0 + g) : 8u;
            }
          const uint32_t st = cs % CS;
          ok = __all_sync(0xffffffffu, wait(B_C_FULL + st, (cs / CS) & 1, 64u));   // the warp goes on as one
          if (!ok) break;
          uint4 v[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t ch = uint32_t((2 * j + h) * 2 + e);
              const uint32_t addr = sc + st * C_BYTES + uint32_t(srow) * 128u + ((ch ^ uint32_t(srow & 7)) << 4);
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(v[j][e].x), "=r"(v[j][e].y), "=r"(v[j][e].z), "=r"(v[j][e].w)
                           : "r"(addr));
            }
          __syncwarp();
          if (lane == 0) tcx::mbar_arrive(bar(B_C_EMPTY + st));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int kb = 4 * c + 2 * j + h;
            if (kb >= kend) break;
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t s2 = scale_pair(s[j][e]), z2 = offset_pair(z[j][e]);
              const uint32_t word[4] = {v[j][e].x, v[j][e].y, v[j][e].z, v[j][e].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t o[4];
                decode(word[i], z2, s2, o);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[16 * e + 4 * i + k] = o[k];
              }
            }
            const uint32_t it = it0 + uint32_t(r * a.nk_l + kb), as = it % AS;
            ok = __all_sync(0xffffffffu, wait(B_A_EMPTY + as, ((it / AS) & 1) ^ 1, 128u));
            if (!ok) break;
            tcx::tc_fence_after();
            tcx::tmem_st32(tmem + lane_base + kTmemA + as * 32, w);
            tcx::tmem_st_wait();
            tcx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(lead_bar(B_A_FULL + as));
          }
        }
      }
      it0 += uint32_t(a.shards * a.nk_l);
    }
  } else if (warp >= 12) {
    // ---- epilogue ----
    const int q = warp & 3;
    uint32_t u = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles && ok; tile += pairs, ++u) {
      ok = __all_sync(0xffffffffu, wait(B_ACC_FULL + (u & 1), (u >> 1) & 1, 256u));
      if (!ok) break;
      tcx::tc_fence_after();
      const int p = tile % a.p_tiles, m0 = tile / a.p_tiles * a.bn, m1 = min(m0 + a.bn, a.M);
      const uint32_t d = tmem + (uint32_t(32 * q) << 16) + (u & 1) * kMaxTokens;
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
      for (int c = 0; c < a.bn; c += 32) {
        uint32_t v[32];
        tmem_ld32_arrived(d + c, v);
        if (SILU) {
          // lanes 0-15 hold the gate, 16-31 the up of output (lane & 15); the halves take tokens in turn
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float give = __uint_as_float(lane < 16 ? v[i + 1] : v[i]);
            const float got = __shfl_xor_sync(0xffffffffu, give, 16);
            const float gate = lane < 16 ? __uint_as_float(v[i]) : got;
            const float up = lane < 16 ? got : __uint_as_float(v[i + 1]);
            const int m = m0 + c + i + (lane >> 4);
            if (have && m < m1) a.out[int64_t(m) * a.ldc + o] = __float2bfloat16_rn(__fdividef(gate, 1.0f + __expf(-gate)) * up);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (have && m0 + c + i < m1) a.out[int64_t(m0 + c + i) * a.ldc + o] = __float2bfloat16_rn(__uint_as_float(v[i]));
        }
      }
      tcx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(lead_bar(B_ACC_EMPTY + (u & 1)));
    }
  }
  __syncwarp();
  tcx::tc_fence_before();
  cluster_sync_all();   // neither CTA leaves while the other may arrive at its barriers or use its TMEM
  if (warp == 1) {
    tcx::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <bool SILU>
static int launch(const CUtensorMap& mx, const CUtensorMap& mc, const TcArgs& a, cudaStream_t st) {
  auto kern = gemm_tc_kernel<SILU>;
  static const cudaError_t set =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTcSmem));
  if (set != cudaSuccess) return set_error(QW_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(set));
  const int tiles = a.p_tiles * a.q_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(2 * std::min(tiles, 76)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
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

int gemm_tc(const bf16* x, const Weights& w, bf16* out, int64_t M, int64_t N, int64_t K, int shards, int tp, bool silu,
            cudaStream_t st) {
  const int64_t K_l = K / shards;
  TcArgs a{};
  a.out = out;
  a.w = w;
  a.rows = N;
  a.ldc = silu ? N / 2 : N;
  a.i_l = silu ? N / 2 / tp : 0;
  a.M = int(M);
  a.q_tiles = int((M + kMaxTokens - 1) / kMaxTokens);
  a.bn = int((M + a.q_tiles - 1) / a.q_tiles + 15) / 16 * 16;
  a.q_tiles = int((M + a.bn - 1) / a.bn);
  a.shard_tiles = silu ? int((a.i_l + kRows - 1) / kRows) : 0;
  const int64_t p_tiles = silu ? int64_t(tp) * a.shard_tiles : (N + 2 * kRows - 1) / (2 * kRows);
  if (p_tiles * a.q_tiles >= (int64_t(1) << 31)) return set_error(QW_ERR_SHAPE, "qw_w4_gemm: too many output tiles");
  a.p_tiles = int(p_tiles);
  a.shards = shards;
  a.nk_l = int((K_l + 63) / 64);
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
  return silu ? launch<true>(mx, mc, a, st) : launch<false>(mx, mc, a, st);
}

}  // namespace w4

unsigned int take_w4_errors() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, w4::g_w4_error, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(w4::g_w4_error, &zero, sizeof(zero));
  return v;
}

}  // namespace qw
