// Linear layers with 4-bit weights, few tokens: weight streaming with warp-level MMA.
//
// out[m, n] = sum_k x[m, k] w[n, k], w decoded from its code, scale and zero point in registers (w4.cuh) and fed to
// mma.sync m16n8k16 as the A operand: 16 weight rows against 8 tokens, fp32 sums.  A warp's sums of its part of K are
// added over the warps of a row tile in shared memory, in slice order.
// Bound: the operands' way through L1, then the chain of a chunk.  A chunk of 16 rows x 128 columns is 8 MMAs, and one
// occupies an SM sub-partition for 8 cycles (measured in a loop of them alone), 64 in all; decoding takes 128 of the
// half-rate bf16 pipe and 112 of the integer pipe beside it.  1 x 28672 x 8192 (117 MB of codes): 31.5 us, 3.8 TB/s, against
// 17.9 for its bytes and 6.2 for its MMAs; L1 is at 85% of its peak there (codes cross it on their way into shared memory
// and out of it, scales in loads of two bytes a row, tokens again for each row tile), the tensor pipe at 22%.  8 x 151936 x
// 1024, its tokens in shared memory: 24.9 us against 12.6 and 4.1, no unit above 53% (issue slots).  1 x 4096 x 1024: 2.4 us
// in a graph, launch and latency.
#include "w4.cuh"

namespace qw {

template <typename T>
int launch_gather_rows(const void* src, int64_t n_src, const int32_t* idx, int64_t n, int64_t H, void* out,
                       cudaStream_t st);
template <typename T>
int launch_argmax(const void* logits, int64_t M, int64_t V, int64_t* out, cudaStream_t st);

namespace w4 {

int check_weights(const char* who, const void* codes, const void* scales, int64_t N, int64_t K, int group);
Weights make_weights(const void* codes, const void* scales, const void* zeros, int64_t K, int group);
int gemm_tc(const bf16* x, const Weights& w, bf16* out, int64_t M, int64_t N, int64_t K, int shards, int tp, bool silu,
            int early, cudaStream_t st);
int64_t tc_steps(int64_t N, int64_t K_l, int silu_shards, int shards);

struct GemvArgs {
  const bf16* x;         // [M, K], at most 8 NT tokens
  bf16* out;             // [M, ldc]
  Weights w;             // of one shard's rows
  int64_t rows;          // N: rows of a shard (row split), of the matrix (column)
  int64_t ldc;
  int64_t i_l;           // SiluAndMul: outputs of a shard
  int64_t tiles;         // row tiles of 16 (SiluAndMul: 8 gate and their 8 up rows)
  int M, K;
  int pieces, pieces_l;  // pieces of K, of a shard's K
  int early;             // the weights may be read ahead of the programmatic wait
  int split;             // warps that share a row tile, each every split-th chunk of 128 columns
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kWarps = 8;
// a warp's shared memory: DEPTH chunks of codes, in whose place its sums come at the end
constexpr size_t gemv_warp_smem(int nt, int r, int depth) {
  const size_t codes = size_t(depth) * r * 1024, sums = size_t(16) * r * (nt * 8 + 1) * 4;
  return ((codes > sums ? codes : sums) + 15) / 16 * 16;
}

// A warp takes R tiles of 16 weight rows and every split-th chunk of 128 columns; lane (g, t) = (lane / 4,
// lane % 4) holds the 32 columns of piece t of rows g and g + 8.  The k index of an MMA may be any
// permutation that weights and tokens share, so a lane's own columns are its k values: no shuffles.
// The codes of DEPTH chunks are in flight at once, the first ones ahead of the programmatic wait
// (QW_W4_WEIGHTS_READY): each lane copies asynchronously to shared memory what it reads there itself, so that the depth
// costs no registers and nothing waits for another lane.
// WHOLE: a shard's columns are whole chunks, so that nothing in the loop has a condition of its own lane.
// XS: the tokens lie in shared memory behind the rings, 16 bytes (8 columns, word i of a piece) of lane (g, t) at
// [chunk][n][i][lane]: a read has no bank conflict, while a load of 8 tokens from memory touches 16 lines.  For warps
// that walk through all of K (split 1), which all read them.
template <int NT, int R, int DEPTH, bool SILU, bool ZEROS, bool WHOLE, bool XS>
__global__ void __launch_bounds__(kWarps * 32) gemv_kernel(GemvArgs a) {
  extern __shared__ __align__(16) uint8_t gemv_dyn[];
  constexpr size_t WARP_SMEM = gemv_warp_smem(NT, R, DEPTH);
  auto sum_at = [&](int w, int row, int n) -> float& {
    return reinterpret_cast<float*>(gemv_dyn + w * WARP_SMEM)[row * (NT * 8 + 1) + n];
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int per_cta = kWarps / a.split, sl = warp % a.split;
  const int64_t tile0 = int64_t(blockIdx.x) * per_cta * R, tile = tile0 + warp / a.split * R;
  const uint32_t magic = code_magic();
  // this lane's piece within its shard, pieces from it to the end of K, pieces to the next one
  int lu = 4 * sl + t, left = a.pieces - lu;
  const int advance = 4 * a.split;
  // rows g and g + 8 of each tile (SiluAndMul: gate and up of output g): codes and scales at the next piece.
  // A row that is not there reads row 0 and is not stored.
  const uint8_t* cp[R][2];
  const uint16_t* sp[R][2];
  const uint8_t* zp[R][2];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    int64_t row[2];
    if (SILU) {
      const int64_t o = (tile + q) * 8 + g, r = o / a.i_l;
      row[0] = tile + q < a.tiles ? o + r * a.i_l : 0;
      row[1] = tile + q < a.tiles ? row[0] + a.i_l : 0;
    } else {
      row[0] = (tile + q) * 16 + g;
      row[1] = row[0] + 8;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (row[e] >= a.rows) row[e] = 0;
      cp[q][e] = a.w.codes + row[e] * a.w.row_bytes + int64_t(lu) * 16;
      sp[q][e] = reinterpret_cast<const uint16_t*>(a.w.scales) + row[e] * a.w.groups + (lu >> a.w.group_shift);
      zp[q][e] = a.w.zeros + row[e] * a.w.groups + (lu >> a.w.group_shift);
    }
  }
  const int64_t to_shard_c = (a.rows - 1) * a.w.row_bytes, to_shard_s = (a.rows - 1) * a.w.groups;
  const uint32_t ring = smem_u32(gemv_dyn + warp * WARP_SMEM) + uint32_t(lane) * 16u;
  struct Scales {
    uint32_t s[R][2], z[R][2];
  };
  // codes of the next chunk to ring slot d, its scales to b
  auto load = [&](int d, Scales& b) {
    while (lu >= a.pieces_l && left > 0) {   // on to the next shard's rows
      lu -= a.pieces_l;
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cp[q][e] += to_shard_c;
          sp[q][e] += to_shard_s;
          zp[q][e] += to_shard_s;
        }
    }
    const int step = WHOLE ? advance >> a.w.group_shift
                           : ((lu + advance) >> a.w.group_shift) - (lu >> a.w.group_shift);
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (!WHOLE) {
          b.s[q][e] = 0;
          b.z[q][e] = 8;
        }
        if (left > 0) {
          cp_async16(ring + uint32_t((d * R + q) * 2 + e) * 512u, cp[q][e]);
          b.s[q][e] = __ldg(sp[q][e]);
          if (ZEROS) b.z[q][e] = __ldg(zp[q][e]);
        }
        cp[q][e] += 16 * advance;
        sp[q][e] += step;
        if (ZEROS) zp[q][e] += step;
      }
    cp_async_commit();
    lu += advance;
    left -= advance;
  };
  float acc[R][NT][4];
#pragma unroll
  for (int q = 0; q < R; ++q)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[q][n][0] = acc[q][n][1] = acc[q][n][2] = acc[q][n][3] = 0.0f;
  if (!a.early) pdl_wait();
  Scales sc[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, sc[d]);
  if (a.early) pdl_wait();
  pdl_trigger();
  // this lane's token of each group of 8; past the last one it is token 0, whose sums there are not stored
  const bf16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = n * 8 + g;
    xp[n] = a.x + int64_t(tok < a.M ? tok : 0) * a.K + (4 * sl + t) * kPiece;
  }
  const uint32_t xsm = smem_u32(gemv_dyn) + uint32_t(kWarps * WARP_SMEM);
  if (XS) {
    for (int e = threadIdx.x; e < a.pieces / 4 * NT * 128; e += kWarps * 32) {
      const int tok = (e >> 7) % NT * 8 + ((e >> 2) & 7), k = (e >> 7) / NT * 128 + (e & 3) * 32 + ((e >> 5) & 3) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (tok < a.M) v = *reinterpret_cast<const uint4*>(a.x + int64_t(tok) * a.K + k);
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(xsm + uint32_t(e) * 16u), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    }
    __syncthreads();
  }
  for (int u0 = 4 * sl; u0 < a.pieces; u0 += advance * DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int u = u0 + advance * d;
      if (u >= a.pieces) break;
      const bool in = WHOLE || u + t < a.pieces;
      uint4 x[4][NT];
      auto load_x = [&](int i) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (XS) {
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x[i][n].x), "=r"(x[i][n].y), "=r"(x[i][n].z), "=r"(x[i][n].w)
                         : "r"(xsm + uint32_t((((u >> 2) * NT + n) * 4 + i) * 32 + lane) * 16u)
                         : "memory");
            continue;
          }
          if (!WHOLE) x[i][n] = make_uint4(0, 0, 0, 0);
          if (in) x[i][n] = __ldg(reinterpret_cast<const uint4*>(xp[n] + 8 * i));
        }
      };
      constexpr int AHEAD = XS ? 2 : NT <= 2 ? 4 : NT <= 6 ? 2 : 1;   // words of tokens in flight
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) load_x(i);
      cp_async_wait<DEPTH - 1>();
      uint4 c[R][2];
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(c[q][e].x), "=r"(c[q][e].y), "=r"(c[q][e].z), "=r"(c[q][e].w)
                       : "r"(ring + uint32_t((d * R + q) * 2 + e) * 512u)
                       : "memory");
          if (!WHOLE && !in) c[q][e] = make_uint4(0, 0, 0, 0);   // nothing was copied there
        }
      const Scales& b = sc[d];
      uint32_t s2[R][2], z2[R][2];
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) s2[q][e] = scale_pair(b.s[q][e]), z2[q][e] = offset_pair(ZEROS ? b.z[q][e] : 8u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          uint32_t pa[4], pb[4];
          const uint32_t wa = i == 0 ? c[q][0].x : i == 1 ? c[q][0].y : i == 2 ? c[q][0].z : c[q][0].w;
          const uint32_t wb = i == 0 ? c[q][1].x : i == 1 ? c[q][1].y : i == 2 ? c[q][1].z : c[q][1].w;
          decode(wa, magic, z2[q][0], s2[q][0], pa);
          decode(wb, magic, z2[q][1], s2[q][1], pb);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816(acc[q][n], pa[0], pb[0], pa[1], pb[1], x[i][n].x, x[i][n].y);
            mma_16816(acc[q][n], pa[2], pb[2], pa[3], pb[3], x[i][n].z, x[i][n].w);
          }
        }
        if (i + AHEAD < 4) load_x(i + AHEAD);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) xp[n] += advance * kPiece;
      load(d, sc[d]);
    }
  }
  cp_async_wait<0>();   // nothing is on its way into the places of the sums
  __syncwarp();
#pragma unroll
  for (int q = 0; q < R; ++q)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      sum_at(warp, 16 * q + g, n * 8 + 2 * t) = acc[q][n][0];
      sum_at(warp, 16 * q + g, n * 8 + 2 * t + 1) = acc[q][n][1];
      sum_at(warp, 16 * q + g + 8, n * 8 + 2 * t) = acc[q][n][2];
      sum_at(warp, 16 * q + g + 8, n * 8 + 2 * t + 1) = acc[q][n][3];
    }
  __syncthreads();
  constexpr int out_rows = SILU ? 8 : 16;   // of a tile
  const int total = per_cta * R * out_rows, live = a.M;
  for (int e = threadIdx.x; e < total * live; e += kWarps * 32) {
    const int j = e % total, n = e / total, lt = j / out_rows, r = j % out_rows;
    const int64_t o = (tile0 + lt) * out_rows + r;
    if (o >= (SILU ? a.rows / 2 : a.rows)) continue;
    float v = 0.0f, up = 0.0f;
    for (int s = 0; s < a.split; ++s) {   // in slice order
      const int w = lt / R * a.split + s, row = lt % R * 16 + r;
      v += sum_at(w, row, n);
      if (SILU) up += sum_at(w, row + 8, n);
    }
    if (SILU) v = __fdividef(v, 1.0f + __expf(-v)) * up;
    a.out[int64_t(n) * a.ldc + o] = __float2bfloat16_rn(v);
  }
}

// warps that share a unit of row tiles: up to 8, while the CTAs run at once (`resident` of them on an SM)
static int gemv_split(int64_t units, int chunks, int resident) {
  int split = kWarps;
  while (split > 1 && (split > chunks || units * split > 152 * kWarps * int64_t(resident))) split >>= 1;
  return split;
}

// 9 to 64 tokens: whether the tcgen05 kernel is expected to be done first.  Both sides from measurements: a step of
// 256 rows x 128 columns takes a pair of SMs 0.39 us, the launch and its ends about 5; here 2.5 us and 0.21, 0.39, 0.46,
// 0.46, 0.6 and 0.78 us for each 2^20 weights with 2, 3, 4, 5, 6 and 8 groups of 8 tokens.  us there and here:
// 8192 x 8192, 16 tokens 19.5 / 17.3, 24 19.9 / 26.5, 64 21.0 / 49.2; 4096 x 4096, 24 11.5 / 9.1, 64 12.4 / 16.8;
// 4096 x 1024, 64 8.3 / 7.5; 151936 x 1024, 16 32.3 / 34.5, 64 33.3 / 146.
static bool tc_is_faster(int nt, int64_t N, int64_t K, int64_t K_l, int silu_shards, int shards) {
  static const double per_mega[9] = {0, 0, 0.21, 0.39, 0.46, 0.46, 0.6, 0.78, 0.78};
  const double here = 2.5 + per_mega[nt] * double(N) * double(K) / (1 << 20);
  return 5.0 + 0.39 * double(tc_steps(N, K_l, silu_shards, shards)) < here;
}

template <int NT, int R, int DEPTH, bool SILU, bool ZEROS, bool WHOLE, bool XS>
static int start_gemv(const GemvArgs& a, int64_t units, size_t smem, cudaStream_t st) {
  auto kern = gemv_kernel<NT, R, DEPTH, SILU, ZEROS, WHOLE, XS>;
  if (smem > 48 * 1024) {
    static const cudaError_t set = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (set != cudaSuccess) return set_error(QW_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(set));
  }
  const int per_cta = kWarps / a.split;
  launch_pdl(kern, dim3(unsigned((units + per_cta - 1) / per_cta)), kWarps * 32, smem, st, a);
  return check_launch("w4 gemv");
}

template <int NT, int R, int DEPTH, bool SILU, bool ZEROS, bool WHOLE>
static int launch_gemv(GemvArgs a, cudaStream_t st) {
  constexpr size_t smem = kWarps * gemv_warp_smem(NT, R, DEPTH);
  static_assert(smem <= 128 * 1024, "");
  static const int resident = [&] {
    auto kern = gemv_kernel<NT, R, DEPTH, SILU, ZEROS, WHOLE, false>;
    int n = 0;
    if (smem > 48 * 1024) cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kWarps * 32, smem) == cudaSuccess && n > 0 ? n : 1;
  }();
  const int chunks = (a.pieces + 3) / 4;
  const int64_t units = (a.tiles + R - 1) / R;
  a.split = gemv_split(units, chunks, resident);
  if constexpr (WHOLE && NT <= 2) {
    // us without and with them there: 8 x 151936 x 1024 26.5 / 24.9, 16 x 100000 x 1024 31.2 / 27.4; 8 x 60000 x 4096 (64 KB
    // of a CTA) 39.0 / 40.4; two tokens or one touch few lines anyway
    const size_t x_bytes = size_t(chunks) * NT * 2048;
    if (a.split == 1 && a.M > 2 && x_bytes <= 32 * 1024)
      return start_gemv<NT, R, DEPTH, SILU, ZEROS, WHOLE, true>(a, units, smem + x_bytes, st);
  }
  return start_gemv<NT, R, DEPTH, SILU, ZEROS, WHOLE, false>(a, units, smem, st);
}

template <int NT, int R, int DEPTH, bool WHOLE>
static int launch_gemv(const GemvArgs& a, bool silu, cudaStream_t st) {
  if (a.w.zeros != nullptr)
    return silu ? launch_gemv<NT, R, DEPTH, true, true, WHOLE>(a, st) : launch_gemv<NT, R, DEPTH, false, true, WHOLE>(a, st);
  return silu ? launch_gemv<NT, R, DEPTH, true, false, WHOLE>(a, st) : launch_gemv<NT, R, DEPTH, false, false, WHOLE>(a, st);
}

static int linear(const bf16* x, const void* codes, const void* scales, const void* zeros, bf16* out, int64_t M, int64_t N,
                  int64_t K, int group, int tp, int mode, int epi, int flags, cudaStream_t st) {
  const int64_t K_l = mode == QW_GEMM_ROW_REDUCE ? K / tp : K;
  GemvArgs a{};
  const bool silu = epi == QW_EPI_SILU_MUL;
  a.x = x;
  a.out = out;
  a.w = make_weights(codes, scales, zeros, K_l, group);
  a.rows = N;
  a.ldc = silu ? N / 2 : N;
  a.i_l = silu ? N / 2 / tp : 0;
  a.tiles = silu ? N / 16 : (N + 15) / 16;
  a.M = int(M);
  a.early = flags & QW_W4_WEIGHTS_READY;
  a.K = int(K);
  a.pieces = int(K / kPiece);
  a.pieces_l = int(K_l / kPiece);
  const int shards = mode == QW_GEMM_ROW_REDUCE ? tp : 1, nt = int((M + 7) / 8);
  const bool whole = a.pieces_l % 4 == 0;
  if (nt > 8 || (nt > 1 && tc_is_faster(nt, N, K, K_l, silu ? tp : 0, shards)) || (nt > 1 && !whole))
    return gemm_tc(x, a.w, out, M, N, K, shards, tp, silu, a.early, st);
  if (!whole) return launch_gemv<1, 1, 2, false>(a, silu, st);
  switch (nt) {
    case 1: {
      // Two row tiles a warp halve the tokens' traffic through L1 (8 x 16 lines a load), one tile leaves more warps and
      // shorter ones; four chunks in flight pay only where a warp has many.  us with one tile and 2 or 4 chunks, two and 2:
      // 8 x 151936 x 1024 29.3 / 31.1 / 26.3, 4 x 8192 x 8192 14.2 / 18.7 / 12.3, 1 x 28672 x 8192 38.0 / 30.2 / 35.5,
      // 1 x 4096 x 4096 6.1 / 7.0 / 6.2, 8 x 1024 x 2048 2.6 / 2.7 / 3.2, 1 x 4096 x 1024 2.5 / 2.9 / 2.5.
      const int chunks = a.pieces / 4, each = chunks / gemv_split(a.tiles, chunks, 3);
      if (M > 2 && each >= 4) return launch_gemv<1, 2, 2, true>(a, silu, st);
      return each >= 16 ? launch_gemv<1, 1, 4, true>(a, silu, st) : launch_gemv<1, 1, 2, true>(a, silu, st);
    }
    case 2: return launch_gemv<2, 2, 2, true>(a, silu, st);
    case 3: return launch_gemv<3, 2, 2, true>(a, silu, st);
    case 4: return launch_gemv<4, 2, 2, true>(a, silu, st);
    case 5: return launch_gemv<5, 2, 2, true>(a, silu, st);
    case 6: return launch_gemv<6, 2, 2, true>(a, silu, st);
    default: return launch_gemv<8, 2, 2, true>(a, silu, st);
  }
}

// argmax over rows of bf16 logits of any width, lowest index on ties (as qw_argmax; NaN is passed over)
__global__ void __launch_bounds__(1024) argmax_kernel(const bf16* __restrict__ logits, int64_t V, int64_t* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sv[32];
  __shared__ int64_t si[32];
  const bf16* p = logits + int64_t(blockIdx.x) * V;
  float best = -INFINITY;
  int64_t at = V;
  auto take = [&](float ob, int64_t oi) {
    if (ob > best || (ob == best && oi < at)) { best = ob; at = oi; }
  };
  for (int64_t i = threadIdx.x; i < V; i += 1024) {
    const float f = __bfloat162float(p[i]);
    if (f > best) { best = f; at = i; }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) take(__shfl_xor_sync(0xffffffffu, best, o), __shfl_xor_sync(0xffffffffu, at, o));
  if ((threadIdx.x & 31) == 0) { sv[threadIdx.x >> 5] = best; si[threadIdx.x >> 5] = at; }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) take(sv[w], si[w]);
    out[blockIdx.x] = at < V ? at : 0;
  }
}

}  // namespace w4
}  // namespace qw

using namespace qw;

static inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

extern "C" size_t qw_w4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int tp, int mode, int epilogue) {
  (void)M, (void)N, (void)K, (void)tp, (void)mode, (void)epilogue;
  return 0;
}

extern "C" int qw_w4_gemm(const void* A, const void* codes, const void* scales, const void* zeros, void* C, int64_t M,
                          int64_t N, int64_t K, int group, int tp, int mode, int epilogue, void* workspace,
                          size_t workspace_bytes, int dtype, int flags, void* stream) {
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "qw_w4_gemm: dtype %d", dtype);
  if (flags & ~QW_W4_WEIGHTS_READY) return set_error(QW_ERR_INVALID_ARG, "qw_w4_gemm: flags %d", flags);
  if (M < 0 || N <= 0 || K <= 0 || tp <= 0) return set_error(QW_ERR_INVALID_ARG, "qw_w4_gemm: bad sizes");
  if (mode != QW_GEMM_COLUMN && mode != QW_GEMM_ROW_REDUCE)
    return set_error(QW_ERR_INVALID_ARG, "qw_w4_gemm: mode %d", mode);
  if (epilogue != QW_EPI_NONE && epilogue != QW_EPI_SILU_MUL)
    return set_error(QW_ERR_INVALID_ARG, "qw_w4_gemm: epilogue %d", epilogue);
  if (epilogue == QW_EPI_SILU_MUL && mode != QW_GEMM_COLUMN)
    return set_error(QW_ERR_INVALID_ARG, "qw_w4_gemm: SiluAndMul needs the column (gate_up) layout");
  if (mode == QW_GEMM_ROW_REDUCE && K % tp) return set_error(QW_ERR_SHAPE, "qw_w4_gemm: K=%lld %% tp=%d", (long long)K, tp);
  if (mode == QW_GEMM_COLUMN && N % tp) return set_error(QW_ERR_SHAPE, "qw_w4_gemm: N=%lld %% tp=%d", (long long)N, tp);
  if (epilogue == QW_EPI_SILU_MUL && N % (16 * int64_t(tp)))
    return set_error(QW_ERR_SHAPE, "qw_w4_gemm: gate_up width %lld not 2*tp*I_l with I_l a multiple of 8", (long long)N);
  if (M >= (int64_t(1) << 21)) return set_error(QW_ERR_SHAPE, "qw_w4_gemm: 2^21 tokens or more");
  if (M == 0) return QW_OK;
  const int64_t K_l = mode == QW_GEMM_ROW_REDUCE ? K / tp : K;
  if (K >= (int64_t(1) << 31)) return set_error(QW_ERR_SHAPE, "qw_w4_gemm: dimension too large");
  const int rc = w4::check_weights("qw_w4_gemm", codes, scales, N, K_l, group);
  if (rc) return rc;
  if (!A || !C || !al16(A) || !al16(C)) return set_error(QW_ERR_INVALID_ARG, "qw_w4_gemm: null or misaligned A or C");
  (void)workspace, (void)workspace_bytes;
  return w4::linear(static_cast<const bf16*>(A), codes, scales, zeros, static_cast<bf16*>(C), M, N, K, group, tp, mode,
                    epilogue, flags, static_cast<cudaStream_t>(stream));
}

extern "C" size_t qw_w4_lm_head_workspace_size(int64_t n_out, int64_t V, int64_t H, int tp) {
  if (n_out <= 0 || V <= 0 || H <= 0) return 0;
  (void)tp;
  return kCounterBytes + (size_t(n_out) * size_t(H) * 2 + 255) / 256 * 256;
}

extern "C" int qw_w4_lm_head(const void* hidden, int64_t T, const int32_t* last_idx, int64_t n_out, const void* codes,
                             const void* scales, const void* zeros, int64_t V, int64_t H, int group, int tp, void* logits,
                             int64_t* next_tokens, void* workspace, size_t workspace_bytes, int dtype, int flags,
                             void* stream) {
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "qw_w4_lm_head: dtype %d", dtype);
  if (flags & ~QW_W4_WEIGHTS_READY) return set_error(QW_ERR_INVALID_ARG, "qw_w4_lm_head: flags %d", flags);
  if (T < 0 || n_out < 0 || V <= 0 || H <= 0 || tp <= 0) return set_error(QW_ERR_INVALID_ARG, "qw_w4_lm_head: bad sizes");
  if (V % tp) return set_error(QW_ERR_SHAPE, "qw_w4_lm_head: V=%lld %% tp=%d", (long long)V, tp);
  if (n_out == 0) return QW_OK;
  if (n_out >= (int64_t(1) << 21)) return set_error(QW_ERR_SHAPE, "qw_w4_lm_head: 2^21 rows or more");
  if (!last_idx && n_out > T) return set_error(QW_ERR_SHAPE, "qw_w4_lm_head: n_out > T without last_idx");
  const int rc = w4::check_weights("qw_w4_lm_head", codes, scales, V, H, group);
  if (rc) return rc;
  if (!hidden || !logits || !al16(hidden) || !al16(logits))
    return set_error(QW_ERR_INVALID_ARG, "qw_w4_lm_head: null or misaligned hidden or logits");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* x = hidden;
  const size_t need = qw_w4_lm_head_workspace_size(n_out, V, H, tp);
  if ((last_idx || next_tokens) && (!workspace || workspace_bytes < need || !al16(workspace)))
    return set_error(QW_ERR_WORKSPACE, "qw_w4_lm_head: workspace of %zu bytes needed", need);
  if (last_idx) {
    uint8_t* rows = static_cast<uint8_t*>(workspace) + kCounterBytes;
    const int e = launch_gather_rows<bf16>(hidden, T, last_idx, n_out, H, rows, st);
    if (e) return e;
    x = rows;
  }
  int e = w4::linear(static_cast<const bf16*>(x), codes, scales, zeros, static_cast<bf16*>(logits), n_out, V, H, group, 1,
                     QW_GEMM_COLUMN, QW_EPI_NONE, flags, st);
  if (e || !next_tokens) return e;
  if (V % 8 == 0) return launch_argmax<bf16>(logits, n_out, V, next_tokens, st);   // whole 16-byte pieces
  launch_pdl(w4::argmax_kernel, unsigned(n_out), 1024, 0, st, static_cast<const bf16*>(logits), V, next_tokens);
  return check_launch("qw_w4_lm_head");
}
