// Matrix product of bfloat16 operands on the tensor cores (tcgen05, fp32
// accumulators in tensor memory), D[m][n] = sum_k A[m][k]·B[n][k], with the
// linear layer's epilogue.
//
// A persistent CTA walks over 128 x BN output tiles.  One warp issues the TMA
// loads of 64-element K blocks into a ring of shared-memory stages, one
// issues the MMAs, eight take finished accumulators out of tensor memory;
// two accumulators alternate, so a tile's epilogue runs under the next
// tile's products.
//
// Operands.  Every operand is a [P][mid][inner] view with `inner` contiguous,
// cut along `inner` into chunks of I elements (I = 64, 32 or 16, the span of
// one swizzled shared-memory row of 2·I bytes); a position has ceil(inner / I)
// chunks, and the chunks of all positions are numbered through.  Either
//   - K lies along the chunks (K-major): a stage holds 64 / I chunks of the
//     tile's rows, [chunk][row][I]; or
//   - the rows of the tile do (MN-major): a stage holds the tile's rows / I
//     chunks of 64 K values, [chunk][k][I].
// Plain matrices are the P = 1 case.  The channel-batch-first tensors come
// in with inner = N: a 3-dimensional TMA box of N batch items, channels and
// whole positions lands as the tile that the MMA reads, whatever N is.
// Everything outside the view reads as zero, in both operands.
#pragma once

#include <cuda.h>

#include "mqv_layer_common.cuh"
#include "mqv_linear_act.cuh"
#include "mqv_ptx.cuh"

namespace mqv {

constexpr int kGemmBM = 128, kGemmBK = 64;
constexpr int kGemmEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;
// epilogue staging: 32 rows x 16 columns per warp, rows 20 floats apart so
// that 16-byte accesses of eight lanes fall in different banks
constexpr int kGemmEpiPitch = 20;
constexpr int kGemmEpiBytes = kGemmEpiWarps * 32 * kGemmEpiPitch * 4;

// How one operand's chunks are fetched.
struct GemmOperand {
  int chunk;                   // I
  int per_pos;                 // chunks per position
  int box;                     // chunks per TMA box: all of a stage's, or 1
  int mn_major;
};

struct GemmTcArgs {
  GemmOperand a, b;
  int tiles_m, tiles_n, splits, kblocks;
  // output element (row, column c of chunk q = c / col_chunk):
  //   (q / col_per_pos)·pos + row·row_stride + (q % col_per_pos)·col_chunk + c % col_chunk
  int64_t M, pos, row_stride;
  int64_t col_inner, col_pos;  // extent of a position's columns, positions
  int col_chunk, col_per_pos;
  Epilogue e;
  float* part;                 // fp32 sums of split s at part + s·part_stride; null: one split, epilogue here
  int64_t part_stride;
  uint32_t* err;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// One stage's share of an operand: `rows` tile rows from chunk or row
// `row0`, K block kb.
__device__ __forceinline__ void gemm_load(const GemmOperand& o, const CUtensorMap* map, uint32_t dst, int rows, int row0,
                                          int kb, uint64_t* bar) {
  const int chunks = (o.mn_major ? rows : kGemmBK) / o.chunk;
  const int first = o.mn_major ? row0 / o.chunk : kb * chunks;
  const int mid = o.mn_major ? kb * kGemmBK : row0;
  const uint32_t bytes = (o.mn_major ? kGemmBK : rows) * o.chunk * 2;
  for (int c = 0; c < chunks; c += o.box) {
    const int q = first + c, p = q / o.per_pos;
    tma_load_3d(dst + c * bytes, map, (q - p * o.per_pos) * o.chunk, mid, p, bar);
  }
}

// Shared-memory descriptor without the start address: swizzle span 2·I bytes,
// 8-row groups 16·I bytes apart, and (MN-major) chunks 64·I elements apart.
__device__ __forceinline__ uint64_t gemm_desc(const GemmOperand& o) {
  const uint64_t lbo = o.mn_major ? (kGemmBK * o.chunk * 2) >> 4 : 1;
  const uint64_t sbo = (16 * o.chunk) >> 4;
  const uint64_t swizzle = o.chunk == 64 ? 2 : o.chunk == 32 ? 4 : 6;
  return (lbo << 16) | (sbo << 32) | (uint64_t{1} << 46) | (swizzle << 61);
}

// Offset (in 16-byte units) of 16-element K step s within a stage's operand.
__device__ __forceinline__ uint32_t gemm_step(const GemmOperand& o, int rows, int s) {
  const int k = s * 16;
  const int bytes = o.mn_major ? k * o.chunk * 2 : (k / o.chunk) * rows * o.chunk * 2 + (k % o.chunk) * 2;
  return bytes >> 4;
}

struct GemmTile {
  int m, n, split;
};

// Tile order: the M tiles of eight N tiles at a time, so that CTAs that run
// together share operand tiles in L2.
__device__ __forceinline__ GemmTile gemm_tile(const GemmTcArgs& g, int t) {
  GemmTile r;
  const int per = g.tiles_m * g.tiles_n;
  r.split = t / per;
  t -= r.split * per;
  const int band = t / (8 * g.tiles_m), n0 = band * 8;
  const int width = min(8, g.tiles_n - n0);
  t -= band * 8 * g.tiles_m;
  r.m = t / width;
  r.n = n0 + t % width;
  return r;
}

template <int BN>
constexpr int gemm_stage_bytes = (kGemmBM + BN) * kGemmBK * 2;
template <int BN>
constexpr int gemm_stages = BN == 256 ? 4 : 6;
template <int BN>
constexpr int gemm_smem = 1024 + gemm_stages<BN> * gemm_stage_bytes<BN> + kGemmEpiBytes + 256;

template <int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ GemmTcArgs g) {
  constexpr int kStages = gemm_stages<BN>, kStageBytes = gemm_stage_bytes<BN>;
  constexpr uint32_t kABytes = kGemmBM * kGemmBK * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  float* stage_epi = reinterpret_cast<float*>(smem + kStages * kStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes + kGemmEpiBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, kGemmEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tiles = g.tiles_m * g.tiles_n * g.splits;
  // K blocks of split s: an even share, the first kblocks % splits one more
  const int share = g.kblocks / g.splits, extra = g.kblocks % g.splits;

  if (warp == 0 && lane == 0) {
    // ---- TMA producer
    uint32_t it = 0;
    bool live = true;
    for (int t = blockIdx.x; t < tiles && live; t += gridDim.x) {
      const GemmTile tl = gemm_tile(g, t);
      const int k0 = tl.split * share + min(tl.split, extra), k1 = k0 + share + (tl.split < extra);
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = it % kStages;
        if (it >= kStages && !mbar_wait_bounded(empty + s, (it / kStages - 1) & 1, g.err, 1)) {
          live = false;
          break;
        }
        const uint32_t dst = smem_u32(smem + s * kStageBytes);
        mbar_arrive_expect_tx(full + s, kStageBytes);
        gemm_load(g.a, &map_a, dst, kGemmBM, tl.m * kGemmBM, kb, full + s);
        gemm_load(g.b, &map_b, dst + kABytes, BN, tl.n * BN, kb, full + s);
      }
    }
    if (!live)                    // given up: the copies in flight still land in this CTA's memory
      for (uint32_t j = it < kStages ? 0 : it - kStages; j < it; ++j)
        mbar_wait_bounded(full + j % kStages, (j / kStages) & 1, g.err, 2);
  } else if (warp == 1 && lane == 0) {
    // ---- MMA issuer
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(g.a.mn_major) << 15) |
                           (static_cast<uint32_t>(g.b.mn_major) << 16) | (static_cast<uint32_t>(BN >> 3) << 17) |
                           (static_cast<uint32_t>(kGemmBM >> 4) << 24);
    const uint64_t da = gemm_desc(g.a), db = gemm_desc(g.b);
    uint32_t sa[4], sb[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      sa[s] = gemm_step(g.a, kGemmBM, s);
      sb[s] = gemm_step(g.b, BN, s);
    }
    uint32_t it = 0, nt = 0;
    bool live = true;
    for (int t = blockIdx.x; t < tiles && live; t += gridDim.x, ++nt) {
      const GemmTile tl = gemm_tile(g, t);
      const int kn = share + (tl.split < extra);
      const int buf = nt & 1;
      if (nt >= 2 && !mbar_wait_bounded(acc_empty + buf, (nt / 2 - 1) & 1, g.err, 4)) {
        live = false;
        break;
      }
      tc_fence_after();
      for (int k = 0; k < kn; ++k, ++it) {
        const int s = it % kStages;
        if (!mbar_wait_bounded(full + s, (it / kStages) & 1, g.err, 2)) {
          live = false;
          break;
        }
        tc_fence_after();
        const uint32_t base = smem_u32(smem + s * kStageBytes) >> 4;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma_f16_ss(tmem + buf * BN, da | (base + sa[q]), db | (base + (kABytes >> 4) + sb[q]), idesc, k > 0 || q > 0);
        mma_commit(empty + s);
      }
      mma_commit(acc_full + buf);
    }
  } else if (warp >= 2) {
    // ---- epilogue: warp w reads tensor-memory lanes 32·(w % 4).., half of the columns
    const int quad = warp & 3, half = (warp - 2) >> 2;
    float* st = stage_epi + (warp - 2) * 32 * kGemmEpiPitch;
    uint32_t nt = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++nt) {
      const GemmTile tl = gemm_tile(g, t);
      const int buf = nt & 1;
      if (!mbar_wait_bounded(acc_full + buf, (nt / 2) & 1, g.err, 4)) break;
      tc_fence_after();
      const int64_t row0 = static_cast<int64_t>(tl.m) * kGemmBM + quad * 32;
      float* part = g.part ? g.part + tl.split * g.part_stride : nullptr;
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem + buf * BN + (static_cast<uint32_t>(quad * 32) << 16) + c, r);
        tmem_ld_wait();
        if (c + 16 == (half + 1) * (BN / 2)) {
          // the accumulator is read: the MMA warp may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty + buf);
        }
        __syncwarp();             // the staging rows are free
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(st + lane * kGemmEpiPitch + 4 * j) =
              make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                          __uint_as_float(r[4 * j + 3]));
        __syncwarp();
        // column group: 16 columns of one chunk
        const int col = tl.n * BN + c, q = col / g.col_chunk, p = q / g.col_per_pos;
        const int64_t n0 = static_cast<int64_t>(q - p * g.col_per_pos) * g.col_chunk + col % g.col_chunk;
        if (p >= g.col_pos) continue;
        const int64_t base = p * g.pos + n0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2), cc = (lane & 3) * 4;
          const float4 v4 = *reinterpret_cast<const float4*>(st + rr * kGemmEpiPitch + cc);
          float v[4] = {v4.x, v4.y, v4.z, v4.w};
          const int64_t row = row0 + rr, n = n0 + cc;
          if (row < g.M && n < g.col_inner)
            epilogue_store4(g.e, part, base + row * g.row_stride + cc, row, n, g.col_inner - n, v);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * BN);
}

}  // namespace mqv
