// Matrix product of bfloat16 operands on the tensor cores (tcgen05, fp32
// accumulators in tensor memory), D[m][n] = sum_k A[m][k]·B[n][k], with the
// linear layer's epilogue.
//
// Persistent CTAs walk over the output tiles.  One warp issues the TMA loads
// of 64-element K blocks into a ring of shared-memory stages, one issues the
// MMAs, eight take finished accumulators out of tensor memory; two
// accumulators alternate, so a tile's epilogue runs under the next tile's
// products.  PAIR: two CTAs of a cluster share one 256 x BN tile
// (tcgen05 cta_group::2): each loads its own 128 rows of A and half of B's
// rows, and the first CTA issues the MMAs for both, which halves the operand
// traffic from L2 per product.  Otherwise a CTA has a 128 x BN tile.
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
//
// What bounds it: with many K blocks the operand bytes that come from L2 (a CTA
// takes 32 KB a K block for its part of the pair's tile and for a 128 x 128
// tile, 24 KB for a 128 x 64 one, in 0.34, 0.28 and 0.255 us, so the pair's
// tile, with two to four times the products for them, is the fast one: 8192
// tokens 4096 -> 4096 from a cold L2 in 165 us, 1.67 PFLOP/s, 0.98 of the
// measured bfloat16 burst rate; one after another under the power cap 215 us,
// as cuBLAS); with few the epilogue (a 256 x 256 tile 4.1 us, about 9.3 with
// GELU and a kept pre-activation).
//
// Outputs.  FAST, when the output's rows are 16-byte aligned: an epilogue
// thread has 32 columns of one row in registers; bias and activation are
// applied there, the residual comes and the results leave through swizzled
// shared-memory tiles of 32 rows x 32 columns by TMA, which clips what is
// outside.  Otherwise the sums are turned through shared memory so that a
// warp stores runs of columns, with bounds checks.
#pragma once

#include <cuda.h>

#include "mqv_layer_common.cuh"
#include "mqv_linear_act.cuh"
#include "mqv_ptx.cuh"

namespace mqv {

constexpr int kGemmBM = 128, kGemmBK = 64;
constexpr int kGemmEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;
// Epilogue staging per warp.  FAST: up to 4 KB of y (32 x 32 fp32) and 2 KB of
// z, two buffers of each where they fit.  Otherwise 32 rows x 16 columns,
// rows 20 floats apart so that 16-byte accesses of eight lanes fall in
// different banks.
constexpr int kGemmEpiPitch = 20;
template <bool FAST>
constexpr int kGemmEpiWarpBytes = FAST ? 8192 : 32 * kGemmEpiPitch * 4;

// How one operand's chunks are fetched.
struct GemmOperand {
  int chunk;                   // I
  int per_pos;                 // chunks per position
  int box;                     // chunks per TMA box: all of a stage's, or 1
  int mn_major;
};

struct GemmMaps {
  CUtensorMap a, b;
  CUtensorMap d, z, residual;  // FAST: y or the partial sums, z, residual
};

struct GemmTcArgs {
  GemmOperand a, b;
  int tiles_m, tiles_n, splits, kblocks;
  int tail_width;              // N tiles of the last band (see gemm_tile)
  int run;                     // K blocks summed by one accumulator at most (see gemm_add_runs)
  FastDiv by_split, by_band, by_tail, by_pos;   // divisions by tiles of a split, of a band, tail_width, col_per_pos
  // output element (row, column c of chunk q = c / col_chunk):
  //   (q / col_per_pos)·pos + row·row_stride + (q % col_per_pos)·col_chunk + c % col_chunk
  int64_t M, pos, row_stride;
  int64_t col_inner, col_pos;  // extent of a position's columns, positions
  int col_chunk, col_shift, col_per_pos;       // col_chunk = 1 << col_shift
  Epilogue e;
  float* part;                 // fp32 sums of split s at part + s·part_stride; null: one split, epilogue here
  int64_t part_stride;
  uint32_t* err;
};

// PAIR: `bar` may be the other CTA's, as a shared::cluster address.
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
            "r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// True in one lane of the (converged) warp.  The code around the issuing
// instructions stays uniform over the warp, which their operands want.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// The whole warp waits, bounded as mbar_wait_bounded, and leaves as one: loads
// and stores of tensor memory want all of its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code,
                                          long long limit = 1ll << 32) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
    if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
      atomicOr(err, code);
      return false;
    }
  return true;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address of `bar` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void gemm_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    mma_f16_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
}

// Arrive on `bar` (PAIR: of both CTAs) once the MMAs issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void gemm_commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    mma_commit(bar);
}

template <bool PAIR>
__device__ __forceinline__ void gemm_tmem_alloc(uint32_t* slot, uint32_t cols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  }
}

template <bool PAIR>
__device__ __forceinline__ void gemm_tmem_free(uint32_t tmem, uint32_t cols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  else
    tmem_dealloc(tmem, cols);
}

// The producer's place in one operand, `rows` tile rows a stage: the chunk
// that the next stage starts at, as (x, p), and the other coordinate.  What a
// stage costs the one issuing thread bounds the whole kernel, so every
// division and product is made once, here.
struct GemmCursor {
  int x, p, mid;
  int boxes, dx, dp, wrap;     // boxes a stage; from one box to the next
  uint32_t bytes;              // of a box
  int dmid;                    // to the next K block; 0: along the chunks
  int per_stage, per_pos, chunk;

  __device__ __forceinline__ GemmCursor(const GemmOperand& o, int rows) {
    const int chunks = (o.mn_major ? rows : kGemmBK) / o.chunk;
    boxes = chunks / o.box;
    bytes = (o.mn_major ? kGemmBK : rows) * o.chunk * o.box * 2;
    dx = o.per_pos == 1 ? 0 : o.chunk;
    dp = o.per_pos == 1 ? o.box : 0;
    wrap = o.per_pos == 1 ? 1 << 30 : o.per_pos * o.chunk;
    dmid = o.mn_major ? kGemmBK : 0;
    per_stage = kGemmBK / o.chunk;
    per_pos = o.per_pos;
    chunk = o.chunk;
  }

  // To tile row `row0` and K block kb.
  __device__ __forceinline__ void seek(int row0, int kb) {
    const int q = dmid ? row0 / chunk : kb * per_stage;
    p = q / per_pos;
    x = (q - p * per_pos) * chunk;
    mid = dmid ? kb * kGemmBK : row0;
  }

  // Loads the stage's share of the K block (in the lane that is elected) and
  // goes on to the next.
  template <bool PAIR>
  __device__ __forceinline__ void load(const CUtensorMap* map, uint32_t dst, uint32_t bar, bool elected) {
    int cx = x, cp = p;
    for (int i = 0; i < boxes; ++i) {
      if (elected) tma_load_3d<PAIR>(dst, map, cx, mid, cp, bar);
      dst += bytes;
      cx += dx;
      cp += dp;
      if (cx >= wrap) {
        cx = 0;
        ++cp;
      }
    }
    mid += dmid;
    if (!dmid) {
      x = cx;
      p = cp;
    }
  }
};

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
  r.split = fdiv(t, g.by_split);
  t -= r.split * g.tiles_m * g.tiles_n;
  const int band = fdiv(t, g.by_band), n0 = band * 8;
  t -= band * 8 * g.tiles_m;
  if (n0 + 8 <= g.tiles_n) {
    r.m = t >> 3;
    r.n = n0 + (t & 7);
  } else {
    r.m = fdiv(t, g.by_tail);
    r.n = n0 + t - r.m * g.tail_width;
  }
  return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map), "r"(src),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the newest N groups have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A staged tile of 32 rows x 32 columns: pieces of `width` columns (of one
// chunk), [piece][row][width], with the swizzle of the rows' size.
// Vectors of 16 bytes; a row's are at `off` for the lane that holds it.
template <int ELEM>
struct GemmStaged {
  static constexpr int kVecs = 2 * ELEM;
  static constexpr uint32_t kBytes = 1024 * ELEM;
  int width;
  uint32_t off[kVecs];

  __device__ __forceinline__ GemmStaged(int chunk, int lane) {
    width = chunk < 32 ? 16 : 32;
    const int shift = (chunk < 32 ? 4 : 5) + (ELEM == 4 ? 2 : 1);    // row bytes = 1 << shift
    const uint32_t mask = (1u << shift) - 16;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const uint32_t b = j * 16, piece = b >> shift;
      const uint32_t a = (piece << (shift + 5)) + (lane << shift) + (b - (piece << shift));
      off[j] = a ^ ((a >> 3) & mask);
    }
  }
};

// A place among the output columns: batch item or channel n of position p.
struct GemmColumn {
  int n, p;
  __device__ __forceinline__ void seek(const GemmTcArgs& g, int col) {
    const int q = col >> g.col_shift;
    p = fdiv(q, g.by_pos);
    n = ((q - p * g.col_per_pos) << g.col_shift) + (col & (g.col_chunk - 1));
  }
  __device__ __forceinline__ void next(const GemmTcArgs& g, int by) {
    n += by;
    if (n >= g.col_per_pos * g.col_chunk) {
      n = 0;
      ++p;
    }
  }
};

// TMA of one staged tile (a load into it or a store from it), rows from row0;
// one box where a chunk is a whole position, else one per piece.
template <bool LOAD, int ELEM>
__device__ __forceinline__ void gemm_move(const GemmTcArgs& g, const CUtensorMap* map, int width, uint32_t smem,
                                          GemmColumn c, int row0, int split, uint64_t* bar) {
  const int step = g.col_per_pos == 1 ? 32 : width;
  for (int i = 0; i < 32; i += step) {
    const uint32_t at = smem + i * 32 * ELEM;
    if constexpr (LOAD)
      tma_load_4d(at, map, c.n, row0, c.p, split, bar);
    else
      tma_store_4d(map, at, c.n, row0, c.p, split);
    if (step < 32) c.next(g, width);
  }
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Stages the lane's row of 32 values as BF16 or fp32.
template <bool BF>
__device__ __forceinline__ void stage_row(uint32_t tile, const GemmStaged<BF ? 2 : 4>& st, const float (&v)[32]) {
  if constexpr (BF) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4(tile + st.off[j], pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                   pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      st_shared_v4(tile + st.off[j], __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                   __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
  }
}

// One warp's share of a finished tile, FAST: rows row0 .. row0 + 31 of
// columns col0 .. col0 + COLS - 1 (of the tile's tensor-memory columns from
// `tmem`), y (or the partial sums) as BF16 or fp32.  `used` counts the staged
// tiles this warp has filled; `bars`: its two residual barriers; `acc`: the
// barrier of the accumulator, waited for here; `bias_s`: 32 floats of the
// warp's own shared memory; `release` is called once the accumulator is read.
// 0, or if a wait gave up 1 + the residual loads, from `used` on, that it left
// in flight.
template <int COLS, bool BF, typename F>
__device__ __forceinline__ int gemm_epilogue_fast(const GemmTcArgs& g, const GemmMaps& maps, uint32_t tmem, uint32_t smem,
                                                  int row0, int col0, int split, uint32_t& used, uint64_t* bars,
                                                  uint64_t* acc, uint32_t acc_parity, float* bias_s, F release) {
  const int lane = threadIdx.x & 31;
  const GemmStaged<BF ? 2 : 4> sy(g.col_chunk, lane);
  const GemmStaged<2> sz(g.col_chunk, lane);
  const bool part = g.part != nullptr;
  const bool keep_z = !part && g.e.z.p, res = !part && g.e.residual;
  const bool bias_row = !part && g.e.bias && g.e.bias_on_row, bias_col = !part && g.e.bias && !g.e.bias_on_row;
  // y tiles: four or (with z) two of 2 KB, or two or (with z) one of 4 KB; z in
  // the upper half of the warp's 8 KB
  const bool two = BF || !keep_z;
  const uint32_t ring = (BF ? 4 : 2) / (keep_z ? 2 : 1) - 1;
  GemmColumn c;
  c.seek(g, col0);
  auto y_tile = [&](uint32_t i) { return smem + (i & ring) * sy.kBytes; };
  auto z_tile = [&](uint32_t i) { return smem + 4096 + (two ? (i & 1) * 2048 : 0); };
  auto load_residual = [&](GemmColumn at, uint32_t i) {
    mbar_arrive_expect_tx(bars + (i & 1), sy.kBytes);
    gemm_move<true, BF ? 2 : 4>(g, &maps.residual, sy.width, y_tile(i), at, row0, 0, bars + (i & 1));
  };
  // what can be had before the products are done: the bias (a lane's row's, or
  // its column of the first step) and, with two buffers, the first step's
  // residual; later steps' bias and residual are loaded one step ahead
  auto column_bias = [&](int k) {
    const int64_t n = static_cast<int64_t>(col0) + k + lane;
    return bias_col && k < COLS && n < g.col_inner ? __ldg(g.e.bias + n) : 0.f;
  };
  float bias = bias_row ? (row0 + lane < g.M ? __ldg(g.e.bias + row0 + lane) : 0.f) : column_bias(0);
  if (res && two && lane == 0) {
    if (ring == 3)
      bulk_wait_read<3>();
    else
      bulk_wait_read<1>();
    load_residual(c, used);
  }
  if (!warp_wait(acc, acc_parity, g.err, 4)) return 1 + (res && two);
  tc_fence_after();
  // not unrolled: the steps' code would not stay in the instruction cache
#pragma unroll 1
  for (int k = 0; k < COLS; k += 32, ++used) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(tmem + k, r);
    GemmColumn nx = c;
    nx.next(g, sy.width);
    if (sy.width < 32) nx.next(g, sy.width);
    if (lane == 0) {
      // this step's buffers (with a residual to come, the next step's too) are
      // free once the stores from them have read them
      if (ring == 3)
        bulk_wait_read<2>();
      else if (two && !res)
        bulk_wait_read<1>();
      else
        bulk_wait_read<0>();
      if (res && !two) load_residual(c, used);
      if (res && two && k + 32 < COLS) load_residual(nx, used + 1);
    }
    if (bias_col) {
      bias_s[lane] = bias;
      bias = column_bias(k + 32);
    }
    tmem_ld_wait();
    if (k + 32 == COLS) {
      tc_fence_before();
      release();
    }
    __syncwarp();
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
    if (bias_col) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 b = *reinterpret_cast<const float4*>(bias_s + 4 * j);
        v[4 * j] += b.x, v[4 * j + 1] += b.y, v[4 * j + 2] += b.z, v[4 * j + 3] += b.w;
      }
    } else if (bias_row) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += bias;
    }
    if (keep_z) stage_row<true>(z_tile(used), sz, v);
    if (!part) act_values(v, g.e.act);
    const uint32_t y = y_tile(used);
    if (res) {
      // barrier `used & 1` completes once every second step
      if (!warp_wait(bars + (used & 1), (used >> 1) & 1, g.err, 2)) return 2 + (two && k + 32 < COLS);
#pragma unroll
      for (int j = 0; j < (BF ? 4 : 8); ++j) {
        const uint4 t = ld_shared_v4(y + sy.off[j]);
        if constexpr (BF) {
          v[8 * j] += bf16_lo(t.x), v[8 * j + 1] += bf16_hi(t.x), v[8 * j + 2] += bf16_lo(t.y), v[8 * j + 3] += bf16_hi(t.y);
          v[8 * j + 4] += bf16_lo(t.z), v[8 * j + 5] += bf16_hi(t.z), v[8 * j + 6] += bf16_lo(t.w), v[8 * j + 7] += bf16_hi(t.w);
        } else {
          v[4 * j] += __uint_as_float(t.x), v[4 * j + 1] += __uint_as_float(t.y);
          v[4 * j + 2] += __uint_as_float(t.z), v[4 * j + 3] += __uint_as_float(t.w);
        }
      }
    }
    stage_row<BF>(y, sy, v);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (row0 < g.M && c.p < g.col_pos) {
        if (keep_z) gemm_move<false, 2>(g, &maps.z, sz.width, z_tile(used), c, row0, 0, nullptr);
        gemm_move<false, BF ? 2 : 4>(g, &maps.d, sy.width, y, c, row0, split, nullptr);
      }
      bulk_commit();
    }
    c = nx;
  }
  return 0;
}

// The tensor cores' running sum truncates: each step of 16 products loses up
// to a step of the sum, 2·2^-24, and always towards zero, so the loss grows with
// the length (positive products, mean loss in units of 2^-24 of the sum: 512
// 1.8, 1024 11, 4096 169, 8192 504; 2-norm of the error on noise 4.7e-7, 1.0e-6,
// 4.4e-6, 9.1e-6).  Sums are therefore made in runs of g.run K blocks; the
// epilogue warps add the runs' sums in registers, rounding to nearest, and put
// the total in the place of the last run's accumulator.  The tensor cores go
// on meanwhile with the other accumulator.  Results kept in fp32, runs of 512
// products: 4.8e-7 off over any length, three to four times what fp32 products
// rounded to nearest are for a few hundred; runs of 1024: 9.9e-7, and 4 %
// faster (8192 tokens 4096 -> 4096, weight gradient: 196 and 188 us).  Results
// in bfloat16, runs of 32768.  `tmem`: the first
// accumulator at the warp's lanes and columns; `nt` counts the CTA's runs.
// False if a wait gave up.
template <int BN, int COLS, typename F>
__device__ __forceinline__ bool gemm_add_runs(const GemmTcArgs& g, uint32_t tmem, int runs, uint32_t& nt,
                                              uint64_t* acc_full, F release) {
  float sum[COLS];
#pragma unroll
  for (int i = 0; i < COLS; ++i) sum[i] = 0.f;
  for (int run = 0; run < runs; ++run) {
    const int buf = nt & 1;
    if (!warp_wait(acc_full + buf, (nt / 2) & 1, g.err, 4)) return false;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < COLS; k += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + buf * BN + k, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[k + i] += __uint_as_float(r[i]);
    }
    if (run + 1 < runs) {
      tc_fence_before();
      release(buf);
      ++nt;
    }
  }
#pragma unroll
  for (int k = 0; k < COLS; k += 32) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(sum[k + i]);
    tmem_st_32x32b_x32(tmem + (nt & 1) * BN + k, r);
  }
  tmem_st_wait();
  return true;
}

// The same without TMA: half of the tile's columns from col0, 16 at a time
// through the warp's staging rows `st`.
template <int COLS, typename F>
__device__ __forceinline__ void gemm_epilogue_any(const GemmTcArgs& g, uint32_t tmem, float* st, int row0, int col0,
                                                  int split, F release) {
  const int lane = threadIdx.x & 31;
  float* part = g.part ? g.part + split * g.part_stride : nullptr;
  GemmColumn c;
  c.seek(g, col0);
#pragma unroll 1
  for (int k = 0; k < COLS; k += 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(tmem + k, r);
    tmem_ld_wait();
    if (k + 16 == COLS) {
      tc_fence_before();
      release();
    }
    __syncwarp();                 // the staging rows are free
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(st + lane * kGemmEpiPitch + 4 * j) =
          make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                      __uint_as_float(r[4 * j + 3]));
    __syncwarp();
    if (c.p < g.col_pos) {
      const int64_t base = c.p * g.pos + c.n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = i * 8 + (lane >> 2), cc = (lane & 3) * 4;
        const float4 v4 = *reinterpret_cast<const float4*>(st + rr * kGemmEpiPitch + cc);
        float v[4] = {v4.x, v4.y, v4.z, v4.w};
        const int64_t row = row0 + rr, n = c.n + cc;
        if (row < g.M && n < g.col_inner)
          epilogue_store4(g.e, part, base + row * g.row_stride + cc, row, n, g.col_inner - n, v);
      }
    }
    c.next(g, 16);
  }
}

// warp_wait's timeout on its own: two barriers, one that has been arrived at,
// which is not to set anything, and one that nothing arrives at.
__global__ void warp_wait_selftest_kernel(uint32_t* err, uint32_t code, uint32_t wrong, long long limit) {
  __shared__ uint64_t bars[2];
  if (threadIdx.x == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    fence_mbar_init();
    mbar_arrive(bars);
  }
  __syncwarp();
  if (!warp_wait(bars, 0, err, wrong, limit) || warp_wait(bars + 1, 0, err, code, limit)) atomicOr(err, wrong);
}

template <int BN, bool PAIR>
constexpr int gemm_b_rows = PAIR ? BN / 2 : BN;
template <int BN, bool PAIR>
constexpr int gemm_stage_bytes = (kGemmBM + gemm_b_rows<BN, PAIR>) * kGemmBK * 2;
template <int BN, bool PAIR>
constexpr int gemm_stages = 163840 / gemm_stage_bytes<BN, PAIR>;
template <int BN, bool PAIR, bool FAST>
constexpr int gemm_smem = 1024 + gemm_stages<BN, PAIR> * gemm_stage_bytes<BN, PAIR> +
                          kGemmEpiWarps * kGemmEpiWarpBytes<FAST> + 1536;

// RUNS: the sums may go in several runs of K blocks.
template <int BN, bool PAIR, bool FAST, bool RUNS>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_tc_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmTcArgs g) {
  constexpr int kStages = gemm_stages<BN, PAIR>, kStageBytes = gemm_stage_bytes<BN, PAIR>;
  constexpr int kBRows = gemm_b_rows<BN, PAIR>, kCtas = PAIR ? 2 : 1;
  constexpr uint32_t kABytes = kGemmBM * kGemmBK * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  // the staging comes first: its tiles are aligned to 1 KB
  uint8_t* stage_epi = smem;
  smem += (kGemmEpiWarps * kGemmEpiWarpBytes<FAST> + 1023) / 1024 * 1024;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* res_full = acc_empty + 2;
  float* bias_s = reinterpret_cast<float*>(res_full + 2 * kGemmEpiWarps);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bias_s + 32 * kGemmEpiWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, kCtas * kGemmEpiWarps);
    }
    for (int w = 0; w < 2 * kGemmEpiWarps; ++w) mbar_init(res_full + w, 1);
    fence_mbar_init();
  }
  if (warp == 1) gemm_tmem_alloc<PAIR>(tmem_slot, 2 * BN);
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the kernel that adds split sums may be set up from here on; it waits for
  // this one's end before it reads them
  pdl_launch_dependents();

  const int tiles = g.tiles_m * g.tiles_n * g.splits;
  const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas;
  // K blocks of split s: an even share, the first kblocks % splits one more
  const int share = g.kblocks / g.splits, extra = g.kblocks % g.splits;

  if (warp == 0) {
    // ---- TMA producer; the stages of a pair are full when both CTAs' bytes
    // have arrived, counted on the first CTA's barriers
    GemmCursor ca(g.a, kGemmBM), cb(g.b, kBRows);
    const uint32_t smem0 = smem_u32(smem), bar0 = PAIR ? cluster_addr(full, 0) : smem_u32(full);
    int s = 0;
    uint32_t round = 0;           // times the ring has been filled
    bool live = true;
    for (int t = first; t < tiles && live; t += step) {
      const GemmTile tl = gemm_tile(g, t);
      const int k0 = tl.split * share + min(tl.split, extra), k1 = k0 + share + (tl.split < extra);
      ca.seek((tl.m * kCtas + rank) * kGemmBM, k0);
      cb.seek(tl.n * BN + rank * kBRows, k0);
      for (int kb = k0; kb < k1; ++kb) {
        if (round > 0 && !warp_wait(empty + s, (round - 1) & 1, g.err, 1)) {
          live = false;
          break;
        }
        const uint32_t dst = smem0 + s * kStageBytes, bar = bar0 + 8 * s;
        const bool elected = elect_one();
        if (rank == 0 && elected) mbar_arrive_expect_tx(full + s, kCtas * kStageBytes);
        ca.load<PAIR>(&maps.a, dst, bar, elected);
        cb.load<PAIR>(&maps.b, dst + kABytes, bar, elected);
        if (++s == kStages) {
          s = 0;
          ++round;
        }
      }
    }
    if (!live && rank == 0)       // given up: the copies in flight still land in shared memory
      for (int j = 0; j < kStages; ++j) {
        const int fills = static_cast<int>(round) + (j < s);
        if (fills > 0) warp_wait(full + j, (fills - 1) & 1, g.err, 2);
      }
    // the last release of each stage is an arrival on this CTA's barriers, from
    // the other one's products in a pair: it is waited for before they go
    for (int j = 0; j < kStages && live; ++j) {
      const int fills = static_cast<int>(round) + (j < s);
      if (fills > 0) live = warp_wait(empty + j, (fills - 1) & 1, g.err, 1);
    }
  } else if (warp == 1 && rank == 0) {
    // ---- MMA issuer
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(g.a.mn_major) << 15) |
                           (static_cast<uint32_t>(g.b.mn_major) << 16) | (static_cast<uint32_t>(BN >> 3) << 17) |
                           (static_cast<uint32_t>((kCtas * kGemmBM) >> 4) << 24);
    const uint64_t da = gemm_desc(g.a), db = gemm_desc(g.b);
    uint32_t sa[4], sb[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      sa[s] = gemm_step(g.a, kGemmBM, s);
      sb[s] = gemm_step(g.b, kBRows, s);
    }
    const uint32_t base0 = smem_u32(smem) >> 4;
    uint32_t nt = 0, round = 0;
    int s = 0;
    bool live = true;
    for (int t = first; t < tiles && live; t += step) {
      const GemmTile tl = gemm_tile(g, t);
      const int kn = share + (tl.split < extra);
      for (int k0 = 0; k0 < kn && live; k0 += RUNS ? g.run : kn, ++nt) {
        const int buf = nt & 1, end = RUNS ? min(k0 + g.run, kn) : kn;
        if (nt >= 2 && !warp_wait(acc_empty + buf, (nt / 2 - 1) & 1, g.err, 4)) {
          live = false;
          break;
        }
        tc_fence_after();
        for (int k = k0; k < end; ++k) {
          if (!warp_wait(full + s, round & 1, g.err, 2)) {
            live = false;
            break;
          }
          tc_fence_after();
          const uint32_t base = base0 + s * (kStageBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              gemm_mma<PAIR>(tmem + buf * BN, da | (base + sa[q]), db | (base + (kABytes >> 4) + sb[q]), idesc,
                             k > k0 || q > 0);
            gemm_commit<PAIR>(empty + s);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ++round;
          }
        }
        if (elect_one()) gemm_commit<PAIR>(acc_full + buf);
        __syncwarp();
      }
    }
  } else if (warp >= 2) {
    // ---- epilogue: warp w reads tensor-memory lanes 32·(w % 4).., half of the columns
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* st = stage_epi + (warp - 2) * kGemmEpiWarpBytes<FAST>;
    uint32_t nt = 0, used = 0;
    for (int t = first; t < tiles; t += step, ++nt) {
      const GemmTile tl = gemm_tile(g, t);
      const int row0 = (tl.m * kCtas + rank) * kGemmBM + quad * 32;
      const int c0 = half * (BN / 2);
      const uint32_t acc0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0;
      // an accumulator is read: the MMA warp may overwrite it
      auto release_buf = [&](int b) {
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_cluster(cluster_addr(acc_empty + b, 0));
          else
            mbar_arrive(acc_empty + b);
        }
      };
      if constexpr (RUNS) {
        const int kn = share + (tl.split < extra);
        if (kn > g.run && !gemm_add_runs<BN, BN / 2>(g, acc0, (kn + g.run - 1) / g.run, nt, acc_full, release_buf)) break;
      }
      const int buf = nt & 1;
      const uint32_t acc = acc0 + buf * BN;
      auto release = [&] { release_buf(buf); };
      if constexpr (FAST) {
        const bool bf = !g.part && g.e.d.bf16;
        uint64_t* bars = res_full + 2 * (warp - 2);
        float* bias = bias_s + 32 * (warp - 2);
        const int col0 = tl.n * BN + c0;
        const int gone = bf ? gemm_epilogue_fast<BN / 2, true>(g, maps, acc, smem_u32(st), row0, col0, tl.split, used, bars,
                                                               acc_full + buf, (nt / 2) & 1, bias, release)
                            : gemm_epilogue_fast<BN / 2, false>(g, maps, acc, smem_u32(st), row0, col0, tl.split, used, bars,
                                                                acc_full + buf, (nt / 2) & 1, bias, release);
        if (gone) {               // given up: the loads in flight still land in shared memory
          for (uint32_t i = used; i < used + gone - 1; ++i) warp_wait(bars + (i & 1), (i >> 1) & 1, g.err, 2);
          break;
        }
      } else {
        if (!warp_wait(acc_full + buf, (nt / 2) & 1, g.err, 4)) break;
        tc_fence_after();
        gemm_epilogue_any<BN / 2>(g, acc, reinterpret_cast<float*>(st), row0, tl.n * BN + c0, tl.split, release);
      }
    }
    if (FAST && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync_all();           // also: no CTA leaves while the other may still signal its barriers
  else
    __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (warp == 1) gemm_tmem_free<PAIR>(tmem, 2 * BN);
}

}  // namespace mqv
