// Layer norm over the channels of a [P][C][N] tensor, forward and backward.
//   mean = sum_c x / C, rstd = (sum_c (x - mean)^2 / C + eps)^(-1/2),
//   y = (x - mean)·rstd·gamma + beta;
//   with xh = (x - mean)·rstd and g = gamma·gy:
//   gx = rstd·(g - sum_c g / C - xh·sum_c (g·xh) / C),
//   ggamma[c] = sum_{p,n} gy·xh, gbeta[c] = sum_{p,n} gy.
// Memory-bound: each tensor is read once into registers and written once.
// The variance is summed around the mean (a second pass over the registers),
// so a large common offset costs no precision; all sums are fp32.
//   - Rows (N = 1): a group of threads takes a row at a time, a thread K
//     vectors of 8 consecutive channels, or E scalars where rows are no whole
//     number of vectors.
//   - Tiles (N > 1): a group takes the C x TN tile of one position and TN
//     batch items; a thread K vectors of 4 batch items (or scalars), `rows`
//     channels apart, so a warp's loads are runs of whole tile rows.
// What bounds these kernels besides memory is the number of instructions an
// element costs: threads hold many elements, so that the reductions' cost is
// spread, arithmetic is on pairs (fma.rn.f32x2 and its kin: two IEEE
// operations an instruction), and addresses are stepped, not multiplied.
// Rows of vectors are on their way, D rows ahead (three, or one where
// three do not fit), into slots of shared memory that only the thread itself
// uses: loads stay in flight across the reductions, and no barrier is needed
// for them.  Scalars are loaded into registers a row ahead, where there are
// some left.
// The backward groups run over many rows or tiles and keep their channels'
// parameter gradients in registers; a block adds its groups' in order and
// writes one partial row, and column_sum_kernel adds the rows in a fixed order.
//
// Measured, L2 flushed: forward 16384 x 4096 bfloat16 47 us (5.7 TB/s, 0.88 of
// the copy rate), 80 x 80 pixels of 64 channels at batch 16, fp32 to bfloat16,
// 8.7 us (0.72); backward 8192 x 4096 50 us (4.0 TB/s, 0.62: instruction issue
// and latency at the 512 threads an SM that the registers allow), 56 x 56
// pixels of 128 channels at batch 64 in fp32 60 us (0.79), 28 x 28 20 us (2.65
// tiles a group: the last round is not full).  8 instead of 16 values a thread
// at twice the threads are slower (64 us for 8192 x 4096 backward), so are 80
// registers for a third block (76 us, spills), or a prefetch of tiles (no gain).
// The backward instances of 1024 threads (rows of more than 8192 channels and
// the tiles beside them) have 64 registers and spill, 372 to 1124 bytes a
// thread: 3000 x 16384 196 us, where the bytes take 46.
#pragma once

#include "mqv_layer_common.cuh"
#include "mqv_ptx.cuh"

namespace mqv {

struct LnArgs {
  int64_t N;
  int C;
  float eps;
  const float *gamma, *beta;   // null: 1 and 0
  float *mean, *rstd;          // [P][N]; null in the forward pass: not kept
  TensorIn x, gy;
  TensorOut out;               // y, or gx
  float* part;                 // backward: [gridDim.x][2][C]; null: no parameter gradients
  int group;                   // threads of a group, whole warps
  int units;                   // rows or tiles
  // tiles
  int tn, tiles;               // batch items per tile, tiles along the batch
  FastDiv by_tiles;
  int lanes, rows;             // threads along a tile row, channels per step
};

// The threads of one group and its barrier.  MANY: a block may hold several
// groups of more than a warp, each with a barrier of its own (an SM has 64 of
// them, so such blocks are few); otherwise a group is a warp or the block.
template <bool MANY>
struct LnGroup {
  int size, index, tid;
  __device__ __forceinline__ explicit LnGroup(int group) : size(group), index(threadIdx.x / group) {
    tid = threadIdx.x - index * group;
  }
  __device__ __forceinline__ void sync() const {
    if (size == 32)
      __syncwarp();
    else if (MANY)
      asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(size) : "memory");
    else
      __syncthreads();
  }
};

// M sums over a group; every thread gets them.  buf: 32·M floats of the
// group's own, not those of the call before.
template <int M, typename G>
__device__ __forceinline__ void group_sum(const G& g, float (&v)[M], float* buf) {
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = warp_sum(v[m]);
  if (g.size == 32) return;
  const int w = g.tid >> 5, lane = g.tid & 31, warps = g.size >> 5;
  if (lane == 0)
#pragma unroll
    for (int m = 0; m < M; ++m) buf[32 * m + w] = v[m];
  g.sync();
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = warp_sum(lane < warps ? buf[32 * m + lane] : 0.f);
}

// ------------------------------------------------------- vectors as pairs

// V fp32 elements from p as pairs.
template <int H>
__device__ __forceinline__ void load_vector(const float* p, pair_t (&v)[H]) {
#pragma unroll
  for (int i = 0; i < H / 2; ++i) {
    const float4 t = __ldg(reinterpret_cast<const float4*>(p) + i);
    v[2 * i] = pair(t.x, t.y);
    v[2 * i + 1] = pair(t.z, t.w);
  }
}

template <bool VEC, int V, bool BF>
__device__ __forceinline__ void store_pairs(char* p, int64_t apart, bool second, const pair_t (&v)[V / 2]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i == 0 || second) {
        const float e = i ? hi(v[0]) : lo(v[0]);
        if constexpr (BF)
          reinterpret_cast<__nv_bfloat16*>(p)[i * apart] = __float2bfloat16_rn(e);
        else
          reinterpret_cast<float*>(p)[i * apart] = e;
      }
  } else if constexpr (BF) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16(lo(v[i]), hi(v[i]));
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(lo(v[2 * i]), hi(v[2 * i]), lo(v[2 * i + 1]), hi(v[2 * i + 1]));
  }
}

// K vectors of 8 or 4 elements, `step` elements apart, those whose bit in
// `mask` is set; zeros for the others.  All loads are issued before the first
// value is used, and the type is tested once, around them.
template <int V, int K>
__device__ __forceinline__ void load_vectors(const TensorIn& t, int64_t i, int64_t step, uint32_t mask,
                                             pair_t (&v)[K][V / 2]) {
  if (t.bf16) {
    const char* p = static_cast<const char*>(t.p) + i * 2;
    uint32_t w[K][V / 2];
#pragma unroll
    for (int k = 0; k < K; ++k, p += step * 2) {
#pragma unroll
      for (int q = 0; q < V / 2; ++q) w[k][q] = 0;
      if (mask >> k & 1) {
        if constexpr (V == 8) {
          const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
          w[k][0] = r.x, w[k][1] = r.y, w[k][2] = r.z, w[k][3] = r.w;
        } else {
          const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
          w[k][0] = r.x, w[k][1] = r.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int q = 0; q < V / 2; ++q) v[k][q] = pair(bf16_lo(w[k][q]), bf16_hi(w[k][q]));
  } else {
    const char* p = static_cast<const char*>(t.p) + i * 4;
    float4 r[K][V / 4];
#pragma unroll
    for (int k = 0; k < K; ++k, p += step * 4)
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        r[k][q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mask >> k & 1) r[k][q] = __ldg(reinterpret_cast<const float4*>(p) + q);
      }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        v[k][2 * q] = pair(r[k][q].x, r[k][q].y);
        v[k][2 * q + 1] = pair(r[k][q].z, r[k][q].w);
      }
  }
}

// n single elements, `step` elements apart, as they are stored.  The loads are
// unconditional, of the tensor's first element where the bit in `mask` is not
// set, so that none waits for another.
template <int n>
__device__ __forceinline__ void load_raw(const TensorIn& t, int64_t i, int64_t step, uint32_t mask, uint32_t (&h)[n]) {
  if (t.bf16) {
#pragma unroll
    for (int k = 0; k < n; ++k, i += step) h[k] = __ldg(static_cast<const uint16_t*>(t.p) + (mask >> k & 1 ? i : 0));
  } else {
#pragma unroll
    for (int k = 0; k < n; ++k, i += step) h[k] = __ldg(static_cast<const uint32_t*>(t.p) + (mask >> k & 1 ? i : 0));
  }
}

// Their values, zeros where the bit in `mask` is not set.
template <int n>
__device__ __forceinline__ void raw_values(const TensorIn& t, uint32_t mask, const uint32_t (&h)[n], float (&f)[n]) {
  const int shift = t.bf16 ? 16 : 0;
#pragma unroll
  for (int k = 0; k < n; ++k) f[k] = mask >> k & 1 ? __uint_as_float(h[k] << shift) : 0.f;
}

template <int n>
__device__ __forceinline__ void load_scalars(const TensorIn& t, int64_t i, int64_t step, uint32_t mask, float (&f)[n]) {
  uint32_t h[n];
  load_raw<n>(t, i, step, mask, h);
  raw_values<n>(t, mask, h, f);
}

// A row thread's K vectors of 8, or 2·K scalars.
template <bool VEC, int V, int K>
__device__ __forceinline__ void load_all(const TensorIn& t, int64_t i, int64_t step, uint32_t mask, pair_t (&v)[K][V / 2]) {
  if constexpr (VEC) {
    load_vectors<V, K>(t, i, step, mask, v);
  } else {
    float f[2 * K];
    load_scalars<2 * K>(t, i, step, mask, f);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k][0] = pair(f[2 * k], f[2 * k + 1]);
  }
}

template <bool VEC, int V, int K>
__device__ __forceinline__ void store_all(const TensorOut& t, int64_t i, int64_t step, uint32_t mask,
                                          const pair_t (&v)[K][V / 2]) {
  const int64_t hop = VEC ? step : 2 * step;
  if (t.bf16) {
    char* p = static_cast<char*>(t.p) + i * 2;
#pragma unroll
    for (int k = 0; k < K; ++k, p += hop * 2)
      if (mask >> (VEC ? k : 2 * k) & 1) store_pairs<VEC, V, true>(p, step, mask >> (2 * k + 1) & 1, v[k]);
  } else {
    char* p = static_cast<char*>(t.p) + i * 4;
#pragma unroll
    for (int k = 0; k < K; ++k, p += hop * 4)
      if (mask >> (VEC ? k : 2 * k) & 1) store_pairs<VEC, V, false>(p, step, mask >> (2 * k + 1) & 1, v[k]);
  }
}

// Bits of the `n` items, `step` apart from `first`, that are below `end`.
__device__ __forceinline__ uint32_t items_below(int first, int step, int n, int end) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) m |= static_cast<uint32_t>(first + i * step < end) << i;
  return m;
}

// --------------------------------------------------- prefetched row vectors
//
// A thread's K vectors of 8 elements of one tensor, as 16-byte pieces; piece j
// of the block's thread t lies at (j·blockDim + t)·16 in the tensor's slot.

template <int K>
__device__ __forceinline__ void slot_fetch(const TensorIn& t, int64_t i, int step, uint32_t mask, uint32_t slot) {
  const uint32_t hop = blockDim.x * 16;
  slot += threadIdx.x * 16;
  if (t.bf16) {
    const char* p = static_cast<const char*>(t.p) + i * 2;
#pragma unroll
    for (int k = 0; k < K; ++k, p += step * 2)
      if (mask >> k & 1) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + k * hop), "l"(p) : "memory");
  } else {
    const char* p = static_cast<const char*>(t.p) + i * 4;
#pragma unroll
    for (int k = 0; k < K; ++k, p += step * 4)
      if (mask >> k & 1) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + 2 * k * hop), "l"(p) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + (2 * k + 1) * hop), "l"(p + 16) : "memory");
      }
  }
}

template <int K>
__device__ __forceinline__ void slot_read(const TensorIn& t, uint32_t mask, uint32_t slot, pair_t (&v)[K][4]) {
  const uint32_t hop = blockDim.x * 16;
  slot += threadIdx.x * 16;
  if (t.bf16) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (mask >> k & 1) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(slot + k * hop) : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
      }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (mask >> k & 1) {
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[k][0]), "=l"(v[k][1]) : "r"(slot + 2 * k * hop) : "memory");
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[k][2]), "=l"(v[k][3]) : "r"(slot + (2 * k + 1) * hop) : "memory");
      }
  }
}

__device__ __forceinline__ void slot_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest D - 1 groups have arrived.
template <int D>
__device__ __forceinline__ void slot_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory"); }
__device__ __forceinline__ void slot_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ------------------------------------------------------------------- rows
//
// VEC: K vectors of V = 8 channels a thread, else K pairs of scalars (V = 2).

// D: rows in flight; B: blocks an SM that the registers must allow; KEEP:
// gamma and beta stay in registers, where there are some left, else they are
// read again for each row (from L1); EXACT: every thread has all K vectors,
// and nothing is tested.
template <bool VEC, int K, int T, int B, int D, bool KEEP, bool EXACT>
__global__ void __launch_bounds__(T, B) ln_fwd_row_kernel(const LnArgs a) {
  constexpr int V = VEC ? 8 : 2, kItems = VEC ? K : 2 * K;
  extern __shared__ __align__(16) uint8_t slots[];
  __shared__ float bufs[T / 32][2][32];
  const LnGroup<false> grp(a.group);
  const int groups = blockDim.x / grp.size;
  const int C = a.C, step = grp.size * (VEC ? V : 1), c0 = grp.tid * (VEC ? V : 1);
  const float inv = 1.f / C;
  const uint32_t mask = EXACT ? ~0u : items_below(c0, step, kItems, C);
  const uint32_t s0 = smem_u32(slots), slot_bytes = K * blockDim.x * (a.x.bf16 ? 16 : 32);
  const int first = blockIdx.x * groups + grp.index, hop = gridDim.x * groups;
  auto fetch = [&](int p, uint32_t slot) {
    if constexpr (VEC) {
      if (p < a.units) slot_fetch<K>(a.x, static_cast<int64_t>(p) * C + c0, step, mask, slot);
      slot_commit();
    }
  };
  pair_t gam[K][V / 2], bet[K][V / 2];
  auto parameters = [&] {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        gam[k][i] = pair(1.f, 1.f);
        bet[k][i] = 0;
      }
    if (a.gamma) load_all<VEC, V, K>(TensorIn{a.gamma, 0}, c0, step, mask, gam);
    if (a.beta) load_all<VEC, V, K>(TensorIn{a.beta, 0}, c0, step, mask, bet);
  };
  if constexpr (KEEP) parameters();
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(first + i * hop, s0 + i * slot_bytes);
  // a row's scalars are loaded a row ahead where registers allow (2000 x 8191:
  // 34 us, 39 without; 8192 x 255: 6.3 and 6.6; with three blocks of 256
  // threads, 4097 x 1023: 13 us, 11 without)
  constexpr bool kAhead = !VEC && (K == 4 || T == 512);
  constexpr int kRaw = kAhead ? 2 * K : 1;
  uint32_t next[kRaw];
  auto ahead = [&](int p) {
    if constexpr (kAhead)
      if (p < a.units) load_raw<kRaw>(a.x, static_cast<int64_t>(p) * C + c0, step, mask, next);
  };
  ahead(first);
  int turn = 0;
  for (int p = first; p < a.units; p += hop) {
    const int64_t at = static_cast<int64_t>(p) * C + c0;
    const uint32_t slot = s0 + turn * slot_bytes;
    turn = turn + 1 < D ? turn + 1 : 0;
    pair_t v[K][V / 2];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) v[k][i] = 0;
    if constexpr (VEC) {
      slot_wait<D>();
      slot_read<K>(a.x, mask, slot, v);
    } else if constexpr (kAhead) {
      float f[kRaw];
      raw_values<kRaw>(a.x, mask, next, f);
#pragma unroll
      for (int k = 0; k < K; ++k) v[k][0] = pair(f[2 * k], f[2 * k + 1]);
    } else {
      load_all<VEC, V, K>(a.x, at, step, mask, v);
    }
    ahead(p + hop);
    pair_t t = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) t = add2(t, v[k][i]);
    float s[1] = {lo(t) + hi(t)};
    group_sum(grp, s, bufs[grp.index][0]);
    fetch(p + D * hop, slot);               // what was there is in registers
    const float mean = s[0] * inv;
    const pair_t minus = pair(-mean, -mean);
    t = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (mask >> (VEC ? k : 2 * k) & 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[k][i] = add2(v[k][i], minus);
        if (!VEC && !(mask >> (2 * k + 1) & 1)) v[k][0] = pair(lo(v[k][0]), 0.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) t = fma2(v[k][i], v[k][i], t);
      }
    s[0] = lo(t) + hi(t);
    group_sum(grp, s, bufs[grp.index][1]);
    const float rstd = rsqrtf(s[0] * inv + a.eps);
    if (grp.tid == 0 && a.mean) {
      a.mean[p] = mean;
      a.rstd[p] = rstd;
    }
    const pair_t r2 = pair(rstd, rstd);
    if constexpr (!KEEP) parameters();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) v[k][i] = fma2(mul2(v[k][i], r2), gam[k][i], bet[k][i]);
    store_all<VEC, V, K>(a.out, at, step, mask, v);
  }
}

// A block's partial row: the groups' sums of a channel added in their order.
// `put(acc)` adds the calling thread's own sums to acc[2][C].
template <typename G, typename F>
__device__ __forceinline__ void write_partial(const LnArgs& a, const G& grp, int turns, int turn, float* acc, F put) {
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.C; i += blockDim.x) acc[i] = 0.f;
  __syncthreads();
  const int groups = blockDim.x / grp.size;
  for (int g = 0; g < groups; ++g)
    for (int t = 0; t < turns; ++t) {
      if (grp.index == g && turn == t) put(acc);
      __syncthreads();
    }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
  for (int i = threadIdx.x; i < 2 * a.C; i += blockDim.x) part[i] = acc[i];
}

template <bool VEC, int K, int T, int B, int D, bool EXACT>
__global__ void __launch_bounds__(T, B) ln_bwd_row_kernel(const LnArgs a) {
  constexpr int V = VEC ? 8 : 2, kItems = VEC ? K : 2 * K;
  extern __shared__ __align__(16) uint8_t slots[];
  __shared__ float bufs[T / 32][2][64];
  const LnGroup<true> grp(a.group);
  const int groups = blockDim.x / grp.size;
  const int C = a.C, step = grp.size * (VEC ? V : 1), c0 = grp.tid * (VEC ? V : 1);
  const float inv = 1.f / C;
  const uint32_t mask = EXACT ? ~0u : items_below(c0, step, kItems, C);
  const uint32_t s0 = smem_u32(slots), x_bytes = K * blockDim.x * (a.x.bf16 ? 16 : 32);
  const uint32_t slot_bytes = x_bytes + K * blockDim.x * (a.gy.bf16 ? 16 : 32);
  const int first = blockIdx.x * groups + grp.index, hop = gridDim.x * groups;
  auto fetch = [&](int p, uint32_t slot) {
    if constexpr (VEC) {
      if (p < a.units) {
        const int64_t at = static_cast<int64_t>(p) * C + c0;
        slot_fetch<K>(a.x, at, step, mask, slot);
        slot_fetch<K>(a.gy, at, step, mask, slot + x_bytes);
      }
      slot_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(first + i * hop, s0 + i * slot_bytes);
  // ag, ab: sums of gy·xh and gy.  Vectors of gamma come in again for each row
  // (from L1), which leaves the registers to more warps; scalars would wait for
  // one another, and are kept
  pair_t ag[K][V / 2], ab[K][V / 2], gam[VEC ? 1 : K][V / 2];
  if constexpr (!VEC) {
#pragma unroll
    for (int k = 0; k < K; ++k) gam[k][0] = pair(1.f, 1.f);
    if (a.gamma) load_all<VEC, V, K>(TensorIn{a.gamma, 0}, c0, step, mask, gam);
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) ag[k][i] = ab[k][i] = 0;
  // a row's statistics, and its scalars, are loaded a row ahead (8192 x 4096:
  // 50 us, 55 without; 4097 x 1023: 15 and 20; 2000 x 4095: 24 and 36); not
  // with sixteen scalars a thread, which leave no registers for it (2000 x
  // 8191: 69 us, 64 without)
  constexpr bool kStats = VEC || K <= 4, kAhead = !VEC && K <= 4;
  constexpr int kRaw = kAhead ? 2 * K : 1;
  float mean_next = 0.f, rstd_next = 0.f;
  uint32_t x_next[kRaw], g_next[kRaw];
  auto ahead = [&](int p) {
    if (!kStats || p >= a.units) return;
    mean_next = __ldg(a.mean + p);
    rstd_next = __ldg(a.rstd + p);
    if constexpr (kAhead) {
      const int64_t at = static_cast<int64_t>(p) * C + c0;
      load_raw<kRaw>(a.x, at, step, mask, x_next);
      load_raw<kRaw>(a.gy, at, step, mask, g_next);
    }
  };
  ahead(first);
  int turn = 0, odd = 0;
  for (int p = first; p < a.units; p += hop, odd ^= 1) {
    const int64_t at = static_cast<int64_t>(p) * C + c0;
    const uint32_t slot = s0 + turn * slot_bytes;
    turn = turn + 1 < D ? turn + 1 : 0;
    const float mean = kStats ? mean_next : __ldg(a.mean + p), rstd = kStats ? rstd_next : __ldg(a.rstd + p);
    pair_t x[K][V / 2], g[K][V / 2];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) x[k][i] = g[k][i] = 0;
    if constexpr (VEC) {
      slot_wait<D>();
      slot_read<K>(a.x, mask, slot, x);
      slot_read<K>(a.gy, mask, slot + x_bytes, g);
    } else if constexpr (kAhead) {
      float f[kRaw];
      raw_values<kRaw>(a.x, mask, x_next, f);
#pragma unroll
      for (int k = 0; k < K; ++k) x[k][0] = pair(f[2 * k], f[2 * k + 1]);
      raw_values<kRaw>(a.gy, mask, g_next, f);
#pragma unroll
      for (int k = 0; k < K; ++k) g[k][0] = pair(f[2 * k], f[2 * k + 1]);
    } else {
      load_all<VEC, V, K>(a.x, at, step, mask, x);
      load_all<VEC, V, K>(a.gy, at, step, mask, g);
    }
    ahead(p + hop);
    const pair_t minus = pair(-mean, -mean), r2 = pair(rstd, rstd);
    pair_t t1 = 0, t2 = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        x[k][i] = mul2(add2(x[k][i], minus), r2);          // outside the row: gy is 0
        ag[k][i] = fma2(g[k][i], x[k][i], ag[k][i]);
        ab[k][i] = add2(ab[k][i], g[k][i]);
      }
    if constexpr (!VEC) {
#pragma unroll
      for (int k = 0; k < K; ++k) g[k][0] = mul2(g[k][0], gam[k][0]);
    } else if (a.gamma) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (mask >> k & 1) {
          pair_t w[V / 2];
          load_vector(a.gamma + c0 + k * step, w);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) g[k][i] = mul2(g[k][i], w[i]);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        t1 = add2(t1, g[k][i]);
        t2 = fma2(g[k][i], x[k][i], t2);
      }
    float s[2] = {lo(t1) + hi(t1), lo(t2) + hi(t2)};
    group_sum(grp, s, bufs[grp.index][odd]);
    fetch(p + D * hop, slot);
    const pair_t m1 = pair(-s[0] * inv, -s[0] * inv), m2 = pair(-s[1] * inv, -s[1] * inv);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) g[k][i] = mul2(r2, fma2(x[k][i], m2, add2(g[k][i], m1)));
    store_all<VEC, V, K>(a.out, at, step, mask, g);
  }
  slot_wait_all();
  pdl_launch_dependents();
  if (!a.part) return;
  write_partial(a, grp, 1, 0, reinterpret_cast<float*>(slots), [&](float* acc) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = c0 + (VEC ? k * step + e : (2 * k + e) * step);
        if (c < C) {
          acc[c] += e & 1 ? hi(ag[k][e / 2]) : lo(ag[k][e / 2]);
          acc[C + c] += e & 1 ? hi(ab[k][e / 2]) : lo(ab[k][e / 2]);
        }
      }
  });
}

// ------------------------------------------------------------------ tiles
//
// VEC: a thread's items are vectors of V = 4 batch items, else single ones
// (V = 1, held as half a pair).

template <int M>
__device__ __forceinline__ void read_floats(const float* p, float (&v)[M]) {
  if constexpr (M % 4 == 0) {
#pragma unroll
    for (int q = 0; q < M / 4; ++q) {
      const float4 f = reinterpret_cast<const float4*>(p)[q];
      v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = p[m];
  }
}

// Floats that tile_sum needs for `values` sums a thread: the warps' sums and
// their totals where the lanes divide a warp, else the threads' sums.
__host__ __device__ inline bool tile_sum_by_warps(int lanes) { return lanes <= 32 && (lanes & (lanes - 1)) == 0; }
__host__ __device__ inline int tile_sum_floats(int lanes, int size, int values) {
  return values * (tile_sum_by_warps(lanes) ? (size / 32 + 1) * lanes : size);
}

// Sums M values over the threads of a group that share a tile column (same
// thread index modulo `lanes`); every active thread gets its column's sums.
// buf: tile_sum_floats of the group's own, not those of the call before.
template <int M, typename G>
__device__ __forceinline__ void tile_sum(float (&v)[M], const G& g, int lanes, int rows, float* buf) {
  if (tile_sum_by_warps(lanes)) {
    // lanes divide a warp: first over the warp, then over the warps
    for (int o = 16; o >= lanes; o >>= 1)
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    const int warps = g.size >> 5;
    if (warps == 1) return;
    const int w = g.tid >> 5, l = g.tid & 31;
    if (l < lanes)
#pragma unroll
      for (int m = 0; m < M; ++m) buf[(w * lanes + l) * M + m] = v[m];
    g.sync();
    const int c = l & (lanes - 1), width = lanes * M;
    if (warps > 4) {
      // many warps: each sum by one thread, then read by all
      float* total = buf + warps * width;
      for (int i = g.tid; i < width; i += g.size) {
        float f = 0.f;
        for (int k = 0; k < warps; ++k) f += buf[k * width + i];
        total[i] = f;
      }
      g.sync();
      read_floats<M>(total + c * M, v);
      return;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = 0.f;
    for (int i = 0; i < warps; ++i) {
      float t[M];
      read_floats<M>(buf + i * width + c * M, t);
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += t[m];
    }
    return;
  }
  const int t = g.tid, r = t / lanes;
  const bool act = r < rows;
  if (act)
#pragma unroll
    for (int m = 0; m < M; ++m) buf[m * g.size + t] = v[m];
  for (int n = rows; n > 1;) {
    const int half = (n + 1) / 2;
    g.sync();
    if (r < n - half)
#pragma unroll
      for (int m = 0; m < M; ++m) buf[m * g.size + t] += buf[m * g.size + t + half * lanes];
    n = half;
  }
  g.sync();
  if (act)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = buf[m * g.size + t % lanes];
}

// V values as pairs, and back.
template <int V>
__device__ __forceinline__ void spread(const pair_t (&t)[(V + 1) / 2], float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = e & 1 ? hi(t[e / 2]) : lo(t[e / 2]);
}
template <int V>
__device__ __forceinline__ void gather(const float* v, pair_t (&t)[(V + 1) / 2]) {
#pragma unroll
  for (int e = 0; e < V; e += 2) t[e / 2] = pair(v[e], e + 1 < V ? v[e + 1] : 0.f);
}

// K items of V elements, `step` elements apart.
template <int V, int K>
__device__ __forceinline__ void load_items(const TensorIn& t, int64_t i, int64_t step, uint32_t mask,
                                           pair_t (&v)[K][(V + 1) / 2]) {
  if constexpr (V == 4) {
    load_vectors<4, K>(t, i, step, mask, v);
  } else {
    float f[K];
    load_scalars<K>(t, i, step, mask, f);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k][0] = pair(f[k], 0.f);
  }
}
template <int V, int K>
__device__ __forceinline__ void store_items(const TensorOut& t, int64_t i, int64_t step, uint32_t mask,
                                            const pair_t (&v)[K][(V + 1) / 2]) {
  if constexpr (V == 4) {
    store_all<true, 4, K>(t, i, step, mask, v);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k, i += step)
      if (mask >> k & 1) store_vec<1>(t, i, {lo(v[k][0])});
  }
}

// EXACT: every thread has all K items of every tile.
template <int V, int K, int T, bool EXACT>
__global__ void __launch_bounds__(T) ln_fwd_tile_kernel(const LnArgs a) {
  constexpr int H = (V + 1) / 2;
  extern __shared__ __align__(16) float sums[];
  const LnGroup<false> grp(a.group);
  const int u = blockIdx.x * (blockDim.x / grp.size) + grp.index;
  if (u >= a.units) return;                        // a whole group
  const int C = a.C, r = grp.tid / a.lanes, l = grp.tid - r * a.lanes;
  const float inv = 1.f / C;
  const int p = fdiv(u, a.by_tiles);
  const int64_t n = static_cast<int64_t>(u - p * a.tiles) * a.tn + l * V;
  const int sum_floats = tile_sum_floats(a.lanes, grp.size, V);
  float* buf = sums + grp.index * 2 * sum_floats;
  const uint32_t mask = EXACT ? ~0u : r < a.rows && l * V < a.tn && n < a.N ? items_below(r, a.rows, K, C) : 0;
  const int64_t at = (static_cast<int64_t>(p) * C + r) * a.N + n, step = a.rows * a.N;
  pair_t v[K][H], t[H];
  load_items<V, K>(a.x, at, step, mask, v);
  float m[V], q[V];
#pragma unroll
  for (int i = 0; i < H; ++i) t[i] = 0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < H; ++i) t[i] = add2(t[i], v[k][i]);
  spread<V>(t, m);
  tile_sum<V>(m, grp, a.lanes, a.rows, buf);
  float minus[V];
#pragma unroll
  for (int e = 0; e < V; ++e) minus[e] = -(m[e] *= inv);
  pair_t mp[H];
  gather<V>(minus, mp);
#pragma unroll
  for (int i = 0; i < H; ++i) t[i] = 0;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (mask >> k & 1)
#pragma unroll
      for (int i = 0; i < H; ++i) {
        v[k][i] = add2(v[k][i], mp[i]);
        t[i] = fma2(v[k][i], v[k][i], t[i]);
      }
  spread<V>(t, q);
  tile_sum<V>(q, grp, a.lanes, a.rows, buf + sum_floats);
#pragma unroll
  for (int e = 0; e < V; ++e) q[e] = rsqrtf(q[e] * inv + a.eps);
  if (mask && r == 0 && a.mean)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      a.mean[p * a.N + n + e] = m[e];
      a.rstd[p * a.N + n + e] = q[e];
    }
  gather<V>(q, mp);
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (mask >> k & 1) {
      const int c = r + k * a.rows;
      const float g = a.gamma ? __ldg(a.gamma + c) : 1.f, b = a.beta ? __ldg(a.beta + c) : 0.f;
#pragma unroll
      for (int i = 0; i < H; ++i) v[k][i] = fma2(mul2(v[k][i], mp[i]), pair(g, g), pair(b, b));
    }
  store_items<V, K>(a.out, at, step, mask, v);
}

template <int V, int K, int T, int B, bool EXACT>
__global__ void __launch_bounds__(T, B) ln_bwd_tile_kernel(const LnArgs a) {
  constexpr int H = (V + 1) / 2;
  extern __shared__ __align__(16) float sums[];
  const LnGroup<true> grp(a.group);
  const int groups = blockDim.x / grp.size;
  const int C = a.C, r = grp.tid / a.lanes, l = grp.tid - r * a.lanes;
  const float inv = 1.f / C;
  const int64_t step = a.rows * a.N;
  const int sum_floats = tile_sum_floats(a.lanes, grp.size, 2 * V);
  float* buf = sums + grp.index * 2 * sum_floats;  // two, used in turn
  const uint32_t items = EXACT ? ~0u : r < a.rows && l * V < a.tn ? items_below(r, a.rows, K, C) : 0;
  float w[K];
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = a.gamma && (items >> k & 1) ? __ldg(a.gamma + r + k * a.rows) : 1.f;
  float ag[K], ab[K];
#pragma unroll
  for (int k = 0; k < K; ++k) ag[k] = ab[k] = 0.f;
  int turn = 0;
  for (int u = blockIdx.x * groups + grp.index; u < a.units; u += gridDim.x * groups, turn ^= 1) {
    const int p = fdiv(u, a.by_tiles);
    const int64_t n = static_cast<int64_t>(u - p * a.tiles) * a.tn + l * V;
    const uint32_t mask = EXACT || n < a.N ? items : 0;
    const int64_t at = (static_cast<int64_t>(p) * C + r) * a.N + n;
    pair_t x[K][H], g[K][H], mp[H], qp[H], t1[H], t2[H];
    load_items<V, K>(a.x, at, step, mask, x);
    load_items<V, K>(a.gy, at, step, mask, g);
    float m[V], q[V];
    if (mask) {
      load_f32<V>(a.mean, p * a.N + n, m);
      load_f32<V>(a.rstd, p * a.N + n, q);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) m[e] = q[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = -m[e];
    gather<V>(m, mp);
    gather<V>(q, qp);
#pragma unroll
    for (int i = 0; i < H; ++i) t1[i] = t2[i] = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const pair_t wk = pair(w[k], w[k]);
      pair_t tg = 0, tb = 0;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        x[k][i] = mul2(add2(x[k][i], mp[i]), qp[i]);       // outside: gy is 0
        tg = fma2(g[k][i], x[k][i], tg);
        tb = add2(tb, g[k][i]);
        g[k][i] = mul2(g[k][i], wk);
        t1[i] = add2(t1[i], g[k][i]);
        t2[i] = fma2(g[k][i], x[k][i], t2[i]);
      }
      ag[k] += lo(tg) + hi(tg);
      ab[k] += lo(tb) + hi(tb);
    }
    float s[2 * V], s1[V], s2[V];
    spread<V>(t1, s1);
    spread<V>(t2, s2);
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = s1[e], s[V + e] = s2[e];
    tile_sum<2 * V>(s, grp, a.lanes, a.rows, buf + turn * sum_floats);
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) s[e] *= -inv;
    gather<V>(s, t1);
    gather<V>(s + V, t2);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < H; ++i) g[k][i] = mul2(qp[i], fma2(x[k][i], t2[i], add2(g[k][i], t1[i])));
    store_items<V, K>(a.out, at, step, mask, g);
  }
  pdl_launch_dependents();
  if (!a.part) return;
  // a channel's sums over the lanes of its row, then over the groups
  int turns = a.lanes;
  if (tile_sum_by_warps(a.lanes)) {
    for (int o = a.lanes >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        ag[k] += __shfl_xor_sync(0xffffffffu, ag[k], o);
        ab[k] += __shfl_xor_sync(0xffffffffu, ab[k], o);
      }
    turns = 1;
  }
  write_partial(a, grp, turns, l, sums, [&](float* acc) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = r + k * a.rows;
      if (r < a.rows && c < C) {
        acc[c] += ag[k];
        acc[C + c] += ab[k];
      }
    }
  });
}

}  // namespace mqv
