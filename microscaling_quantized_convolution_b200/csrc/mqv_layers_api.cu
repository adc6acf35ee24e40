// C ABI of the BF16 layers around the quantized convolutions (declared in
// include/mqv.h): layer norm and the linear layer.  Argument validation and
// launch geometry; the arithmetic is in mqv_norm.cuh and mqv_linear.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "mqv.h"
#include "mqv_gemm.cuh"
#include "mqv_host.h"
#include "mqv_linear.cuh"
#include "mqv_norm.cuh"

namespace {

using namespace mqv;

constexpr int kSms = 148;
constexpr int64_t kMaxChannels = 16384;             // layer norm: a position's channels in one block's registers
constexpr int64_t kMaxElements = int64_t{1} << 37;            // TMA strides stay below 2^40 bytes
constexpr int64_t kMaxColumns = (int64_t{1} << 31) - (1 << 16);   // with a tile's overhang still an int

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t b) { return ceil_div(b, 256) * 256; }
int64_t type_size(int32_t t) { return t == MQV_BF16 ? 2 : 4; }

mqv_status check_type(int32_t t, const char* name) {
  if (t != MQV_F32 && t != MQV_BF16) return fail(MQV_ERR_INVALID_ARG, "%s: unknown element type %d", name, t);
  return MQV_OK;
}

// A device buffer of a call: what it is, where, how many bytes; `out` when the
// call writes it, `need` when it may not be null.
struct Buf {
  const char* name;
  const void* p;
  int64_t bytes;
  bool out, need;
};

// Pointers present and 16-byte aligned, no written buffer overlapping another,
// except that `alias` may be exactly the buffer of `of` (element-wise reads
// and writes of the same element by one thread).
mqv_status check_buffers(std::initializer_list<Buf> bufs, const char* alias = nullptr, const char* of = nullptr) {
  for (const Buf& b : bufs) {
    if (b.need && b.bytes > 0 && !b.p) return fail(MQV_ERR_INVALID_ARG, "%s: null pointer", b.name);
    if (b.p && !aligned16(b.p)) return fail(MQV_ERR_INVALID_ARG, "%s must be 16-byte aligned", b.name);
  }
  for (const Buf& a : bufs)
    for (const Buf& b : bufs) {
      if (!a.out || &a == &b || !a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) continue;
      const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
      if (x >= y + b.bytes || y >= x + a.bytes) continue;
      if (alias && x == y && a.bytes == b.bytes && !b.out && a.name == alias && b.name == of) continue;
      return fail(MQV_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
    }
  return MQV_OK;
}

mqv_status check_workspace(const void* ws, size_t have, int64_t need) {
  if (need > 0 && (!ws || have < static_cast<size_t>(need) || !aligned16(ws)))
    return fail(MQV_ERR_WORKSPACE, "workspace of %lld bytes required", (long long)need);
  return MQV_OK;
}

mqv_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ok() : cuda_fail(e, what);
}

// Where a pass goes: to a stream or, for the test hooks, into the text of the
// kernel instances that it would launch.
struct Target {
  cudaStream_t st;
  char* text;                  // null: launch
  size_t size;
  __attribute__((format(printf, 2, 3))) cudaError_t name(const char* fmt, ...) const {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, size, fmt, ap);
    va_end(ap);
    return cudaSuccess;
  }
};

template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<bool> (&done)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  done[dev] = e == cudaSuccess;
  return e;
}

// Launch configuration with the attribute of a programmatic dependent.
struct DependentLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  DependentLaunch(unsigned grid, unsigned block, cudaStream_t st) {
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

void launch_column_sum(const float* part, int64_t rows, int64_t n, int pairs, float* out0, float* out1,
                       cudaStream_t st) {
  DependentLaunch l((unsigned)ceil_div(n * pairs, 32), 1024, st);
  cudaLaunchKernelEx(&l.cfg, column_sum_kernel, part, (int)rows, n, pairs, out0, out1);   // its error: launched()
}

// ------------------------------------------------------------- layer norm

// Launch geometry of one direction: values and items per thread, threads of a
// group, groups of a block and (N > 1) the tile.
struct LnPlan {
  int v, k, group, groups;     // v: vector width; rows of scalars (v = 1) hold 2·k
  int tn, tiles, lanes, rows;
  bool exact;                  // every thread has all its items
  int64_t units, blocks;
  int threads() const { return group * groups; }
};

mqv_status plan_ln(const mqv_ln_desc* d, bool bwd, LnPlan* pl) {
  if (!d) return fail(MQV_ERR_INVALID_ARG, "null descriptor");
  if (d->P < 0 || d->C <= 0 || d->N <= 0 || d->reserved)
    return fail(MQV_ERR_INVALID_ARG, "layer norm of [%lld][%lld][%lld]: P >= 0, C and N > 0, reserved 0 required",
                (long long)d->P, (long long)d->C, (long long)d->N);
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(MQV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (d->C > kMaxChannels)
    return fail(MQV_ERR_UNSUPPORTED, "%lld channels: at most %lld", (long long)d->C, (long long)kMaxChannels);
  if (d->N > kMaxColumns || d->P > kMaxColumns / d->N || (d->P > 0 && d->C > kMaxElements / (d->P * d->N)))
    return fail(MQV_ERR_UNSUPPORTED, "tensor [%lld][%lld][%lld] too large", (long long)d->P, (long long)d->C,
                (long long)d->N);
  *pl = {};
  if (d->N == 1) {
    // 16 values per thread, which with their parameters (and backward the
    // parameters' gradients) is what registers hold at 512 to 768 threads an
    // SM; 8 for short rows, and for scalars backward, where the next row's then
    // fit in registers too (4097 x 1023: 15 us against 21)
    pl->v = d->C % 8 == 0 ? 8 : 1;
    const int e = d->C <= 256 || (bwd && pl->v == 1 && d->C <= 4096) ? 8 : 16;
    pl->k = pl->v == 8 ? e / 8 : e / 2;
    pl->group = (int)(ceil_div(ceil_div(d->C, e), 32) * 32);
    pl->exact = pl->v == 8 && d->C == (int64_t)pl->group * e;
    pl->units = d->P;
  } else {
    // K items of 4 (or 1) batch items a thread; the widest tile (up to 64
    // batch items) whose channels fit in 512 threads, or in 1024 once its
    // rows are down to 16 items
    for (int v : {4, 1}) {
      if (d->N % v || pl->group) continue;
      const int k = v == 1 ? 16 : 8;
      for (int64_t tiles = ceil_div(d->N, 64);; tiles *= 2) {
        const int64_t tn = ceil_div(ceil_div(d->N, tiles), v) * v;
        const int64_t lanes = tn / v, group = ceil_div(lanes * ceil_div(d->C, k), 32) * 32;
        if (group <= 512 || (group <= 1024 && tn <= 16)) {
          pl->v = v;
          pl->k = k;
          pl->group = (int)group;
          pl->tn = (int)tn;
          pl->tiles = (int)ceil_div(d->N, tn);
          pl->lanes = (int)lanes;
          pl->rows = (int)std::min<int64_t>(group / lanes, d->C);
          pl->exact = v == 4 && d->N % tn == 0 && lanes * pl->rows == group && (int64_t)pl->rows * k == d->C;
          break;
        }
        if (tn <= v) break;
      }
    }
    if (!pl->group) return fail(MQV_ERR_UNSUPPORTED, "%lld channels", (long long)d->C);
    pl->units = d->P * pl->tiles;
  }
  // Rows, and tiles backward, run as many blocks as fit (768 threads an SM
  // forward, 512 backward, or one block), each over many units.  Backward,
  // blocks of 256 threads hold several groups, since each block's partial row
  // is to be added.
  pl->groups = bwd ? std::max(1, 256 / pl->group) : pl->group == 32 ? 4 : 1;
  pl->blocks = ceil_div(pl->units, pl->groups);
  if (bwd || d->N == 1) {
    const int64_t fit = pl->threads() > 256 ? 1 : (bwd ? 512 : 768) / pl->threads();
    pl->blocks = std::min<int64_t>(pl->blocks, kSms * fit);
  }
  return MQV_OK;
}

template <typename K>
cudaError_t launch_ln_kernel(K kernel, const LnArgs& a, const LnPlan& pl, int64_t smem, std::atomic<bool> (&done)[kMaxDevices],
                             cudaStream_t st) {
  const cudaError_t e = allow_smem(kernel, 200 * 1024, done);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)pl.blocks, pl.threads(), (size_t)smem, st>>>(a);
  return cudaGetLastError();
}

int64_t slot_bytes(const TensorIn& t, const LnPlan& pl, int depth) {
  return pl.v == 8 ? (int64_t)depth * pl.k * pl.threads() * (t.bf16 ? 16 : 32) : 0;
}

template <bool VEC, int K, int T, int B, bool KEEP, bool EXACT = false>
cudaError_t launch_ln_fwd_rows(const LnArgs& a, const LnPlan& pl, const Target& to) {
  if (to.text) return to.name("launch_ln_fwd_rows<%d, %d, %d, %d, %d, %d>", VEC, K, T, B, KEEP, EXACT);
  static std::atomic<bool> done[kMaxDevices] = {};
  return launch_ln_kernel(ln_fwd_row_kernel<VEC, K, T, B, 3, KEEP, EXACT>, a, pl, slot_bytes(a.x, pl, 3), done, to.st);
}

// The partial row is put together where the slots (or tiles' sums) were.
template <bool VEC, int K, int T, int B, int D, bool EXACT = false>
cudaError_t launch_ln_bwd_rows(const LnArgs& a, const LnPlan& pl, const Target& to) {
  if (to.text) return to.name("launch_ln_bwd_rows<%d, %d, %d, %d, %d, %d>", VEC, K, T, B, D, EXACT);
  static std::atomic<bool> done[kMaxDevices] = {};
  return launch_ln_kernel(ln_bwd_row_kernel<VEC, K, T, B, D, EXACT>, a, pl,
                          std::max(slot_bytes(a.x, pl, D) + slot_bytes(a.gy, pl, D), 2 * (int64_t)a.C * 4), done, to.st);
}

template <int V, int K, int T, bool EXACT = false>
cudaError_t launch_ln_fwd_tiles(const LnArgs& a, const LnPlan& pl, const Target& to) {
  if (to.text) return to.name("launch_ln_fwd_tiles<%d, %d, %d, %d>", V, K, T, EXACT);
  static std::atomic<bool> done[kMaxDevices] = {};
  const int64_t sums = (int64_t)pl.groups * 2 * 4 * tile_sum_floats(pl.lanes, pl.group, V);
  return launch_ln_kernel(ln_fwd_tile_kernel<V, K, T, EXACT>, a, pl, sums, done, to.st);
}

template <int V, int K, int T, int B, bool EXACT = false>
cudaError_t launch_ln_bwd_tiles(const LnArgs& a, const LnPlan& pl, const Target& to) {
  if (to.text) return to.name("launch_ln_bwd_tiles<%d, %d, %d, %d, %d>", V, K, T, B, EXACT);
  static std::atomic<bool> done[kMaxDevices] = {};
  const int64_t sums = (int64_t)pl.groups * 2 * 4 * tile_sum_floats(pl.lanes, pl.group, 2 * V);
  return launch_ln_kernel(ln_bwd_tile_kernel<V, K, T, B, EXACT>, a, pl, std::max(sums, 2 * (int64_t)a.C * 4), done, to.st);
}

// Instances: EXACT ones for the usual widths, the others for the rest.
cudaError_t launch_ln_fwd(const LnArgs& a, const LnPlan& pl, bool rows, const Target& to) {
  const int t = pl.threads();
  if (rows && pl.v == 8) {
    if (pl.k == 1) return launch_ln_fwd_rows<true, 1, 128, 6, true>(a, pl, to);
    if (t <= 256)
      return pl.exact ? launch_ln_fwd_rows<true, 2, 256, 3, true, true>(a, pl, to)
                      : launch_ln_fwd_rows<true, 2, 256, 3, true>(a, pl, to);
    return t <= 512 ? launch_ln_fwd_rows<true, 2, 512, 1, true>(a, pl, to)
                    : launch_ln_fwd_rows<true, 2, 1024, 1, false>(a, pl, to);
  }
  if (rows) {
    if (pl.k == 4) return launch_ln_fwd_rows<false, 4, 128, 6, true>(a, pl, to);
    return t <= 256   ? launch_ln_fwd_rows<false, 8, 256, 3, true>(a, pl, to)
           : t <= 512 ? launch_ln_fwd_rows<false, 8, 512, 1, true>(a, pl, to)
                      : launch_ln_fwd_rows<false, 8, 1024, 1, false>(a, pl, to);
  }
  if (pl.v == 4) {
    if (t > 512) return launch_ln_fwd_tiles<4, 8, 1024>(a, pl, to);
    return pl.exact ? launch_ln_fwd_tiles<4, 8, 512, true>(a, pl, to) : launch_ln_fwd_tiles<4, 8, 512>(a, pl, to);
  }
  return t <= 512 ? launch_ln_fwd_tiles<1, 16, 512>(a, pl, to) : launch_ln_fwd_tiles<1, 16, 1024>(a, pl, to);
}

cudaError_t launch_ln_bwd(const LnArgs& a, const LnPlan& pl, bool rows, const Target& to) {
  const int t = pl.threads();
  if (rows && pl.v == 8) {
    if (pl.k == 1) return launch_ln_bwd_rows<true, 1, 256, 2, 3>(a, pl, to);
    if (t <= 256)
      return pl.exact ? launch_ln_bwd_rows<true, 2, 256, 2, 3, true>(a, pl, to)
                      : launch_ln_bwd_rows<true, 2, 256, 2, 3>(a, pl, to);
    return t <= 512 ? launch_ln_bwd_rows<true, 2, 512, 1, 3>(a, pl, to)
                    : launch_ln_bwd_rows<true, 2, 1024, 1, 1>(a, pl, to);
  }
  if (rows) {
    if (pl.k == 4)
      return t <= 256 ? launch_ln_bwd_rows<false, 4, 256, 2, 1>(a, pl, to)
                      : launch_ln_bwd_rows<false, 4, 512, 1, 1>(a, pl, to);
    // from 4097 channels on: 288 threads or more
    return t <= 512 ? launch_ln_bwd_rows<false, 8, 512, 1, 1>(a, pl, to)
                    : launch_ln_bwd_rows<false, 8, 1024, 1, 1>(a, pl, to);
  }
  if (pl.v == 4) {
    if (t > 512) return launch_ln_bwd_tiles<4, 8, 1024, 1>(a, pl, to);
    if (t > 256) return launch_ln_bwd_tiles<4, 8, 512, 1>(a, pl, to);
    return pl.exact ? launch_ln_bwd_tiles<4, 8, 256, 2, true>(a, pl, to) : launch_ln_bwd_tiles<4, 8, 256, 2>(a, pl, to);
  }
  return t <= 512 ? launch_ln_bwd_tiles<1, 16, 512, 1>(a, pl, to) : launch_ln_bwd_tiles<1, 16, 1024, 1>(a, pl, to);
}

LnArgs ln_args(const mqv_ln_desc* d, const LnPlan& pl, const void* x, int32_t x_type, const float* gamma) {
  LnArgs a = {};
  a.N = d->N;
  a.C = (int)d->C;
  a.eps = d->eps;
  a.gamma = gamma;
  a.x = {x, x_type == MQV_BF16};
  a.group = pl.group;
  a.units = (int)pl.units;
  a.tn = pl.tn;
  a.tiles = pl.tiles;
  a.by_tiles = make_fastdiv(std::max(1, pl.tiles));
  a.lanes = pl.lanes;
  a.rows = pl.rows;
  return a;
}

int64_t ln_bwd_ws(const mqv_ln_desc* d, const LnPlan& pl) { return align256(pl.blocks * 2 * d->C * 4); }

// ----------------------------------------------------------- linear layer

mqv_status check_lin(const mqv_lin_desc* d) {
  if (!d) return fail(MQV_ERR_INVALID_ARG, "null descriptor");
  if (d->P < 0 || d->Cin <= 0 || d->Cout <= 0 || d->N <= 0 || d->reserved)
    return fail(MQV_ERR_INVALID_ARG,
                "linear layer [%lld][%lld -> %lld][%lld]: P >= 0, Cin, Cout and N > 0, reserved 0 required",
                (long long)d->P, (long long)d->Cin, (long long)d->Cout, (long long)d->N);
  if (d->act < MQV_ACT_NONE || d->act > MQV_ACT_SILU) return fail(MQV_ERR_INVALID_ARG, "unknown activation %d", d->act);
  // a position's columns are padded to whole chunks in the tiles
  const int64_t c = std::max(d->Cin, d->Cout), padded = d->N == 1 ? 1 : ceil_div(d->N, 64) * 64;
  if (c > (1 << 24) || d->N > kMaxColumns - 64 || d->P > kMaxColumns / padded ||
      (d->P > 0 && c > kMaxElements / (d->P * padded)) || d->Cin > kMaxElements / d->Cout)
    return fail(MQV_ERR_UNSUPPORTED, "linear layer [%lld][%lld -> %lld][%lld] too large", (long long)d->P,
                (long long)d->Cin, (long long)d->Cout, (long long)d->N);
  return MQV_OK;
}

struct ActGradPlan {
  int v, lanes, rows, tiles;
  unsigned gx, gy;
};

// For P > 0: the element limit then keeps the blocks below a grid's limit.
ActGradPlan plan_act_grad(const mqv_lin_desc* d) {
  ActGradPlan pl = {};
  int64_t steps;
  pl.tiles = 1;
  if (d->N == 1) {
    pl.v = d->Cout % 8 == 0 ? 8 : 1;
    pl.gx = (unsigned)ceil_div(d->Cout, 32 * pl.v);
    steps = ceil_div(d->P, 8);
  } else {
    pl.v = d->N % 8 == 0 ? 8 : d->N % 4 == 0 ? 4 : 1;
    pl.lanes = (int)std::min<int64_t>(ceil_div(d->N, pl.v), 256);
    pl.rows = 256 / pl.lanes;
    pl.tiles = (int)ceil_div(d->N, (int64_t)pl.lanes * pl.v);
    pl.gx = (unsigned)(ceil_div(d->Cout, pl.rows) * pl.tiles);
    steps = d->P;
  }
  // about eight blocks an SM, four steps a block at least
  const int64_t want = std::max<int64_t>(1, kSms * 8 / pl.gx);
  pl.gy = (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, ceil_div(steps, 4)));
  return pl;
}

template <int V, bool TOKENS>
cudaError_t launch_act_grad_v(const ActGradArgs& a, int act, dim3 grid, cudaStream_t st) {
  switch (act) {
    case MQV_ACT_RELU: act_grad_kernel<V, kActRelu, TOKENS><<<grid, 256, 0, st>>>(a); break;
    case MQV_ACT_GELU: act_grad_kernel<V, kActGelu, TOKENS><<<grid, 256, 0, st>>>(a); break;
    case MQV_ACT_SILU: act_grad_kernel<V, kActSilu, TOKENS><<<grid, 256, 0, st>>>(a); break;
    default: act_grad_kernel<V, kActNone, TOKENS><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_act_grad(const ActGradArgs& a, const ActGradPlan& pl, int act, cudaStream_t st) {
  const dim3 grid(pl.gx, pl.gy);
  if (a.N == 1)
    return pl.v == 8 ? launch_act_grad_v<8, true>(a, act, grid, st) : launch_act_grad_v<1, true>(a, act, grid, st);
  if (pl.v == 8) return launch_act_grad_v<8, false>(a, act, grid, st);
  return pl.v == 4 ? launch_act_grad_v<4, false>(a, act, grid, st) : launch_act_grad_v<1, false>(a, act, grid, st);
}

// A few tokens: the forward pass reads the weights once, without tiles.
// (4096 -> 4096, us: 1 token 12, 4 tokens 15.3, 5 tokens in tiles with K split
// 15.8; 1024 -> 1024: 4.3, 6.3 and 8.6.)
bool few_tokens(const mqv_lin_desc* d, int op) { return op == MQV_OP_FWD && d->N == 1 && d->P <= kFewTokens; }

template <int P, bool ODD>
cudaError_t launch_few_tokens_p(const mqv_lin_desc* d, const Epilogue& e, const void* w, const void* x, const Target& to) {
  constexpr int R = P <= 2 ? 1 : 2;                // rows a warp, which share the tokens' loads
  if (to.text) return to.name("few_tokens_kernel<%d, %d, %d>", P, R, ODD);
  // warps to a row, so that a lane's eight loads at a time are all it has
  int split = 1;
  while (split < kFewThreads / 32 && d->Cin > split * 256 * (8 / R)) split *= 2;
  few_tokens_kernel<P, R, ODD><<<(unsigned)ceil_div(d->Cout, R * (kFewThreads / 32 / split)), kFewThreads, 0, to.st>>>(
      e, static_cast<const uint16_t*>(w), static_cast<const uint16_t*>(x), (int)d->Cin, (int)d->Cout, split);
  return cudaGetLastError();
}

template <bool ODD>
cudaError_t launch_few_tokens_odd(const mqv_lin_desc* d, const Epilogue& e, const void* w, const void* x, const Target& to) {
  switch (d->P) {
    case 1: return launch_few_tokens_p<1, ODD>(d, e, w, x, to);
    case 2: return launch_few_tokens_p<2, ODD>(d, e, w, x, to);
    case 3: return launch_few_tokens_p<3, ODD>(d, e, w, x, to);
    default: return launch_few_tokens_p<4, ODD>(d, e, w, x, to);
  }
}

cudaError_t launch_few_tokens(const mqv_lin_desc* d, const Epilogue& e, const void* w, const void* x, const Target& to) {
  return d->Cin % 8 == 0 ? launch_few_tokens_odd<false>(d, e, w, x, to) : launch_few_tokens_odd<true>(d, e, w, x, to);
}

// ---- products on the tensor cores

// A [pos][mid][inner] view of an operand, rows of `inner` elements.
struct GemmView {
  int64_t pos, mid, inner;
  bool mn_major;               // the tile's rows lie along inner, else K does
  int64_t pitch() const { return ceil_div(inner, 8) * 8; }
  bool copied() const { return inner % 8 != 0; }
  int64_t copy_bytes() const { return copied() ? align256(pos * mid * pitch() * 2) : 0; }
  // a plain MN-major matrix of whole 64-element chunks: the chunks are taken
  // as positions, so that one box brings a stage's share
  bool chunked() const { return pos == 1 && mn_major && inner % 64 == 0; }
};

// One pass as D = A·B^T over the views; D's columns are contiguous.
struct GemmPlan {
  GemmView a, b;
  GemmOperand oa, ob;
  int64_t M;
  int bn;
  bool pair;
  GemmTcArgs args;
  int64_t out_elems, part_bytes, ws_bytes;
};

// The chunk size of an inner extent: the largest whose padding stays within
// an eighth, else the largest of those with the least padding (batch 20, gw
// of 128 x 128 over 400 pixels: 24.2 us in chunks of 32, 24.9 in chunks of 16).
int chunk_of(int64_t inner) {
  int best = 64;
  for (int c : {64, 32, 16}) {
    if (ceil_div(inner, c) * c * 8 <= inner * 9) return c;
    if (ceil_div(inner, c) * c < ceil_div(inner, best) * best) best = c;
  }
  return best;
}

GemmOperand operand_of(const GemmView& v, int rows, bool batch) {
  GemmOperand o;
  o.chunk = batch ? chunk_of(v.inner) : 64;
  o.per_pos = v.chunked() ? 1 : (int)ceil_div(v.inner, o.chunk);
  o.mn_major = v.mn_major;
  o.box = (batch || v.chunked()) && o.per_pos == 1 ? (v.mn_major ? rows : kGemmBK) / o.chunk : 1;
  return o;
}

// The tile and the split of K with the least time by a model of the measured
// times (us): `kBase` for launch, first loads and last epilogue, and for each
// wave of tiles `start` and `block` for each K block, or `epilogue` where that
// takes longer.  Measured (and modelled) for 8192 tokens, us in 256 x 256 tiles
// of two CTAs, 128 x 128 and 128 x 64: 64 -> 4096 34, 31, 32 (33, 33, 35); 256
// -> 4096 36, 34, 53 (33, 33, 54); 1024 -> 4096 50, 78, 140 (50, 78, 140); for
// 2048 tokens 64 -> 1024 9.6, 6.8, 6.0 (8.6, 6.5, 6.7).  256 x 128 tiles of two
// CTAs were never faster than 128 x 128.  A split writes and reads fp32
// partial sums and takes a second kernel (1024 tokens 2048 -> 128 in 128 x 64
// tiles: split eight ways 9.9 us, four ways 10.1).  The model knows neither the
// bytes of the outputs nor what the epilogue does beside storing them, and is
// short by that: 1600 x 16 pixels 512 -> 128 with an fp32 residual 10.6 us
// modelled, 15.3 measured, 8187 tokens 1024 -> 4096 50 modelled, 55 measured
// plain, 70 with GELU and a kept pre-activation.
void choose_tile(GemmPlan* pl, int64_t kblocks, int64_t vcols) {
  struct Tile {
    int bn;
    bool pair;
    double start, block, epilogue;
  };
  static constexpr Tile kTiles[] = {{256, true, 1.1, .34, 4.1}, {128, false, .8, .28, 2.0}, {64, false, .75, .255, 1.1}};
  constexpr double kBase = 4.5;
  double best = 0;
  for (const Tile& t : kTiles) {
    const int64_t units = t.pair ? kSms / 2 : kSms;
    const int64_t tiles = std::max<int64_t>(1, ceil_div(pl->M, t.pair ? 2 * kGemmBM : kGemmBM) * ceil_div(vcols, t.bn));
    const int64_t fill = std::max<int64_t>(1, std::min(units / tiles, kblocks / 2));
    for (int64_t s : {int64_t{1}, int64_t{2}, int64_t{4}, int64_t{8}, int64_t{16}, int64_t{32}, fill}) {
      if (s > fill) continue;
      const double wave = std::max(t.start + ceil_div(kblocks, s) * t.block, t.epilogue);
      double us = kBase + ceil_div(tiles * s, units) * wave;
      if (s > 1) us += 2.5 + s * pl->out_elems * 4 / 2.2e6;
      if (best == 0 || us < best) {
        best = us;
        pl->bn = t.bn;
        pl->pair = t.pair;
        pl->args.splits = (int)s;
      }
    }
  }
}

void plan_gemm(const mqv_lin_desc* d, int op, GemmPlan* pl) {
  const bool tokens = d->N == 1;
  // a [P][C][N] tensor: rows of channels for tokens, of batch items otherwise
  auto tensor = [&](int64_t C, bool mn) {
    return tokens ? GemmView{1, d->P, C, mn} : GemmView{d->P, C, d->N, mn};
  };
  GemmTcArgs& g = pl->args;
  g = {};
  int64_t kdim = 0;            // channels contracted over; 0: the columns
  int64_t cols;
  bool batch_a = false, batch_b = false;
  if (op == MQV_OP_WGRAD) {
    pl->a = tensor(d->Cout, tokens);
    pl->b = tensor(d->Cin, tokens);
    batch_a = batch_b = !tokens;
    pl->M = d->Cout;
    cols = d->Cin;
  } else {
    const int64_t out = op == MQV_OP_FWD ? d->Cout : d->Cin;
    kdim = op == MQV_OP_FWD ? d->Cin : d->Cout;
    const GemmView w{1, d->Cout, d->Cin, op == MQV_OP_DGRAD};
    if (tokens) {
      pl->a = tensor(kdim, false);
      pl->b = w;
      pl->M = d->P;
      cols = out;
    } else {
      pl->a = w;
      pl->b = tensor(kdim, true);
      batch_b = true;
      pl->M = out;
      cols = 0;
    }
  }
  const bool col_batch = op != MQV_OP_WGRAD && !tokens;
  g.M = pl->M;
  g.col_chunk = col_batch ? chunk_of(d->N) : 64;
  g.col_shift = g.col_chunk == 64 ? 6 : g.col_chunk == 32 ? 5 : 4;
  g.col_inner = col_batch ? d->N : cols;
  g.col_pos = col_batch ? d->P : 1;
  g.col_per_pos = (int)ceil_div(g.col_inner, g.col_chunk);
  g.row_stride = g.col_inner;
  g.pos = col_batch ? pl->M * d->N : 0;
  g.e.vec4 = g.col_inner % 4 == 0;
  g.e.bias_on_row = col_batch;
  pl->out_elems = pl->M * g.col_inner * g.col_pos;
  const int64_t vcols = g.col_pos * g.col_per_pos * g.col_chunk;
  const int64_t kblocks = kdim ? ceil_div(kdim, kGemmBK)
                          : batch_a ? ceil_div(d->P * ceil_div(d->N, chunk_of(d->N)), kGemmBK / chunk_of(d->N))
                                    : ceil_div(d->P, kGemmBK);
  choose_tile(pl, kblocks, vcols);
  g.tiles_m = (int)ceil_div(pl->M, pl->pair ? 2 * kGemmBM : kGemmBM);
  g.tiles_n = (int)ceil_div(vcols, pl->bn);
  g.tail_width = g.tiles_n % 8 ? g.tiles_n % 8 : 8;
  g.by_split = make_fastdiv(std::max<int64_t>(1, (int64_t)g.tiles_m * g.tiles_n));
  g.by_band = make_fastdiv(std::max<int64_t>(1, (int64_t)g.tiles_m * 8));
  g.by_tail = make_fastdiv(g.tail_width);
  g.by_pos = make_fastdiv(std::max(1, g.col_per_pos));
  pl->oa = operand_of(pl->a, kGemmBM, batch_a);
  pl->ob = operand_of(pl->b, pl->pair ? pl->bn / 2 : pl->bn, batch_b);
  g.a = pl->oa;
  g.b = pl->ob;
  g.kblocks = (int)kblocks;
  g.part_stride = ceil_div(pl->out_elems, 4) * 4;
  pl->part_bytes = g.splits > 1 ? align256(g.splits * g.part_stride * 4) : 0;
  pl->ws_bytes = pl->part_bytes + pl->a.copy_bytes() + pl->b.copy_bytes();
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn tensor_map_encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

mqv_status encode(CUtensorMap* map, bool f32, int rank, const void* p, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box) {
  const EncodeFn fn = tensor_map_encoder();
  if (!fn) return fail(MQV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from this driver");
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const unsigned span = box[0] * (f32 ? 4 : 2);
  const CUresult r = fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                        const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        span == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                        : span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_32B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MQV_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)r);
  return MQV_OK;
}

mqv_status encode_operand(CUtensorMap* map, const void* p, const GemmView& v, const GemmOperand& o, int rows) {
  const bool ch = v.chunked();
  const cuuint64_t dims[3] = {(cuuint64_t)(ch ? 64 : v.inner), (cuuint64_t)v.mid, (cuuint64_t)(ch ? v.inner / 64 : v.pos)};
  const cuuint64_t strides[2] = {(cuuint64_t)v.pitch() * 2, (cuuint64_t)(ch ? 64 : v.pitch() * v.mid) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)o.chunk, (cuuint32_t)(o.mn_major ? kGemmBK : rows), (cuuint32_t)o.box};
  return encode(map, false, 3, p, dims, strides, box);
}

// An output (or the residual) in staged tiles of 32 rows x 32 columns; the
// fourth dimension is the split of the partial sums.
mqv_status encode_output(CUtensorMap* map, const void* p, bool f32, const GemmTcArgs& g) {
  const int64_t size = f32 ? 4 : 2, width = std::min(g.col_chunk, 32);
  const int64_t row = g.row_stride * size, pos = g.M * row;
  const cuuint64_t dims[4] = {(cuuint64_t)g.col_inner, (cuuint64_t)g.M, (cuuint64_t)g.col_pos, (cuuint64_t)g.splits};
  const cuuint64_t strides[3] = {(cuuint64_t)row, (cuuint64_t)pos, (cuuint64_t)(g.splits > 1 ? g.part_stride * size : 16)};
  const cuuint32_t box[4] = {(cuuint32_t)width, 32, (cuuint32_t)(g.col_per_pos == 1 ? 32 / width : 1), 1};
  return encode(map, f32, 4, p, dims, strides, box);
}

template <int BN, bool PAIR, bool FAST, bool RUNS>
cudaError_t launch_gemm_tile(const GemmPlan& pl, const GemmMaps& maps, const Target& to) {
  if (to.text)
    return to.name("gemm_tc_kernel<%d, %d, %d, %d>%s%s%s", BN, PAIR, FAST, RUNS,
                   pl.args.splits == 1 ? "" : pl.args.e.vec4 ? " split_sum_kernel<4>" : " split_sum_kernel<1>",
                   pl.a.copied() ? " copy a" : "", pl.b.copied() ? " copy b" : "");
  static std::atomic<bool> done[kMaxDevices] = {};
  auto kernel = gemm_tc_kernel<BN, PAIR, FAST, RUNS>;
  const cudaError_t e = allow_smem(kernel, gemm_smem<BN, PAIR, FAST>, done);
  if (e != cudaSuccess) return e;
  constexpr int kCtas = PAIR ? 2 : 1;
  const int64_t tiles = (int64_t)pl.args.tiles_m * pl.args.tiles_n * pl.args.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)(std::min<int64_t>(tiles, kSms / kCtas) * kCtas);
  cfg.blockDim = kGemmThreads;
  cfg.dynamicSmemBytes = gemm_smem<BN, PAIR, FAST>;
  cfg.stream = to.st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, pl.args);
}

template <bool FAST, bool RUNS>
cudaError_t launch_gemm_form(const GemmPlan& pl, const GemmMaps& maps, const Target& to) {
  if (pl.pair) return launch_gemm_tile<256, true, FAST, RUNS>(pl, maps, to);
  return pl.bn == 128 ? launch_gemm_tile<128, false, FAST, RUNS>(pl, maps, to)
                      : launch_gemm_tile<64, false, FAST, RUNS>(pl, maps, to);
}

// Rows of whole 16-byte vectors, in bfloat16 too: outputs go by TMA.
bool fast_output(const GemmPlan& pl) { return pl.args.col_inner % 8 == 0; }

// K blocks that an accumulator sums at most (see gemm_add_runs): 512 products
// for results kept in fp32, 32768 for bfloat16 ones, whose sums then lose a
// sixteenth of their rounding at most (in one run of 262144 positive products,
// half of it).  A tile whose sum takes two runs does not have its epilogue
// under the next tile's products: in runs of 16384, 2048 tokens 32768 -> 2048
// took 241 us, 225 in one.
int run_length(bool bf16) { return bf16 ? 512 : 8; }

cudaError_t launch_gemm(const GemmPlan& pl, const GemmMaps& maps, const Target& to) {
  const bool runs = ceil_div(pl.args.kblocks, pl.args.splits) > pl.args.run;
  if (fast_output(pl)) return runs ? launch_gemm_form<true, true>(pl, maps, to) : launch_gemm_form<true, false>(pl, maps, to);
  return runs ? launch_gemm_form<false, true>(pl, maps, to) : launch_gemm_form<false, false>(pl, maps, to);
}

// Copies an operand whose rows are unaligned to its place in the workspace.
void repitch(const GemmView& v, const void* src, const void* dst, cudaStream_t st) {
  if (!v.copied()) return;
  const int64_t rows = v.pos * v.mid;
  int per = 1;
  while (per < 32 && per * 8 < v.inner) per *= 2;
  repitch_kernel<<<(unsigned)std::min<int64_t>(ceil_div(rows, 256 / per), kSms * 32), 256, 0, st>>>(
      static_cast<const uint16_t*>(src), static_cast<uint16_t*>(const_cast<void*>(dst)), rows, (int)v.inner,
      (int)v.pitch(), per);
}

// The pass `op` with A and B at a and b, and epilogue e (its d, z, residual,
// bias and act).
mqv_status run_gemm(const mqv_lin_desc* d, int op, const void* a, const void* b, const Epilogue& e, void* ws,
                    cudaStream_t st) {
  GemmPlan pl;
  plan_gemm(d, op, &pl);
  GemmTcArgs& g = pl.args;
  if (pl.out_elems == 0) return ok();
  if (g.kblocks == 0) {          // a weight gradient over no columns
    const cudaError_t ce = cudaMemsetAsync(e.d.p, 0, (size_t)pl.out_elems * 4, st);
    return ce == cudaSuccess ? ok() : cuda_fail(ce, "linear layer gradient");
  }
  const Epilogue plan_e = g.e;
  g.e = e;
  g.e.vec4 = plan_e.vec4;
  g.e.bias_on_row = plan_e.bias_on_row;
  g.run = run_length(g.e.d.bf16);
  char* w = static_cast<char*>(ws);
  if (g.splits > 1) g.part = reinterpret_cast<float*>(w);
  w += pl.part_bytes;
  const void* ta = pl.a.copied() ? w : a;          // what the tensor maps point at
  w += pl.a.copy_bytes();
  const void* tb = pl.b.copied() ? w : b;
  mqv_status s = device_error_word(&g.err);
  if (s) return s;
  GemmMaps maps;
  if ((s = encode_operand(&maps.a, ta, pl.a, pl.oa, kGemmBM)) ||
      (s = encode_operand(&maps.b, tb, pl.b, pl.ob, pl.pair ? pl.bn / 2 : pl.bn)))
    return s;
  if (fast_output(pl)) {
    if ((s = encode_output(&maps.d, g.part ? g.part : g.e.d.p, g.part || !g.e.d.bf16, g))) return s;
    if (!g.part && g.e.z.p && (s = encode_output(&maps.z, g.e.z.p, false, g))) return s;
    if (!g.part && g.e.residual && (s = encode_output(&maps.residual, g.e.residual, !g.e.d.bf16, g))) return s;
  }
  repitch(pl.a, a, ta, st);
  repitch(pl.b, b, tb, st);
  const cudaError_t ce = launch_gemm(pl, maps, {st, nullptr, 0});
  if (ce != cudaSuccess) return cuda_fail(ce, "linear layer launch");
  if (g.splits > 1) {
    const int64_t inner = g.e.bias_on_row ? g.col_inner : 1, channels = g.e.bias_on_row ? pl.M : g.col_inner;
    const int v = g.e.vec4 ? 4 : 1;
    const unsigned blocks = (unsigned)ceil_div(pl.out_elems, 32 * v);
    DependentLaunch l(blocks, 256, st);
    const float* part = g.part;
    const cudaError_t se =
        v == 4 ? cudaLaunchKernelEx(&l.cfg, split_sum_kernel<4>, g.e, part, g.splits, g.part_stride, pl.out_elems, inner, channels)
               : cudaLaunchKernelEx(&l.cfg, split_sum_kernel<1>, g.e, part, g.splits, g.part_stride, pl.out_elems, inner, channels);
    if (se != cudaSuccess) return cuda_fail(se, "linear layer launch");
  }
  return launched("linear layer launch");
}

int64_t lin_ws(const mqv_lin_desc* d, int op) {
  if (op == MQV_OP_ACT_GRAD) {
    if (d->P == 0) return 0;
    const ActGradPlan pl = plan_act_grad(d);
    return align256((int64_t)pl.gy * pl.tiles * d->Cout * 4);
  }
  if (few_tokens(d, op)) return 0;
  GemmPlan pl;
  plan_gemm(d, op, &pl);
  return pl.out_elems && pl.args.kblocks ? pl.ws_bytes : 0;
}

}  // namespace

extern "C" {

mqv_status mqv_ln_fwd(const mqv_ln_desc* d, const void* x, int32_t x_type, const float* gamma, const float* beta,
                      void* y, int32_t y_type, float* mean, float* rstd, void* stream) {
  LnPlan pl;
  mqv_status st = plan_ln(d, false, &pl);
  if (st || (st = check_type(x_type, "x")) || (st = check_type(y_type, "y"))) return st;
  const int64_t cols = d->P * d->N, n = cols * d->C;
  if (!mean != !rstd) return fail(MQV_ERR_INVALID_ARG, "mean and rstd: both or neither");
  if ((st = check_buffers({{"x", x, n * type_size(x_type), false, true},
                           {"gamma", gamma, d->C * 4, false, false},
                           {"beta", beta, d->C * 4, false, false},
                           {"y", y, n * type_size(y_type), true, true},
                           {"mean", mean, cols * 4, true, false},
                           {"rstd", rstd, cols * 4, true, false}},
                          "y", "x")))
    return st;
  if (cols == 0) return ok();
  LnArgs a = ln_args(d, pl, x, x_type, gamma);
  a.beta = beta;
  a.mean = mean;
  a.rstd = rstd;
  a.out = {y, y_type == MQV_BF16};
  const cudaError_t e = launch_ln_fwd(a, pl, d->N == 1, {static_cast<cudaStream_t>(stream), nullptr, 0});
  return e == cudaSuccess ? ok() : cuda_fail(e, "layer norm launch");
}

mqv_status mqv_ln_bwd_workspace_size(const mqv_ln_desc* d, size_t* bytes) {
  LnPlan pl;
  mqv_status st = plan_ln(d, true, &pl);
  if (st) return st;
  if (!bytes) return fail(MQV_ERR_INVALID_ARG, "null output pointer");
  *bytes = (size_t)ln_bwd_ws(d, pl);
  return ok();
}

mqv_status mqv_ln_bwd(const mqv_ln_desc* d, const void* gy, int32_t gy_type, const void* x, int32_t x_type,
                      const float* mean, const float* rstd, const float* gamma, void* gx, int32_t gx_type,
                      float* ggamma, float* gbeta, void* ws, size_t ws_bytes, void* stream) {
  LnPlan pl;
  mqv_status st = plan_ln(d, true, &pl);
  if (st || (st = check_type(gy_type, "gy")) || (st = check_type(x_type, "x")) || (st = check_type(gx_type, "gx")))
    return st;
  const int64_t cols = d->P * d->N, n = cols * d->C;
  if (!ggamma != !gbeta) return fail(MQV_ERR_INVALID_ARG, "ggamma and gbeta: both or neither");
  const int64_t need = ggamma ? ln_bwd_ws(d, pl) : 0;
  if ((st = check_workspace(ws, ws_bytes, need))) return st;
  if ((st = check_buffers({{"gy", gy, n * type_size(gy_type), false, true},
                           {"x", x, n * type_size(x_type), false, true},
                           {"mean", mean, cols * 4, false, true},
                           {"rstd", rstd, cols * 4, false, true},
                           {"gamma", gamma, d->C * 4, false, false},
                           {"gx", gx, n * type_size(gx_type), true, true},
                           {"ggamma", ggamma, d->C * 4, true, false},
                           {"gbeta", gbeta, d->C * 4, true, false},
                           {"ws", ws, need, true, false}},
                          "gx", "gy")))
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LnArgs a = ln_args(d, pl, x, x_type, gamma);
  a.gy = {gy, gy_type == MQV_BF16};
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.out = {gx, gx_type == MQV_BF16};
  a.part = ggamma ? static_cast<float*>(ws) : nullptr;
  if (cols > 0) {
    const cudaError_t e = launch_ln_bwd(a, pl, d->N == 1, {s, nullptr, 0});
    if (e != cudaSuccess) return cuda_fail(e, "layer norm gradient launch");
  }
  if (ggamma) launch_column_sum(a.part, pl.blocks, d->C, 2, ggamma, gbeta, s);
  return launched("layer norm gradient launch");
}

mqv_status mqv_lin_workspace_size(const mqv_lin_desc* d, int32_t op, size_t* bytes) {
  mqv_status st = check_lin(d);
  if (st) return st;
  if (op != MQV_OP_FWD && op != MQV_OP_WGRAD && op != MQV_OP_DGRAD && op != MQV_OP_ACT_GRAD)
    return fail(MQV_ERR_INVALID_ARG, "unknown op %d", op);
  if (!bytes) return fail(MQV_ERR_INVALID_ARG, "null output pointer");
  *bytes = (size_t)lin_ws(d, op);
  return ok();
}

mqv_status mqv_lin_fwd(const mqv_lin_desc* d, const void* w, const void* x, const float* bias, const void* residual,
                       void* z, void* y, int32_t y_type, void* ws, size_t ws_bytes, void* stream) {
  mqv_status st = check_lin(d);
  if (st || (st = check_type(y_type, "y"))) return st;
  const int64_t cols = d->P * d->N, n = cols * d->Cout, need = lin_ws(d, MQV_OP_FWD);
  if ((st = check_workspace(ws, ws_bytes, need))) return st;
  if ((st = check_buffers({{"w", w, d->Cout * d->Cin * 2, false, true},
                           {"x", x, cols * d->Cin * 2, false, true},
                           {"bias", bias, d->Cout * 4, false, false},
                           {"residual", residual, n * type_size(y_type), false, false},
                           {"z", z, n * 2, true, false},
                           {"y", y, n * type_size(y_type), true, true},
                           {"ws", ws, need, true, false}},
                          "y", "residual")))
    return st;
  Epilogue e = {};
  e.d = {y, y_type == MQV_BF16};
  e.z = {z, 1};
  e.residual = residual;
  e.bias = bias;
  e.act = d->act;
  if (few_tokens(d, MQV_OP_FWD) && cols > 0) {
    const cudaError_t ce = launch_few_tokens(d, e, w, x, {static_cast<cudaStream_t>(stream), nullptr, 0});
    return ce == cudaSuccess ? ok() : cuda_fail(ce, "linear layer launch");
  }
  return run_gemm(d, MQV_OP_FWD, d->N == 1 ? x : w, d->N == 1 ? w : x, e, ws, static_cast<cudaStream_t>(stream));
}

mqv_status mqv_lin_act_grad(const mqv_lin_desc* d, const void* gy, int32_t gy_type, const void* z, void* gz,
                            float* gbias, void* ws, size_t ws_bytes, void* stream) {
  mqv_status st = check_lin(d);
  if (st || (st = check_type(gy_type, "gy"))) return st;
  const int64_t cols = d->P * d->N, n = cols * d->Cout;
  if (!gz && !gbias)             // nothing to write: the rule only where there is something, as empty tensors are null
    return cols > 0 ? fail(MQV_ERR_INVALID_ARG, "gz and gbias: one at least") : ok();
  const int64_t need = gbias ? lin_ws(d, MQV_OP_ACT_GRAD) : 0;
  if ((st = check_workspace(ws, ws_bytes, need))) return st;
  const bool act = d->act != MQV_ACT_NONE;
  if ((st = check_buffers({{"gy", gy, n * type_size(gy_type), false, true},
                           {"z", act ? z : nullptr, n * 2, false, act},
                           {"gz", gz, n * 2, true, false},
                           {"gbias", gbias, d->Cout * 4, true, false},
                           {"ws", ws, need, true, false}},
                          "gz", "gy")))
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const ActGradPlan pl = cols > 0 ? plan_act_grad(d) : ActGradPlan{};
  ActGradArgs a = {};
  a.gy = {gy, gy_type == MQV_BF16};
  a.z = act ? z : nullptr;
  a.gz = {gz, 1};
  a.part = gbias ? static_cast<float*>(ws) : nullptr;
  a.P = d->P;
  a.N = d->N;
  a.C = (int)d->Cout;
  a.lanes = pl.lanes;
  a.rows = pl.rows;
  a.tiles = pl.tiles;
  if (cols > 0) {
    const cudaError_t e = launch_act_grad(a, pl, d->act, s);
    if (e != cudaSuccess) return cuda_fail(e, "activation gradient launch");
  }
  if (gbias) launch_column_sum(a.part, (int64_t)pl.gy * pl.tiles, d->Cout, 1, gbias, nullptr, s);
  return launched("activation gradient launch");
}

mqv_status mqv_lin_dgrad(const mqv_lin_desc* d, const void* w, const void* gz, void* gx, int32_t gx_type, void* ws,
                         size_t ws_bytes, void* stream) {
  mqv_status st = check_lin(d);
  if (st || (st = check_type(gx_type, "gx"))) return st;
  const int64_t cols = d->P * d->N, need = lin_ws(d, MQV_OP_DGRAD);
  if ((st = check_workspace(ws, ws_bytes, need))) return st;
  if ((st = check_buffers({{"w", w, d->Cout * d->Cin * 2, false, true},
                           {"gz", gz, cols * d->Cout * 2, false, true},
                           {"gx", gx, cols * d->Cin * type_size(gx_type), true, true},
                           {"ws", ws, need, true, false}})))
    return st;
  Epilogue e = {};
  e.d = {gx, gx_type == MQV_BF16};
  return run_gemm(d, MQV_OP_DGRAD, d->N == 1 ? gz : w, d->N == 1 ? w : gz, e, ws, static_cast<cudaStream_t>(stream));
}

mqv_status mqv_lin_wgrad(const mqv_lin_desc* d, const void* gz, const void* x, float* gw, void* ws, size_t ws_bytes,
                         void* stream) {
  mqv_status st = check_lin(d);
  if (st) return st;
  const int64_t cols = d->P * d->N, need = lin_ws(d, MQV_OP_WGRAD);
  if ((st = check_workspace(ws, ws_bytes, need))) return st;
  if ((st = check_buffers({{"gz", gz, cols * d->Cout * 2, false, true},
                           {"x", x, cols * d->Cin * 2, false, true},
                           {"gw", gw, d->Cout * d->Cin * 4, true, true},
                           {"ws", ws, need, true, false}})))
    return st;
  Epilogue e = {};
  e.d = {gw, 0};
  return run_gemm(d, MQV_OP_WGRAD, gz, x, e, ws, static_cast<cudaStream_t>(stream));
}

mqv_status mqv_selftest_warp_wait_timeout(int64_t limit_cycles, void* stream) {
  if (limit_cycles < 1 || limit_cycles > (int64_t{1} << 32))
    return fail(MQV_ERR_INVALID_ARG, "limit_cycles %lld outside 1 .. 2^32", (long long)limit_cycles);
  uint32_t* err = nullptr;
  const mqv_status st = device_error_word(&err);
  if (st) return st;
  warp_wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(err, 8, 16, limit_cycles);
  return launched("self-test launch");
}

mqv_status mqv_selftest_ln_instance(const mqv_ln_desc* d, int32_t bwd, char* text, size_t bytes) {
  LnPlan pl;
  const mqv_status st = plan_ln(d, bwd != 0, &pl);
  if (st) return st;
  if (!text || !bytes) return fail(MQV_ERR_INVALID_ARG, "null output buffer");
  const Target to = {nullptr, text, bytes};
  text[0] = 0;
  if (d->P > 0) (bwd ? launch_ln_bwd : launch_ln_fwd)(LnArgs{}, pl, d->N == 1, to);
  return ok();
}

mqv_status mqv_selftest_lin_instance(const mqv_lin_desc* d, int32_t op, int32_t out_type, char* text, size_t bytes) {
  mqv_status st = check_lin(d);
  if (st || (st = check_type(out_type, "output"))) return st;
  if (op != MQV_OP_FWD && op != MQV_OP_WGRAD && op != MQV_OP_DGRAD) return fail(MQV_ERR_INVALID_ARG, "unknown op %d", op);
  if (!text || !bytes) return fail(MQV_ERR_INVALID_ARG, "null output buffer");
  const Target to = {nullptr, text, bytes};
  text[0] = 0;
  if (d->P == 0) return ok();
  if (few_tokens(d, op)) {
    launch_few_tokens(d, Epilogue{}, nullptr, nullptr, to);
  } else {
    GemmPlan pl;
    plan_gemm(d, op, &pl);
    pl.args.run = run_length(out_type == MQV_BF16 && op != MQV_OP_WGRAD);
    launch_gemm(pl, GemmMaps{}, to);
  }
  return ok();
}

}  // extern "C"
