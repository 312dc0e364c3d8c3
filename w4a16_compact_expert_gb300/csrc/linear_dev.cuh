// What the matrix products share (linear.cu, linear_blocks.cu): instructions of
// the tensor cores and of TMA, the pipelines' waits, activations, epilogue
// stores, tensor maps and the choice of cluster sizes.
#pragma once
#include <cuda.h>
#include <type_traits>

#include "block.h"

namespace lin {

// The status word of a translation unit's kernels.
static __device__ DevStatus g_block_status;

constexpr int kChunk = 128;   // bytes of K per pipeline stage and row

struct LinearArgs {
  const float *xs, *ws, *bias;
  const void* res;
  void* out;
  long long ld_res, ld_out;
  int T, N, K;       // K in elements
  int act;
  uint32_t idesc;    // MMA instruction descriptor without its M and N fields
  int vec;           // 4: four neighbouring outputs can be read and written at once, else 1
  // the self-test's: which warps stop early (GIVE_UP_*), and the limit of the others' waits
  int give_up;
  long long limit;
};
enum { GIVE_UP_MMA = 1, GIVE_UP_LOADS = 2, GIVE_UP_ODD_LOADS = 3, GIVE_UP_FINISH = 4 };
constexpr int kGiveUpAt = 2;   // chunks before they stop

// a / (1 + e^-a), relative error up to (2 |a| + 8) 2^-24; 0 where e^-a passes
// 2^126 and the result is smaller than 87 2^-126.
DEV_INLINE float silu(float a) { return a * blk::fast_rcp(1.f + blk::fast_exp(-a)); }

// a Phi(a) of two values with the normal distribution's tail Phi(-|a|) =
// e^(-a^2 / 2) (c1 t + .. + c7 t^7), t = 1 / (1 + 0.35 |a|): the form of formula
// 26.2.17 of Abramowitz and Stegun, Handbook of Mathematical Functions, with
// coefficients fitted in 64 bits (reweighted least squares over 0 <= |a| <= 14)
// to a relative error of 1.4e-7 near 0 that may grow to 4.2e-6 far out; the
// book's five terms are as near at 0 and 2 % off at a = -9.  Taken from the
// tail's side, so that large negative a keep their relative accuracy: as
// evaluated here 6.3e-6 down to a = -8 and 9.4e-6 at -12, where the rounding of
// a^2 / 2 shows; the result is 0 below a = -13.
DEV_INLINE float2 gelu(float2 a) {
  auto both = [](float c) { return make_float2(c, c); };
  const float2 d = blk::fma2(both(0.35f), make_float2(fabsf(a.x), fabsf(a.y)), both(1.f));
  const float2 t = make_float2(blk::fast_rcp(d.x), blk::fast_rcp(d.y));
  float2 p = blk::fma2(t, both(0.0456598994f), both(-0.188426584f));
  p = blk::fma2(t, p, both(0.217169923f));
  p = blk::fma2(t, p, both(0.00426009167f));
  p = blk::fma2(t, p, both(0.145026514f));
  p = blk::fma2(t, p, both(0.136507087f));
  p = blk::fma2(t, p, both(0.139803139f));
  const float2 e = blk::mul2(blk::mul2(a, a), both(-0.72134752f));   // -a^2 / 2 log2 e
  const float2 tail = blk::mul2(blk::mul2(t, p), make_float2(blk::fast_exp2(e.x), blk::fast_exp2(e.y)));
  const float2 head = blk::fma2(tail, both(-1.f), both(1.f));
  return blk::mul2(a, make_float2(a.x > 0.f ? head.x : tail.x, a.y > 0.f ? head.y : tail.y));
}

// (1 + tanh u) / 2 = 1 / (1 + e^-2u); relative error up to (18 |u| + 8) 2^-24, 0
// where e^-2u passes 2^126.
DEV_INLINE float gelu_tanh(float a) {
  const float u = 0.7978845608f * fmaf(0.044715f * a, a * a, a);
  return a * blk::fast_rcp(1.f + blk::fast_exp(-2.f * u));
}

// The switch stands outside the values' loop: one branch per value kept a
// thread's values from overlapping (a 256 x 256 tile's epilogue took 7.5 us).
template <int N>
DEV_INLINE void activate(float (&v)[N], int act) {
  switch (act) {
    case MOE_W4A16_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays
      break;
    case MOE_W4A16_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 g = gelu(make_float2(v[i], v[i + 1]));
        v[i] = g.x;
        v[i + 1] = g.y;
      }
      break;
    case MOE_W4A16_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = gelu_tanh(v[i]);
      break;
    case MOE_W4A16_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = silu(v[i]);
      break;
    default: break;
  }
}

// The warp that issues the MMAs runs converged, every lane with the same
// values, and one elected lane executes the instruction: descriptors and
// addresses then live in uniform registers.  Inside an `if (lane == 0)` each
// MMA cost 75 cycles of issue, whatever its N.
DEV_INLINE uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}

#define UMMA_ASM(group, kind)                                                                       \
  asm volatile(                                                                                     \
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"                      \
      " @q tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem), \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc), "r"(leader)                                   \
      : "memory")

template <bool F8, int GROUP>
DEV_INLINE void umma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc,
                     uint32_t leader) {
  if constexpr (GROUP == 1 && F8) UMMA_ASM("1", "f8f6f4");
  else if constexpr (GROUP == 1) UMMA_ASM("1", "f16");
  else if constexpr (F8) UMMA_ASM("2", "f8f6f4");
  else UMMA_ASM("2", "f16");
}

// Arrives on `bar` once the MMAs issued so far are done; the pair form at its
// place in the CTAs of the mask.
DEV_INLINE void commit_one(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
DEV_INLINE void commit_pair(uint64_t* bar, uint32_t mask, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)mask), "r"(leader)
      : "memory");
}

// The same for the warp that loads: the elected lane expects `bytes` and fetches.
DEV_INLINE void expect_bytes(uint32_t bar, uint32_t bytes, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
// TMA box -> this CTA's shared memory; GROUP 2: counted by the barrier at the
// cluster address `bar`, in either CTA of the pair.
template <int GROUP>
DEV_INLINE void fetch(uint32_t dst, const CUtensorMap* tmap, int c0, int r0, uint32_t bar, uint32_t leader) {
  if constexpr (GROUP == 1)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
        " @q cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(r0), "r"(bar), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
        " @q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(r0), "r"(bar), "r"(leader)
        : "memory");
}

// Starts a box on its way into the L2 cache.  Allowed before the grids ahead
// have finished, whatever they write: the L2 is where their writes go too.
DEV_INLINE void prefetch_box(const CUtensorMap* tmap, int c0, int r0, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %3, 0;\n"
      " @q cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n}\n" ::"l"(tmap),
      "r"(c0), "r"(r0), "r"(leader)
      : "memory");
}

DEV_INLINE void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// The end of the epilogue for Q quads of outputs: quad q holds the columns n,
// n + step, .. n + 3 step of token t[q] (step 1: neighbours, read and written
// at once).  live[q] says whether the quad exists.  Written without branches
// per quad: each cost a thread 50-100 cycles, and a 256 x 256 tile's
// epilogue 7.5 us.
template <typename O, int Q>
DEV_INLINE void store_quads(const LinearArgs& a, const int (&t)[Q], const bool (&live)[Q], int n, int step,
                            const float (&v)[Q * 4]) {
  O* const out = static_cast<O*>(a.out);
  const O* const res = static_cast<const O*>(a.res);
  if (step == 1) {
    blk::Pack<O, 4> o[Q];
    if (res) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (live[q]) {   // past the L1, which the shared memory leaves almost nothing
          using V = typename std::conditional<sizeof(O) == 4, uint4, uint2>::type;
          *reinterpret_cast<V*>(&o[q]) = __ldcg(reinterpret_cast<const V*>(res + (size_t)t[q] * a.ld_res + n));
        }
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[q].v[j] = blk::from_float<O>(v[4 * q + j] + blk::to_float(o[q].v[j]));
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[q].v[j] = blk::from_float<O>(v[4 * q + j]);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (live[q]) *reinterpret_cast<blk::Pack<O, 4>*>(out + (size_t)t[q] * a.ld_out + n) = o[q];
  } else {
    bool in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) in[j] = n + j * step < a.N;
    O o[Q * 4];
    if (res) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (live[q] && in[j]) o[4 * q + j] = res[(size_t)t[q] * a.ld_res + n + j * step];
#pragma unroll
      for (int i = 0; i < Q * 4; ++i) o[i] = blk::from_float<O>(v[i] + blk::to_float(o[i]));
    } else {
#pragma unroll
      for (int i = 0; i < Q * 4; ++i) o[i] = blk::from_float<O>(v[i]);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (live[q] && in[j]) out[(size_t)t[q] * a.ld_out + n + j * step] = o[4 * q + j];
  }
}

// Scales or biases of the columns n + j step; those past N repeat the last.
struct Four {
  float v[4];
};
DEV_INLINE Four load_columns(const LinearArgs& a, const float* p, int n, int step) {
  Four f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = p[min(n + j * step, a.N - 1)];
  return f;
}

// Scales, bias and activation of Q quads; g holds the (gate) sums, u the up
// sums, already times the token's x_scale.  w(up), b(up): the scales and biases
// of the quads' columns (up: of the up rows), asked for one after the other as
// they are needed.
template <bool GATED, int Q, typename W, typename Bi>
DEV_INLINE void activate_quads(const LinearArgs& a, W w, Bi b, float (&g)[Q * 4], float (&u)[GATED ? Q * 4 : 1]) {
  if (a.ws) {
    const Four f = w(false);
#pragma unroll
    for (int i = 0; i < Q * 4; ++i) g[i] *= f.v[i % 4];
    if constexpr (GATED) {
      const Four h = w(true);
#pragma unroll
      for (int i = 0; i < Q * 4; ++i) u[i] *= h.v[i % 4];
    }
  }
  if (a.bias) {
    const Four f = b(false);
#pragma unroll
    for (int i = 0; i < Q * 4; ++i) g[i] += f.v[i % 4];
    if constexpr (GATED) {
      const Four h = b(true);
#pragma unroll
      for (int i = 0; i < Q * 4; ++i) u[i] += h.v[i % 4];
    }
  }
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < Q * 4; ++i) g[i] = silu(g[i]) * u[i];
  } else {
    activate(g, a.act);
  }
}

// How a CTA ends.  The waits of the pipelines are bounded; whoever gives up
// leaves its loop, and the others' waits run out in turn.  Either way nothing
// may be on its way to a CTA's shared memory, and no MMA in flight, when it
// ends (a pair: when both do, at their last cluster barrier):
//   - the warp that multiplies waits for the MMAs it issued;
//   - the warp that loads waits for the last release of every stage it filled
//     (a stage is released once its MMAs have read it, so its copies have
//     landed too).  Where the multiplying warp stopped first none comes; when
//     this wait runs out, a second has passed since the last copy was issued.
// These waits are over by the time the epilogue is, and keep their full limit
// in the self-test.
template <int STAGES>
DEV_INLINE void wait_released(uint64_t* empty, int filled) {
  for (int s = 0; s < STAGES && s < filled; ++s) {
    const int last = (filled - 1 - s) / STAGES;   // the stage's last fill, counted from 0
    if (!mbar_wait_bounded(&empty[s], (uint32_t)(last & 1), &g_block_status)) break;
  }
}

// The pipelines' waits.
template <bool TEST>
DEV_INLINE bool wait_for(uint64_t* bar, uint32_t parity, const LinearArgs& a) {
  return mbar_wait_limit(bar, parity, &g_block_status, TEST ? a.limit : MOE_WAIT_CYCLES);
}

struct Pipe {   // stage index and phase parity of a ring
  int i = 0;
  uint32_t ph = 0;
  DEV_INLINE void next(int n) {
    if (++i == n) {
      i = 0;
      ph ^= 1u;
    }
  }
};

DEV_INLINE void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
DEV_INLINE void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 32 rows of one warp, turned: `buf` holds [32 rows][8 units of 4 columns] with
// unit u of row r at u ^ (r & 7), so that neither the writes (a row per lane)
// nor the reads (8 lanes along a row) meet in a bank.  GATED: units 0-3 are
// gate, 4-7 the matching up columns, 4 lanes a row.  A lane finishes 4
// columns of 8 (GATED: 4) rows, 64- or 128-byte pieces of a row per store;
// outputs that cannot be stored four at a time have a lane's columns
// kLanes apart, so that the lanes' single stores still lie side by side.
// cw, cb: the scales and biases of this warp's columns of the tile, fetched
// ahead; chunk: which 32 (GATED: 16) of them.
template <bool GATED, typename O>
DEV_INLINE void finish_turned(const LinearArgs& a, const float* buf, int t0, int n0, int lane, const Four& cw,
                              const Four& cb, int chunk) {
  constexpr int kLanes = GATED ? 4 : 8;    // lanes along a row
  constexpr int kPass = GATED ? 4 : 8, kRows = 32 / kPass;
  const bool wide = a.vec == 4 && n0 + 4 * kLanes <= a.N;
  const int u = lane % kLanes, step = wide ? 1 : kLanes, c = wide ? 4 * u : u;
  // rows of a pass; GATED: neighbours in a quarter warp are 4 rows apart, else
  // their units would share banks
  const int i = lane / kLanes, r0 = GATED ? (i >> 1) + (i & 1) * 4 : i;
  float v[kPass * 4], w[GATED ? kPass * 4 : 1];
  if (wide) {
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int r = r0 + p * kRows;
      const float4 g = *reinterpret_cast<const float4*>(buf + r * 32 + ((u ^ (r & 7)) * 4));
      v[4 * p] = g.x, v[4 * p + 1] = g.y, v[4 * p + 2] = g.z, v[4 * p + 3] = g.w;
      if constexpr (GATED) {
        const float4 h = *reinterpret_cast<const float4*>(buf + r * 32 + (((u + 4) ^ (r & 7)) * 4));
        w[4 * p] = h.x, w[4 * p + 1] = h.y, w[4 * p + 2] = h.z, w[4 * p + 3] = h.w;
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int r = r0 + p * kRows;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int cc = c + j * step;
        v[4 * p + j] = buf[r * 32 + (((cc >> 2) ^ (r & 7)) * 4) + (cc & 3)];
        if constexpr (GATED) w[4 * p + j] = buf[r * 32 + ((((cc >> 2) + 4) ^ (r & 7)) * 4) + (cc & 3)];
      }
    }
  }
  auto columns = [&](const Four& of, bool up) {
    Four f;
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = __shfl_sync(0xffffffffu, of.v[j], (up ? 16 : 0) + chunk * kLanes + u);
    return f;
  };
  activate_quads<GATED, kPass>(
      a, [&](bool up) { return columns(cw, up); }, [&](bool up) { return columns(cb, up); }, v, w);
  int t[kPass];
  bool live[kPass];
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    t[p] = t0 + r0 + p * kRows;
    live[p] = t[p] < a.T;
  }
  store_quads<O, kPass>(a, t, live, n0 + c, step, v);
}

// ------------------------------------------------------------ tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    cudaGetLastError();
    return static_cast<EncodeTiledFn>(nullptr);
  }();
  return fn;
}

// [rows][cols] of 1- or 2-byte elements with a row stride in bytes; boxes of
// box_rows rows x 128 bytes, 128-byte swizzle, zeros out of range.
inline bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int elem, int64_t stride,
                 int box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {(cuuint32_t)(kChunk / elem), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// Asked about below in the place of the kernels of its shape, never launched:
// for a kernel that allocates tensor memory the occupancy query answers one
// CTA per SM, whatever it allocates.
static __global__ void __launch_bounds__(640) shape_kernel() {}

// Clusters of CTAs of this shape that can be resident at once.  GPCs hold a
// whole number of clusters: at one CTA per SM 76 of 2 but 36 of 4, at two 152 of
// 2, 97 of 3, 74 of 4, 36 of 8.
inline cudaError_t active_clusters(int threads, size_t smem, int cluster, int* n) {
  const void* kernel = (const void*)shape_kernel;
  cudaError_t e = opt_in_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
  return e == cudaSuccess && *n < 1 ? cudaErrorLaunchOutOfResources : e;
}

// CTAs of a cluster share a tile's K chunks.  The split that ends first, each
// CTA costing its chunks and about four chunks' time for its start, its share
// of the sum and its stores, and half as much again per chunk where CTAs have
// to share SMs.  alone[s], shared[s]: clusters of s that run at once with one
// and with two CTAs per SM.  (W [2048][5632], 16 tiles, 15 clusters of 8 and 23
// of 6 alone: T = 32 from the L2 6.3 us split by 8, 5.4 by 6; from memory 8.3 and 8.7.)
inline int split_of(int tiles, int nk, const int (&alone)[9], const int (&shared)[9]) {
  int best = 1;
  long long cost = -1;
  for (int s = 1; s <= 8 && s <= nk; ++s) {
    const long long rounds = (tiles + shared[s] - 1) / shared[s], chunks = (nk + s - 1) / s;
    const long long c = rounds * (chunks * (tiles > alone[s] ? 3 : 2) + 8);
    if (cost < 0 || c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

inline int elem_size(int dtype) { return dtype == MOE_W4A16_E4M3 ? 1 : dtype == MOE_W4A16_F32 ? 4 : 2; }


}  // namespace lin
