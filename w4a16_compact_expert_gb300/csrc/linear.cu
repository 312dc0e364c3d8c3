// moe_w4a16_linear: out = act(x_scale w_scale x W^T + bias) + residual on the
// 5th-generation tensor cores (tcgen05.mma, FP32 accumulators in TMEM), for
// FP16, BF16 and E4M3 operands.  A 128-byte row of a K chunk is 64 16-bit or
// 128 8-bit values and one MMA takes 32 bytes of it, so the pipeline is the
// same for all three.
//
// linear_narrow_kernel (up to 64 tokens; bound by reading W once): W is the
// MMA's A operand (128 weight rows, M), the tokens are N (16, 32 or 64 of
// them), so a few tokens waste little of the tensor core.  The K chunks of a
// tile are split over the S CTAs of a cluster; every CTA sends its FP32 part
// of a token's row to that token's owner in the cluster, which adds the parts
// in rank order and finishes the row (no workspace, no atomics, one launch).
// For SWIGLU the 128 rows are 64 gate rows and the matching 64 up rows.
// W [11264][2048] FP16, one token: 9.5 us, 4.8 TB/s; W [8192][28672] 6.8 TB/s.
//
// linear_wide_kernel (more tokens; bound by the tensor cores, or by the few
// tiles of a short problem): persistent CTA pairs (cta_group::2) over tiles
// of 256 tokens x 256, 128 or 64 weight rows, two accumulators, so that one
// tile's epilogue runs under the next tile's MMAs.
// T = 2048, W [11264][2048]: E4M3 37.4 us (2,530 TFLOP/s; 34 in a loop of this
// call alone), FP16 56 us (1,690); T = 4096, W [2048][5632] FP16 69 us (1,370).
#include <cuda.h>
#include <type_traits>

#include "block.h"

namespace {

__device__ DevStatus g_block_status;

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
enum { GIVE_UP_MMA = 1, GIVE_UP_LOADS = 2, GIVE_UP_ODD_LOADS = 3 };
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

// ------------------------------------------------------------------ narrow
template <int NT>
struct NarrowCfg {
  static constexpr int kA = 128 * kChunk, kB = NT * kChunk, kStage = kA + kB;
  // The parts that this CTA receives, [sending rank][token][row]: at most 7
  // tokens' room is lost to rounding.  Up to 32 tokens they have a place of
  // their own, so that a CTA can send before the receiver has finished; for
  // 64 they go over the stages.
  static constexpr int kRecv = (NT + 7) * 128 * 4;
  static constexpr bool kOwnRecv = NT <= 32;
  static constexpr int kBudget = 110 * 1024;   // two CTAs per SM
  static constexpr int kStages = (kBudget - (kOwnRecv ? kRecv : 0)) / kStage;
  static constexpr int kRing = kStages * kStage;
  static_assert(kOwnRecv || kRecv <= kRing, "the parts fit over the stages");
  static constexpr int kRecvAt = kOwnRecv ? kRing : 0;
  static constexpr int kBarAt = kRing + (kOwnRecv ? kRecv : 0);
  static constexpr int kSmem = kBarAt + (2 * kStages + 1) * 8 + 16 + 1024;
  static constexpr uint32_t kCols = NT < 32 ? 32 : NT;
  static constexpr int kThreads = 192;   // warp 0 loads, warp 1 multiplies, warps 2-5 empty the accumulator
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

DEV_INLINE void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
DEV_INLINE void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <bool F8, bool GATED, int NT, bool TEST>
__global__ void __launch_bounds__(192, 2)
    linear_narrow_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, int out_dtype, int S, int prefetch) {
  using C = NarrowCfg<NT>;
  constexpr int kElem = F8 ? 128 : 64;   // K values per chunk
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int FT = GATED ? 64 : 128;   // output features per tile
  const int rank = blockIdx.x % S, n0 = blockIdx.x / S * FT;   // T <= NT: a tile holds all tokens
  const int nk = (a.K + kElem - 1) / kElem;
  // rank r takes the chunks r, r + S, ..: the cluster reads neighbouring
  // 128-byte pieces of a weight row at about the same time
  const int mine = (nk - rank + S - 1) / S;

  if (threadIdx.x == 32) {
    prefetch_map(&tmW);
    prefetch_map(&tmX);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 0 && prefetch) {   // the weights of the first stages, while the grid before drains
    const uint32_t leader = elect_lane();
    for (int i = 0; i < C::kStages && i < mine; ++i) {
      prefetch_box(&tmW, (rank + i * S) * kElem, n0, leader);
      if (GATED) prefetch_box(&tmW, (rank + i * S) * kElem, a.N + n0, leader);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The trigger comes after the allocation: the next grid starts only when
  // every CTA of this one has its tensor memory, so a CTA that holds some
  // while it waits here never keeps the grid before from getting its own.
  pdl_wait();
  pdl_trigger();
  if (C::kOwnRecv && S > 1) cluster_arrive();   // this CTA runs: its place for parts can be written

  bool ok = true;
  if (warp == 0) {
    Pipe p;
    const uint32_t leader = elect_lane(), ring = smem_u32(smem), bars = smem_u32(full);
    int issued = 0;
    for (; issued < mine; ++issued) {
      if (TEST && issued == kGiveUpAt && (a.give_up == GIVE_UP_LOADS || (a.give_up == GIVE_UP_ODD_LOADS && (rank & 1)))) break;
      if (!wait_for<TEST>(&empty[p.i], p.ph ^ 1u, a)) break;
      const int c0 = (rank + issued * S) * kElem;
      const uint32_t dst = ring + (uint32_t)(p.i * C::kStage), bar = bars + (uint32_t)(p.i * 8);
      expect_bytes(bar, (uint32_t)C::kStage, leader);
      fetch<1>(dst, &tmW, c0, n0, bar, leader);
      if (GATED) fetch<1>(dst + FT * kChunk, &tmW, c0, a.N + n0, bar, leader);
      fetch<1>(dst + C::kA, &tmX, c0, 0, bar, leader);
      p.next(C::kStages);
    }
    wait_released<C::kStages>(empty, issued);
    __syncwarp();
  } else if (warp == 1) {
    Pipe p;
    const uint32_t leader = elect_lane();
    const uint32_t idesc = a.idesc | ((uint32_t)(NT >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t d = __reduce_or_sync(0xffffffffu, tmem);   // the same in every lane, and known to be
    const uint64_t desc0 = sw128_desc(smem_u32(smem));        // its address field counts 16 bytes
    for (int k = 0; k < mine; ++k) {
      if (TEST && k == kGiveUpAt && a.give_up == GIVE_UP_MMA) break;
      if (!wait_for<TEST>(&full[p.i], p.ph, a)) break;
      tc_fence_after();
      const uint64_t ad = desc0 + (uint64_t)(p.i * (C::kStage / 16)), bd = ad + C::kA / 16;
#pragma unroll
      for (int j = 0; j < 4; ++j)   // 32 bytes of K each
        umma<F8, 1>(d, ad + (uint64_t)(2 * j), bd + (uint64_t)(2 * j), idesc, (uint32_t)((k | j) != 0), leader);
      commit_one(&empty[p.i], leader);
      p.next(C::kStages);
    }
    commit_one(done, leader);
    mbar_wait_bounded(done, 0, &g_block_status);
    __syncwarp();
  } else {
    ok = __all_sync(0xffffffffu, wait_for<TEST>(done, 0, a));   // every stage has been consumed
  }

  // Token c of the tile belongs to rank c % S: every CTA sends its part of c's
  // row there, as slot c / S, and the owner adds the parts in rank order.
  if (S > 1) {
    if (!C::kOwnRecv) cluster_arrive();   // this CTA's stages are free
    cluster_wait();
  } else if (!C::kOwnRecv) {
    __syncthreads();
  }
  const int nt = min(NT, a.T), cap = (NT + S - 1) / S;
  const uint32_t recv = smem_u32(smem + C::kRecvAt);
  if (warp >= 2) {
    const int q = warp & 3, row = q * 32 + lane;
    tc_fence_after();
    if (ok) {
      int owner = 0;
      uint32_t at = recv + (uint32_t)((rank * cap * 128 + row) * 4);
      for (int c0 = 0; c0 < nt; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (c0 + j < nt) {
            uint32_t addr;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(at), "r"(owner));
            st_cluster_f32(addr, __uint_as_float(v[j]));
          }
          if (++owner == S) {
            owner = 0;
            at += 512;
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }

  // The quads of this CTA's tokens: neighbouring columns where the output
  // allows wide stores, else kQ apart, so that the lanes' single stores still
  // lie side by side.  A thread's quads are of one column group.
  constexpr int kQ = FT / 4, kBatch = NT > 16 ? 2 : 1, kSweep = C::kThreads / kQ;
  static_assert(C::kThreads % kQ == 0, "a thread keeps its columns");
  const bool wide = a.vec == 4 && n0 + FT <= a.N;
  const int step = wide ? 1 : kQ, f = (int)(threadIdx.x % kQ) * (wide ? 4 : 1), n = n0 + f;
  const int own = (nt - rank + S - 1) / S;   // tokens of this CTA
  const float* parts = reinterpret_cast<const float*>(smem + C::kRecvAt) + f;
  if (n < a.N) {
    Four cw[GATED ? 2 : 1], cb[GATED ? 2 : 1];   // of the gate rows, of the up rows
#pragma unroll
    for (int up = 0; up <= GATED; ++up) {
      if (a.ws) cw[up] = load_columns(a, a.ws + up * a.N, n, step);
      if (a.bias) cb[up] = load_columns(a, a.bias + up * a.N, n, step);
    }
    for (int s = (int)threadIdx.x / kQ; s < own; s += kSweep * kBatch) {
      int t[kBatch];
      bool live[kBatch];
      float v[kBatch * 4] = {}, up[GATED ? kBatch * 4 : 1] = {};
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int sl = s + q * kSweep;
        live[q] = sl < own;
        t[q] = min(sl, own - 1) * S + rank;
        const float* p = parts + min(sl, own - 1) * 128;
        if (wide) {
#pragma unroll 4
          for (int r = 0; r < S; ++r, p += cap * 128) {
            const float4 g = *reinterpret_cast<const float4*>(p);
            v[4 * q] += g.x, v[4 * q + 1] += g.y, v[4 * q + 2] += g.z, v[4 * q + 3] += g.w;
            if constexpr (GATED) {
              const float4 h = *reinterpret_cast<const float4*>(p + FT);
              up[4 * q] += h.x, up[4 * q + 1] += h.y, up[4 * q + 2] += h.z, up[4 * q + 3] += h.w;
            }
          }
        } else {
#pragma unroll 4
          for (int r = 0; r < S; ++r, p += cap * 128)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[4 * q + j] += p[j * kQ];
              if constexpr (GATED) up[4 * q + j] += p[FT + j * kQ];
            }
        }
        if (a.xs) {
          const float xs = a.xs[t[q]];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[4 * q + j] *= xs;
            if constexpr (GATED) up[4 * q + j] *= xs;
          }
        }
      }
      activate_quads<GATED, kBatch>(
          a, [&](bool of_up) { return cw[GATED && of_up]; }, [&](bool of_up) { return cb[GATED && of_up]; }, v, up);
      if (out_dtype == MOE_W4A16_F16) store_quads<__half, kBatch>(a, t, live, n, step, v);
      else if (out_dtype == MOE_W4A16_BF16) store_quads<__nv_bfloat16, kBatch>(a, t, live, n, step, v);
      else store_quads<float, kBatch>(a, t, live, n, step, v);
    }
  }
}

// -------------------------------------------------------------------- wide
// A pair of CTAs shares one tile of 256 tokens x BN weight rows: each loads
// its 128 token rows and half of the weight rows, the first issues the MMAs of
// both, and each finishes its 128 tokens.
template <int BN>
struct WideCfg {
  static constexpr int kA = 128 * kChunk;   // the 128 token rows of this CTA
  static constexpr int kB = BN / 2 * kChunk;   // this CTA's half of the weight rows
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = 192 * 1024 / kStage;
  static constexpr int kEpiWarps = 8, kParts = kEpiWarps / 4;   // kParts warps per TMEM lane quarter
  static constexpr int kTurn = 32 * 32 * 4;   // per epilogue warp: 32 rows x 32 FP32 columns
  static constexpr int kBars = 2 * kStages + 5;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * kTurn + kBars * 8 + 16 + 1024;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;   // warp 0 loads, warp 1 multiplies, the others finish
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

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

template <bool F8, bool GATED, int BN, typename O, bool TEST>
__global__ void __launch_bounds__(WideCfg<BN>::kThreads, 1)
    linear_wide_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmX) {
  using C = WideCfg<BN>;
  constexpr int kElem = F8 ? 128 : 64;
  constexpr uint32_t kCols = 2 * BN;      // two accumulators
  constexpr int FT = GATED ? BN / 2 : BN;   // output features per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* turn = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage + C::kEpiWarps * C::kTurn);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* last = acc_empty + 2;            // every MMA of the pair is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(last + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int mtiles = (a.T + 255) / 256, tiles = mtiles * ((a.N + FT - 1) / FT);
  const int nk = (a.K + kElem - 1) / kElem;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;

  if (threadIdx.x == 32) {
    prefetch_map(&tmW);
    prefetch_map(&tmX);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 2 * C::kEpiWarps);
    }
    mbar_init(last, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();   // after the allocation: see the narrow kernel
  pdl_trigger();

  if (warp == 0) {
    Pipe p;
    bool ok = true;
    int issued = 0;
    const uint32_t leader = elect_lane(), ring = smem_u32(smem), bars = smem_u32(full), bars0 = map_to_rank(full, 0);
    for (int tile = first; tile < tiles && ok; tile += step) {
      const int m0 = (tile % mtiles) * 256 + rank * 128, n0 = tile / mtiles * FT;
      const int b0 = rank == 0 ? n0 : GATED ? a.N + n0 : n0 + BN / 2;   // this CTA's weight rows
      for (int k = 0; k < nk; ++k) {
        if ((TEST && issued == kGiveUpAt && (a.give_up == GIVE_UP_LOADS || (a.give_up == GIVE_UP_ODD_LOADS && rank))) ||
            !wait_for<TEST>(&empty[p.i], p.ph ^ 1u, a)) {
          ok = false;
          break;
        }
        const uint32_t dst = ring + (uint32_t)(p.i * C::kStage), bar0 = bars0 + (uint32_t)(p.i * 8);
        if (rank == 0) expect_bytes(bars + (uint32_t)(p.i * 8), (uint32_t)(2 * C::kStage), leader);
        fetch<2>(dst, &tmX, k * kElem, m0, bar0, leader);
        fetch<2>(dst + C::kA, &tmW, k * kElem, b0, bar0, leader);
        ++issued;
        p.next(C::kStages);
      }
    }
    wait_released<C::kStages>(empty, issued);
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      Pipe p, acc;
      bool ok = true;
      const uint32_t leader = elect_lane();
      const uint32_t idesc = a.idesc | ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
      const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
      const uint64_t desc0 = sw128_desc(smem_u32(smem));
      for (int tile = first; tile < tiles && ok; tile += step) {
        if (!wait_for<TEST>(&acc_empty[acc.i], acc.ph ^ 1u, a)) break;
        tc_fence_after();
        const uint32_t d = tm + (uint32_t)(acc.i * BN);
        for (int k = 0; k < nk; ++k) {
          if ((TEST && k == kGiveUpAt && a.give_up == GIVE_UP_MMA) || !wait_for<TEST>(&full[p.i], p.ph, a)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + (uint64_t)(p.i * (C::kStage / 16)), bd = ad + C::kA / 16;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma<F8, 2>(d, ad + (uint64_t)(2 * j), bd + (uint64_t)(2 * j), idesc, (uint32_t)((k | j) != 0), leader);
          commit_pair(&empty[p.i], 3, leader);
          p.next(C::kStages);
        }
        if (ok) commit_pair(&acc_full[acc.i], 3, leader);
        acc.next(2);
      }
      commit_pair(last, 1, leader);
      mbar_wait_bounded(last, 0, &g_block_status);
    }
    __syncwarp();
  } else {
    // a TMEM lane (token) per thread; the kParts warps of a lane quarter share
    // the tile's output features
    const int q = warp & 3, h = (warp - 2) >> 2;
    float* buf = turn + (warp - 2) * (C::kTurn / 4);
    Pipe acc;
    for (int tile = first; tile < tiles; tile += step) {
      const int t0 = (tile % mtiles) * 256 + rank * 128 + q * 32, n0 = tile / mtiles * FT;
      constexpr int kStep = GATED ? 16 : 32, kLanes = kStep / 4, kPart = FT / C::kParts;
      // Under the tile's MMAs: this warp's part of the residual starts towards
      // the L2 (a lane takes a row), and its rows' scales (one to a lane) and its
      // columns' scales and biases are fetched, four to a lane: lane chunk kLanes
      // + u holds those of lane u of the chunk's rows (GATED: of the gate rows in
      // the lanes below 16, of the up rows above).  T = 2048, N = 2048, K = 1024
      // FP16 with residual 14.4 -> 13.1 us, with bias 11.8 -> 11.5; T = 2048, N =
      // 4096, K = 2048 E4M3 18.8 -> 17.0; SWIGLU N = 5632 E4M3 35.5 -> 33.1, with
      // bias 40.6 -> 35.0 (loops of one call; E4M3 SWIGLU among others 37.8 -> 37.6).
      if (a.res && t0 + lane < a.T) {
        const int n = n0 + h * kPart, left = min(kPart, a.N - n);
        const O* p = static_cast<const O*>(a.res) + (size_t)(t0 + lane) * a.ld_res + n;
        for (int c = 0; c < left; c += 128 / (int)sizeof(O)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c) : "memory");
      }
      const float xs = a.xs && t0 + lane < a.T ? a.xs[t0 + lane] : 1.f;
      Four cw = {}, cb = {};
      static_assert(kPart / 4 <= (GATED ? 16 : 32), "a lane for every four columns");
      const int cl = GATED ? lane & 15 : lane, up = GATED && lane >= 16 ? a.N : 0;
      if (cl < kPart / 4) {
        const int cn = n0 + h * kPart + cl / kLanes * kStep;
        const bool wide = a.vec == 4 && cn + kStep <= a.N;
        const int n = cn + cl % kLanes * (wide ? 4 : 1), apart = wide ? 1 : kLanes;
        if (a.ws) cw = load_columns(a, a.ws + up, n, apart);
        if (a.bias) cb = load_columns(a, a.bias + up, n, apart);
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, wait_for<TEST>(&acc_full[acc.i], acc.ph, a))) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc.i * BN) + ((uint32_t)(q * 32) << 16);
      for (int c0 = h * kPart; c0 < (h + 1) * kPart; c0 += kStep) {   // kStep output features at a time
        if (t0 >= a.T || n0 + c0 >= a.N) break;   // the same for the whole warp
        uint32_t v[32];
        if constexpr (GATED) {
          uint32_t g[16], w[16];
          tmem_ld16(d + (uint32_t)c0, g);
          tmem_ld16(d + (uint32_t)(BN / 2 + c0), w);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = g[j];
            v[16 + j] = w[j];
          }
        } else {
          tmem_ld32(d + (uint32_t)c0, v);
          tmem_wait_ld();
        }
        if (a.xs) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * xs);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(buf + lane * 32 + ((j ^ (lane & 7)) * 4)) =
              make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        __syncwarp();
        finish_turned<GATED, O>(a, buf, t0, n0 + c0, lane, cw, cb, (c0 - h * kPart) / kStep);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         map_to_rank(&acc_empty[acc.i], 0))
                     : "memory");
      acc.next(2);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // nothing is on its way to either CTA (see wait_released)
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

// ------------------------------------------------------------ tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
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
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int elem, int64_t stride,
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

// -------------------------------------------------------------- host side
struct Problem {
  LinearArgs a;
  const void *x, *w;
  int64_t ld_x, ld_w;   // bytes
  int elem, out_dtype, num_sms, dev;
};

constexpr int kMaxDevices = 64;

// Asked about below in the place of the kernels of its shape, never launched:
// for a kernel that allocates tensor memory the occupancy query answers one
// CTA per SM, whatever it allocates.
__global__ void __launch_bounds__(320) shape_kernel() {}

// Clusters of CTAs of this shape that can be resident at once.  GPCs hold a
// whole number of clusters: at one CTA per SM 76 of 2 but 36 of 4, at two 152 of
// 2, 97 of 3, 74 of 4, 36 of 8.
cudaError_t active_clusters(int threads, size_t smem, int cluster, int* n) {
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
int split_of(int tiles, int nk, const int (&alone)[9], const int (&shared)[9]) {
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

template <bool F8, bool GATED, int NT, bool TEST = false>
cudaError_t launch_narrow(const Problem& p, cudaStream_t st) {
  using C = NarrowCfg<NT>;
  constexpr int FT = GATED ? 64 : 128;
  CUtensorMap mw, mx;
  if (!encode_rows(&mw, p.w, GATED ? 2ll * p.a.N : p.a.N, p.a.K, p.elem, p.ld_w, FT) ||
      !encode_rows(&mx, p.x, p.a.T, p.a.K, p.elem, p.ld_x, NT))
    return cudaErrorInvalidValue;
  auto kernel = linear_narrow_kernel<F8, GATED, NT, TEST>;
  const cudaError_t e = opt_in_smem((const void*)kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = (p.a.N + FT - 1) / FT;
  const int nk = (p.a.K + kChunk / p.elem - 1) / (kChunk / p.elem);
  // asked once per device; racing first calls ask twice and store the same
  static std::atomic<int> known[kMaxDevices][2][9];
  int fit[2][9];
  for (int two = 0; two < 2; ++two)
    for (int s = 1; s <= 8; ++s) {
      int& n = fit[two][s];
      n = known[p.dev][two][s].load(std::memory_order_relaxed);
      if (!n) {
        const cudaError_t q = active_clusters(C::kThreads, two ? C::kSmem : 200 * 1024, s, &n);
        if (q != cudaSuccess) return q;
        known[p.dev][two][s].store(n, std::memory_order_relaxed);
      }
    }
  const int S = split_of(tiles, nk, fit[0], fit[1]);
  // Grids of more CTAs than SMs keep the memory busy to their end, and the next
  // grid's prefetch takes over there (W [11264][2048] FP16 9.8 -> 9.3 us);
  // smaller ones it holds up (W [2048][5632] 8.9 -> 9.6, [64][2048] 3.2 -> 4.1).
  const int prefetch = tiles * S > p.num_sms;
  return launch_pdl(kernel, dim3((unsigned)(tiles * S)), dim3(C::kThreads), C::kSmem, st, S, p.a, mw, mx, p.out_dtype, S,
                    prefetch);
}

template <bool F8, bool GATED, int BN, typename O, bool TEST = false>
cudaError_t launch_wide_o(const Problem& p, cudaStream_t st) {
  using C = WideCfg<BN>;
  CUtensorMap mw, mx;
  if (!encode_rows(&mw, p.w, GATED ? 2ll * p.a.N : p.a.N, p.a.K, p.elem, p.ld_w, BN / 2) ||
      !encode_rows(&mx, p.x, p.a.T, p.a.K, p.elem, p.ld_x, 128))
    return cudaErrorInvalidValue;
  auto kernel = linear_wide_kernel<F8, GATED, BN, O, TEST>;
  cudaError_t e = opt_in_smem((const void*)kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  static std::atomic<int> resident[kMaxDevices];   // clusters that run at once, asked once per device
  int n = resident[p.dev].load(std::memory_order_relaxed);
  if (!n) {
    e = active_clusters(C::kThreads, C::kSmem, 2, &n);
    if (e != cudaSuccess) return e;
    resident[p.dev].store(n, std::memory_order_relaxed);
  }
  constexpr int FT = GATED ? BN / 2 : BN;
  const long long tiles = (long long)((p.a.T + 255) / 256) * ((p.a.N + FT - 1) / FT);
  if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(kernel, dim3((unsigned)((tiles < n ? tiles : n) * 2)), dim3(C::kThreads), C::kSmem, st, 2, p.a, mw,
                    mx);
}

template <bool F8, bool GATED, int BN>
cudaError_t launch_wide(const Problem& p, cudaStream_t st) {
  return p.out_dtype == MOE_W4A16_F16    ? launch_wide_o<F8, GATED, BN, __half>(p, st)
         : p.out_dtype == MOE_W4A16_BF16 ? launch_wide_o<F8, GATED, BN, __nv_bfloat16>(p, st)
                                         : launch_wide_o<F8, GATED, BN, float>(p, st);
}

// The tile width of the wide kernel: rounds of tiles over the resident
// clusters, times a tile's time.  A K chunk takes a pair 0.29 us at 256 weight
// rows, 0.17 at 128 and 0.14 at 64 (below 128 the warps that fetch and issue
// set the pace), a launch and its last epilogue 2.6, 1.7 and 1.2 us: in units
// of 5 ns.  Measured at N = K = 2048 with 256 / 128 / 64 rows: T = 512 14.2 /
// 9.0 / 8.2 us, T = 1024 14.5 / 10.1 / 12.8, T = 4096 24.6 / 26.3 / 36.0.
template <bool GATED>
int wide_rows(const Problem& p) {
  const long long nk = (p.a.K + kChunk / p.elem - 1) / (kChunk / p.elem);
  const long long slots = p.num_sms / 2;
  const int rows[3] = {256, 128, 64}, chunk[3] = {58, 34, 28}, fixed[3] = {520, 340, 240};
  int best = 0;
  long long cost = -1;
  for (int i = 0; i < 3; ++i) {
    const int ft = GATED ? rows[i] / 2 : rows[i];
    const long long tiles = (long long)((p.a.T + 255) / 256) * ((p.a.N + ft - 1) / ft);
    const long long c = (tiles + slots - 1) / slots * nk * chunk[i] + fixed[i];
    if (cost < 0 || c < cost) {
      cost = c;
      best = rows[i];
    }
  }
  return best;
}

// Up to 64 tokens the narrow kernel (N = K = 2048: T = 64 5.5 us, the wide one
// 7.1; with a 128-token tile T = 128 took it 10.7, the wide one 7.3).
template <bool F8, bool GATED>
cudaError_t launch_gated(const Problem& p, cudaStream_t st) {
  if (p.a.T <= 16) return launch_narrow<F8, GATED, 16>(p, st);
  if (p.a.T <= 32) return launch_narrow<F8, GATED, 32>(p, st);
  if (p.a.T <= 64) return launch_narrow<F8, GATED, 64>(p, st);
  const int rows = wide_rows<GATED>(p);
  return rows == 256   ? launch_wide<F8, GATED, 256>(p, st)
         : rows == 128 ? launch_wide<F8, GATED, 128>(p, st)
                       : launch_wide<F8, GATED, 64>(p, st);
}

template <bool F8>
cudaError_t launch_linear(const Problem& p, cudaStream_t st) {
  return p.a.act == MOE_W4A16_ACT_SWIGLU ? launch_gated<F8, true>(p, st) : launch_gated<F8, false>(p, st);
}

int elem_size(int dtype) { return dtype == MOE_W4A16_E4M3 ? 1 : dtype == MOE_W4A16_F32 ? 4 : 2; }

// give_up nonzero: the self-test, with the limit of its waits.
moe_w4a16_status run_linear(const char* op, const moe_w4a16_linear_config* cfg, int64_t T, const void* x, const void* w,
                            const float* x_scale, const float* w_scale, const float* bias, const void* residual,
                            void* out, moe_w4a16_stream_t stream, int give_up, int64_t limit) {
  if (!cfg) return blk::reject(op, "cfg is NULL");
  const moe_w4a16_linear_config c = *cfg;
  const bool f8 = c.in_dtype == MOE_W4A16_E4M3;
  if (c.in_dtype != MOE_W4A16_F16 && c.in_dtype != MOE_W4A16_BF16 && !f8)
    return blk::reject(op, "in_dtype must be F16, BF16 or E4M3");
  if (c.out_dtype != MOE_W4A16_F16 && c.out_dtype != MOE_W4A16_BF16 && c.out_dtype != MOE_W4A16_F32)
    return blk::reject(op, "out_dtype must be F16, BF16 or F32");
  if (c.act < MOE_W4A16_ACT_NONE || c.act > MOE_W4A16_ACT_SWIGLU) return blk::reject(op, "unknown activation");
  if (c.reserved) return blk::reject(op, "reserved must be 0");
  if (c.n < 1 || c.n > (1 << 29) || c.k < 1 || c.k > (1 << 24))   // at 2^24 a tile's chunks take
    return blk::reject(op, "n outside [1, 2^29] or k outside [1, 2^24]");   // 0.1-0.2 s, a wait gives up after 1 s
  if (T < 0 || T > (1 << 30)) return blk::reject(op, "T outside [0, 2^30]");
  const int es = elem_size(c.in_dtype), os = elem_size(c.out_dtype);
  int64_t ld_x = c.ld_x ? c.ld_x : c.k, ld_w = c.ld_w ? c.ld_w : c.k;
  const int64_t ld_out = c.ld_out ? c.ld_out : c.n, ld_res = c.ld_residual ? c.ld_residual : c.n;
  if (ld_x < c.k || ld_w < c.k || ld_out < c.n || ld_res < c.n)
    return blk::reject(op, "a row stride is below the row length");
  // a single row has no stride to speak of: any that the tensor map takes
  if (T < 2) ld_x = (c.k + 15ll) / 16 * 16;
  if (c.n == 1 && c.act != MOE_W4A16_ACT_SWIGLU) ld_w = (c.k + 15ll) / 16 * 16;
  if (ld_x * es % 16 || ld_w * es % 16) return blk::reject(op, "the row strides of x and W must be multiples of 16 bytes");
  if (ld_x * es >= (1ll << 40) || ld_w * es >= (1ll << 40)) return blk::reject(op, "a row stride is too large");
  if (T == 0) return MOE_W4A16_OK;
  if (!x || !w || !out) return blk::reject(op, "NULL x, w or out");
  if (f8 && (!x_scale || !w_scale)) return blk::reject(op, "E4M3 needs x_scale and w_scale");
  if (!f8 && (x_scale || w_scale)) return blk::reject(op, "x_scale and w_scale go with E4M3 only");
  if (!blk::aligned(x, 16) || !blk::aligned(w, 16)) return blk::reject(op, "x and w must be 16-byte aligned");
  if (!blk::aligned(x_scale, 4) || !blk::aligned(w_scale, 4) || !blk::aligned(bias, 4) || !blk::aligned(out, os) ||
      !blk::aligned(residual, os))
    return blk::reject(op, "a pointer is not aligned to its type");
  if (out == x || out == w) return blk::reject(op, "out must not alias x or w");
  Problem p;
  p.x = x;
  p.w = w;
  p.ld_x = ld_x * es;
  p.ld_w = ld_w * es;
  p.elem = es;
  p.out_dtype = c.out_dtype;
  p.num_sms = blk::current_sms(&p.dev);
  if (p.num_sms < 1) return blk::launch_failed(op, cudaErrorNoDevice);
  p.a.xs = x_scale;
  p.a.ws = w_scale;
  p.a.bias = bias;
  p.a.res = residual;
  p.a.out = out;
  p.a.ld_res = ld_res;
  p.a.ld_out = ld_out;
  p.a.T = (int)T;
  p.a.N = c.n;
  p.a.K = c.k;
  p.a.act = c.act;
  // FP32 accumulator; operand formats: kind::f16 0 = FP16, 1 = BF16; kind::f8f6f4 0 = E4M3
  const uint32_t fmt = c.in_dtype == MOE_W4A16_BF16 ? 1u : 0u;
  p.a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10);
  const size_t vb = 4 * (size_t)os;
  p.a.vec = blk::aligned(out, vb) && ld_out % 4 == 0 && (!residual || (blk::aligned(residual, vb) && ld_res % 4 == 0)) ? 4 : 1;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  p.a.give_up = give_up;
  p.a.limit = limit;
  const cudaError_t e = give_up ? (T <= 16 ? launch_narrow<false, false, 16, true>(p, st)
                                           : launch_wide_o<false, false, 128, __half, true>(p, st))
                        : f8    ? launch_linear<true>(p, st)
                                : launch_linear<false>(p, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
}

}  // namespace

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_linear(const moe_w4a16_linear_config* cfg, int64_t T,
                                                           const void* x, const void* w, const float* x_scale,
                                                           const float* w_scale, const float* bias,
                                                           const void* residual, void* out,
                                                           moe_w4a16_stream_t stream) try {
  return run_linear("linear", cfg, T, x, w, x_scale, w_scale, bias, residual, out, stream, 0, 0);
} catch (...) {   // the host's heap is full
  return MOE_W4A16_ERR_OOM;
}

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_selftest_linear(const moe_w4a16_linear_config* cfg, int64_t T,
                                                                    const void* x, const void* w, void* out,
                                                                    int32_t which, int64_t limit_cycles,
                                                                    moe_w4a16_stream_t stream) try {
  const char* op = "selftest_linear";
  if (!cfg) return blk::reject(op, "cfg is NULL");
  if (cfg->in_dtype != MOE_W4A16_F16 || cfg->out_dtype != MOE_W4A16_F16 || cfg->act != MOE_W4A16_ACT_NONE)
    return blk::reject(op, "takes F16 in and out and no activation");
  if (T < 1 || (T > 16 && T <= 64)) return blk::reject(op, "T outside [1, 16] and (64, 2^30]");
  if (which < 0 || which > 2) return blk::reject(op, "which outside [0, 2]");
  if (limit_cycles < 1000 || limit_cycles > MOE_WAIT_CYCLES) return blk::reject(op, "limit_cycles outside [1000, 2^31]");
  return run_linear(op, cfg, T, x, w, nullptr, nullptr, nullptr, nullptr, out, stream, GIVE_UP_MMA + which, limit_cycles);
} catch (...) {
  return MOE_W4A16_ERR_OOM;
}

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_block_status(void) {
  const char* op = "block_status";
  DevStatus s;
  memset(&s, 0, sizeof s);
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&s, g_block_status, sizeof s);
  if (e == cudaSuccess && s.flags) {
    const DevStatus zero = {};
    e = cudaMemcpyToSymbol(g_block_status, &zero, sizeof zero);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return blk::launch_failed(op, e);
  if (s.flags & STATUS_TIMEOUT) {
    set_handle_free_error("block_status: a bounded device wait gave up");
    return MOE_W4A16_ERR_TIMEOUT;
  }
  return MOE_W4A16_OK;
}
