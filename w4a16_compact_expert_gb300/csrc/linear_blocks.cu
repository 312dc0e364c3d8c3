// moe_w4a16_linear_blocks: out = act(x W^T + bias) + residual of E4M3 operands
// with FP32 scales in blocks, x one per row and 128 of K, W one per 128 rows
// and 128 of K.  With d_b the product over the K block b,
//   acc[t][m] = sum_b x_scale[t][b] w_scale[m / 128][b] d_b[t][m].
// A K block is one 128-byte chunk of the pipeline.  The tensor cores multiply
// a chunk into an accumulator of its own (FP32, tensor memory), and the
// epilogue's warps add it, scaled, to sums in registers while the next chunk is
// being multiplied into another.  A thread's tensor memory lane is a token
// (wide kernel), whose scale it needs once per chunk and 128 columns.
//
// linear_blocks_narrow_kernel (up to 64 tokens, 48 with SWIGLU; bound by reading W
// once): as linear_narrow_kernel, W as the 128-row operand, the K chunks of a tile
// dealt to the CTAs of a cluster, parts added by a token's owner in rank order.  A
// tile holds 128 features (SWIGLU: 128 gate and 128 up rows in two accumulators),
// one block of scales of the output.  8 tokens through W [50304][2048] take 18.2 us
// (5.6 TB/s), one through SWIGLU [11264][2048] 5.8, 8 through [2048][5632] 5.7: the
// last two, whose W lies in the L2 there (from memory about 7), on the time of a
// launch and one trip through the pipeline.  More tokens send more between the CTAs,
// four bytes a store: 17 through SWIGLU [11264][2048] 7.2, 48 11.9 (33 to 48 also
// spill 120 bytes a thread).
//
// linear_blocks_wide_kernel (more tokens): as linear_wide_kernel, CTA pairs over
// tiles of 256 tokens x BN weight rows, but the accumulators (two of 256 columns,
// four of fewer) go round by chunks instead of tiles.  A chunk's MMAs take 512
// cycles at 256 columns, but a chunk takes 820: waking up for its accumulator,
// reading, adding (the packed FP32 FMAs 270) and handing it back, one after the
// other in each warp.  The warps that add also finish the tile, and no chunk is added
// meanwhile (3.0 of a tile's 9.7 us at K = 2048 by the rule of wide_rows).  At a
// tile's end the sums go back into the last chunk's accumulator, so that the rest of
// the epilogue is a loop over columns: out of registers it has to be unrolled, and
// its instructions no longer fit the cache.  2048 tokens through SWIGLU [11264][2048]
// to E4M3 take 51 us (1.84 PFLOP/s), 4096 through [2048][5632] to FP16 46 (2.0
// PFLOP/s), a residual added 52.  Furthest from their bytes and operations are 65 to
// 256 tokens (tiles hold 256, K is not split: SWIGLU [11264][2048] 12.5 to 13.1 us,
// [2048][5632] 11.6) and short K, where the end of a tile is most of it (4096 tokens,
// [32768][512] to FP16 150 us).  At 128 and 256 rows up to 32 bytes of a thread's sums
// and addresses are spilled.
#include "linear_dev.cuh"

namespace {

using namespace lin;

struct BlockArgs {
  LinearArgs a;   // without scales: they are in the sums
  const float *xs, *ws;
  long long ld_xs, ld_ws;
  int kb, nb;     // blocks of K; of the output features
  int xs_vec, ws_vec;   // four neighbouring scales of a row can be read at once
  float* qs;      // scales of an E4M3 output
  int wide_rows;  // every 32 bytes of a row of the output (and the residual) can be stored at once
};
struct E4M3 {
  uint8_t v;
};

constexpr float kTiny = 1.17549435e-38f;   // 2^-126: a scale below it is 0, its values too

// A row's scales of the chunks k, .. k + 3 (vec: kb is a multiple of 4); those
// past the last repeat it.
DEV_INLINE float4 load_scales(const float* row, int k, int kb, int vec) {
  if (vec) return *reinterpret_cast<const float4*>(row + k);
  return make_float4(row[min(k, kb - 1)], row[min(k + 1, kb - 1)], row[min(k + 2, kb - 1)], row[min(k + 3, kb - 1)]);
}
DEV_INLINE float lane4(const float4& f, int i) { return i == 0 ? f.x : i == 1 ? f.y : i == 2 ? f.z : f.w; }

// Waits for the tensor memory loads of this thread; r is not read before.
DEV_INLINE void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
DEV_INLINE void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
DEV_INLINE float2 pair_at(const uint32_t (&r)[N], int j) {
  return make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}

// Arrives at a cluster address, by one lane for its warp.  Nothing but tensor
// memory changes hands: every lane's reads of it have returned (wait::ld) before the
// __syncwarp in front of the arrival, so nothing that follows can overwrite what
// is still to be read, and tcgen05.fence::before_thread_sync orders them before it.
// A release at cluster scope waits for the thread's other memory accesses too:
// 2048 tokens through SWIGLU [11264][2048] 93 us instead of 53.
DEV_INLINE void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The MMAs of one K chunk into a fresh accumulator.
template <int GROUP>
DEV_INLINE void multiply_chunk(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t leader) {
#pragma unroll
  for (int j = 0; j < 4; ++j)   // 32 bytes of K each
    umma<true, GROUP>(d, ad + (uint64_t)(2 * j), bd + (uint64_t)(2 * j), idesc, (uint32_t)(j != 0), leader);
}

// ------------------------------------------------------------------ narrow
// PER: CTAs that share an SM.
template <bool GATED, int NT, int PER>
struct NarrowCfg {
  static constexpr int P = GATED ? 2 : 1;
  static constexpr int kA = P * 128 * kChunk, kB = NT * kChunk, kStage = kA + kB;
  // the parts that this CTA receives, [sending rank][token][gate, up][row]
  static constexpr int kRecv = (NT + 7) * P * 128 * 4;
  static constexpr bool kOwnRecv = kRecv <= 24 * 1024 && !GATED;   // else over the stages
  static constexpr int kScales = 4 * 2 * P * NT * 4;   // per multiplying-out warp: two chunks' scales of the tokens
  static constexpr int kBudget = PER == 2 ? 110 * 1024 : 73 * 1024;
  static constexpr int kStages = (kBudget - (kOwnRecv ? kRecv : 0) - kScales) / kStage;
  static constexpr int kRing = kStages * kStage;
  static_assert(kStages >= 2 && (kOwnRecv || kRecv <= kRing), "the parts fit over the stages");
  static constexpr int kRecvAt = kOwnRecv ? kRing : 0;
  static constexpr int kScaleAt = kRing + (kOwnRecv ? kRecv : 0);
  static constexpr int kBarAt = kScaleAt + kScales;
  static constexpr int kSmem = kBarAt + (2 * kStages + 5) * 8 + 16 + 1024;
  static constexpr uint32_t kCols = 2 * P * NT < 32 ? 32 : 2 * P * NT;
  static constexpr int kThreads = 192;   // warp 0 loads, warp 1 multiplies, warps 2-5 add up
  static_assert(PER * (kSmem + 1024) <= 228 * 1024, "they fit");
  static_assert(PER == 3 || kSmem + 1024 >= 85 * 1024, "in clusters: see WideCfg");
};

// One token's 128 features of a tile, four to a lane: scaled, rounded to E4M3
// and stored.  v of a column past N does not count.
DEV_INLINE void store_e4m3_row(const BlockArgs& b, int t, int n0, int lane, const float (&v)[4]) {
  const LinearArgs& a = b.a;
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n0 + 4 * lane + j < a.N) m = fmaxf(m, fabsf(v[j]));   // NaN is left out, its value carries it
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float c = m * (1.f / 448.f);
  if (c < kTiny) c = 0.f;
  const float inv = c > 0.f ? __fdividef(1.f, c) : 0.f;
  if (lane == 0) b.qs[(size_t)t * b.nb + n0 / 128] = c;
  uint8_t* out = static_cast<uint8_t*>(a.out) + (size_t)t * a.ld_out + n0 + 4 * lane;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; j += 2)
    w |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[j] * inv, v[j + 1] * inv), __NV_SATFINITE, __NV_E4M3) << (8 * j);
  if (a.vec == 4 && n0 + 4 * lane + 4 <= a.N) {
    *reinterpret_cast<uint32_t*>(out) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n0 + 4 * lane + j < a.N) out[j] = (uint8_t)(w >> (8 * j));
  }
}

template <bool GATED, int NT, int PER, bool TEST>
__global__ void __launch_bounds__(192, PER)
    linear_blocks_narrow_kernel(const __grid_constant__ BlockArgs b, const __grid_constant__ CUtensorMap tmW,
                                const __grid_constant__ CUtensorMap tmX, int out_dtype, int S, int prefetch) {
  using C = NarrowCfg<GATED, NT, PER>;
  constexpr int P = C::P;
  const LinearArgs& a = b.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* last = acc_empty + 2;            // every MMA is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(last + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % S, n0 = blockIdx.x / S * 128;   // T <= NT: a tile holds all tokens
  const int mine = (b.kb - rank + S - 1) / S;                   // chunks rank, rank + S, ..

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
      mbar_init(&acc_empty[s], 4);
    }
    mbar_init(last, 1);
    fence_mbar_init();
  }
  if (warp == 0 && prefetch) {   // the weights of the first stages, while the grid before drains
    const uint32_t leader = elect_lane();
    for (int i = 0; i < C::kStages && i < mine; ++i) {
      prefetch_box(&tmW, (rank + i * S) * 128, n0, leader);
      if (GATED) prefetch_box(&tmW, (rank + i * S) * 128, a.N + n0, leader);
    }
  }
  __syncwarp();   // tensor memory and cluster barriers want the warp converged, here and below
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();   // after the allocation: see linear_narrow_kernel
  pdl_trigger();
  if (C::kOwnRecv && S > 1) cluster_arrive();   // this CTA runs: its place for parts can be written

  const int nt = min(NT, a.T), cap = (NT + S - 1) / S;
  bool ok = true;
  float2 acc[P * NT / 2];   // warps 2-5: the sums of a weight row, gate then up, over the tokens
  if (warp == 0) {
    Pipe p;
    const uint32_t leader = elect_lane(), ring = smem_u32(smem), bars = smem_u32(full);
    int issued = 0;
    for (; issued < mine; ++issued) {
      if (TEST && issued == kGiveUpAt && (a.give_up == GIVE_UP_LOADS || (a.give_up == GIVE_UP_ODD_LOADS && (rank & 1)))) break;
      if (!wait_for<TEST>(&empty[p.i], p.ph ^ 1u, a)) break;
      const int c0 = (rank + issued * S) * 128;
      const uint32_t dst = ring + (uint32_t)(p.i * C::kStage), bar = bars + (uint32_t)(p.i * 8);
      expect_bytes(bar, (uint32_t)C::kStage, leader);
      fetch<1>(dst, &tmW, c0, n0, bar, leader);
      if (GATED) fetch<1>(dst + 128 * kChunk, &tmW, c0, a.N + n0, bar, leader);
      fetch<1>(dst + C::kA, &tmX, c0, 0, bar, leader);
      p.next(C::kStages);
    }
    wait_released<C::kStages>(empty, issued);
    __syncwarp();
  } else if (warp == 1) {
    Pipe p, c;
    const uint32_t leader = elect_lane();
    const uint32_t idesc = a.idesc | ((uint32_t)(NT >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);   // the same in every lane, and known to be
    const uint64_t desc0 = sw128_desc(smem_u32(smem));
    for (int k = 0; k < mine; ++k) {
      if (TEST && k == kGiveUpAt && a.give_up == GIVE_UP_MMA) break;
      if (!wait_for<TEST>(&acc_empty[c.i], c.ph ^ 1u, a)) break;
      if (!wait_for<TEST>(&full[p.i], p.ph, a)) break;
      tc_fence_after();
      const uint64_t ad = desc0 + (uint64_t)(p.i * (C::kStage / 16)), bd = ad + C::kA / 16;
#pragma unroll
      for (int i = 0; i < P; ++i)
        multiply_chunk<1>(tm + (uint32_t)((c.i * P + i) * NT), ad + (uint64_t)(i * 128 * kChunk / 16), bd, idesc, leader);
      commit_one(&empty[p.i], leader);
      commit_one(&acc_full[c.i], leader);
      p.next(C::kStages);
      c.next(2);
    }
    commit_one(last, leader);
    mbar_wait_bounded(last, 0, &g_block_status);
    __syncwarp();
  } else {
    const int q = warp & 3;
    float* sc = reinterpret_cast<float*>(smem + C::kScaleAt) + (warp - 2) * (2 * P * NT);
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll
    for (int i = 0; i < P * NT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    // the scales of a chunk: a lane's tokens times the gate's and the up's block, two chunks ahead
    constexpr int NX = NT > 32 ? 2 : 1;
    const int blk = n0 / 128;
    float xr[2][NX], wr[2][P];
    auto fetch_scales = [&](int slot, int i) {
      const int k = min(rank + i * S, b.kb - 1);
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        const int t = lane + 32 * j;
        xr[slot][j] = t < nt ? b.xs[(size_t)t * b.ld_xs + k] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < P; ++j) wr[slot][j] = b.ws[(size_t)(blk + j * b.nb) * b.ld_ws + k];
    };
    fetch_scales(0, 0);
    fetch_scales(1, 1);
    Pipe c;
    auto chunk = [&](int slot, int k) {
      float* s = sc + slot * (P * NT);
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < NX; ++i)
          if (lane + 32 * i < NT) s[j * NT + lane + 32 * i] = xr[slot][i] * wr[slot][j];
      __syncwarp();
      fetch_scales(slot, k + 2);
      ok = __all_sync(0xffffffffu, wait_for<TEST>(&acc_full[c.i], c.ph, a));
      if (!ok) return;
      tc_fence_after();
      const uint32_t d = lanes + (uint32_t)(c.i * P * NT);
#pragma unroll
      for (int g = 0; g < P * NT / 16; ++g) {
        uint32_t v[16];
        tmem_ld16(d + (uint32_t)(g * 16), v);
        wait_ld(v);
        if (g == P * NT / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[c.i]);
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 f = *reinterpret_cast<const float4*>(s + g * 16 + 2 * j);
          acc[g * 8 + j] = blk::fma2(pair_at(v, j), make_float2(f.x, f.y), acc[g * 8 + j]);
          acc[g * 8 + j + 1] = blk::fma2(pair_at(v, j + 1), make_float2(f.z, f.w), acc[g * 8 + j + 1]);
        }
      }
      c.next(2);
    };
    for (int k = 0; k < mine && ok; k += 2) {
      chunk(0, k);
      if (ok && k + 1 < mine) chunk(1, k + 1);
    }
  }

  // Token c of the tile belongs to rank c % S: every CTA sends its part of c's
  // rows there, as slot c / S, and the owner adds the parts in rank order.
  __syncwarp();
  if (S > 1) {
    if (!C::kOwnRecv) cluster_arrive();   // this CTA's stages are free
    cluster_wait();
  } else if (!C::kOwnRecv) {
    __syncthreads();
  }
  if (warp >= 2 && ok) {
    const uint32_t recv = smem_u32(smem + C::kRecvAt) + (uint32_t)(rank * cap * P * 512 + ((warp & 3) * 32 + lane) * 4);
    int owner = 0;
    uint32_t at = recv;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      if (c < nt) {
        uint32_t addr;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(at), "r"(owner));
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 v = acc[(i * NT + c) / 2];
          st_cluster_f32(addr + (uint32_t)(i * 512), c & 1 ? v.y : v.x);
        }
      }
      if (++owner == S) {
        owner = 0;
        at += P * 512;
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }

  // A warp finishes a token's 128 features, four to a lane: neighbours where the
  // output takes wide stores, else 32 apart, so that single stores lie side by side.
  const bool quant = out_dtype == MOE_W4A16_E4M3;
  const bool wide = quant || (a.vec == 4 && n0 + 128 <= a.N);
  const int step = wide ? 1 : 32, f = lane * (wide ? 4 : 1), n = n0 + f;
  const int own = (nt - rank + S - 1) / S;   // tokens of this CTA
  const float* parts = reinterpret_cast<const float*>(smem + C::kRecvAt) + f;
  const bool in = quant || n < a.N;
  Four cb[P] = {};
  if (a.bias && n < a.N) {
#pragma unroll
    for (int i = 0; i < P; ++i) cb[i] = load_columns(a, a.bias + i * a.N, n, step);
  }
  for (int s = warp; s < own; s += C::kThreads / 32) {
    const int t[1] = {s * S + rank};
    const bool live[1] = {in};
    float v[4] = {}, up[GATED ? 4 : 1] = {};
    const float* p = parts + s * (P * 128);
#pragma unroll 2
    for (int r = 0; r < S; ++r, p += cap * P * 128) {
      if (wide) {
        const float4 g = *reinterpret_cast<const float4*>(p);
        v[0] += g.x, v[1] += g.y, v[2] += g.z, v[3] += g.w;
        if constexpr (GATED) {
          const float4 h = *reinterpret_cast<const float4*>(p + 128);
          up[0] += h.x, up[1] += h.y, up[2] += h.z, up[3] += h.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] += p[j * 32];
          if constexpr (GATED) up[j] += p[128 + j * 32];
        }
      }
    }
    activate_quads<GATED, 1>(
        a, [&](bool) { return Four{}; }, [&](bool of_up) { return cb[GATED && of_up]; }, v, up);
    if (quant) store_e4m3_row(b, t[0], n0, lane, v);
    else if (!in) continue;
    else if (out_dtype == MOE_W4A16_F16) store_quads<__half, 1>(a, t, live, n, step, v);
    else if (out_dtype == MOE_W4A16_BF16) store_quads<__nv_bfloat16, 1>(a, t, live, n, step, v);
    else store_quads<float, 1>(a, t, live, n, step, v);
  }
}

// -------------------------------------------------------------------- wide
template <int BN>
struct WideCfg {
  static constexpr int kA = 128 * kChunk;      // the 128 token rows of this CTA
  static constexpr int kB = BN / 2 * kChunk;   // this CTA's half of the weight rows
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = 192 * 1024 / kStage > 6 ? 6 : 192 * 1024 / kStage;
  static constexpr int kEpiWarps = 8;
  static constexpr int kTurn = 32 * 32 * 4;   // per epilogue warp: 32 rows x 32 FP32 columns
  // Accumulators.  From a chunk's commit until the next MMAs into the same columns
  // pass some 900 cycles (wake up, read and add, arrive, wake up); 256 columns
  // have room for two only, whose MMAs take 512.
  static constexpr int kAccs = BN == 256 ? 2 : 4;
  static constexpr int kBars = 2 * kStages + 2 * kAccs + 4 + 1;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * kTurn + kBars * 8 + 16 + 1024;
  // Warp 0 loads, warp 1 multiplies, warps 4-11 add up and finish.  Three warps
  // share a scheduler's 16384 registers, 168 each at launch; the first warpgroup
  // leaves all but 40 of its threads' to the others (40 + 2 x 232 = 3 x 168),
  // which hold up to 128 sums and 32 values on their way.
  static constexpr int kThreads = 128 + kEpiWarps * 32;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  // The CTAs of a pair, and of a narrow kernel's cluster, wait for one another with
  // tensor memory in hand.  A pair shares no SM with another pair nor with a CTA of
  // a cluster (two of which have tensor memory enough), so that none of them waits
  // for what another one holds.
  static_assert(kSmem + 1024 + 85 * 1024 > 228 * 1024, "alone on an SM but for CTAs without a cluster");
};

// 32 bytes of a row, loaded and stored at once: full sectors, whatever the rows'
// distance.
DEV_INLINE void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
DEV_INLINE void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// The end of the epilogue for a thread's 16 gate and 16 up sums of a token, the
// features from n on.  A lane stores its own row, in whole 32-byte sectors
// (2048 tokens, [11264][2048]: 50 us; turned first, as other outputs are, 54.
// Without the gate the two are as fast, and with few columns turning is faster).
template <typename O>
DEV_INLINE void finish_rows(const LinearArgs& a, const uint32_t (&s)[2][16], int t, int n) {
  constexpr int kWords = 16 * (int)sizeof(O) / 4, kPer = 4 / (int)sizeof(O);
  float v[16], u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __uint_as_float(s[0][i]);
    u[i] = __uint_as_float(s[1][i]);
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] += a.bias[n + i];
      u[i] += a.bias[a.N + n + i];
    }
  }
  const bool live = t < a.T;
  union {
    uint32_t w[kWords / 8][8];
    O o[16];
  } x = {};
  if (a.res && live) {
#pragma unroll
    for (int i = 0; i < kWords / 8; ++i)
      load32(static_cast<const O*>(a.res) + (size_t)t * a.ld_res + n + i * 8 * kPer, x.w[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    x.o[i] = blk::from_float<O>(silu(v[i]) * u[i] + (a.res ? blk::to_float(x.o[i]) : 0.f));
  if (live) {
#pragma unroll
    for (int i = 0; i < kWords / 8; ++i) store32(static_cast<O*>(a.out) + (size_t)t * a.ld_out + n + i * 8 * kPer, x.w[i]);
  }
  __syncwarp();   // rows past T: the caller's next loads of tensor memory want the warp converged
}

// Up to 32 rows of up to 32 bytes from `turn` (9 words a row), by a warp.  A call:
// inlined, it makes the other columns' loop slower (4096^3 76 us instead of 73).
__device__ __noinline__ void store_bytes(const uint32_t* turn, uint8_t* at, long long ld, int rows, int cols, bool words) {
  const int lane = threadIdx.x & 31;
  if (words && cols >= 32) {
    const int f = lane % 8;
#pragma unroll 2
    for (int r = lane / 8; r < rows; r += 4) *reinterpret_cast<uint32_t*>(at + r * ld + 4 * f) = turn[r * 9 + f];
  } else if (lane < cols) {
#pragma unroll 2
    for (int r = 0; r < rows; ++r) at[r * ld + lane] = reinterpret_cast<const uint8_t*>(turn)[r * 36 + lane];
  }
}

// A thread's kF features of a token (the sums are in tensor memory) to E4M3 with
// the scale of their block, which a thread has whole (kF = 128) or shares with
// the same lane of the quarter's other warp: first the features' values back
// into the place of their (gate) sums and the largest, then scaled and stored.
// The two warps meet at `pair`, a wait with a limit as all of them: a named barrier
// would wait for ever for a warp that gave up.  Where it runs out the status says
// so, and the values of the tile count for nothing.
template <bool GATED, int kF, bool TEST, typename Column>
DEV_INLINE void finish_e4m3(const BlockArgs& b, uint32_t d, Column column, int t, int n0, float* row_max,
                            uint32_t* turn, int h, int q, uint64_t* pair, int parity) {
  static_assert(kF == 64 || kF == 128, "one or two warps to a block");
  const LinearArgs& a = b.a;
  const int lane = threadIdx.x & 31;
  float m = 0.f;
#pragma unroll 1
  for (int c = 0; c < kF; c += 16) {
    const int n = n0 + c;
    uint32_t g[16], w[16];
    tmem_ld16(d + column(c), g);
    if (GATED) tmem_ld16(d + column(kF + c), w);
    wait_ld(g);
    if (GATED) wait_ld(w);
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(g[j]);
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] += a.bias[min(n + j, a.N - 1)];
    }
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float up = __uint_as_float(w[j]);
        if (a.bias) up += a.bias[a.N + min(n + j, a.N - 1)];
        v[j] = silu(v[j]) * up;
      }
    } else {
      activate(v, a.act);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (n + j >= a.N) v[j] = 0.f;
      m = fmaxf(m, fabsf(v[j]));   // NaN is left out, its value carries it
      g[j] = __float_as_uint(v[j]);
    }
    tmem_st16(d + column(c), g);
  }
  tmem_wait_st();
  if (kF < 128) {
    row_max[h * 128 + q * 32 + lane] = m;
    __syncwarp();
    if (lane == 0) mbar_arrive(pair);
    wait_for<TEST>(pair, (uint32_t)parity, a);
    __syncwarp();
    m = fmaxf(m, row_max[(h ^ 1) * 128 + q * 32 + lane]);
  }
  float s = m * (1.f / 448.f);
  if (s < kTiny) s = 0.f;
  const float inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
  const bool live = t < a.T;
  if (live && n0 < a.N && (kF == 128 || h == 0)) b.qs[(size_t)t * b.nb + n0 / 128] = s;
  __syncwarp();   // the loads of tensor memory below want the warp converged
  uint8_t* out = static_cast<uint8_t*>(a.out) + (size_t)t * a.ld_out + n0;
#pragma unroll 1
  for (int c = 0; c < kF && n0 + c < a.N; c += 32) {
    uint32_t g[2][16], w[8];
    tmem_ld16(d + column(c), g[0]);
    tmem_ld16(d + column(c + 16), g[1]);
    wait_ld(g[0]);
    wait_ld(g[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t* p = &g[j / 4][4 * (j % 4)];
      const float2 lo = make_float2(__uint_as_float(p[0]) * inv, __uint_as_float(p[1]) * inv);
      const float2 hi = make_float2(__uint_as_float(p[2]) * inv, __uint_as_float(p[3]) * inv);
      w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
             (uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16;
    }
    if (b.wide_rows && n0 + c + 32 <= a.N) {
      if (live) store32(out + c, w);
      __syncwarp();
    } else {
      // other rows are turned, so that the lanes of a store lie side by side, in
      // words or in bytes (T = 2274, N = 5328, K = 112: 18 us, each lane its own
      // row's bytes 115; T = 333, N = 4001, K = 1424: 10.7 and 27)
#pragma unroll
      for (int j = 0; j < 8; ++j) turn[lane * 9 + j] = w[j];
      __syncwarp();
      store_bytes(turn, static_cast<uint8_t*>(a.out) + (size_t)(t - lane) * a.ld_out + n0 + c, a.ld_out,
                  min(32, a.T - t + lane), a.N - n0 - c, a.vec == 4);
      __syncwarp();
    }
  }
}

template <bool GATED, int BN, typename O, bool TEST>
__global__ void __launch_bounds__(WideCfg<BN>::kThreads, 1)
    linear_blocks_wide_kernel(const __grid_constant__ BlockArgs b, const __grid_constant__ CUtensorMap tmW,
                              const __grid_constant__ CUtensorMap tmX) {
  using C = WideCfg<BN>;
  constexpr bool QUANT = std::is_same<O, E4M3>::value;
  constexpr uint32_t kCols = C::kAccs * BN;
  constexpr int FT = GATED ? BN / 2 : BN;    // output features per tile
  constexpr int kW = BN / 2;                 // sums of a thread; GATED: of kF gate columns, then of their up columns
  constexpr int kF = GATED ? kW / 2 : kW;    // features of a thread
  static_assert(!QUANT || FT % 128 == 0, "a block of the output lies in a tile");
  static_assert(2 * 256 * 4 <= C::kTurn / 2 && 32 * 9 * 4 <= C::kTurn / 2, "both fit");
  const LinearArgs& a = b.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* turn = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
  // E4M3 outputs, which turn in the second half of a warp's place: the halves'
  // largest values, [tile's parity][half][128], in the first
  float* row_max = turn;
  uint64_t* full = reinterpret_cast<uint64_t*>(turn + C::kEpiWarps * (C::kTurn / 4));
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kAccs;
  uint64_t* pairs = acc_empty + C::kAccs;   // [lane quarter] of its two warps, for E4M3 outputs
  uint64_t* last = pairs + 4;               // every MMA of the pair is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(last + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int mtiles = (a.T + 255) / 256, tiles = mtiles * ((a.N + FT - 1) / FT);
  const int nk = b.kb, first = blockIdx.x / 2, step = gridDim.x / 2;

  if (threadIdx.x == 32) {
    prefetch_map(&tmW);
    prefetch_map(&tmX);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kAccs; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 2 * C::kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&pairs[q], 2);
    mbar_init(last, 1);
    fence_mbar_init();
  }
  __syncwarp();
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
  pdl_wait();   // after the allocation: see linear_narrow_kernel
  pdl_trigger();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
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
          fetch<2>(dst, &tmX, k * 128, m0, bar0, leader);
          fetch<2>(dst + C::kA, &tmW, k * 128, b0, bar0, leader);
          ++issued;
          p.next(C::kStages);
        }
      }
      wait_released<C::kStages>(empty, issued);
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      Pipe p, acc;
      bool ok = true;
      const uint32_t leader = elect_lane();
      const uint32_t idesc = a.idesc | ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
      const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
      const uint64_t desc0 = sw128_desc(smem_u32(smem));
      for (int tile = first; tile < tiles && ok; tile += step)
        for (int k = 0; k < nk; ++k) {
          if ((TEST && k == kGiveUpAt && a.give_up == GIVE_UP_MMA) || !wait_for<TEST>(&acc_empty[acc.i], acc.ph ^ 1u, a) ||
              !wait_for<TEST>(&full[p.i], p.ph, a)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + (uint64_t)(p.i * (C::kStage / 16));
          multiply_chunk<2>(tm + (uint32_t)(acc.i * BN), ad, ad + C::kA / 16, idesc, leader);
          commit_pair(&empty[p.i], 3, leader);
          commit_pair(&acc_full[acc.i], 3, leader);
          p.next(C::kStages);
          acc.next(C::kAccs);
        }
      commit_pair(last, 1, leader);
      mbar_wait_bounded(last, 0, &g_block_status);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // a TMEM lane (token) per thread; the two warps of a lane quarter share the columns
    const int q = warp & 3, h = (warp - 4) >> 2;
    float* buf = turn + (warp - 4) * (C::kTurn / 4);
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16), empty0 = map_to_rank(acc_empty, 0);
    // the accumulator's column of this warp's sum i
    auto column = [&](int i) { return (uint32_t)(GATED ? (i < kF ? h * kF + i : BN / 2 + h * kF + i - kF) : h * kW + i); };
    Pipe acc;
    bool ok = true;
    int parity = 0;   // of the tiles finished to E4M3
    for (int tile = first; tile < tiles && ok; tile += step) {
      const int t0 = (tile % mtiles) * 256 + rank * 128 + q * 32, n0 = tile / mtiles * FT + h * kF;   // this warp's
      const int blk = min(n0 / 128, b.nb - 1);
      const float* xs = b.xs + (size_t)min(t0 + lane, a.T - 1) * b.ld_xs;
      const float* ws = b.ws + (size_t)blk * b.ld_ws;
      const float* wu = b.ws + (size_t)(GATED ? blk + b.nb : blk) * b.ld_ws;   // of the up rows
      float2 sum[kW / 2];
#pragma unroll
      for (int i = 0; i < kW / 2; ++i) sum[i] = make_float2(0.f, 0.f);
      float4 nx = load_scales(xs, 0, nk, b.xs_vec), nw = load_scales(ws, 0, nk, b.ws_vec), nu = {};
      if (GATED) nu = load_scales(wu, 0, nk, b.ws_vec);
      for (int k = 0; k < nk && ok; k += 4) {
        const float4 sg = make_float4(nx.x * nw.x, nx.y * nw.y, nx.z * nw.z, nx.w * nw.w);
        const float4 su = make_float4(nx.x * nu.x, nx.y * nu.y, nx.z * nu.z, nx.w * nu.w);
        if (k + 4 < nk) {
          nx = load_scales(xs, k + 4, nk, b.xs_vec);
          nw = load_scales(ws, k + 4, nk, b.ws_vec);
          if (GATED) nu = load_scales(wu, k + 4, nk, b.ws_vec);
        }
#pragma unroll 1
        for (int i = 0; i < 4 && k + i < nk; ++i) {
          ok = __all_sync(0xffffffffu, wait_for<TEST>(&acc_full[acc.i], acc.ph, a));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = lanes + (uint32_t)(acc.i * BN);
          const float fg = lane4(sg, i), fu = lane4(su, i);
          // 16 columns are on their way while 16 are added; the MMAs may have the
          // accumulator back as soon as the last are read (the last chunk's is
          // kept for the sums)
          const bool keep = k + i + 1 == nk;
          uint32_t v[2][16];
          tmem_ld16(d + column(0), v[0]);
          wait_ld(v[0]);
#pragma unroll
          for (int g = 0; g < kW / 16; ++g) {
            if (g + 1 < kW / 16) tmem_ld16(d + column(16 * g + 16), v[(g + 1) & 1]);
            const float f = GATED && 16 * g >= kF ? fu : fg;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sum[g * 8 + j] = blk::fma2(pair_at(v[g & 1], j), make_float2(f, f), sum[g * 8 + j]);
            if (g + 1 < kW / 16) wait_ld(v[(g + 1) & 1]);
            if (g + 2 == kW / 16 && !keep) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_at(empty0 + (uint32_t)(acc.i * 8));
            }
          }
          if (!keep) acc.next(C::kAccs);
        }
      }
      if (!ok || (TEST && a.give_up == GIVE_UP_FINISH && rank == 0 && warp == 4)) break;
      const uint32_t d = lanes + (uint32_t)(acc.i * BN);
#pragma unroll
      for (int g = 0; g < kW / 16; ++g) {
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[2 * j] = __float_as_uint(sum[g * 8 + j].x);
          v[2 * j + 1] = __float_as_uint(sum[g * 8 + j].y);
        }
        tmem_st16(d + column(16 * g), v);
      }
      tmem_wait_st();
      if (t0 < a.T) {   // the same for a lane quarter
        if constexpr (QUANT) {
          finish_e4m3<GATED, kF, TEST>(b, d, column, t0 + lane, n0, row_max + parity * 256,
                                  reinterpret_cast<uint32_t*>(buf) + 512, h, q, &pairs[q], parity);
          parity ^= 1;
        } else {
          constexpr int kStep = GATED ? 16 : 32, kLanes = kStep / 4;
          const bool direct = GATED && b.wide_rows && n0 + kF <= a.N;
#pragma unroll 1
          for (int c = 0; c < kF && n0 + c < a.N; c += kStep) {
            const int n = n0 + c;
            uint32_t v[2][16];
            tmem_ld16(d + column(c), v[0]);
            tmem_ld16(d + column(GATED ? kF + c : c + 16), v[1]);
            wait_ld(v[0]);
            wait_ld(v[1]);
            if (direct) {
              if constexpr (GATED) finish_rows<O>(a, v, t0 + lane, n);
            } else {
              Four cb = {};   // as finish_turned wants them
              const int cl = GATED ? lane & 15 : lane, up = GATED && lane >= 16 ? a.N : 0;
              if (a.bias && cl < kLanes) {
                const bool wide = a.vec == 4 && n + kStep <= a.N;
                cb = load_columns(a, a.bias + up, n + cl * (wide ? 4 : 1), wide ? 1 : kLanes);
              }
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(buf + lane * 32 + ((j ^ (lane & 7)) * 4)) =
                    make_uint4(v[j / 4][4 * (j % 4)], v[j / 4][4 * (j % 4) + 1], v[j / 4][4 * (j % 4) + 2], v[j / 4][4 * (j % 4) + 3]);
              __syncwarp();
              finish_turned<GATED, O>(a, buf, t0, n, lane, Four{}, cb, 0);
              __syncwarp();
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(empty0 + (uint32_t)(acc.i * 8));
      acc.next(C::kAccs);
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

// -------------------------------------------------------------- host side
struct Problem {
  BlockArgs b;
  const void *x, *w;
  int64_t ld_x, ld_w;
  int out_dtype, num_sms, dev;
};

template <bool GATED, int NT, int PER, bool TEST>
cudaError_t launch_narrow_s(const Problem& p, int S, cudaStream_t st) {
  using C = NarrowCfg<GATED, NT, PER>;
  const LinearArgs& a = p.b.a;
  CUtensorMap mw, mx;
  if (!encode_rows(&mw, p.w, GATED ? 2ll * a.N : a.N, a.K, 1, p.ld_w, 128) ||
      !encode_rows(&mx, p.x, a.T, a.K, 1, p.ld_x, NT))
    return cudaErrorInvalidValue;
  auto kernel = linear_blocks_narrow_kernel<GATED, NT, PER, TEST>;
  const cudaError_t e = opt_in_smem((const void*)kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N + 127) / 128;
  const int prefetch = tiles * S > p.num_sms;   // as linear_narrow_kernel
  return launch_pdl(kernel, dim3((unsigned)(tiles * S)), dim3(C::kThreads), C::kSmem, st, S, p.b, mw, mx, p.out_dtype, S,
                    prefetch);
}

// Fewer tiles than SMs are split over clusters.  With more, one CTA to a tile, and
// for up to 16 tokens three to an SM, which evens out what is left in the last
// round (T = 8, W [50304][2048], 393 tiles: 18.4 us, two to an SM 22.1, clusters
// of two 24.9; T = 1, W [28672][8192] 37.0, 37.8, 40.8).
template <bool GATED, int NT, bool TEST = false>
cudaError_t launch_narrow(const Problem& p, cudaStream_t st) {
  using C = NarrowCfg<GATED, NT, 2>;
  const int tiles = (p.b.a.N + 127) / 128;
  if (tiles >= p.num_sms) {
    if constexpr (!GATED && NT == 16 && !TEST) return launch_narrow_s<GATED, NT, 3, TEST>(p, 1, st);
    return launch_narrow_s<GATED, NT, 2, TEST>(p, 1, st);
  }
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
  return launch_narrow_s<GATED, NT, 2, TEST>(p, split_of(tiles, p.b.kb, fit[0], fit[1]), st);
}

template <bool GATED, int BN, typename O, bool TEST = false>
cudaError_t launch_wide_o(const Problem& p, cudaStream_t st) {
  using C = WideCfg<BN>;
  const LinearArgs& a = p.b.a;
  CUtensorMap mw, mx;
  if (!encode_rows(&mw, p.w, GATED ? 2ll * a.N : a.N, a.K, 1, p.ld_w, BN / 2) ||
      !encode_rows(&mx, p.x, a.T, a.K, 1, p.ld_x, 128))
    return cudaErrorInvalidValue;
  auto kernel = linear_blocks_wide_kernel<GATED, BN, O, TEST>;
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
  const long long tiles = (long long)((a.T + 255) / 256) * ((a.N + FT - 1) / FT);
  if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(kernel, dim3((unsigned)((tiles < n ? tiles : n) * 2)), dim3(C::kThreads), C::kSmem, st, 2, p.b, mw,
                    mx);
}

template <bool GATED, int BN>
cudaError_t launch_wide(const Problem& p, cudaStream_t st) {
  if constexpr (BN >= (GATED ? 256 : 128))
    if (p.out_dtype == MOE_W4A16_E4M3) return launch_wide_o<GATED, BN, E4M3>(p, st);
  return p.out_dtype == MOE_W4A16_F16    ? launch_wide_o<GATED, BN, __half>(p, st)
         : p.out_dtype == MOE_W4A16_BF16 ? launch_wide_o<GATED, BN, __nv_bfloat16>(p, st)
                                         : launch_wide_o<GATED, BN, float>(p, st);
}

// The tile width of the wide kernel: rounds of tiles over the resident clusters
// times a tile's time, a K chunk 0.42, 0.29 or 0.19 us at 256, 128 or 64 weight
// rows and the end of a tile 3, 1.5 or 0.8 us, in units of 10 ns.  Measured with
// 256 / 128 / 64 rows: T = 512, N = K = 2048 12.8 / 9.2 / 7.0 us, T = 2048, N =
// 4096 28 / 33 / 34, SWIGLU N = 5632 50 / 64 / 83.  An E4M3 output's block of 128
// features has to lie in a tile.
template <bool GATED>
int wide_rows(const Problem& p) {
  const LinearArgs& a = p.b.a;
  const long long slots = p.num_sms / 2;
  const int rows[3] = {256, 128, 64}, chunk[3] = {42, 29, 19}, end[3] = {300, 150, 80};
  int best = 0;
  long long cost = -1;
  for (int i = 0; i < 3; ++i) {
    const int ft = GATED ? rows[i] / 2 : rows[i];
    if (p.out_dtype == MOE_W4A16_E4M3 && ft < 128) continue;
    const long long tiles = (long long)((a.T + 255) / 256) * ((a.N + ft - 1) / ft);
    const long long c = (tiles + slots - 1) / slots * (p.b.kb * (long long)chunk[i] + end[i]);
    if (cost < 0 || c < cost) {
      cost = c;
      best = rows[i];
    }
  }
  return best;
}

template <bool GATED>
cudaError_t launch_gated(const Problem& p, cudaStream_t st) {
  if (p.b.a.T <= 16) return launch_narrow<GATED, 16>(p, st);
  if (p.b.a.T <= 32) return launch_narrow<GATED, 32>(p, st);
  // 64 tokens, SWIGLU [11264][2048]: 13.6 us, the wide kernel 12.1; 48 12.3 and 12.2;
  // without the gate, W [4096][4096] 9.7 and 9.7, [2048][5632] 8.0 and 11.3
  if (p.b.a.T <= (GATED ? 48 : 64)) return launch_narrow<GATED, 64>(p, st);
  const int rows = wide_rows<GATED>(p);
  return rows == 256   ? launch_wide<GATED, 256>(p, st)
         : rows == 128 ? launch_wide<GATED, 128>(p, st)
                       : launch_wide<GATED, 64>(p, st);
}

}  // namespace

cudaError_t take_linear_blocks_status(DevStatus* s) {
  cudaError_t e = cudaMemcpyFromSymbol(s, g_block_status, sizeof *s);
  if (e == cudaSuccess && s->flags) {
    const DevStatus zero = {};
    e = cudaMemcpyToSymbol(g_block_status, &zero, sizeof zero);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  return e;
}

// give_up nonzero: the self-test, with the limit of its waits.
static moe_w4a16_status run_linear_blocks(const char* op, const moe_w4a16_linear_blocks_config* cfg, int64_t T,
                                          const void* x, const float* x_scale, const void* w, const float* w_scale,
                                          const float* bias, const void* residual, void* out, float* out_scale,
                                          moe_w4a16_stream_t stream, int give_up, int64_t limit) {
  if (!cfg) return blk::reject(op, "cfg is NULL");
  const moe_w4a16_linear_blocks_config c = *cfg;
  if (c.out_dtype < MOE_W4A16_F16 || c.out_dtype > MOE_W4A16_E4M3) return blk::reject(op, "out_dtype must be F16, BF16, F32 or E4M3");
  if (c.act < MOE_W4A16_ACT_NONE || c.act > MOE_W4A16_ACT_SWIGLU) return blk::reject(op, "unknown activation");
  if (c.reserved || c.reserved2) return blk::reject(op, "reserved must be 0");
  if (c.n < 1 || c.n > (1 << 29) || c.k < 1 || c.k > (1 << 24))
    return blk::reject(op, "n outside [1, 2^29] or k outside [1, 2^24]");
  if (T < 0 || T > (1 << 30)) return blk::reject(op, "T outside [0, 2^30]");
  const bool quant = c.out_dtype == MOE_W4A16_E4M3, gated = c.act == MOE_W4A16_ACT_SWIGLU;
  const int os = elem_size(c.out_dtype), kb = (c.k + 127) / 128, nb = (c.n + 127) / 128;
  int64_t ld_x = c.ld_x ? c.ld_x : c.k, ld_w = c.ld_w ? c.ld_w : c.k;
  const int64_t ld_out = c.ld_out ? c.ld_out : c.n, ld_res = c.ld_residual ? c.ld_residual : c.n;
  const int64_t ld_xs = c.ld_x_scale ? c.ld_x_scale : kb, ld_ws = c.ld_w_scale ? c.ld_w_scale : kb;
  if (ld_x < c.k || ld_w < c.k || ld_out < c.n || ld_res < c.n || ld_xs < kb || ld_ws < kb)
    return blk::reject(op, "a row stride is below the row length");
  // a single row has no stride to speak of: any that the tensor map takes
  if (T < 2) ld_x = (c.k + 15ll) / 16 * 16;
  if (c.n == 1 && !gated) ld_w = (c.k + 15ll) / 16 * 16;
  if (ld_x % 16 || ld_w % 16) return blk::reject(op, "the row strides of x and W must be multiples of 16 bytes");
  if (ld_x >= (1ll << 40) || ld_w >= (1ll << 40)) return blk::reject(op, "a row stride is too large");
  if (T == 0) return MOE_W4A16_OK;
  if (!x || !x_scale || !w || !w_scale || !out) return blk::reject(op, "NULL x, x_scale, w, w_scale or out");
  if (quant != (out_scale != nullptr)) return blk::reject(op, "out_scale goes with an E4M3 output");
  if (quant && residual) return blk::reject(op, "an E4M3 output takes no residual");
  if (!blk::aligned(x, 16) || !blk::aligned(w, 16)) return blk::reject(op, "x and w must be 16-byte aligned");
  if (!blk::aligned(x_scale, 4) || !blk::aligned(w_scale, 4) || !blk::aligned(bias, 4) || !blk::aligned(out, os) ||
      !blk::aligned(residual, os) || !blk::aligned(out_scale, 4))
    return blk::reject(op, "a pointer is not aligned to its type");
  if (out == x || out == w) return blk::reject(op, "out must not alias x or w");
  if (quant && (out_scale == x_scale || out_scale == w_scale)) return blk::reject(op, "out_scale must not alias x_scale or w_scale");
  Problem p;
  p.x = x;
  p.w = w;
  p.ld_x = ld_x;
  p.ld_w = ld_w;
  p.out_dtype = c.out_dtype;
  p.num_sms = blk::current_sms(&p.dev);
  if (p.num_sms < 1) return blk::launch_failed(op, cudaErrorNoDevice);
  BlockArgs& b = p.b;
  LinearArgs& a = b.a;
  a.xs = a.ws = nullptr;
  a.bias = bias;
  a.res = residual;
  a.out = out;
  a.ld_res = ld_res;
  a.ld_out = ld_out;
  a.T = (int)T;
  a.N = c.n;
  a.K = c.k;
  a.act = c.act;
  a.idesc = 1u << 4;   // FP32 accumulator; kind::f8f6f4 0 = E4M3
  const size_t vb = 4 * (size_t)os;
  a.vec = blk::aligned(out, vb) && ld_out % 4 == 0 && (!residual || (blk::aligned(residual, vb) && ld_res % 4 == 0)) ? 4 : 1;
  a.give_up = give_up;
  a.limit = limit;
  b.xs = x_scale;
  b.ws = w_scale;
  b.ld_xs = ld_xs;
  b.ld_ws = ld_ws;
  b.kb = kb;
  b.nb = nb;
  b.xs_vec = kb % 4 == 0 && ld_xs % 4 == 0 && blk::aligned(x_scale, 16);
  b.ws_vec = kb % 4 == 0 && ld_ws % 4 == 0 && blk::aligned(w_scale, 16);
  b.qs = out_scale;
  b.wide_rows = blk::aligned(out, 32) && ld_out * os % 32 == 0 &&
                (!residual || (blk::aligned(residual, 32) && ld_res * os % 32 == 0));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = give_up ? (T <= 16 ? launch_narrow<false, 16, true>(p, st) : launch_wide_o<true, 256, E4M3, true>(p, st))
                        : gated ? launch_gated<true>(p, st)
                                : launch_gated<false>(p, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
}

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_linear_blocks(const moe_w4a16_linear_blocks_config* cfg, int64_t T,
                                                                  const void* x, const float* x_scale, const void* w,
                                                                  const float* w_scale, const float* bias,
                                                                  const void* residual, void* out, float* out_scale,
                                                                  moe_w4a16_stream_t stream) try {
  return run_linear_blocks("linear_blocks", cfg, T, x, x_scale, w, w_scale, bias, residual, out, out_scale, stream, 0, 0);
} catch (...) {   // the host's heap is full
  return MOE_W4A16_ERR_OOM;
}

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_selftest_linear_blocks(
    const moe_w4a16_linear_blocks_config* cfg, int64_t T, const void* x, const float* x_scale, const void* w,
    const float* w_scale, void* out, float* out_scale, int32_t which, int64_t limit_cycles,
    moe_w4a16_stream_t stream) try {
  const char* op = "selftest_linear_blocks";
  if (!cfg) return blk::reject(op, "cfg is NULL");
  if (T < 1 || (T > 16 && T <= 64)) return blk::reject(op, "T outside [1, 16] and (64, 2^30]");
  if (T <= 16 ? cfg->out_dtype == MOE_W4A16_E4M3 || cfg->act != MOE_W4A16_ACT_NONE
              : cfg->out_dtype != MOE_W4A16_E4M3 || cfg->act != MOE_W4A16_ACT_SWIGLU)
    return blk::reject(op, "takes no activation and no E4M3 output up to 16 tokens, SWIGLU and E4M3 above 64");
  if (which < 0 || which > (T <= 16 ? 2 : 3)) return blk::reject(op, "which outside [0, 2], above 64 tokens [0, 3]");
  if (limit_cycles < 1000 || limit_cycles > MOE_WAIT_CYCLES) return blk::reject(op, "limit_cycles outside [1000, 2^31]");
  return run_linear_blocks(op, cfg, T, x, x_scale, w, w_scale, nullptr, nullptr, out, out_scale, stream,
                           GIVE_UP_MMA + which, limit_cycles);
} catch (...) {   // the host's heap is full
  return MOE_W4A16_ERR_OOM;
}
