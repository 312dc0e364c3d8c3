// moe_w4a16_token_logprobs: of every row of logits the log probability of a
// given token, the entropy, and the k most likely tokens:
//   M = max x,  S = sum e^(x - M),  ln p_i = x_i - M - ln S,
//   entropy = ln S - sum e^(x - M) (x - M) / S.
//
// Bound by reading the logits once: 4096 rows of 131072 BF16 take 165 us (6.5
// TB/s), with 8 alternatives 208, with 32 232; 64 of 151936 FP32 with 5 alternatives
// 13.2, one of 50304 with 20 5.2, of which the reading is 3.0 and finding them the
// rest.  A row is read by one CTA, or, where there
// are few rows, by the CTAs of a cluster; every thread keeps the running
// maximum m of its values and the two sums relative to it, which are rescaled
// once per batch of values; threads and CTAs join by rescaling to the common
// maximum.
//
// The k largest: a thread's m is the largest of its values so far, and k values
// reach the k-th largest of any groups of threads' maxima.  This threshold is
// found after the 1st, 2nd, 4th, 8th .. batch of values, as the k-th largest of
// 64 groups' maxima: 64 ln(64 / (64 - k)) values reach it where they come in no
// order, 8 for k = 8 and 44 for k = 32.  The 16 bytes around a value that
// reaches it are put aside while they are in registers, about as many
// times 1 + log2(batches) per row; in the end those that still reach it
// are gone through, and their values ordered by counting.  (Picking the single
// values out in the reading loop cost it half as many instructions again.)  Rows
// in which more are put aside than there is room for (values that rise along the
// row) are read once more for what reaches the last threshold; rows in which too
// many or too few are found (ties, masks of the lowest finite value, fewer than k
// values left by the mask) a few times.
//
// What runs once per row is written in short loops: straight code that is new
// to the SM costs some 15 cycles an instruction, waiting for itself.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "block.h"

namespace {

using blk::add2;
using blk::fma2;
using blk::mul2;

struct LogprobArgs {
  const void *x, *tokens;
  float *logprob, *entropy, *top;
  int32_t* ids;
  long long ld;
  int V, k, wide_tokens;
};

constexpr int kMaxTop = 32;
constexpr int kSend = 64;   // candidates that a CTA sends to the cluster's first without ordering them
constexpr float kLog2e = 1.4426950408889634f;
// Stands for a masked value (-inf, NaN) while a row is read: differences to it
// stay finite, and e to their power is 0.  Rows without anything above it are
// read again with care.
template <typename E>
constexpr float kFloor = -1e38f;
template <>
constexpr float kFloor<__half> = -65504.f;

// m: the largest value, s: sum e^(x - m), e: sum e^(x - m) (x - m)
struct Stat {
  float m, s, e;
};

// `a` relative to the larger maximum m.
DEV_INLINE Stat rescale(Stat a, float m) {
  if (a.m == m) return a;
  const float d = a.m - m;
  if (!(d > -100.f) || a.s == 0.f) return Stat{m, 0.f, 0.f};   // e^-100 of at most 2^29 values is nothing beside 1
  const float f = blk::fast_exp2(d * kLog2e);
  return Stat{m, a.s * f, f * (a.e + a.s * d)};
}

// Orders values as unsigned numbers; 0 for what is masked.  -0 equals 0.
DEV_INLINE uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t k = (int)b < 0 ? ~b : b | 0x80000000u;
  return x > -INFINITY ? k : 0u;   // false for NaN
}
constexpr uint32_t kMaskedKey = 0x007fffffu;   // of -inf, below every other
DEV_INLINE float key_value(uint32_t k) { return __uint_as_float((int)k < 0 ? k & 0x7fffffffu : ~k); }
// A candidate: larger values first, then lower places.
DEV_INLINE unsigned long long candidate(uint32_t key, int place) {
  return (unsigned long long)key << 32 | (uint32_t)~place;
}
DEV_INLINE int place_of(unsigned long long c) { return (int)~(uint32_t)c; }

// The join of a warp's (m, s, e): one maximum, one rescaling each, one sum.
DEV_INLINE Stat warp_join(Stat a) {
  const float m = key_value(max(__reduce_max_sync(0xffffffffu, order_key(a.m)), kMaskedKey));
  a = rescale(a, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.e += __shfl_xor_sync(0xffffffffu, a.e, o);
  }
  return Stat{m, a.s, a.e};
}

// Sixteen bytes of a row, on the 16-byte grid in memory.
template <typename E>
struct Win {
  static constexpr int N = 16 / sizeof(E);
  uint4 v;
};
DEV_INLINE uint32_t masked_word(float) { return 0xff800000u; }
DEV_INLINE uint32_t masked_word(__half) { return 0xfc00fc00u; }
DEV_INLINE uint32_t masked_word(__nv_bfloat16) { return 0xff80ff80u; }

DEV_INLINE float2 pair_of(const Win<float>& w, int j) {
  const float* f = reinterpret_cast<const float*>(&w.v);
  return make_float2(f[2 * j], f[2 * j + 1]);
}
// The largest value of a window, no less than the floor (NaN is left out) ..
template <typename H2>
DEV_INLINE float largest_of_pairs(const uint4& v, H2 floor) {
  const H2* p = reinterpret_cast<const H2*>(&v);
  const H2 m = __hmax2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])), floor);
  return fmaxf(__low2float(m), __high2float(m));
}
DEV_INLINE float largest(const Win<float>& w) {
  const float2 a = pair_of(w, 0), b = pair_of(w, 1);
  return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)), kFloor<float>);
}
DEV_INLINE float largest(const Win<__half>& w) { return largest_of_pairs(w.v, __float2half2_rn(kFloor<__half>)); }
DEV_INLINE float largest(const Win<__nv_bfloat16>& w) {
  return largest_of_pairs(w.v, __float2bfloat162_rn(kFloor<__nv_bfloat16>));
}
// .. and a pair of its values, the floor in the place of anything below it and of NaN.
DEV_INLINE float2 floored_pair(const Win<float>& w, int j) {
  const float2 f = pair_of(w, j);
  return make_float2(fmaxf(f.x, kFloor<float>), fmaxf(f.y, kFloor<float>));
}
DEV_INLINE float2 floored_pair(const Win<__half>& w, int j) {
  return __half22float2(__hmax2(reinterpret_cast<const __half2*>(&w.v)[j], __float2half2_rn(kFloor<__half>)));
}
DEV_INLINE float2 floored_pair(const Win<__nv_bfloat16>& w, int j) {
  return __bfloat1622float2(
      __hmax2(reinterpret_cast<const __nv_bfloat162*>(&w.v)[j], __float2bfloat162_rn(kFloor<__nv_bfloat16>)));
}
// The floor as the type holds it.
template <typename E>
DEV_INLINE float floor_of() { return blk::to_float(blk::from_float<E>(kFloor<E>)); }

// What the CTAs of a cluster send to the first.
struct Received {
  Stat stat[8];
  unsigned long long cand[8 * kSend];
};
struct Nothing {};
template <int NT, bool CLUSTER>
struct Shared {
  // windows that can be put aside, and candidates among their values; few where
  // many small CTAs share an SM, whose rows have no more windows.  Rows of 200000
  // FP32 in no order put 284 aside for k = 32, 347 at most (128 threads).
  static constexpr int kWin = NT == 32 ? 128 : 512, kCand = NT == 32 ? 256 : 512;
  static_assert(!CLUSTER || 8 * kSend <= kCand, "the received candidates can all be kept");
  uint4 win[kWin];
  unsigned long long win_max[kWin];   // the window's largest value and its place, as a candidate

  Stat part[32];       // a warp's
  __align__(16) uint32_t group[64];
  uint32_t thr[2], key_max, key_min;
  int win_n, cand_n, kept_n, count[3], warp_n[32];
  unsigned long long best[kMaxTop], cand[kCand], kept[kCand];
  typename std::conditional<CLUSTER, Received, Nothing>::type from;
};

// What a CTA takes of a row: the `windows` whole windows from the place `begin`
// on, and, the first CTA of a row, the `edge` values of the row that no window
// holds, `head` of them at its start.
template <typename E>
struct Part {
  const E* row;
  int V, begin, windows, head, edge;
  DEV_INLINE Win<E> window(int w) const {
    Win<E> r;   // past the L1: read once, but in rows that are read again much later
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.v.x), "=r"(r.v.y), "=r"(r.v.z), "=r"(r.v.w)
                 : "l"(row + begin + (long long)w * Win<E>::N)
                 : "memory");
    return r;
  }
  DEV_INLINE int edge_place(int i) const { return i < head ? i : V - edge + i; }
  // f(value, place) of every value: for what is rare
  template <int NT, typename F>
  DEV_INLINE void each(F f) const {
    if ((int)threadIdx.x < edge) {
      const int c = edge_place(threadIdx.x);
      f(blk::to_float(row[c]), c);
    }
    const uint4* const at = reinterpret_cast<const uint4*>(row + begin);
#pragma unroll 4
    for (int w = threadIdx.x; w < windows; w += NT) {
      const uint4 v = at[w];
#pragma unroll
      for (int j = 0; j < Win<E>::N; ++j) f(blk::to_float(reinterpret_cast<const E*>(&v)[j]), begin + w * Win<E>::N + j);
    }
  }
};

template <int NT, typename Sh>
DEV_INLINE Stat block_join(Stat a, Sh& sh) {
  a = warp_join(a);
  __syncthreads();   // `part` may still be read
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = a;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_join(lane < NT / 32 ? sh.part[lane] : Stat{-INFINITY, 0.f, 0.f});
}

// Any row: nothing left by its mask, infinities, values below the floor.
template <typename E, int NT>
__device__ __noinline__ Stat careful(const Part<E>& p) {
  Stat a = {-INFINITY, 0.f, 0.f};
  p.template each<NT>([&](float x, int) { a.m = fmaxf(a.m, x); });
  if (a.m > -INFINITY)
    p.template each<NT>([&](float x, int) {
      const float d = x == a.m ? 0.f : x - a.m;
      if (d > -100.f) {   // false for what is masked and beside an infinite maximum
        const float q = blk::fast_exp2(d * kLog2e);
        a.s += q;
        a.e = fmaf(q, d, a.e);
      }
    });
  return a;
}

DEV_INLINE int add8(int v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The k-th largest of the maxima of up to 64 groups of neighbouring threads, 0
// where fewer than k have any key: at least k threads' keys reach it.  A
// group's place is counted by the threads of a group.  slot: another one than in
// the call before, which may still be read.
template <int NT, typename Sh>
DEV_INLINE uint32_t threshold(uint32_t key, int k, Sh& sh, int slot) {
  constexpr int NG = NT < 64 ? NT : 64, R = NT / NG;
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = R / 2; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  if (tid % R == 0) sh.group[tid / R] = key;
  if (tid == 0) sh.thr[slot] = 0;
  __syncthreads();
  int larger = 0, equal = 0;
  const uint4* g = reinterpret_cast<const uint4*>(sh.group) + tid % R * (NG / R / 4);
#pragma unroll 2
  for (int i = 0; i < NG / R / 4; ++i) {
    const uint4 v = g[i];
    larger += (v.x > key) + (v.y > key) + (v.z > key) + (v.w > key);
    equal += (v.x == key) + (v.y == key) + (v.z == key) + (v.w == key);
  }
#pragma unroll
  for (int o = R / 2; o > 0; o >>= 1) {
    larger += __shfl_xor_sync(0xffffffffu, larger, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (larger < k && larger + equal >= k) sh.thr[slot] = key;   // every thread of which this holds has the same key
  __syncthreads();
  return sh.thr[slot];
}

// Gives a group's threads entries of a list that lie 64 apart, so that no group
// is left without.
template <int NT>
DEV_INLINE int spread(int tid) {
  constexpr int R = NT < 64 ? 1 : NT / 64;
  return tid % R * 64 + tid / R;
}

// The k largest of the distinct candidates list[0], .. list[n - 1] into sh.best,
// largest first: a candidate's place is counted by eight lanes.
template <int NT, typename Sh>
DEV_INLINE void place_candidates(const unsigned long long* list, int n, int k, Sh& sh) {
  const int tid = threadIdx.x;
#pragma unroll 1
  for (int c0 = 0; c0 < n; c0 += NT / 8) {
    const int c = c0 + tid / 8;
    const unsigned long long mine = c < n ? list[c] : 0;
    int rank = 0;
#pragma unroll 1
    for (int i = tid & 7; i < n; i += 8) rank += list[i] > mine;
    rank = add8(rank);
    if (c < n && (tid & 7) == 0 && rank < k) sh.best[rank] = mine;
  }
  __syncthreads();
}

// The same of the candidates list[0], .. list[n - 1] (0: none), most of which may
// lie below the k-th; their number, at most k, is returned.
template <int NT, typename Sh>
DEV_INLINE int order_candidates(const unsigned long long* list, int n, int k, Sh& sh) {
  const int tid = threadIdx.x;
  if (n > 64) {
    if (tid == 0) sh.kept_n = 0;
    uint32_t key = 0;
#pragma unroll 1
    for (int c = spread<NT>(tid); c < n; c += NT) key = max(key, (uint32_t)(list[c] >> 32));
    const uint32_t thr = max(threshold<NT>(key, k, sh, 0), 1u);
#pragma unroll 1
    for (int c = tid; c < n; c += NT) {
      const unsigned long long mine = list[c];
      if ((uint32_t)(mine >> 32) >= thr) sh.kept[atomicAdd(&sh.kept_n, 1)] = mine;
    }
    __syncthreads();
    n = sh.kept_n;
    list = sh.kept;
  }
  place_candidates<NT>(list, n, k, sh);
  return min(n, k);
}

// Candidates of a part in which too many values crowd at the threshold or too
// few are above the floor: at most kCand into sh.cand, the k largest (or all that
// are not masked) among them, ties to the lower place.  Their number is returned.
// Reads the part twice where at most kCand values are not masked: 1000 rows of
// 131072 BF16 that keep 3 tokens, 20 best, take 244 us (all kept 72).
// from: a number that k keys reach, or 0; where no more do than fit, one reading
// is enough.
template <typename E, int NT, typename Sh>
__device__ __noinline__ int collect_again(const Part<E>& p, int k, uint32_t from, Sh& sh) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (from) {
    if (tid == 0) sh.cand_n = 0;
    __syncthreads();
    p.template each<NT>([&](float x, int c) {
      const uint32_t key = order_key(x);
      // not counted on once too many reach it (one value everywhere)
      if (key >= from && *static_cast<volatile int*>(&sh.cand_n) <= Sh::kCand) {
        const int i = atomicAdd(&sh.cand_n, 1);
        if (i < Sh::kCand) sh.cand[i] = candidate(key, c);
      }
    });
    __syncthreads();
    const int have = sh.cand_n;
    if (have >= k && have <= Sh::kCand) return have;   // the same for the whole CTA
  }
  auto sum = [&](int (&n)[3]) {   // over the CTA
    __syncthreads();
    if (tid < 3) sh.count[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = __reduce_add_sync(0xffffffffu, n[i]);
      if (lane == 0) atomicAdd(&sh.count[i], c);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) n[i] = sh.count[i];
  };
  // the values that are not masked: the largest, the smallest, how many
  uint32_t most = 0, least = 0xffffffffu;
  int n[3] = {};
  p.template each<NT>([&](float x, int) {
    const uint32_t key = order_key(x);
    most = max(most, key);
    if (key) {
      least = min(least, key);
      ++n[0];
    }
  });
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  __syncthreads();
  if (tid == 0) {
    sh.key_max = 0;
    sh.key_min = 0xffffffffu;
  }
  __syncthreads();
  if (lane == 0) {
    atomicMax(&sh.key_max, most);
    atomicMin(&sh.key_min, least);
  }
  __syncthreads();
  most = sh.key_max;
  least = sh.key_min;
  sum(n);
  // What reaches `limit` is collected, where it fits; else all that lies above
  // it, and of those that equal it the first, up to k in all.  The smallest, where
  // few lie above it (few left by the mask, a mask by the lowest value, one value
  // everywhere); else the largest number that k keys reach, found two bits at a
  // time from the first that the keys do not have in common, or the first found
  // that few enough reach.
  uint32_t limit = least;
  int reach = n[0];   // keys that reach `limit`; k or more where there are more than kCand
  if (reach > Sh::kCand) {
    n[0] = n[1] = n[2] = 0;
    p.template each<NT>([&](float x, int) { n[0] += order_key(x) > least; });
    sum(n);
    if (n[0] > Sh::kCand) {
      const int same = __clz(most ^ least) & ~1;
      limit = same == 0 ? 0u : most >> (32 - same) << (32 - same);
      for (int shift = 30 - same; shift >= 0 && reach > Sh::kCand; shift -= 2) {
        n[0] = n[1] = n[2] = 0;
        p.template each<NT>([&](float x, int) {
          const uint32_t key = order_key(x);
#pragma unroll
          for (uint32_t i = 0; i < 3; ++i) n[i] += key >= (limit | (i + 1) << shift);
        });
        sum(n);
        uint32_t step = 0;
#pragma unroll
        for (uint32_t i = 0; i < 3; ++i)
          if (n[i] >= k) {
            step = i + 1;
            reach = n[i];
          }
        limit |= step << shift;
      }
    }
  }
  const bool fits = reach <= Sh::kCand;
  if (tid == 0) sh.cand_n = 0;
  __syncthreads();
  p.template each<NT>([&](float x, int c) {
    const uint32_t key = order_key(x);
    if (key > limit || (fits && key == limit)) {
      const int i = atomicAdd(&sh.cand_n, 1);
      if (i < Sh::kCand) sh.cand[i] = candidate(key, c);
    }
  });
  __syncthreads();
  int have = min(sh.cand_n, Sh::kCand);
  if (fits) return have;   // the same for the whole CTA
  // in the order of the places: the head, the windows, the tail
  const int inner = p.windows * Win<E>::N, all = inner + p.edge;
  for (int c0 = 0; c0 < all && have < k; c0 += NT) {
    const int i = c0 + tid;
    const int c = i < p.head ? i : i < p.head + inner ? p.begin + i - p.head : p.V - all + i;
    const bool hit = i < all && order_key(blk::to_float(p.row[c])) == limit;
    const unsigned votes = __ballot_sync(0xffffffffu, hit);
    __syncthreads();
    if (lane == 0) sh.warp_n[tid >> 5] = __popc(votes);
    __syncthreads();
    int before = have, total = have;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < (tid >> 5)) before += sh.warp_n[w];
      total += sh.warp_n[w];
    }
    before += __popc(votes & ((1u << lane) - 1));
    if (hit && before < k) sh.cand[before] = candidate(limit, c);
    have = min(total, k);
  }
  __syncthreads();
  return have;
}

// Puts a thread's windows that reach thr aside.
template <typename E, int U, typename Sh>
DEV_INLINE void put_aside(const Win<E> (&v)[U], const float (&wm)[U], float thr, int c0, int step, Sh& sh) {
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (wm[u] >= thr) {
      const int at = atomicAdd(&sh.win_n, 1);
      if (at < Sh::kWin) {
        sh.win[at] = v[u].v;
        sh.win_max[at] = candidate(order_key(wm[u]), c0 + u * step);
      }
    }
}

// The values of the windows put aside (and x_edge, the thread's value outside
// the windows) that reach the threshold into sh.cand; their number, which may
// pass kCand.
template <typename E, int NT, typename Sh>
DEV_INLINE int open_windows(const Part<E>& p, int k, uint32_t thr, float x_edge, Sh& sh) {
  constexpr int N = Win<E>::N;
  const int tid = threadIdx.x, n = sh.win_n;
  if (tid == 0) sh.cand_n = 0;
  if (n > 64) {
    uint32_t key = 0;
#pragma unroll 1
    for (int c = spread<NT>(tid); c < n; c += NT) key = max(key, (uint32_t)(sh.win_max[c] >> 32));
    thr = max(thr, threshold<NT>(key, k, sh, 0));
  } else {
    __syncthreads();
  }
#pragma unroll 1
  for (int i = tid; i < n * N; i += NT) {
    const unsigned long long top = sh.win_max[i / N];
    if ((uint32_t)(top >> 32) < thr) continue;
    const uint32_t key = order_key(blk::to_float(reinterpret_cast<const E*>(&sh.win[i / N])[i % N]));
    if (key < thr) continue;
    const int at = atomicAdd(&sh.cand_n, 1);
    if (at < Sh::kCand) sh.cand[at] = candidate(key, place_of(top) + i % N);
  }
  if (tid < p.edge && order_key(x_edge) >= thr) {
    const int at = atomicAdd(&sh.cand_n, 1);
    if (at < Sh::kCand) sh.cand[at] = candidate(order_key(x_edge), p.edge_place(tid));
  }
  __syncthreads();
  return sh.cand_n;
}

DEV_INLINE float log_prob(float x, const Stat& a, float log_s) {
  if (!(x > -INFINITY)) return -INFINITY;
  return x == a.m ? -log_s : x - a.m - log_s;
}

DEV_INLINE void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
// A CTA's own list, where it is too long for its place at the first CTA.
template <int NT, typename Sh>
__device__ __noinline__ int order_here(int n, int k, Sh& sh) {
  return order_candidates<NT>(sh.cand, n, k, sh);
}

template <typename E, int NT, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(NT, NT == 32 ? 24 : 1024 / NT)
    token_logprobs_kernel(const __grid_constant__ LogprobArgs a, int S) {
  using Sh = Shared<NT, CLUSTER>;
  __shared__ Sh sh;
  constexpr int N = Win<E>::N, U = 4;
  const int tid = threadIdx.x, lane = tid & 31, rank = CLUSTER ? blockIdx.x % S : 0;
  const long long t = CLUSTER ? blockIdx.x / S : blockIdx.x;
  Part<E> p;
  p.row = static_cast<const E*>(a.x) + t * a.ld;
  p.V = a.V;
  p.head = min(a.V, (int)((16 - reinterpret_cast<uintptr_t>(p.row) % 16) % 16 / sizeof(E)));
  const int whole = (a.V - p.head) / N;   // windows of the row
  p.edge = rank == 0 ? a.V - whole * N : 0;
  const int w0 = CLUSTER ? (int)((long long)whole * rank / S) : 0;
  p.begin = p.head + w0 * N;
  p.windows = (CLUSTER ? (int)((long long)whole * (rank + 1) / S) : whole) - w0;
  if (rank != 0) p.head = 0;
  if (TOP && tid == 0) sh.win_n = 0;   // before the first batch's barrier
  pdl_wait();
  pdl_trigger();
  if constexpr (CLUSTER) {
    __syncwarp();   // cluster barriers want the warp converged
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }

  const float floor = floor_of<E>();
  Win<E> next[U];
  auto fetch = [&](int w) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t off = masked_word(E{});
      if (w + u * NT < p.windows) next[u] = p.window(w + u * NT);
      else next[u].v = make_uint4(off, off, off, off);
    }
  };
  fetch(tid);
  float x_edge = floor;   // one of the values that no window holds
  if (tid < p.edge) x_edge = fmaxf(blk::to_float(p.row[p.edge_place(tid)]), floor);
  Stat st = {x_edge, x_edge > floor ? 1.f : 0.f, 0.f};
  float x_token = NAN;   // the first thread's: asked for early
  bool has_token = false;
  if (tid == 0 && rank == 0) {
    const long long tok = a.wide_tokens ? static_cast<const long long*>(a.tokens)[t]
                                        : (long long)static_cast<const int32_t*>(a.tokens)[t];
    has_token = tok >= 0 && tok < a.V;
    if (has_token) x_token = blk::to_float(p.row[tok]);
  }
  // every thread takes every batch, with or without values
  const int batches = max(1, (p.windows + U * NT - 1) / (U * NT));
  uint32_t top = 0;
  float thr = 0.f;
  for (int b = 0, w = tid; b < batches; ++b, w += U * NT) {
    Win<E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = next[u];
    if (b + 1 < batches) fetch(w + U * NT);
    float wm[U], bm = floor;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wm[u] = largest(v[u]);
      bm = fmaxf(bm, wm[u]);
    }
    const float m = fmaxf(st.m, bm);
    if (TOP) {
      if ((b & (b + 1)) == 0) {   // what is put aside lies above the floor
        top = max(threshold<NT>(m > floor ? order_key(m) : 0u, a.k, sh, __popc(b) & 1), order_key(floor) + 1);
        thr = key_value(top);
      }
      if (__any_sync(0xffffffffu, bm >= thr)) {
        put_aside<E, U>(v, wm, thr, p.begin + w * N, NT * N, sh);
        __syncwarp();
      }
    }
    const float d0 = fmaxf(st.m - m, -1000.f), r = blk::fast_exp2(d0 * kLog2e);
    float2 s = make_float2(st.s * r, 0.f), e = make_float2(r * (st.e + st.s * d0), 0.f);
    const float2 mm = make_float2(-m, -m), l2 = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < U * N / 2; ++i) {
      const float2 d = add2(floored_pair(v[i / (N / 2)], i % (N / 2)), mm), x2 = mul2(d, l2);
      const float2 q = make_float2(blk::fast_exp2(x2.x), blk::fast_exp2(x2.y));
      s = add2(s, q);
      e = fma2(q, d, e);
    }
    st = Stat{m, s.x + s.y, e.x + e.y};
  }
  Stat all = block_join<NT>(st, sh);
  bool again = false;
  if (!(all.m > floor) || all.m == INFINITY || !(fabsf(all.s) < INFINITY) || !(fabsf(all.e) < INFINITY)) {   // the whole CTA alike
    all = block_join<NT>(careful<E, NT>(p), sh);
    again = true;
  }
  int n = 0;   // the candidates in sh.cand, or, once ordered, in sh.best
  if (TOP && all.m > -INFINITY) {
    const bool lost = sh.win_n > Sh::kWin;   // windows
    if (!again && !lost) {
      n = open_windows<E, NT>(p, a.k, top, x_edge, sh);
      again = n > Sh::kCand || n < a.k;
    }
    if (again || lost) n = collect_again<E, NT>(p, a.k, lost ? top : 0u, sh);
  }

  if constexpr (CLUSTER) {
    const unsigned long long* list = sh.cand;
    if (TOP && n > kSend) {
      n = order_here<NT>(n, a.k, sh);
      list = sh.best;
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // the first CTA runs
    if (TOP && tid < kSend)   // turned by 8 per CTA, so that they spread over order_candidates' groups
      st_cluster_u64(map_to_rank(&sh.from.cand[rank * kSend + (tid + 8 * rank) % kSend], 0), tid < n ? list[tid] : 0);
    if (tid == 0) {
      const uint32_t at = map_to_rank(&sh.from.stat[rank], 0);
      st_cluster_f32(at, all.m);
      st_cluster_f32(at + 4, all.s);
      st_cluster_f32(at + 8, all.e);
    }
    __syncwarp();
    cluster_sync();
    if (rank != 0) return;
    all = warp_join(lane < S ? sh.from.stat[lane] : Stat{-INFINITY, 0.f, 0.f});
    if (TOP && all.m > -INFINITY) n = order_candidates<NT>(sh.from.cand, S * kSend, a.k, sh);
  } else if (TOP && all.m > -INFINITY) {
    n = order_candidates<NT>(sh.cand, n, a.k, sh);
  }

  const float log_s = all.s > 0.f ? logf(all.s) : 0.f;
  if (tid == 0) {
    a.logprob[t] = has_token ? log_prob(x_token, all, log_s) : 0.f;
    a.entropy[t] = all.s > 0.f ? log_s - all.e / all.s : 0.f;
  }
  if (TOP) {
    if (tid < n) {
      const unsigned long long b = sh.best[tid];
      a.ids[t * a.k + tid] = place_of(b);
      a.top[t * a.k + tid] = log_prob(key_value((uint32_t)(b >> 32)), all, log_s);
    }
    // fewer than k unmasked values, all of them chosen: the lowest masked places
    // follow, which are among the first k
    if (n < a.k && tid < 32) {
      bool chosen = tid >= a.k;
      for (int i = 0; i < n; ++i) chosen |= place_of(sh.best[i]) == tid;
      const unsigned free = ~__ballot_sync(0xffffffffu, chosen);
      const int at = n + __popc(free & ((1u << tid) - 1));
      if (!chosen && at < a.k) {
        a.ids[t * a.k + at] = tid;
        a.top[t * a.k + at] = -INFINITY;
      }
    }
  }
}

template <typename E, int NT, bool CLUSTER>
cudaError_t launch_nt(const LogprobArgs& a, long long T, int S, cudaStream_t st) {
  return a.k ? launch_pdl(token_logprobs_kernel<E, NT, true, CLUSTER>, dim3((unsigned)(T * S)), dim3(NT), 0, st, S, a, S)
             : launch_pdl(token_logprobs_kernel<E, NT, false, CLUSTER>, dim3((unsigned)(T * S)), dim3(NT), 0, st, S, a, S);
}

// The CTAs of a row and their threads.  Measured, in us with 20 alternatives
// (without): one row of 50304 FP32 by 1 / 2 / 4 / 8 CTAs of 512 threads 7.7 /
// 7.7 / 6.2 / 5.3 (4.4 / 4.2 / 3.5 / 3.0), of 5000 3.5 / 5.1 (2.0 / 3.1); 64
// rows of 151936 18.8 / 15.0 / 14.6 / 20.1 (16.4 / 11.8 / 10.2 / 14.1).  2048
// rows of 131072 BF16 by 128 / 512 threads 120 / 126 (91 / 94), 512 rows of
// 5000 7.4 / 10.9 (3.9 / 6.2), 64 rows of 5000 5.3 / 3.6 (2.4 / 2.0).  8192
// rows of 500 by 32 / 128 threads 22 / 39 (8.9 / 17); with more than 16
// alternatives a warp's 32 maxima tell too little.  CTAs of 128 threads, eight
// to an SM, fill the SMs unevenly with a few long rows each: 680 rows of 197211 BF16 by
// 128 / 512 threads 100 / 66 (74 / 55), 900 100 / 80 (75 / 65), 1200 104 / 106
// (79 / 85), 512 of 65536 26 / 24 (18 / 16), of 32000 17 / 17 (10 / 10).
template <typename E>
cudaError_t launch_e(const LogprobArgs& a, long long T, int num_sms, cudaStream_t st) {
  const int windows = (int)(a.V / Win<E>::N) + 1;
  int S = 1;
  while (S < 8 && windows > 4096 &&
         ((T * 2 * S <= num_sms && windows >= 2 * S * 1024) || (T * 2 * S <= 2 * num_sms && windows >= 2 * S * 2048)))
    S *= 2;
  if (S > 1) return launch_nt<E, 512, true>(a, T, S, st);
  if (windows <= 128 && T > 8 * num_sms && a.k <= 16) return launch_nt<E, 32, false>(a, T, 1, st);
  if (T <= 2 * num_sms ? windows >= 512 : T <= 6 * num_sms && windows >= 8000) return launch_nt<E, 512, false>(a, T, 1, st);
  return launch_nt<E, 128, false>(a, T, 1, st);
}

}  // namespace

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_token_logprobs(const moe_w4a16_logprobs_config* cfg, int64_t T,
                                                                   const void* logits, const void* tokens,
                                                                   float* logprob, float* entropy, int32_t* topk_ids,
                                                                   float* topk_logprobs, moe_w4a16_stream_t stream) try {
  const char* op = "token_logprobs";
  if (!cfg) return blk::reject(op, "cfg is NULL");
  const moe_w4a16_logprobs_config c = *cfg;
  if (c.dtype != MOE_W4A16_F32 && c.dtype != MOE_W4A16_F16 && c.dtype != MOE_W4A16_BF16)
    return blk::reject(op, "dtype must be F32, F16 or BF16");
  if (c.vocab < 1 || c.vocab > (1 << 28)) return blk::reject(op, "vocab outside [1, 2^28]");
  if (c.top_k < 0 || c.top_k > kMaxTop || c.top_k > c.vocab) return blk::reject(op, "top_k outside [0, min(32, vocab)]");
  if (c.token_bits != 32 && c.token_bits != 64) return blk::reject(op, "token_bits must be 32 or 64");
  if (c.ld_logits != 0 && c.ld_logits < c.vocab) return blk::reject(op, "ld_logits is below vocab");
  if (T < 0 || T > (1 << 27)) return blk::reject(op, "T outside [0, 2^27]");
  if (T == 0) return MOE_W4A16_OK;
  if (!logits || !tokens || !logprob || !entropy) return blk::reject(op, "NULL logits, tokens, logprob or entropy");
  if ((c.top_k > 0) != (topk_ids != nullptr) || (c.top_k > 0) != (topk_logprobs != nullptr))
    return blk::reject(op, "topk_ids and topk_logprobs go with top_k");
  const size_t es = c.dtype == MOE_W4A16_F32 ? 4 : 2;
  if (!blk::aligned(logits, es) || !blk::aligned(tokens, c.token_bits / 8) || !blk::aligned(logprob, 4) ||
      !blk::aligned(entropy, 4) || !blk::aligned(topk_ids, 4) || !blk::aligned(topk_logprobs, 4))
    return blk::reject(op, "a pointer is not aligned to its type");
  LogprobArgs a;
  a.x = logits;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.ids = topk_ids;
  a.top = topk_logprobs;
  a.ld = c.ld_logits ? c.ld_logits : c.vocab;
  a.V = c.vocab;
  a.k = c.top_k;
  a.wide_tokens = c.token_bits == 64;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int num_sms = blk::current_sms();
  if (num_sms < 1) return blk::launch_failed(op, cudaErrorNoDevice);
  const cudaError_t e = c.dtype == MOE_W4A16_F32   ? launch_e<float>(a, T, num_sms, st)
                        : c.dtype == MOE_W4A16_F16 ? launch_e<__half>(a, T, num_sms, st)
                                                   : launch_e<__nv_bfloat16>(a, T, num_sms, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
} catch (...) {   // the host's heap is full
  return MOE_W4A16_ERR_OOM;
}
