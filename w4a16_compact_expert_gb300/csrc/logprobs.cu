// moe_w4a16_token_logprobs: of every row of logits the log probability of a
// given token, the entropy, and the k most likely tokens:
//   M = max x,  S = sum e^(x - M),  ln p_i = x_i - M - ln S,
//   entropy = ln S - sum e^(x - M) (x - M) / S.
//
// Bound by reading the logits once.  A row is read by the CTAs of a cluster
// (one CTA where there are enough rows); every thread keeps the running
// maximum m of its values and the two sums relative to it, which are rescaled
// once per batch of values; threads and CTAs join by rescaling to the common
// maximum.
//
// The k largest need no list while the row is read: a thread's m is the
// largest of its values, and at least k values reach the smallest of k
// threads' maxima.  Only the few threads whose maximum reaches that threshold
// have values to offer; the CTA reads theirs again (from the L2, some percent
// of the row), collects what reaches the threshold and orders it by counting.
// Rows in which too many values reach it (ties, masks of the lowest finite
// value) find the k-th largest value by bisection over its bits instead.
#include <math.h>
#include <string.h>

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
constexpr int kCand = 1024;   // candidates a CTA can collect
constexpr float kLog2e = 1.4426950408889634f;
// Stands for a masked value (-inf, NaN) while a row is read: differences to it
// stay finite, and e to their power is 0.  Rows without anything above it are
// read again with care.
constexpr float kFloor = -1e38f;

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
DEV_INLINE Stat join(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  a = rescale(a, m);
  b = rescale(b, m);
  return Stat{m, a.s + b.s, a.e + b.e};
}

// Orders values as unsigned numbers; 0 for what is masked.  -0 equals 0.
DEV_INLINE uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t k = (int)b < 0 ? ~b : b | 0x80000000u;
  return x > -INFINITY ? k : 0u;   // false for NaN
}
DEV_INLINE float key_value(uint32_t k) { return __uint_as_float((int)k < 0 ? k & 0x7fffffffu : ~k); }

// Sixteen bytes of a row.  Windows lie on the 16-byte grid in memory; the first
// and the last may be partly outside the row and hold -inf there.
template <typename E>
struct Win {
  static constexpr int N = 16 / sizeof(E);
  uint4 v;
};
template <typename E>
DEV_INLINE E masked();
template <>
DEV_INLINE float masked<float>() { return -INFINITY; }
template <>
DEV_INLINE __half masked<__half>() { return __ushort_as_half((unsigned short)0xfc00u); }
template <>
DEV_INLINE __nv_bfloat16 masked<__nv_bfloat16>() { return __ushort_as_bfloat16((unsigned short)0xff80u); }

// The window that starts at value c0 (may be negative).
template <typename E>
DEV_INLINE Win<E> load_window(const E* row, long long c0, int V) {
  constexpr int N = Win<E>::N;
  Win<E> w;
  if (c0 >= 0 && c0 + N <= V) {
    // past the L1: read once, but for the few windows that are read again much later
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.v.x), "=r"(w.v.y), "=r"(w.v.z), "=r"(w.v.w)
                 : "l"(row + c0)
                 : "memory");
  } else {
    E t[N];
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = c0 + j >= 0 && c0 + j < V ? row[c0 + j] : masked<E>();
    memcpy(&w.v, t, 16);
  }
  return w;
}
DEV_INLINE float2 pair_of(const Win<float>& w, int j) {
  const float* f = reinterpret_cast<const float*>(&w.v);
  return make_float2(f[2 * j], f[2 * j + 1]);
}
DEV_INLINE float2 pair_of(const Win<__half>& w, int j) {
  return __half22float2(reinterpret_cast<const __half2*>(&w.v)[j]);
}
DEV_INLINE float2 pair_of(const Win<__nv_bfloat16>& w, int j) {
  return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&w.v)[j]);
}

struct Shared {
  Stat part[32];             // a warp's
  uint32_t thr[32];          // a warp's threshold
  int owners_n, cand_n, count[4];
  int warp_n[32];
  unsigned short owner[1024];
  unsigned long long cand[kCand];
  unsigned long long best[kMaxTop];
  // what the CTAs of a cluster send to the first
  Stat from[8];
  int from_n[8];
  unsigned long long from_best[8][kMaxTop];
};

// A row's windows [w0, w1) belong to this CTA, w0 + tid + j NT to a thread.
template <typename E>
struct Part {
  const E* row;
  int V, m, w0, w1;   // m: values of the first window before the row's start
  DEV_INLINE Win<E> window(int w) const { return load_window<E>(row, (long long)w * Win<E>::N - m, V); }
};

template <int NT>
DEV_INLINE Stat block_join(Stat a, Shared& sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.e = __shfl_xor_sync(0xffffffffu, a.e, o);
    a = join(a, b);
  }
  __syncthreads();   // `part` may still be read
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = a;
  __syncthreads();
  a = sh.part[0];
#pragma unroll
  for (int i = 1; i < NT / 32; ++i) a = join(a, sh.part[i]);
  return a;
}

// Any row: nothing left by its mask, infinities, values below the floor.
template <typename E, int NT>
DEV_INLINE Stat careful(const Part<E>& p, float& tm) {
  tm = -INFINITY;
  for (int w = p.w0 + threadIdx.x; w < p.w1; w += NT) {
    const Win<E> v = p.window(w);
    for (int j = 0; j < Win<E>::N / 2; ++j) {
      const float2 f = pair_of(v, j);
      tm = fmaxf(tm, fmaxf(f.x, f.y));
    }
  }
  Stat a = {tm, 0.f, 0.f};
  if (tm > -INFINITY) {
    for (int w = p.w0 + threadIdx.x; w < p.w1; w += NT) {
      const Win<E> v = p.window(w);
      for (int j = 0; j < Win<E>::N; ++j) {
        const float2 f = pair_of(v, j / 2);
        const float x = j & 1 ? f.y : f.x;
        if (x == tm) {
          a.s += 1.f;
        } else if (x - tm > -100.f) {   // false for what is masked and beside an infinite maximum
          const float d = x - tm, q = blk::fast_exp2(d * kLog2e);
          a.s += q;
          a.e = fmaf(q, d, a.e);
        }
      }
    }
  }
  return a;
}

// Rows whose values crowd: the k largest of the part into sh.best (their
// number is returned), largest first, ties to the lower index.
template <typename E, int NT>
__device__ __noinline__ int select_crowded(const Part<E>& p, int k, Shared& sh) {
  constexpr int N = Win<E>::N;
  const int tid = threadIdx.x, lane = tid & 31;
  // the largest number that k keys reach, two bits at a time; 0: fewer than k are not masked
  uint32_t at = 0;
  for (int shift = 30; shift >= 0; shift -= 2) {
    int n[3] = {};
    for (int w = p.w0 + tid; w < p.w1; w += NT) {
      const Win<E> v = p.window(w);
      for (int j = 0; j < N; ++j) {
        const float2 f = pair_of(v, j / 2);
        const uint32_t key = order_key(j & 1 ? f.y : f.x);
#pragma unroll
        for (uint32_t i = 0; i < 3; ++i) n[i] += key >= (at | (i + 1) << shift);
      }
    }
    __syncthreads();
    if (tid < 3) sh.count[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = __reduce_add_sync(0xffffffffu, n[i]);
      if (lane == 0) atomicAdd(&sh.count[i], c);
    }
    __syncthreads();
    uint32_t step = 0;
    for (uint32_t i = 0; i < 3; ++i)
      if (sh.count[i] >= k) step = i + 1;
    at |= step << shift;
  }
  // what lies above it: fewer than k
  __syncthreads();
  if (tid == 0) sh.cand_n = 0;
  __syncthreads();
  const long long c_end = min((long long)p.V, (long long)p.w1 * N - p.m);
  for (int w = p.w0 + tid; w < p.w1; w += NT) {
    const Win<E> v = p.window(w);
    const int c0 = w * N - p.m;
    for (int j = 0; j < N; ++j) {
      const float2 f = pair_of(v, j / 2);
      const uint32_t key = order_key(j & 1 ? f.y : f.x);
      if (key > at) {
        const int i = atomicAdd(&sh.cand_n, 1);
        if (i < kCand) sh.cand[i] = (unsigned long long)key << 32 | (uint32_t)~(c0 + j);
      }
    }
  }
  __syncthreads();
  const int above = sh.cand_n;
  int n = above;
  // and the first of those that equal it
  if (at != 0) {
    long long c = (long long)p.w0 * N - p.m;
    if (c < 0) c = 0;
    for (; c < c_end && n < k; c += NT) {
      const bool hit = c + tid < c_end && order_key(blk::to_float(p.row[c + tid])) == at;
      const unsigned votes = __ballot_sync(0xffffffffu, hit);
      __syncthreads();
      if (lane == 0) sh.warp_n[tid >> 5] = __popc(votes);
      __syncthreads();
      int before = n, all = n;
      for (int i = 0; i < NT / 32; ++i) {
        if (i < (tid >> 5)) before += sh.warp_n[i];
        all += sh.warp_n[i];
      }
      before += __popc(votes & ((1u << lane) - 1));
      if (hit && before < k) sh.cand[before] = (unsigned long long)at << 32 | (uint32_t)~(uint32_t)(c + tid);
      n = min(all, k);
    }
    __syncthreads();
  }
  if (tid < n) {
    const unsigned long long mine = sh.cand[tid];
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += sh.cand[i] > mine;
    sh.best[rank] = mine;
  }
  __syncthreads();
  return n;
}

// The k largest of the part into sh.best, as select_crowded.  tm: the largest
// of this thread's values (the floor or -inf: nothing above the floor).
template <typename E, int NT>
DEV_INLINE int select_top(const Part<E>& p, int k, float tm, float floor, Shared& sh) {
  constexpr int N = Win<E>::N, kWarps = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31;
  // a warp's n-th largest maximum, n = ceil(k / warps): together at least k values reach the smallest of these
  uint32_t key = tm > floor ? order_key(tm) : 0u;
  const uint32_t own = key;
  uint32_t t = 0;
  for (int i = 0; i < (k + kWarps - 1) / kWarps; ++i) {
    t = __reduce_max_sync(0xffffffffu, key);
    const unsigned at = __ballot_sync(0xffffffffu, key == t);
    if (lane == __ffs(at) - 1) key = 0;
  }
  if (lane == 0) sh.thr[tid >> 5] = t;
  if (tid == 0) sh.owners_n = sh.cand_n = 0;
  __syncthreads();
  uint32_t thr = sh.thr[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) thr = min(thr, sh.thr[i]);
  // no threshold (few values above the floor): every thread's values are looked at
  if (thr == 0 || own >= thr) sh.owner[atomicAdd(&sh.owners_n, 1)] = (unsigned short)tid;
  thr = max(thr, 1u);
  __syncthreads();
  const int owners = sh.owners_n, per = (p.w1 - p.w0 + NT - 1) / NT;
  const long long items = (long long)owners * per;
  constexpr int U = 4;
  for (long long i0 = tid; i0 < items; i0 += U * NT) {
    Win<E> v[U];
    int w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * NT;
      w[u] = i < items ? p.w0 + sh.owner[i % owners] + (int)(i / owners) * NT : p.w1;
      if (w[u] < p.w1) v[u] = p.window(w[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (w[u] >= p.w1) continue;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 f = pair_of(v[u], j / 2);
        const uint32_t kx = order_key(j & 1 ? f.y : f.x);
        if (kx >= thr) {
          const int at = atomicAdd(&sh.cand_n, 1);
          if (at < kCand) sh.cand[at] = (unsigned long long)kx << 32 | (uint32_t)~(w[u] * N - p.m + j);
        }
      }
    }
  }
  __syncthreads();
  const int n = sh.cand_n;
  if (n > kCand) return select_crowded<E, NT>(p, k, sh);
  for (int c = tid; c < n; c += NT) {
    const unsigned long long mine = sh.cand[c];
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += sh.cand[i] > mine;
    if (rank < k) sh.best[rank] = mine;
  }
  __syncthreads();
  return min(n, k);
}

DEV_INLINE float log_prob(float x, const Stat& a, float log_s) {
  if (!(x > -INFINITY)) return -INFINITY;
  return x == a.m ? -log_s : x - a.m - log_s;
}

DEV_INLINE void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename E, int NT>
__global__ void __launch_bounds__(NT) token_logprobs_kernel(const __grid_constant__ LogprobArgs a, int S) {
  __shared__ Shared sh;
  constexpr int N = Win<E>::N, U = 4;
  const int tid = threadIdx.x, rank = blockIdx.x % S;
  const long long t = blockIdx.x / S;
  Part<E> p;
  p.row = static_cast<const E*>(a.x) + t * a.ld;
  p.V = a.V;
  p.m = (int)(reinterpret_cast<uintptr_t>(p.row) % 16 / sizeof(E));
  const long long windows = ((long long)a.V + p.m + N - 1) / N;
  p.w0 = (int)(windows * rank / S);
  p.w1 = (int)(windows * (rank + 1) / S);
  pdl_wait();
  pdl_trigger();
  if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  constexpr float floor = kFloor;
  Stat st = {floor, 0.f, 0.f};
  for (int w = p.w0 + tid; w < p.w1; w += U * NT) {
    Win<E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (w + u * NT < p.w1) v[u] = p.window(w + u * NT);
      else {
        E off[N];
#pragma unroll
        for (int j = 0; j < N; ++j) off[j] = masked<E>();
        memcpy(&v[u].v, off, 16);
      }
    float2 f[U * N / 2];
    float m = st.m;
#pragma unroll
    for (int i = 0; i < U * N / 2; ++i) {
      const float2 q = pair_of(v[i / (N / 2)], i % (N / 2));
      f[i] = make_float2(fmaxf(q.x, floor), fmaxf(q.y, floor));   // NaN too becomes the floor
      m = fmaxf(m, fmaxf(f[i].x, f[i].y));
    }
    const float d0 = fmaxf(st.m - m, -1000.f), r = blk::fast_exp2(d0 * kLog2e);
    float2 s = make_float2(st.s * r, 0.f), e = make_float2(r * (st.e + st.s * d0), 0.f);
    const float2 mm = make_float2(-m, -m), l2 = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < U * N / 2; ++i) {
      const float2 d = add2(f[i], mm), x2 = mul2(d, l2);
      const float2 q = make_float2(blk::fast_exp2(x2.x), blk::fast_exp2(x2.y));
      s = add2(s, q);
      e = fma2(q, d, e);
    }
    st = Stat{m, s.x + s.y, e.x + e.y};
  }
  float tm = st.m;
  Stat all = block_join<NT>(st, sh);
  float low = floor;
  if (!(all.m > floor) || all.m == INFINITY || !(fabsf(all.s) < INFINITY) || !(fabsf(all.e) < INFINITY)) {   // the whole CTA alike
    all = block_join<NT>(careful<E, NT>(p, tm), sh);
    low = -INFINITY;
  }
  int n = a.k ? select_top<E, NT>(p, a.k, tm, low, sh) : 0;

  if (S > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // the first CTA runs
    if (tid < n) st_cluster_u64(map_to_rank(&sh.from_best[rank][tid], 0), sh.best[tid]);
    if (tid == 0) {
      const uint32_t at = map_to_rank(&sh.from[rank], 0);
      st_cluster_f32(at, all.m);
      st_cluster_f32(at + 4, all.s);
      st_cluster_f32(at + 8, all.e);
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(map_to_rank(&sh.from_n[rank], 0)), "r"(n) : "memory");
    }
    cluster_sync();
    if (rank != 0) return;
    all = sh.from[0];
    for (int i = 1; i < S; ++i) all = join(all, sh.from[i]);
    if (a.k) {
      // the k largest of the parts' lists
      int total = 0;
      for (int i = 0; i < S; ++i) total += sh.from_n[i];
      for (int c = tid; c < S * kMaxTop; c += NT) {
        if (c % kMaxTop >= sh.from_n[c / kMaxTop]) continue;
        const unsigned long long mine = sh.from_best[c / kMaxTop][c % kMaxTop];
        int place = 0;
        for (int i = 0; i < S; ++i)
          for (int j = 0; j < sh.from_n[i] && sh.from_best[i][j] > mine; ++j) ++place;
        if (place < a.k) sh.best[place] = mine;
      }
      n = min(total, a.k);
      __syncthreads();
    }
  }
  const float log_s = all.s > 0.f ? logf(all.s) : 0.f;
  if (tid == 0) {
    const long long tok = a.wide_tokens ? static_cast<const long long*>(a.tokens)[t]
                                        : (long long)static_cast<const int32_t*>(a.tokens)[t];
    a.logprob[t] = tok >= 0 && tok < a.V ? log_prob(blk::to_float(p.row[tok]), all, log_s) : 0.f;
    a.entropy[t] = all.s > 0.f ? log_s - all.e / all.s : 0.f;
  }
  if (tid < n) {
    const unsigned long long b = sh.best[tid];
    a.ids[t * a.k + tid] = (int32_t)~(uint32_t)b;
    a.top[t * a.k + tid] = log_prob(key_value((uint32_t)(b >> 32)), all, log_s);
  }
  // fewer than k unmasked values, all of them chosen: the lowest masked places
  // follow, which are among the first k
  if (n < a.k && tid < 32) {
    bool chosen = tid >= a.k;
    for (int i = 0; i < n; ++i) chosen |= (int32_t)~(uint32_t)sh.best[i] == tid;
    const unsigned free = ~__ballot_sync(0xffffffffu, chosen);
    const int at = n + __popc(free & ((1u << tid) - 1));
    if (!chosen && at < a.k) {
      a.ids[t * a.k + at] = tid;
      a.top[t * a.k + at] = -INFINITY;
    }
  }
}

template <typename E, int NT>
cudaError_t launch_nt(const LogprobArgs& a, long long T, int S, cudaStream_t st) {
  return launch_pdl(token_logprobs_kernel<E, NT>, dim3((unsigned)(T * S)), dim3(NT), 0, st, S, a, S);
}

// The CTAs of a row and their threads.
template <typename E>
cudaError_t launch_e(const LogprobArgs& a, long long T, int num_sms, cudaStream_t st) {
  int S = 1;
  while (S < 8 && T * S * 2 <= 4ll * num_sms && a.V / (2 * S) >= 4096) S *= 2;
  if (a.V / S <= 8192) return launch_nt<E, 128>(a, T, S, st);
  return launch_nt<E, 512>(a, T, S, st);
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
