// moe_w4a16_route_scored: expert ids and weights of each token from its
// router logits.  One warp per token; lane l holds the EPL consecutive experts
// l*EPL .., so among equal choices the lowest lane, and in it the lowest
// place, is the lowest expert index.
//
// Selection in 64 bits' sense at 32 bits' price: the FP32 scores carry an
// error of a few units in the last place, so two choices closer than that
// could come out in the wrong order.  The FP32 pass therefore also checks
// every border that decided something (between neighbours of the k chosen,
// between the last chosen and all others, between kept and dropped groups)
// against a bound of that error, and redoes the token in FP64 when one is
// closer.  With no bias the experts are ordered by the logits themselves
// (both scores are increasing in them), which is exact, so only group values
// (sums of two scores) need the check.
#include "block.h"

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;   // tokens per CTA

struct ScoreArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  long long T, ld;
  int E, k, G, top_groups;
  int dtype;
  bool sigmoid, two, renorm;   // two: a group's value is the sum of its two largest choices
  float scale;
};

// Monotonic maps to unsigned keys: a < b <=> key(a) < key(b); 0 is below every
// key of a number (-inf included).  -0 counts as +0.
DEV_INLINE uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
DEV_INLINE unsigned long long key_of(double f) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(f + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
DEV_INLINE uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(kFull, k); }
DEV_INLINE unsigned long long warp_max_key(unsigned long long k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long v = __shfl_xor_sync(kFull, k, o);
    k = v > k ? v : k;
  }
  return k;
}
template <typename R>
DEV_INLINE R warp_add(R v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <typename R>
DEV_INLINE R warp_maximum(R v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const R u = __shfl_xor_sync(kFull, v, o);
    v = u > v ? u : v;
  }
  return v;
}
DEV_INLINE float exp_of(float v) { return expf(v); }
DEV_INLINE double exp_of(double v) { return exp(v); }
DEV_INLINE float div_of(float a, float b) { return __fdividef(a, b); }
DEV_INLINE double div_of(double a, double b) { return a / b; }
template <typename R>
DEV_INLINE R sigmoid_of(R l) {
  return div_of((R)1, (R)1 + exp_of(-l));
}
template <>
DEV_INLINE float sigmoid_of<float>(float l) {   // __fdividef(1, y) is 0 for y above 2^126
  return l > -80.f ? __fdividef(1.f, 1.f + expf(-l)) : expf(l);
}

// One token.  l: this lane's EPL logits (-inf: masked, or no expert).  cell:
// EPL * 32 values of this warp's shared memory (used with groups only).
// FP32: returns true, having written nothing, when a border that decided the
// result is within the error of the scores; the caller then runs FP64.
template <typename R, int EPL>
DEV_INLINE bool choose(const ScoreArgs& a, long long t, const float (&l)[EPL], R* cell) {
  constexpr bool kCheck = sizeof(R) == 4;
  const R kNone = -(R)INFINITY;
  const int lane = threadIdx.x & 31;
  const int e0 = lane * EPL;
  float m = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
  m = warp_maximum(m);   // -inf: every expert is masked
  // the softmax denominator, where a score is needed on its own (with no bias
  // and renormalised weights it cancels)
  const bool grouped = a.G > 1;
  const bool need_score = a.bias || (grouped && a.two);   // to select
  R den = 1;
  if (!a.sigmoid && (need_score || !a.renorm)) {
    R s = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (l[i] != -INFINITY) s += l[i] == m ? (R)1 : exp_of((R)l[i] - (R)m);
    den = warp_add(s);
  }
  auto score_of = [&](float li) -> R {
    if (li == -INFINITY) return (R)0;
    if (a.sigmoid) return sigmoid_of<R>((R)li);
    return li == m ? div_of((R)1, den) : div_of(exp_of((R)li - (R)m), den);
  };
  // c: what the experts are ordered by; v: the choice (group values)
  R c[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    c[i] = (R)l[i];
    if (a.bias) {
      const float b = e0 + i < a.E ? a.bias[e0 + i] : 0.f;
      c[i] = l[i] == -INFINITY || !(b > -INFINITY) ? kNone : score_of(l[i]) + (R)b;
    }
  }
  bool close = false;
  // half of the distance within which two FP32 choices may be in the wrong
  // order is (units of 2^-24): exp and the division 2 + 2 ulp, the softmax
  // sum up to 5 + EPL roundings and its arguments' rounding |l - m| <= 32 at
  // worst where e^(l-m)|l-m| counts, the addition of the bias half an ulp
  const R unit = (R)5.9604645e-8;
  const R slack = a.sigmoid ? (R)(16.f * 5.9604645e-8f) : div_of((R)(96.f * 5.9604645e-8f), den);
  if (grouped) {
    const int per = a.E / a.G;
    const bool two = a.two;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      R v = c[i];
      if (!a.bias && two && v != kNone) v = score_of(l[i]);
      cell[e0 + i] = v;
    }
    __syncwarp();
    // L lanes per group (a power of two), each over every L-th of its experts
    int L = 1;
    while (2 * L * a.G <= 32) L *= 2;
    const int g = lane / L, sub = lane % L;
    R b1 = kNone, b2 = kNone;   // the two largest
    if (g < a.G)
      for (int j = sub; j < per; j += L) {
        const R v = cell[g * per + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
    for (int o = 1; o < L; o <<= 1) {
      const R o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
      const R hi = o1 > b1 ? o1 : b1, lo = o1 > b1 ? b1 : o1;
      const R s2 = o2 > b2 ? o2 : b2;
      b1 = hi;
      b2 = lo > s2 ? lo : s2;
    }
    const R gv = two && b2 != kNone ? b1 + b2 : b1;
    // rank of the group: how many come before it
    int rank = 0;
    for (int o = 0; o < a.G; ++o) {
      const R ov = __shfl_sync(kFull, gv, o * L);
      rank += ov > gv || (ov == gv && o < g);
    }
    const bool kept = g < a.G && rank < a.top_groups;
    const unsigned kb = __ballot_sync(kFull, kept);
    if (kCheck && (a.bias || two)) {
      const R least = -warp_maximum(kept ? -gv : kNone);
      if (g < a.G && !kept && gv != kNone)
        close = least - gv <= 2 * slack + 4 * unit * (least > 0 ? least : -least);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int ge = (e0 + i) / per;
      if (e0 + i < a.E && !((kb >> (ge * L)) & 1u)) c[i] = kNone;
    }
    __syncwarp();
  }
  using Key = decltype(key_of(c[0]));
  Key key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = e0 + i < a.E ? key_of(c[i]) : (Key)0;
  // lane j keeps the j-th choice: its value, logit and expert
  R mine = kNone;
  float my_l = -INFINITY;
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    Key bk = key[0];
    int bi = 0;
    float bl = l[0];
    R bc = c[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = i;
        bl = l[i];
        bc = c[i];
      }
    const Key mk = warp_max_key(bk);
    const int win = __ffs(__ballot_sync(kFull, bk == mk)) - 1;
    const int we = __shfl_sync(kFull, bi, win);
    const float wl = __shfl_sync(kFull, bl, win);
    const R wc = __shfl_sync(kFull, bc, win);
    if (lane == j) {
      mine = wc;
      my_l = wl;
      my_e = win * EPL + we;
    }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == we) key[i] = 0;
    }
  }
  if (kCheck && a.bias) {
    // equal logits under equal biases are a true tie, already in index order
    const float my_b = lane < a.k ? a.bias[my_e] : 0.f;
    const R nc = __shfl_down_sync(kFull, mine, 1);
    const float nl = __shfl_down_sync(kFull, my_l, 1), nb = __shfl_down_sync(kFull, my_b, 1);
    const R ab = mine > 0 ? mine : -mine;
    if (lane + 1 < a.k && nc != kNone && mine - nc <= 2 * slack + 4 * unit * ab && !(nl == my_l && nb == my_b))
      close = true;
    const R kc = __shfl_sync(kFull, mine, a.k - 1);
    const float kl = __shfl_sync(kFull, my_l, a.k - 1), kb = __shfl_sync(kFull, my_b, a.k - 1);
    const R far = 2 * slack + 4 * unit * (kc > 0 ? kc : -kc);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] != 0 && c[i] != kNone && kc - c[i] <= far && !(l[i] == kl && a.bias[e0 + i] == kb)) close = true;
  }
  const bool chosen = lane < a.k && mine != kNone;
  R w = 0;
  if (a.renorm) {
    R s = 0;
    if (a.sigmoid) {
      s = chosen ? score_of(my_l) : (R)0;
    } else {   // the denominator cancels; relative to the largest chosen
      const float top = warp_maximum(chosen ? my_l : -INFINITY);
      if (chosen) s = my_l == top ? (R)1 : exp_of((R)my_l - (R)top);
    }
    const R sum = warp_add(s);
    if (sum > 0) w = div_of(s, sum);
    if (kCheck && sum < (R)1e-30 && warp_maximum(my_l) != -INFINITY) close = true;
  } else if (chosen) {
    w = score_of(my_l);
  }
  if (kCheck && __any_sync(kFull, close)) return true;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_e;
    a.w[t * a.k + lane] = (float)(w * (R)a.scale);
  }
  return false;
}

// The FP64 form, out of line: it runs for a token in some hundreds.
template <int EPL>
__device__ __noinline__ void choose_wide(const ScoreArgs& a, long long t, const float (&l)[EPL], double* cell) {
  choose<double, EPL>(a, t, l, cell);
}

template <typename E, int EPL>
DEV_INLINE void load_logits(const ScoreArgs& a, long long t, float (&l)[EPL]) {
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  const int e0 = (threadIdx.x & 31) * EPL;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float v = e0 + i < a.E ? blk::to_float(row[e0 + i]) : -INFINITY;
    l[i] = v == v ? v : -INFINITY;   // NaN: masked
  }
}

template <typename E, int EPL>
__global__ void __launch_bounds__(kWarps * 32) route_scored_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) double cells[];   // with groups: one double per expert place and warp
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const long long t = (long long)blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  double* cell = cells + warp * EPL * 32;
  float l[EPL];
  load_logits<E, EPL>(a, t, l);
  if (choose<float, EPL>(a, t, l, reinterpret_cast<float*>(cell))) choose_wide<EPL>(a, t, l, cell);
}

template <typename E, int EPL>
cudaError_t launch(const ScoreArgs& a, cudaStream_t st) {
  const size_t smem = a.G > 1 ? (size_t)kWarps * EPL * 32 * sizeof(double) : 0;
  return launch_pdl(route_scored_kernel<E, EPL>, dim3((unsigned)((a.T + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                    smem, st, 1, a);
}

template <typename E>
cudaError_t launch_e(const ScoreArgs& a, cudaStream_t st) {
  return a.E <= 32    ? launch<E, 1>(a, st)
         : a.E <= 64  ? launch<E, 2>(a, st)
         : a.E <= 128 ? launch<E, 4>(a, st)
         : a.E <= 256 ? launch<E, 8>(a, st)
                      : launch<E, 16>(a, st);
}

}  // namespace

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_route_scored(const moe_w4a16_route_config* cfg, int64_t T,
                                                                 const void* logits, const float* bias,
                                                                 int32_t* topk_ids, float* topk_w,
                                                                 moe_w4a16_stream_t stream) {
  const char* op = "route_scored";
  if (!cfg) return blk::reject(op, "cfg is NULL");
  const moe_w4a16_route_config c = *cfg;
  if (c.dtype != MOE_W4A16_F32 && c.dtype != MOE_W4A16_F16 && c.dtype != MOE_W4A16_BF16)
    return blk::reject(op, "dtype must be F32, F16 or BF16");
  if (c.num_experts < 1 || c.num_experts > 512) return blk::reject(op, "num_experts outside [1, 512]");
  if (c.score != MOE_W4A16_SOFTMAX && c.score != MOE_W4A16_SIGMOID)
    return blk::reject(op, "score must be SOFTMAX or SIGMOID");
  if (c.num_groups < 1 || c.num_groups > 32 || c.num_experts % c.num_groups)
    return blk::reject(op, "num_groups must be in [1, 32] and divide num_experts");
  if (c.top_groups < 1 || c.top_groups > c.num_groups) return blk::reject(op, "top_groups outside [1, num_groups]");
  if (c.group_rank != 1 && c.group_rank != 2) return blk::reject(op, "group_rank must be 1 or 2");
  if (c.top_k < 1 || c.top_k > 32 || c.top_k > c.top_groups * (c.num_experts / c.num_groups))
    return blk::reject(op, "top_k outside [1, min(32, top_groups * num_experts / num_groups)]");
  if (!(c.scale > -3.4e38f && c.scale < 3.4e38f)) return blk::reject(op, "scale must be finite");
  if (c.reserved) return blk::reject(op, "reserved must be 0");
  if (c.ld_logits != 0 && c.ld_logits < c.num_experts) return blk::reject(op, "ld_logits is below num_experts");
  if (T < 0 || T > 0x7fffffff) return blk::reject(op, "T outside [0, 2^31)");
  if (T == 0) return MOE_W4A16_OK;
  if (!logits || !topk_ids || !topk_w) return blk::reject(op, "NULL logits, topk_ids or topk_w");
  if (!blk::aligned(logits, c.dtype == MOE_W4A16_F32 ? 4 : 2) || !blk::aligned(bias, 4) ||
      !blk::aligned(topk_ids, 4) || !blk::aligned(topk_w, 4))
    return blk::reject(op, "a pointer is not aligned to its type");
  ScoreArgs a;
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.w = topk_w;
  a.T = T;
  a.ld = c.ld_logits ? c.ld_logits : c.num_experts;
  a.E = c.num_experts;
  a.k = c.top_k;
  a.G = c.num_groups;
  a.top_groups = c.top_groups;
  a.dtype = c.dtype;
  a.sigmoid = c.score == MOE_W4A16_SIGMOID;
  a.two = c.group_rank == 2;
  a.renorm = c.renormalize != 0;
  a.scale = c.scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c.dtype == MOE_W4A16_F32   ? launch_e<float>(a, st)
                        : c.dtype == MOE_W4A16_F16 ? launch_e<__half>(a, st)
                                                   : launch_e<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
}
