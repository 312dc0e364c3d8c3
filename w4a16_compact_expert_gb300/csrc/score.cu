// moe_w4a16_route_scored: expert ids and weights of each token from its
// router logits.  One warp per token; lane l holds the EPL consecutive experts
// l*EPL .., so among equal choices the lowest lane, and in it the lowest
// place, is the lowest expert index.
//
// Bound by instructions and latency (4 bytes of logits an expert cost the
// memory 0.2 us for 2048 tokens of 64 experts): what is kept small is the work
// per round of the k selections.  Each lane sorts the keys of its experts
// once (min/max pairs, no indices), a round is one warp-wide maximum of the
// lanes' heads, a vote for the lowest lane that holds it, and a pop there;
// the k indices are looked up once at the end.
//
// Selection in 64 bits' sense at 32 bits' price: the FP32 scores carry an
// error of a few units in the last place, so two choices closer than that
// could come out in the wrong order.  The FP32 pass therefore also checks
// every border that decided something (between neighbours of the k chosen,
// between the last chosen and all others, between kept and dropped groups)
// against a bound of that error, and decides a closer one in FP64.  Usually
// only the experts at the border are taken up again in FP64, one per lane: a
// whole token in FP64 takes a warp 16 us of dependent operations (when every
// close token went that way, T = 2048, E = 256 with groups took 13.5 us).
// With no bias the FP32 pass orders the experts by the logits themselves (both
// scores are increasing in them), which is exact but for logits whose 64-bit
// scores are equal (sigmoids that round to 1, softmax terms that underflow):
// these tie, so borders between them are close ones too.
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
  int E, k, G, per, top_groups;   // per: experts of a group
  float inv_per;
  bool sigmoid, two, renorm;      // two: a group's value is the sum of its two largest choices
  bool vec;                       // rows can be read 16 bytes at a time
  float scale;
};

// Monotonic maps to unsigned keys: a < b <=> key(a) < key(b); 0 is below every
// key of a number (-inf included).  -0 counts as +0.
DEV_INLINE uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
DEV_INLINE float of_key(uint32_t k) {
  return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}
DEV_INLINE unsigned long long key_of(double f) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(f + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
DEV_INLINE double of_key(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k ^ (1ull << 63)) : ~k));
}
constexpr uint32_t kNone = 0x007fffffu;                          // key of -inf
constexpr unsigned long long kNone64 = 0x000fffffffffffffull;

DEV_INLINE float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

template <typename E>
DEV_INLINE float logit_at(const ScoreArgs& a, long long t, int e) {
  const float v = blk::to_float(static_cast<const E*>(a.logits)[t * a.ld + e]);
  return v == v ? v : -INFINITY;   // NaN: masked
}

// The score of one logit, for the weights (accurate expf).
DEV_INLINE float score_of(const ScoreArgs& a, float l, float m, float den) {
  if (l == -INFINITY) return 0.f;
  if (a.sigmoid) return l > -80.f ? __fdividef(1.f, 1.f + expf(-l)) : expf(l);   // above 2^126 __fdividef gives 0
  return __fdividef(l == m ? 1.f : expf(l - m), den);
}

// The FP64 score of a logit that is not masked; m and den: the softmax's.  One
// copy of exp for both scores; a sigmoid below e^-700 is e^l, where e^-l would
// overflow.
DEV_INLINE double exact_score(bool sigmoid, double l, double m, double den) {
  const bool low = l < -700.0;
  const double x = exp(!sigmoid ? l - m : low ? l : -l);
  return !sigmoid ? (l == m ? 1.0 : x) / den : low ? x : 1.0 / (1.0 + x);
}

// The FP64 choice of one expert, as a key.
__device__ __noinline__ unsigned long long exact_choice(bool sigmoid, float l, float b, double m, double den) {
  if (l == -INFINITY || !(b > -INFINITY)) return kNone64;
  return key_of(exact_score(sigmoid, (double)l, m, den) + (double)b);
}

template <typename E>
__device__ __noinline__ double exact_den(const ScoreArgs& a, long long t, double m) {
  double den = 0;
#pragma unroll 2
  for (int e = threadIdx.x & 31; e < a.E; e += 32) {
    const double l = logit_at<E>(a, t, e);
    den += l == -INFINITY ? 0.0 : l == m ? 1.0 : exp(l - m);
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
  return den;
}

// One token in FP64, written for size: it runs for a token in some hundreds,
// and straight-line code would be fetched from memory each time.  cell: one
// key per expert in this warp's shared memory.
template <typename E>
__device__ __noinline__ void choose_exact(const ScoreArgs& a, long long t, unsigned long long* cell) {
  const int lane = threadIdx.x & 31;
  float mf = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) mf = fmaxf(mf, logit_at<E>(a, t, e));
  double m = warp_max_f(mf), den = 0;
  if (!a.sigmoid) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) {
      const double l = logit_at<E>(a, t, e);
      if (l != -INFINITY) den += l == m ? 1.0 : exp(l - m);
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
  }
  auto score = [&](double l) -> double { return l == -INFINITY ? 0.0 : exact_score(a.sigmoid, l, m, den); };
  const bool grouped = a.G > 1;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const double l = logit_at<E>(a, t, e);
    const float b = a.bias ? a.bias[e] : 0.f;
    cell[e] = l == -INFINITY || !(b > -INFINITY) ? kNone64 : key_of(score(l) + (double)b);
  }
  __syncwarp();
  if (grouped) {
    int L = 1;   // lanes per group, each over every L-th of its experts
    while (2 * L * a.G <= 32) L *= 2;
    const int g = lane / L;
    unsigned long long b1 = 0, b2 = 0;
    if (g < a.G) {
#pragma unroll 1
      for (int j = lane % L; j < a.per; j += L) {
        const unsigned long long v = cell[g * a.per + j];
        if (v > b1) b2 = b1, b1 = v;
        else if (v > b2) b2 = v;
      }
    }
#pragma unroll 1
    for (int o = 1; o < L; o <<= 1) {
      const unsigned long long o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
      const unsigned long long lo = o1 > b1 ? b1 : o1, s2 = o2 > b2 ? o2 : b2;
      b1 = o1 > b1 ? o1 : b1;
      b2 = lo > s2 ? lo : s2;
    }
    const unsigned long long gv = a.two && b2 > kNone64 ? key_of(of_key(b1) + of_key(b2)) : b1;
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o < a.G; ++o) {
      const unsigned long long ov = __shfl_sync(kFull, gv, o * L);
      rank += ov > gv || (ov == gv && o < g);
    }
    const unsigned kept = __ballot_sync(kFull, g < a.G && rank < a.top_groups);
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32)
      if (!((kept >> ((e / a.per) * L)) & 1u)) cell[e] = kNone64;
    __syncwarp();
  }
  unsigned long long mine = 0;
  int my_e = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    unsigned long long bk = 0;
    int be = 0;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32)
      if (cell[e] > bk) bk = cell[e], be = e;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long ok = __shfl_xor_sync(kFull, bk, o);
      const int oe = __shfl_xor_sync(kFull, be, o);
      if (ok > bk || (ok == bk && oe < be)) bk = ok, be = oe;
    }
    if (lane == j) mine = bk, my_e = be;
    if (lane == 0) cell[be] = 0;
    __syncwarp();
  }
  const bool chosen = lane < a.k && mine > kNone64;
  const float my_l = chosen ? logit_at<E>(a, t, my_e) : -INFINITY;
  double sum = 1.0;
  if (a.renorm && !a.sigmoid) {   // the denominator cancels; relative to the largest chosen, so that none is lost
    m = warp_max_f(my_l);
    den = 1.0;
  }
  const double s = score((double)my_l);
  if (a.renorm) {
    sum = s;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_e;
    a.w[t * a.k + lane] = sum > 0 ? (float)(s / sum * (double)a.scale) : 0.f;
  }
}

template <int N>
DEV_INLINE uint32_t key_at(const uint32_t (&k)[N], int i) {   // without an indexed register file
  uint32_t r = k[0];
#pragma unroll
  for (int j = 1; j < N; ++j) r = i == j ? k[j] : r;
  return r;
}

template <int N>
DEV_INLINE void sort_down(uint32_t (&k)[N]) {   // bitonic: largest first
#pragma unroll
  for (int size = 2; size <= N; size *= 2)
#pragma unroll
    for (int gap = size / 2; gap > 0; gap /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = i ^ gap;
        if (j > i) {
          const uint32_t hi = max(k[i], k[j]), lo = min(k[i], k[j]);
          const bool down = (i & size) == 0;
          k[i] = down ? hi : lo;
          k[j] = down ? lo : hi;
        }
      }
}

template <typename E, int EPL>
DEV_INLINE void load_logits(const ScoreArgs& a, long long t, float (&l)[EPL]) {
  const E* row = static_cast<const E*>(a.logits) + t * a.ld;
  const int e0 = (threadIdx.x & 31) * EPL;
  constexpr int kVec = 16 / (int)sizeof(E) < EPL ? 16 / (int)sizeof(E) : EPL;
  if (a.vec && e0 + EPL <= a.E) {
#pragma unroll
    for (int i = 0; i < EPL; i += kVec) {
      const auto p = *reinterpret_cast<const blk::Pack<E, kVec>*>(row + e0 + i);
#pragma unroll
      for (int j = 0; j < kVec; ++j) l[i + j] = blk::to_float(p.v[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = e0 + i < a.E ? blk::to_float(row[e0 + i]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = l[i] == l[i] ? l[i] : -INFINITY;   // NaN: masked
}

// True, with nothing written, where the token has to be done in FP64 as a whole:
// a close border between groups that do not lie on whole lanes, more close
// experts than lanes, scores that FP32 cannot hold, or logits that differ where
// their scores may not.
template <typename E, int EPL>
DEV_INLINE bool choose(const ScoreArgs& a, long long t, uint32_t* cell) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  float l[EPL];
  load_logits<E, EPL>(a, t, l);
  float m = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
  const bool grouped = a.G > 1, scored = a.bias || (grouped && a.two);
  // the softmax denominator, where a score is needed on its own (with no bias
  // and renormalised weights it cancels)
  float den = 1.f;
  if (!a.sigmoid) {
    m = warp_max_f(m);   // -inf: every expert is masked
    if (scored || !a.renorm) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) s += l[i] == -INFINITY ? 0.f : l[i] == m ? 1.f : blk::fast_exp(l[i] - m);
      den = warp_sum(s);
    }
  }
  // A score's error in units of 2^-24.  Sigmoid, at most 8: e^-l is off by
  // 1.5 |l| + 4, which counts s (1 - s) times (1.4), the sum by 1, the
  // quotient by 4.  Softmax, at most 48 / den: the exponential 2.5 |l - m| + 4
  // times itself (5), the denominator 21 additions and as much again (26), its
  // reciprocal and the product 5.  `slack` is that of two scores; a choice adds
  // half an ulp.
  const float unit = 5.9604645e-8f;
  const float slack = (a.sigmoid ? 16.f : __fdividef(96.f, den)) * unit;
  const float inv_den = __fdividef(1.f, den);
  // what the experts are ordered by
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float c = l[i];
    if (a.bias) {
      const float b = e0 + i < a.E ? a.bias[e0 + i] : 0.f;
      const float s = a.sigmoid ? blk::fast_rcp(1.f + blk::fast_exp(fminf(-l[i], 80.f)))
                                : (l[i] == m ? 1.f : blk::fast_exp(l[i] - m)) * inv_den;
      c = l[i] == -INFINITY || !(b > -INFINITY) ? -INFINITY : s + b;
    }
    key[i] = e0 + i < a.E ? key_of(c) : 0u;
  }
  // With no bias: may the 64-bit scores of two logits c0 > c1 be equal (or come
  // out the other way round)?  Where their relative difference (softmax: c0 -
  // c1; sigmoid: (c0 - c1)(1 - score), or more than half of it) comes near the
  // roundings of FP64, some 2^-51 of 1 (softmax: of 1 + |l - m|), or the terms
  // leave its range.  `suspect` sees from c0 alone that it is not so: FP32
  // logits that differ lie farther apart.
  auto suspect = [&](float c0) -> bool {
    return fabsf(c0) < 1e-4f || (a.sigmoid ? c0 > 16.f || c0 < -700.f : m - c0 > 700.f);
  };
  auto saturated = [&](float c0, float c1) -> bool {
    const float rel = a.sigmoid ? fminf(c0 - c1, 1.f) * blk::fast_rcp(1.f + blk::fast_exp(c1))
                                : (c0 - c1) * blk::fast_rcp(1.f + (m - c1));
    return c0 > c1 && (rel <= 1.4e-14f || (a.sigmoid ? 0.f : m) - c0 > 700.f);
  };
  double den64 = -1.0;   // the softmax denominator in FP64, once asked for
  uint32_t srt[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) srt[i] = key[i];
  sort_down(srt);
  if (grouped) {
    // the two largest of a group: from the sorted lanes where a group is a
    // power of two of whole lanes, else over shared memory
    const int lanes = a.per / EPL;
    const bool whole = lanes * EPL == a.per && (lanes & (lanes - 1)) == 0;
    uint32_t b1, b2;
    int L, g;   // lanes that share a group's value, this lane's group
    if (whole) {
      L = lanes;
      g = lane / L;
      b1 = srt[0];
      b2 = EPL > 1 ? srt[EPL > 1 ? 1 : 0] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) cell[e0 + i] = key[i];
      __syncwarp();
      L = 1;
      while (2 * L * a.G <= 32) L *= 2;
      g = lane / L;
      b1 = b2 = 0u;
      if (g < a.G)
        for (int j = lane % L; j < a.per; j += L) {
          const uint32_t v = cell[g * a.per + j];
          b2 = max(b2, min(b1, v));
          b1 = max(b1, v);
        }
      __syncwarp();
    }
    for (int o = 1; o < L; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
      b2 = max(min(b1, o1), max(b2, o2));
      b1 = max(b1, o1);
    }
    // What ranks the groups: logits, or half their value (so that no sum
    // overflows; an infinite one counts as twice the largest number) with a bound of
    // its FP32 error: half of `slack` for each choice's score, and the roundings
    // of the choices and of their sum, a unit each and taken twice, which count
    // by the choices' own size: of opposite sign they may cancel.
    const float largest = 3.402823466e38f;
    float gv = of_key(max(b1, kNone)), err = 0.f;
    const bool none = gv == -INFINITY;
    if (scored) {
      float v2 = a.two ? of_key(max(b2, kNone)) : -INFINITY;
      if (!a.bias && !none) {   // keys of logits: their scores
        gv = score_of(a, gv, m, den);
        if (v2 != -INFINITY) v2 = score_of(a, v2, m, den);
      }
      if (a.two && gv == INFINITY) v2 = gv;   // infinite, whatever the other
      gv = fminf(gv, largest);
      err = 0.25f * slack + 2.f * unit * fminf(fabsf(gv), largest);
      gv *= 0.5f;
      if (v2 != -INFINITY) {
        v2 = fminf(v2, largest);
        err += 0.25f * slack + 2.f * unit * fabsf(v2);
        gv += 0.5f * v2;
      }
    }
    int rank = 0;   // how many groups come before
    for (int o = 0; o < a.G; ++o) {
      const float ov = __shfl_sync(kFull, gv, o * L);
      rank += ov > gv || (ov == gv && o < g);
    }
    bool kept = g < a.G && rank < a.top_groups;
    if (scored) {
      // the 64-bit value lies between lo and hi; a kept group that may lie below
      // a dropped one makes the border a close one
      const float lo = gv - err, hi = gv + err;
      const float least = -warp_max_f(kept ? -lo : -INFINITY), most = warp_max_f(g < a.G && !kept ? hi : -INFINITY);
      if (most != -INFINITY && least <= most) {   // the same in every lane
        if (!whole) return true;
        // the groups on either side of the border in FP64, from their experts
        // that may be among the largest
        if (!a.sigmoid && den64 < 0.0) den64 = exact_den<E>(a, t, (double)m);
        const bool border = g < a.G && !none && (kept ? lo <= most : hi >= least);
        const float low = of_key(max(a.two ? b2 : b1, kNone));
        unsigned long long x1 = 0ull, x2 = 0ull;
        for (int i = 0; i < EPL; ++i) {
          const uint32_t ki = border && e0 + i < a.E ? key_at(key, i) : 0u;
          const bool may = ki > kNone && !(of_key(ki) < low - (a.bias ? slack + 4.f * unit * fabsf(low) : 0.f));   // also at low = inf
          if (__any_sync(kFull, may) && may) {
            const unsigned long long x =
                exact_choice(a.sigmoid, logit_at<E>(a, t, e0 + i), a.bias ? a.bias[e0 + i] : 0.f, (double)m, den64);
            x2 = max(x2, min(x1, x));
            x1 = max(x1, x);
          }
        }
        for (int o = 1; o < L; o <<= 1) {
          const unsigned long long o1 = __shfl_xor_sync(kFull, x1, o), o2 = __shfl_xor_sync(kFull, x2, o);
          x2 = max(min(x1, o1), max(x2, o2));
          x1 = max(x1, o1);
        }
        const unsigned long long gx = !border ? key_of(2.0 * (double)gv)
                                      : a.two && x2 > kNone64 ? key_of(of_key(x1) + of_key(x2)) : x1;
        rank = 0;
        for (int o = 0; o < a.G; ++o) {
          const unsigned long long ov = __shfl_sync(kFull, gx, o * L);
          rank += ov > gx || (ov == gx && o < g);
        }
        kept = g < a.G && rank < a.top_groups;
      }
    } else if (__any_sync(kFull, kept && !none && suspect(gv))) {
      const float least = -warp_max_f(kept ? -gv : -INFINITY), most = warp_max_f(g < a.G && !kept ? gv : -INFINITY);
      if (__any_sync(kFull, g < a.G && !none && most != -INFINITY && (kept ? saturated(gv, most) : saturated(least, gv))))
        return true;
    }
    const unsigned kb = __ballot_sync(kFull, kept);
    // the experts of dropped groups are not eligible
    if (whole) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (!kept) key[i] = min(key[i], kNone);
        if (!kept) srt[i] = min(srt[i], kNone);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int ge = (int)(((float)(e0 + i) + 0.5f) * a.inv_per);
        if (!((kb >> min(ge * L, 31)) & 1u)) key[i] = min(key[i], kNone);
        srt[i] = key[i];
      }
      sort_down(srt);
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) cell[e0 + i] = key[i];
  __syncwarp();
  // lane j keeps the j-th choice: its key and the lane that held it
  uint32_t mine = 0u;
  int my_lane = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t mk = __reduce_max_sync(kFull, srt[0]);
    const int win = __ffs(__ballot_sync(kFull, srt[0] == mk)) - 1;
    if (lane == j) {
      mine = mk;
      my_lane = win;
    }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i + 1 < EPL; ++i) srt[i] = srt[i + 1];
      srt[EPL - 1] = 0u;
    }
  }
  // its expert: of the winner lane's places with that key, the one after those
  // that earlier choices took
  const unsigned same = __match_any_sync(kFull, lane < a.k ? mine : 0u) & __match_any_sync(kFull, my_lane);
  int skip = __popc(same & ((1u << lane) - 1u));
  int my_e = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool eq = cell[my_lane * EPL + i] == mine && !found;
    if (eq && skip == 0) {
      found = true;
      my_e = my_lane * EPL + i;
    }
    skip -= eq;
  }
  bool chosen = lane < a.k && mine > kNone;
  if (a.bias) {
    const float c = of_key(max(mine, kNone)), next = __shfl_down_sync(kFull, c, 1);
    const float kc = __shfl_sync(kFull, c, a.k - 1), head = of_key(max(srt[0], kNone));
    const float far = slack + 4.f * unit * fabsf(kc);
    const bool near1 = lane + 1 < a.k && next != -INFINITY && c - next <= slack + 4.f * unit * fabsf(c);
    const bool near2 = head != -INFINITY && kc - head <= far;
    if (__any_sync(kFull, near1 || near2)) {
      // The chosen and every expert as near to the last of them, one per lane,
      // ordered by their FP64 choices.
      int total = a.k;
      unsigned taken = 0u;   // this lane's chosen places
      for (int j = 0; j < a.k; ++j) {
        const int e = __shfl_sync(kFull, my_e, j);
        if (e >= e0 && e < e0 + EPL) taken |= 1u << (e - e0);
      }
      for (int i = 0; i < EPL; ++i) {
        const uint32_t ki = cell[e0 + i];
        const bool may = near2 && ki > kNone && !((taken >> i) & 1u) && kc - of_key(ki) <= far;
        unsigned who = __ballot_sync(kFull, may);
        for (; who; who &= who - 1, ++total) {
          if (total >= 32) return true;
          if (lane == total) my_e = (__ffs(who) - 1) * EPL + i;
        }
      }
      if (!a.sigmoid && den64 < 0.0) den64 = exact_den<E>(a, t, (double)m);
      const bool in = lane < total && (lane >= a.k || chosen);
      unsigned long long x = 0ull;
      if (in) x = exact_choice(a.sigmoid, logit_at<E>(a, t, my_e), a.bias[my_e], (double)m, den64);
      else if (lane < a.k) x = kNone64;   // fills, behind all others in their order
      int rank = 0;
      for (int o = 0; o < total; ++o) {
        const unsigned long long ox = __shfl_sync(kFull, x, o);
        const int oe = __shfl_sync(kFull, my_e, o);
        rank += ox > x || (ox == x && oe < my_e);
      }
      __syncwarp();
      if (lane < total && rank < a.k) cell[rank] = (uint32_t)my_e | (in ? 0x80000000u : 0u);
      __syncwarp();
      if (lane < a.k) {
        my_e = (int)(cell[lane] & 0x7fffffffu);
        chosen = cell[lane] >> 31;
      }
    }
  } else if (__any_sync(kFull, chosen && suspect(of_key(mine)))) {
    const float c = of_key(max(mine, kNone)), next = __shfl_down_sync(kFull, c, 1), kc = __shfl_sync(kFull, c, a.k - 1);
    float rest = -INFINITY;   // of this lane's others the largest below the last chosen (at equal ones the index decided)
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float v = of_key(max(srt[i], kNone));
      if (v < kc) rest = fmaxf(rest, v);
    }
    if (__any_sync(kFull, (lane + 1 < a.k && next != -INFINITY && saturated(c, next)) ||
                              (rest != -INFINITY && saturated(kc, rest))))
      return true;
  }
  const float my_l = chosen ? logit_at<E>(a, t, my_e) : -INFINITY;
  float w = 0.f;
  if (a.renorm) {
    float s = 0.f;
    if (a.sigmoid) {
      s = score_of(a, my_l, 0.f, 1.f);
    } else {   // the denominator cancels; relative to the largest chosen
      const float top = warp_max_f(my_l);
      if (chosen) s = my_l == top ? 1.f : expf(my_l - top);
    }
    const float sum = warp_sum(s);
    if (sum > 0.f) w = __fdividef(s, sum);
    if (sum < 1e-30f && __any_sync(kFull, chosen)) return true;   // scores below FP32's range
  } else {
    w = score_of(a, my_l, m, den);
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_e;
    a.w[t * a.k + lane] = w * a.scale;
  }
  return false;
}

// CTAs per SM (registers) as measured best at T = 16384: 256 experts in groups
// with a bias 18.1 us with 4, 20.8 with 6; 64 experts 7.5 with 6, 8.5 with 4
// (19.3 and 8.0 since groups carry their own bounds and ties are looked for).
template <int EPL>
constexpr int kCtas = EPL <= 2 ? 6 : EPL == 4 ? 5 : EPL == 8 ? 4 : 3;

template <typename E, int EPL>
__global__ void __launch_bounds__(kWarps * 32, kCtas<EPL>) route_scored_kernel(const __grid_constant__ ScoreArgs a) {
  __shared__ unsigned long long cells[kWarps][EPL * 32];
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const long long t = (long long)blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  if (choose<E, EPL>(a, t, reinterpret_cast<uint32_t*>(cells[warp]))) {
    __syncwarp();
    choose_exact<E>(a, t, cells[warp]);
  }
}

template <typename E, int EPL>
cudaError_t launch(const ScoreArgs& a, cudaStream_t st) {
  return launch_pdl(route_scored_kernel<E, EPL>, dim3((unsigned)((a.T + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0,
                    st, 1, a);
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
                                                                 moe_w4a16_stream_t stream) try {
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
  a.per = c.num_experts / c.num_groups;
  a.inv_per = 1.0f / (float)a.per;
  a.top_groups = c.top_groups;
  a.sigmoid = c.score == MOE_W4A16_SIGMOID;
  a.two = c.group_rank == 2;
  a.renorm = c.renormalize != 0;
  a.scale = c.scale;
  const int es = c.dtype == MOE_W4A16_F32 ? 4 : 2;
  a.vec = blk::aligned(logits, 16) && a.ld * es % 16 == 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c.dtype == MOE_W4A16_F32   ? launch_e<float>(a, st)
                        : c.dtype == MOE_W4A16_F16 ? launch_e<__half>(a, st)
                                                   : launch_e<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
} catch (...) {   // the host's heap is full
  return MOE_W4A16_ERR_OOM;
}
