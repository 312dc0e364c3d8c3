// moe_w4a16_add_rmsnorm: s = x + residual, n = s / sqrt(mean s^2 + eps) * w,
// and n in E4M3 with one scale per row.
//
// Bound by memory: per value 2 + 2 bytes read and 2 + 2 (+ 1) written.  A row
// is read once, its sum stays in registers (FP32) between the one reduction
// and the stores, and the E4M3 scale needs no second reduction: |n| = |s w| r
// with the row's positive r = 1/sqrt(...), hence max|n| = r max|s w|, and
// max|s w| is reduced together with the sum of squares.  What has to be kept
// small is the instruction count (at 28 a value the SMs, not the memory, set
// the time): values go in pairs through the packed FP32 operations, and a
// thread has up to 32 of a row, which spreads the row's fixed cost.
#include "block.h"

namespace {

using blk::Pack;
using blk::add2;
using blk::fma2;
using blk::mul2;

struct NormArgs {
  const void *x, *res, *w;
  void *res_out, *y;
  uint8_t* q;
  float* q_scale;
  long long T, ld_x, ld_res, ld_res_out, ld_y, ld_q;
  int H;
  float eps, inv_h;
};

// How a row's values are read and written, eight (a window) at a time:
enum Access {
  kAligned,   // every window of every tensor is a 16-byte vector
  kPeeled,    // windows lie on the 16-byte grid of the row in memory, m values
              // before the row's start (the same m for every tensor): the
              // first and the last are partly outside and go by single values,
              // so do the weights
  kSingle     // everything by single values
};

template <typename E>
using Win = Pack<E, 8>;

DEV_INLINE float2 pair_of(const Win<__half>& w, int j) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w.v[2 * j]));
}
DEV_INLINE float2 pair_of(const Win<__nv_bfloat16>& w, int j) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.v[2 * j]));
}
// Two neighbouring values of E / of E4M3 (saturating).
DEV_INLINE void pair_to(Win<__half>& w, int j, float2 f) { *reinterpret_cast<__half2*>(&w.v[2 * j]) = __float22half2_rn(f); }
DEV_INLINE void pair_to(Win<__nv_bfloat16>& w, int j, float2 f) {
  *reinterpret_cast<__nv_bfloat162*>(&w.v[2 * j]) = __float22bfloat162_rn(f);
}
DEV_INLINE void pair_to(Win<uint8_t>& w, int j, float2 f) {
  *reinterpret_cast<__nv_fp8x2_storage_t*>(&w.v[2 * j]) = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// Window values [c0, c0 + 8) of a row of H at `row`; outside the row: 0.
template <Access A, typename E>
DEV_INLINE void load_window(Win<E>& w, const E* row, int c0, int H) {
  if (A != kSingle && c0 >= 0 && c0 + 8 <= H) {
    w = *reinterpret_cast<const Win<E>*>(row + c0);
  } else if (A != kAligned) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w.v[j] = (unsigned)(c0 + j) < (unsigned)H ? row[c0 + j] : E{};
  } else {
    w = Win<E>{};
  }
}
template <Access A, typename E>
DEV_INLINE void store_window(const Win<E>& w, E* row, int c0, int H) {
  if (A != kSingle && c0 >= 0 && c0 + 8 <= H) {
    *reinterpret_cast<Win<E>*>(row + c0) = w;
  } else if (A != kAligned) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((unsigned)(c0 + j) < (unsigned)H) row[c0 + j] = w.v[j];
  }
}

// s = x + res of a thread's V windows, its sum of squares, and with q the
// largest |s w|.
template <typename E, int V>
DEV_INLINE void row_sums(const NormArgs& a, const Win<E> (&xv)[V], const Win<E> (&rv)[V], const float2 (&w)[V * 4],
                         float2 (&s)[V * 4], float& ss, float& mx) {
#pragma unroll
  for (int i = 0; i < V * 4; ++i) s[i] = pair_of(xv[i / 4], i % 4);
  if (a.res) {
#pragma unroll
    for (int i = 0; i < V * 4; ++i) s[i] = add2(s[i], pair_of(rv[i / 4], i % 4));
  }
  float2 sq = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < V * 4; ++i) sq = fma2(s[i], s[i], sq);
  ss = sq.x + sq.y;
  mx = 0.f;
  if (a.q) {   // fmaxf leaves NaN out; n and q carry it
#pragma unroll
    for (int i = 0; i < V * 4; ++i) {
      const float2 n = mul2(s[i], w[i]);
      mx = fmaxf(mx, fmaxf(fabsf(n.x), fabsf(n.y)));
    }
  }
}

// Adds (ss, mx) up over the nt threads of a row: `part` holds a pair per warp
// of the CTA; w0 is the row's first warp.
DEV_INLINE void reduce_row(float& ss, float& mx, bool want_mx, int nt, int tx, float2* part, int w0) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < nt) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (want_mx) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < nt) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (nt > 32) {
    if ((tx & 31) == 0) part[w0 + (tx >> 5)] = make_float2(ss, mx);
    __syncthreads();
    ss = mx = 0.f;
#pragma unroll 4
    for (int i = 0; i < (nt >> 5); ++i) {
      const float2 p = part[w0 + i];
      ss += p.x;
      mx = fmaxf(mx, p.y);
    }
  }
}

// The stores of a row: s, n and q of a thread's windows.
template <Access A, typename E, int V>
DEV_INLINE void finish_row(const NormArgs& a, E* s_row, E* y_row, uint8_t* q_row, float* scale, const int (&c0)[V],
                           const float2 (&w)[V * 4], float2 (&s)[V * 4], float ss, float mx) {
  const float r = rsqrtf(fmaf(ss, a.inv_h, a.eps));
  if (a.res_out) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Win<E> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) pair_to(o, j, s[i * 4 + j]);
      store_window<A>(o, s_row, c0[i], a.H);
    }
  }
  const float2 rr = make_float2(r, r);
#pragma unroll
  for (int i = 0; i < V * 4; ++i) s[i] = mul2(mul2(s[i], rr), w[i]);
  if (a.y) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Win<E> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) pair_to(o, j, s[i * 4 + j]);
      store_window<A>(o, y_row, c0[i], a.H);
    }
  }
  if (a.q) {
    float c = mx * r * (1.0f / 448.0f);
    if (c < 1.17549435e-38f) c = 0.f;   // below 2^-126 the reciprocal would overflow
    const float inv = c > 0.f ? __fdividef(1.0f, c) : 0.f;
    if (scale) *scale = c;
    const float2 ii = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Win<uint8_t> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) pair_to(o, j, mul2(s[i * 4 + j], ii));
      store_window<A>(o, q_row, c0[i], a.H);
    }
  }
}

// The place of a row's first value on the 16-byte grid, in values.
template <Access A, typename E>
DEV_INLINE int grid_place(const E* row) {
  return A == kPeeled ? (int)((reinterpret_cast<uintptr_t>(row) / sizeof(E)) & 7) : 0;
}

// A thread's weights in FP32; no weight: 1.
template <Access A, typename E, int V>
DEV_INLINE void load_weights(const NormArgs& a, const int (&c0)[V], float2 (&w)[V * 4]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.w) {
      Win<E> wv = {};
      if (c0[i] < a.H) load_window<A == kPeeled ? kSingle : A>(wv, static_cast<const E*>(a.w), c0[i], a.H);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i * 4 + j] = pair_of(wv, j);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i * 4 + j] = make_float2(1.f, 1.f);
    }
  }
}

// Few rows: a row (short rows: several) per CTA.  V windows of a row per
// thread; blockDim.x threads per row (a power of two below 32, else a
// multiple of 32), blockDim.y rows per CTA, MT threads at most.
template <typename E, Access A, int V, int MT>
__global__ void __launch_bounds__(MT) add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float2 part[32];
  const int nt = blockDim.x, tx = threadIdx.x, H = a.H;
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < a.T;
  const E* const x = static_cast<const E*>(a.x) + t * a.ld_x;
  const int m = grid_place<A>(x);
  pdl_wait();
  pdl_trigger();
  Win<E> xv[V], rv[V];
  float2 w[V * 4];
  int c0[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c0[i] = (i * nt + tx) * 8 - m;
    xv[i] = rv[i] = Win<E>{};
    if (live && c0[i] < H) {
      load_window<A>(xv[i], x, c0[i], H);
      if (a.res) load_window<A>(rv[i], static_cast<const E*>(a.res) + t * a.ld_res, c0[i], H);
    }
  }
  load_weights<A, E, V>(a, c0, w);
  float2 s[V * 4];
  float ss, mx;
  row_sums<E, V>(a, xv, rv, w, s, ss, mx);
  reduce_row(ss, mx, a.q != nullptr, nt, tx, part, threadIdx.y * (nt >> 5));
  if (live)
    finish_row<A, E, V>(a, static_cast<E*>(a.res_out) + t * a.ld_res_out, static_cast<E*>(a.y) + t * a.ld_y,
                        a.q + t * a.ld_q, tx == 0 ? a.q_scale + t : nullptr, c0, w, s, ss, mx);
}

// Many rows: a persistent CTA takes every gridDim.x-th one.  Each thread
// fetches its own windows `ahead` (2 or 3) rows ahead with 16-byte asynchronous
// copies into its own shared memory, so loads stay in flight over the
// reduction and the stores and no thread waits for another's copies; the
// weights stay in registers.  Peeled rows: gridDim.x is a multiple of 8, so
// all rows of a CTA lie alike on the 16-byte grid.
// T = 16383, H = 4096 BF16: 44.6 us, 6.0 TB/s (a CTA per row, 28 instructions
// a value: 85 us); T = 16384, H = 2048 FP16, residual and E4M3: 56 us, 5.4 TB/s.
template <int V>
constexpr int kStreamThreads = V == 1 ? 1280 : V == 2 ? 1024 : 640;   // per SM, as the registers allow

template <typename E, Access A, int V, int MT>
__global__ void __launch_bounds__(MT, kStreamThreads<V> / MT) add_rmsnorm_stream_kernel(
    const __grid_constant__ NormArgs a, int ahead) {
  extern __shared__ __align__(16) uint8_t ring_raw[];   // [ahead + 1][V * (1 or 2)][threads] windows
  __shared__ float2 part[2][32];
  const int nt = blockDim.x, tx = threadIdx.x, H = a.H;
  const uint32_t row_bytes = (uint32_t)(V * (a.res ? 2 : 1) * nt * 16);   // of a row in the ring
  const uint32_t mine = smem_u32(ring_raw) + (uint32_t)tx * 16;
  const long long step = gridDim.x;
  long long t = blockIdx.x;
  const E* xf = static_cast<const E*>(a.x) + t * a.ld_x;   // the next row to fetch
  const E* rf = static_cast<const E*>(a.res) + t * a.ld_res;
  const int m = grid_place<A>(xf);
  int c0[V];
  bool in[V];   // the whole window lies inside the row
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c0[i] = (i * nt + tx) * 8 - m;
    in[i] = c0[i] >= 0 && c0[i] + 8 <= H;
  }
  pdl_wait();
  pdl_trigger();
  int left = (int)((a.T - t + step - 1) / step);   // rows of this CTA still to fetch
  auto fetch_row = [&](uint32_t slot) {
    if (left > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (in[i]) {
          const uint32_t d = mine + slot * row_bytes + (uint32_t)(i * nt * 16);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(xf + c0[i]) : "memory");
          if (a.res)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + (uint32_t)(V * nt * 16)), "l"(rf + c0[i])
                         : "memory");
        }
    }
    --left;
    xf += step * a.ld_x;
    rf += step * a.ld_res;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const E *x = xf, *res = rf;   // the row in work
  E* s_row = static_cast<E*>(a.res_out) + t * a.ld_res_out;
  E* y_row = static_cast<E*>(a.y) + t * a.ld_y;
  uint8_t* q_row = a.q + t * a.ld_q;
  for (int k = 0; k < ahead; ++k) fetch_row(k);
  float2 w[V * 4];
  load_weights<A, E, V>(a, c0, w);
  uint32_t slot = 0;
  for (int flip = 0; t < a.T; t += step, flip ^= 1) {
    fetch_row(slot == 0 ? ahead : slot - 1);
    if (ahead == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
    Win<E> xv[V], rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint8_t* d = ring_raw + slot * row_bytes + (uint32_t)((i * nt + tx) * 16);
      xv[i] = rv[i] = Win<E>{};
      if (in[i]) {
        xv[i] = *reinterpret_cast<const Win<E>*>(d);
        if (a.res) rv[i] = *reinterpret_cast<const Win<E>*>(d + V * nt * 16);
      } else if (A == kPeeled && c0[i] < H) {   // over the row's start or end: read when its turn comes
        load_window<kSingle>(xv[i], x, c0[i], H);
        if (a.res) load_window<kSingle>(rv[i], res, c0[i], H);
      }
    }
    float2 s[V * 4];
    float ss, mx;
    row_sums<E, V>(a, xv, rv, w, s, ss, mx);
    reduce_row(ss, mx, a.q != nullptr, nt, tx, part[flip], 0);   // the other half is free: everyone is past its barrier
    finish_row<A, E, V>(a, s_row, y_row, q_row, tx == 0 ? a.q_scale + t : nullptr, c0, w, s, ss, mx);
    slot = slot == ahead ? 0 : slot + 1;
    x += step * a.ld_x;
    res += step * a.ld_res;
    s_row += step * a.ld_res_out;
    y_row += step * a.ld_y;
    q_row += step * a.ld_q;
  }
}

int row_threads(int windows, int V) {
  const int nt = (windows + V - 1) / V;
  if (nt > 32) return (nt + 31) / 32 * 32;
  int p = 1;
  while (p < nt) p *= 2;
  return p;
}

template <typename E, Access A, int V, int MT>
cudaError_t launch_rows(const NormArgs& a, int windows, cudaStream_t st) {
  const int nt = row_threads(windows, V), rows = nt >= 128 ? 1 : 128 / nt;
  const long long grid = (a.T + rows - 1) / rows;
  return launch_pdl(add_rmsnorm_kernel<E, A, V, MT>, dim3((unsigned)grid), dim3(nt, rows), 0, st, 1, a);
}

template <typename E, Access A, int V, int MT>
cudaError_t launch_stream(const NormArgs& a, int windows, int num_sms, cudaStream_t st) {
  const int nt = row_threads(windows, V);
  const size_t row = (size_t)V * (a.res ? 2 : 1) * nt * 16, fixed = 1024 + sizeof(float2) * 64;
  // three rows ahead where that does not cost a CTA
  const size_t room = 220 * 1024;
  long long per_sm = kStreamThreads<V> / MT * MT / nt;
  const int ahead = per_sm * (4 * row + fixed) <= room ? 3 : 2;
  const size_t smem = (ahead + 1) * row;
  if (per_sm * (long long)(smem + fixed) > (long long)room) per_sm = (long long)(room / (smem + fixed));
  auto kernel = add_rmsnorm_stream_kernel<E, A, V, MT>;
  const cudaError_t e = opt_in_smem((const void*)kernel, smem + sizeof(float2) * 64);   // the static part counts too
  if (e != cudaSuccess) return e;
  const long long grid = a.T < per_sm * num_sms ? a.T : per_sm * num_sms / 8 * 8;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(nt), smem, st, 1, a, ahead);
}

// The split of a row over threads.  It follows from H and the alignment (and,
// for the streaming kernel, from there being enough rows for it), so the same
// row gives the same bits within each of the two kernels.
template <typename E, Access A>
cudaError_t launch_a(const NormArgs& a, int num_sms, cudaStream_t st) {
  const int windows = (a.H + (A == kPeeled ? 14 : 7)) / 8;   // a peeled row of H can touch one more
  if constexpr (A != kSingle) {
    // from 4 rows per SM on (T = 2048, H = 2048: 8.7 us, a CTA per row 10.2),
    // peeled from 16 on (T = 2048, H = 1001: 8.2 and 7.3); short rows go
    // several to a CTA
    if (windows > 96 && a.T >= (A == kAligned ? 4ll : 16ll) * num_sms) {
      if (windows <= 160) return launch_stream<E, A, 1, 160>(a, windows, num_sms, st);
      if (windows <= 320) return launch_stream<E, A, 2, 160>(a, windows, num_sms, st);
      if (windows <= 640) return launch_stream<E, A, 4, 160>(a, windows, num_sms, st);
      if (windows <= 1280) return launch_stream<E, A, 4, 320>(a, windows, num_sms, st);
      return launch_stream<E, A, 4, 640>(a, windows, num_sms, st);
    }
  }
  if (windows <= 256) return launch_rows<E, A, 1, 256>(a, windows, st);
  if (windows <= 512) return launch_rows<E, A, 1, 512>(a, windows, st);
  if (windows <= 1024) return launch_rows<E, A, 2, 512>(a, windows, st);
  return launch_rows<E, A, 5, 512>(a, windows, st);
}

template <typename E>
cudaError_t launch_e(const NormArgs& a, Access acc, int num_sms, cudaStream_t st) {
  return acc == kAligned  ? launch_a<E, kAligned>(a, num_sms, st)
         : acc == kPeeled ? launch_a<E, kPeeled>(a, num_sms, st)
                          : launch_a<E, kSingle>(a, num_sms, st);
}

// Peeled: every tensor in use starts its row t at the same place of the 16-byte
// (E4M3: 8-byte) grid.
Access access_of(const NormArgs& a) {
  const uintptr_t m = reinterpret_cast<uintptr_t>(a.x) / 2;
  auto same = [&](const void* p, long long ld, int size) {
    return !p || (((reinterpret_cast<uintptr_t>(p) / size - m) & 7) == 0 && ((ld - a.ld_x) & 7) == 0);
  };
  if (!same(a.res, a.ld_res, 2) || !same(a.res_out, a.ld_res_out, 2) || !same(a.y, a.ld_y, 2) || !same(a.q, a.ld_q, 1))
    return kSingle;
  return (m & 7) == 0 && a.ld_x % 8 == 0 && a.H % 8 == 0 && (!a.w || blk::aligned(a.w, 16)) ? kAligned : kPeeled;
}

}  // namespace

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_add_rmsnorm(
    const moe_w4a16_rmsnorm_config* cfg, int64_t T, const void* x, const void* residual, const void* weight,
    void* residual_out, void* y, void* q, float* q_scale, moe_w4a16_stream_t stream) try {
  const char* op = "add_rmsnorm";
  if (!cfg) return blk::reject(op, "cfg is NULL");
  const moe_w4a16_rmsnorm_config c = *cfg;
  if (c.dtype != MOE_W4A16_F16 && c.dtype != MOE_W4A16_BF16) return blk::reject(op, "dtype must be F16 or BF16");
  if (c.hidden < 1 || c.hidden > 16384) return blk::reject(op, "hidden outside [1, 16384]");
  if (!(c.eps >= 0.f) || c.eps > 3.4e38f) return blk::reject(op, "eps must be finite and >= 0");
  if (c.reserved) return blk::reject(op, "reserved must be 0");
  if (T < 0 || T > 0x7fffffff) return blk::reject(op, "T outside [0, 2^31)");
  const int64_t lds[5] = {c.ld_x, c.ld_residual, c.ld_residual_out, c.ld_y, c.ld_q};
  for (int64_t ld : lds)
    if (ld != 0 && ld < c.hidden) return blk::reject(op, "a row stride is below hidden");
  if (T == 0) return MOE_W4A16_OK;
  if (!residual_out && !y && !q) return blk::reject(op, "no output given");
  if (!q != !q_scale) return blk::reject(op, "q and q_scale go together");
  if (!x) return blk::reject(op, "x is NULL");
  if (!blk::aligned(x, 2) || !blk::aligned(residual, 2) || !blk::aligned(weight, 2) ||
      !blk::aligned(residual_out, 2) || !blk::aligned(y, 2) || !blk::aligned(q_scale, 4))
    return blk::reject(op, "a pointer is not aligned to its type");
  NormArgs a;
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.res_out = residual_out;
  a.y = y;
  a.q = static_cast<uint8_t*>(q);
  a.q_scale = q_scale;
  a.T = T;
  a.H = c.hidden;
  a.eps = c.eps;
  a.inv_h = 1.0f / (float)c.hidden;
  a.ld_x = c.ld_x ? c.ld_x : c.hidden;
  a.ld_res = c.ld_residual ? c.ld_residual : c.hidden;
  a.ld_res_out = c.ld_residual_out ? c.ld_residual_out : c.hidden;
  a.ld_y = c.ld_y ? c.ld_y : c.hidden;
  a.ld_q = c.ld_q ? c.ld_q : c.hidden;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Access acc = access_of(a);
  const int num_sms = blk::current_sms();
  if (num_sms < 1) return blk::launch_failed(op, cudaErrorNoDevice);
  const cudaError_t e = c.dtype == MOE_W4A16_F16 ? launch_e<__half>(a, acc, num_sms, st)
                                                     : launch_e<__nv_bfloat16>(a, acc, num_sms, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
} catch (...) {   // the host's heap is full
  return MOE_W4A16_ERR_OOM;
}
