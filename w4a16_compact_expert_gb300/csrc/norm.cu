// moe_w4a16_add_rmsnorm: s = x + residual, n = s / sqrt(mean s^2 + eps) * w,
// and n in E4M3 with one scale per row.
//
// Bound by memory: per value 2 + 2 bytes read and 2 + 2 (+ 1) written, about
// 6 flops.  So a row is read once, its sum stays in registers (FP32) between
// the one reduction and the stores, and the E4M3 scale needs no second
// reduction: |n| = |s w| * r with the row's positive r = 1/sqrt(...), hence
// max|n| = r max|s w|, and max|s w| is reduced together with the sum of squares.
#include "block.h"

namespace {

using blk::Pack;

struct NormArgs {
  const void *x, *res, *w;
  void *res_out, *y;
  uint8_t* q;
  float* q_scale;
  long long T, ld_x, ld_res, ld_res_out, ld_y, ld_q;
  int H;
  float eps;
};

// P values of a row per thread, in packs of W; blockDim.x threads per row
// (a multiple of 32), blockDim.y rows per CTA, MT threads at most.  The split depends on H and
// the alignment only, so a row's result does not depend on the batch.
template <typename E, int W, int P, int MT>
__global__ void __launch_bounds__(MT) add_rmsnorm_kernel(NormArgs a) {
  constexpr int V = P / W;
  using PE = Pack<E, W>;
  __shared__ float part_ss[32], part_mx[32];
  const int nt = blockDim.x, tx = threadIdx.x;
  const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < a.T;
  pdl_wait();
  pdl_trigger();
  PE xv[V], rv[V], wv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * nt + tx) * W;
    if (live && col < a.H) {
      xv[i] = *reinterpret_cast<const PE*>(static_cast<const E*>(a.x) + t * a.ld_x + col);
      if (a.res) rv[i] = *reinterpret_cast<const PE*>(static_cast<const E*>(a.res) + t * a.ld_res + col);
      if (a.w) wv[i] = *reinterpret_cast<const PE*>(static_cast<const E*>(a.w) + col);
    }
  }
  float s[P];
  float ss = 0.f, mx = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * nt + tx) * W;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float v = 0.f;
      if (live && col < a.H) {
        v = blk::to_float(xv[i].v[j]);
        if (a.res) v += blk::to_float(rv[i].v[j]);
        const float vw = a.w ? v * blk::to_float(wv[i].v[j]) : v;
        ss = fmaf(v, v, ss);
        mx = fmaxf(mx, fabsf(vw));   // fmaxf leaves NaN out; n and q carry it
      }
      s[i * W + j] = v;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (nt > 32) {
    const int wpr = nt >> 5, w0 = threadIdx.y * wpr;
    if ((tx & 31) == 0) {
      part_ss[w0 + (tx >> 5)] = ss;
      part_mx[w0 + (tx >> 5)] = mx;
    }
    __syncthreads();
    ss = mx = 0.f;
    for (int i = 0; i < wpr; ++i) {
      ss += part_ss[w0 + i];
      mx = fmaxf(mx, part_mx[w0 + i]);
    }
  }
  if (!live) return;
  const float r = 1.0f / sqrtf(ss / (float)a.H + a.eps);
  float c = 0.f, inv = 0.f;
  if (a.q) {
    c = mx * r * (1.0f / 448.0f);
    if (c < 1.17549435e-38f) c = 0.f;   // below 2^-126 the reciprocal would overflow
    inv = c > 0.f ? 1.0f / c : 0.f;
    if (tx == 0) a.q_scale[t] = c;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * nt + tx) * W;
    if (col >= a.H) continue;
    PE so, yo;
    Pack<uint8_t, W> qo;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float v = s[i * W + j];
      const float n = a.w ? v * r * blk::to_float(wv[i].v[j]) : v * r;
      so.v[j] = blk::from_float<E>(v);
      yo.v[j] = blk::from_float<E>(n);
      qo.v[j] = (uint8_t)__nv_cvt_float_to_fp8(n * inv, __NV_SATFINITE, __NV_E4M3);
    }
    if (a.res_out) *reinterpret_cast<PE*>(static_cast<E*>(a.res_out) + t * a.ld_res_out + col) = so;
    if (a.y) *reinterpret_cast<PE*>(static_cast<E*>(a.y) + t * a.ld_y + col) = yo;
    if (a.q) *reinterpret_cast<Pack<uint8_t, W>*>(a.q + t * a.ld_q + col) = qo;
  }
}

template <typename E, int W, int P, int MT>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  int nt = ((a.H + P - 1) / P + 31) / 32 * 32;
  const int rows = nt >= 128 ? 1 : 128 / nt;
  const long long grid = (a.T + rows - 1) / rows;
  return launch_pdl(add_rmsnorm_kernel<E, W, P, MT>, dim3((unsigned)grid), dim3(nt, rows), 0, st, 1, a);
}

template <typename E, int W>
cudaError_t launch_w(const NormArgs& a, cudaStream_t st) {
  if (a.H <= 2048) return launch<E, W, 8, 256>(a, st);
  if (a.H <= 8192) return launch<E, W, 16, 512>(a, st);
  return launch<E, W, 16, 1024>(a, st);
}

template <typename E>
cudaError_t launch_e(const NormArgs& a, int w, cudaStream_t st) {
  return w == 8 ? launch_w<E, 8>(a, st) : w == 4 ? launch_w<E, 4>(a, st) : w == 2 ? launch_w<E, 2>(a, st)
                                                                                  : launch_w<E, 1>(a, st);
}

// The widest pack (8, 4, 2 or 1 elements) that divides the row and every
// stride and pointer in use.
int pack_width(const NormArgs& a) {
  for (int w = 8; w > 1; w >>= 1) {
    const size_t b = 2 * (size_t)w;
    bool ok = a.H % w == 0 && blk::aligned(a.x, b) && a.ld_x % w == 0 && (!a.w || blk::aligned(a.w, b));
    ok = ok && (!a.res || (blk::aligned(a.res, b) && a.ld_res % w == 0));
    ok = ok && (!a.res_out || (blk::aligned(a.res_out, b) && a.ld_res_out % w == 0));
    ok = ok && (!a.y || (blk::aligned(a.y, b) && a.ld_y % w == 0));
    ok = ok && (!a.q || (blk::aligned(a.q, (size_t)w) && a.ld_q % w == 0));
    if (ok) return w;
  }
  return 1;
}

}  // namespace

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_add_rmsnorm(
    const moe_w4a16_rmsnorm_config* cfg, int64_t T, const void* x, const void* residual, const void* weight,
    void* residual_out, void* y, void* q, float* q_scale, moe_w4a16_stream_t stream) {
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
  a.ld_x = c.ld_x ? c.ld_x : c.hidden;
  a.ld_res = c.ld_residual ? c.ld_residual : c.hidden;
  a.ld_res_out = c.ld_residual_out ? c.ld_residual_out : c.hidden;
  a.ld_y = c.ld_y ? c.ld_y : c.hidden;
  a.ld_q = c.ld_q ? c.ld_q : c.hidden;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int w = pack_width(a);
  const cudaError_t e = c.dtype == MOE_W4A16_F16 ? launch_e<__half>(a, w, st) : launch_e<__nv_bfloat16>(a, w, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
}
