// moe_w4a16_linear: out = act(x_scale w_scale x W^T + bias) + residual on the
// 5th-generation tensor cores (tcgen05.mma, FP32 accumulators in TMEM), for
// FP16, BF16 and E4M3 operands.  A 128-byte row of a K chunk is 64 16-bit or
// 128 8-bit values and one MMA takes 32 bytes of it, so the pipeline is the
// same for all three.
//
// linear_narrow_kernel: W is the MMA's A operand (128 weight rows, M), the
// tokens are N (16, 32, 64 or 128 of them), so a few tokens waste little of
// the tensor core and the kernel streams W.  The K chunks of a tile are split
// over the S CTAs of a cluster; every CTA leaves its FP32 part in its own
// shared memory and the parts are added in rank order through distributed
// shared memory, each CTA finishing its share of the tile (no workspace, no
// atomics, one launch).  For SWIGLU the 128 rows are 64 gate rows and the
// matching 64 up rows.
#include <cuda.h>

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
  uint32_t idesc;    // MMA instruction descriptor without its N field
  int vec;           // 4: four neighbouring outputs can be read and written at once, else 1
};

DEV_INLINE float gelu_tanh(float a) { return 0.5f * a * (1.f + tanhf(0.7978845608f * (a + 0.044715f * a * a * a))); }

DEV_INLINE float activate(float a, int act) {
  switch (act) {
    case MOE_W4A16_ACT_RELU: return a > 0.f ? a : (a == a ? 0.f : a);
    case MOE_W4A16_ACT_GELU: return 0.5f * a * (1.f + erff(a * 0.70710678f));
    case MOE_W4A16_ACT_GELU_TANH: return gelu_tanh(a);
    case MOE_W4A16_ACT_SILU: return a / (1.f + __expf(-a));
    default: return a;
  }
}

template <bool F8>
DEV_INLINE void umma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  if (F8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
  else
    umma_f16_ss(d_tmem, a_desc, b_desc, idesc, acc);
}

// Four neighbouring outputs of a row: residual and store, V of them valid.
template <typename O>
DEV_INLINE void finish4(const LinearArgs& a, int t, int n, const float (&v)[4]) {
  O* op = static_cast<O*>(a.out) + (size_t)t * a.ld_out + n;
  const O* rp = a.res ? static_cast<const O*>(a.res) + (size_t)t * a.ld_res + n : nullptr;
  if (a.vec == 4 && n + 4 <= a.N) {
    blk::Pack<O, 4> o, r;
    if (rp) r = *reinterpret_cast<const blk::Pack<O, 4>*>(rp);
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = blk::from_float<O>(rp ? v[i] + blk::to_float(r.v[i]) : v[i]);
    *reinterpret_cast<blk::Pack<O, 4>*>(op) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) op[i] = blk::from_float<O>(rp ? v[i] + blk::to_float(rp[i]) : v[i]);
  }
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
  static constexpr int kStages = (104 * 1024) / kStage;   // two CTAs per SM
  static constexpr int kPart = NT * 128 * 4;              // FP32 part of the tile, over the stages when they are done
  static constexpr int kRing = kStages * kStage > kPart ? kStages * kStage : kPart;
  static constexpr int kSmem = kRing + (2 * kStages + 1) * 8 + 16 + 1024;
  static constexpr uint32_t kCols = NT < 32 ? 32 : NT;
  static constexpr int kThreads = 192;   // warp 0 loads, warp 1 multiplies, warps 2-5 empty the accumulator
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <bool F8, int NT>
__global__ void __launch_bounds__(192, 2)
    linear_narrow_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, int out_dtype, int S) {
  using C = NarrowCfg<NT>;
  constexpr int kElem = F8 ? 128 : 64;   // K values per chunk
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool gated = a.act == MOE_W4A16_ACT_SWIGLU;
  const int FT = gated ? 64 : 128;   // output features per tile
  // the CTAs of a cluster are neighbours in x; then the token tiles of one
  // weight tile, so that W comes from L2 after its first reader
  const int rank = blockIdx.x % S, tile = blockIdx.x / S;
  const int ntt = (a.T + NT - 1) / NT;
  const int t0 = (tile % ntt) * NT, n0 = (tile / ntt) * FT;
  const int nk = (a.K + kElem - 1) / kElem;
  const int k0 = (int)((long long)nk * rank / S), k1 = (int)((long long)nk * (rank + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  // tensor memory is taken after the wait and before the trigger: no grid
  // holds any while it waits for one that still has to allocate
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      Pipe p;
      int k = k0;
      for (; k < k1; ++k) {
        if (!mbar_wait_bounded(&empty[p.i], p.ph ^ 1u, &g_block_status)) break;
        uint8_t* dst = smem + p.i * C::kStage;
        mbar_expect_tx(&full[p.i], (uint32_t)C::kStage);
        if (gated) {
          tma_load_2d(dst, &tmW, k * kElem, n0, &full[p.i]);
          tma_load_2d(dst + 64 * kChunk, &tmW, k * kElem, a.N + n0, &full[p.i]);
        } else {
          tma_load_2d(dst, &tmW, k * kElem, n0, &full[p.i]);
        }
        tma_load_2d(dst + C::kA, &tmX, k * kElem, t0, &full[p.i]);
        p.next(C::kStages);
      }
      if (k < k1) {   // gave up: the copies in flight land before the CTA ends
        const int issued = k - k0;
        for (int s = 0; s < C::kStages && s < issued; ++s) {
          const int last = s + (issued - 1 - s) / C::kStages * C::kStages;
          mbar_wait_bounded(&full[s], (uint32_t)((last / C::kStages) & 1), &g_block_status);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      Pipe p;
      const uint32_t idesc = a.idesc | ((uint32_t)(NT >> 3) << 17);
      for (int k = k0; k < k1; ++k) {
        if (!mbar_wait_bounded(&full[p.i], p.ph, &g_block_status)) break;
        tc_fence_after();
        const uint32_t base = smem_u32(smem + p.i * C::kStage);
        const uint64_t ad = sw128_desc(base), bd = sw128_desc(base + C::kA);
#pragma unroll
        for (int j = 0; j < 4; ++j)   // 32 bytes of K each; the address field counts 16 bytes
          umma<F8>(tmem, ad + (uint64_t)(2 * j), bd + (uint64_t)(2 * j), idesc, (uint32_t)(k > k0 || j > 0));
        umma_commit(&empty[p.i]);
        p.next(C::kStages);
      }
      umma_commit(done);
    }
    __syncwarp();
  } else {
    // the accumulator -> this CTA's part [token][weight row]; every stage has
    // been consumed once `done` completes
    const bool ok = mbar_wait_bounded(done, 0, &g_block_status);
    tc_fence_after();
    const int q = warp & 3, row = q * 32 + lane;
    float* part = reinterpret_cast<float*>(smem) + row;
    const int nt = min(NT, a.T - t0);
    if (ok)
      for (int c0 = 0; c0 < nt; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c0 + j) * 128] = __uint_as_float(v[j]);
      }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (S > 1) cluster_sync();

  // four neighbouring features of a token at a time, spread over the cluster
  const int nt = min(NT, a.T - t0), fq = FT / 4;
  const uint32_t part = smem_u32(smem);
  for (int i = rank * C::kThreads + threadIdx.x; i < nt * fq; i += S * C::kThreads) {
    const int tt = i / fq, f = (i % fq) * 4, t = t0 + tt, n = n0 + f;
    if (n >= a.N) continue;
    float v[2][4] = {};
    const uint32_t off = part + (uint32_t)(tt * 128 + f) * 4u;
    for (int r = 0; r < S; ++r) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !gated) break;
        uint32_t addr;
        float p0, p1, p2, p3;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(off + h * 256u), "r"(r));
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(p0), "=f"(p1), "=f"(p2), "=f"(p3)
                     : "r"(addr)
                     : "memory");
        v[h][0] += p0;
        v[h][1] += p1;
        v[h][2] += p2;
        v[h][3] += p3;
      }
    }
    const float xs = a.xs ? a.xs[t] : 1.f;
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int nn = min(n + j, a.N - 1);
      float g = v[0][j];
      if (a.ws) g *= xs * a.ws[nn];
      if (a.bias) g += a.bias[nn];
      if (gated) {
        float u = v[1][j];
        if (a.ws) u *= xs * a.ws[a.N + nn];
        if (a.bias) u += a.bias[a.N + nn];
        o[j] = g / (1.f + __expf(-g)) * u;
      } else {
        o[j] = activate(g, a.act);
      }
    }
    if (out_dtype == MOE_W4A16_F16) finish4<__half>(a, t, n, o);
    else if (out_dtype == MOE_W4A16_BF16) finish4<__nv_bfloat16>(a, t, n, o);
    else finish4<float>(a, t, n, o);
  }
  if (S > 1) cluster_sync();   // nobody leaves while its part is read
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
  int elem, out_dtype, num_sms;
};

// CTAs of a cluster share a tile's K chunks.  The split that ends first, with
// `slots` CTAs at a time and each costing its chunks and about four chunks'
// time for its start, its share of the sum and its stores.
int split_of(int tiles, int nk, int slots) {
  int best = 1;
  long long cost = -1;
  for (int s = 1; s <= 8 && s <= nk; ++s) {
    const long long waves = ((long long)tiles * s + slots - 1) / slots;
    const long long c = waves * ((nk + s - 1) / s + 4);
    if (cost < 0 || c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

template <bool F8, int NT>
cudaError_t launch_narrow(const Problem& p, cudaStream_t st) {
  using C = NarrowCfg<NT>;
  const bool gated = p.a.act == MOE_W4A16_ACT_SWIGLU;
  const int FT = gated ? 64 : 128;
  CUtensorMap mw, mx;
  if (!encode_rows(&mw, p.w, gated ? 2ll * p.a.N : p.a.N, p.a.K, p.elem, p.ld_w, FT) ||
      !encode_rows(&mx, p.x, p.a.T, p.a.K, p.elem, p.ld_x, NT))
    return cudaErrorInvalidValue;
  auto kernel = linear_narrow_kernel<F8, NT>;
  cudaError_t e = opt_in_smem((const void*)kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((p.a.N + FT - 1) / FT) * ((p.a.T + NT - 1) / NT);
  const int nk = (p.a.K + kChunk / p.elem - 1) / (kChunk / p.elem);
  const int S = tiles > (1 << 24) ? 1 : split_of((int)tiles, nk, 2 * p.num_sms);
  if (tiles * S > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(kernel, dim3((unsigned)(tiles * S)), dim3(C::kThreads), C::kSmem, st, S, p.a, mw, mx, p.out_dtype, S);
}

template <bool F8>
cudaError_t launch_linear(const Problem& p, cudaStream_t st) {
  if (p.a.T <= 16) return launch_narrow<F8, 16>(p, st);
  if (p.a.T <= 32) return launch_narrow<F8, 32>(p, st);
  if (p.a.T <= 64) return launch_narrow<F8, 64>(p, st);
  return launch_narrow<F8, 128>(p, st);
}

int elem_size(int dtype) { return dtype == MOE_W4A16_E4M3 ? 1 : dtype == MOE_W4A16_F32 ? 4 : 2; }

// SM count of the current device, asked once per device.
int current_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  if (!sms[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) cudaGetLastError();
    sms[dev] = n;
  }
  return sms[dev];
}

}  // namespace

extern "C" MOE_W4A16_API moe_w4a16_status moe_w4a16_linear(const moe_w4a16_linear_config* cfg, int64_t T,
                                                           const void* x, const void* w, const float* x_scale,
                                                           const float* w_scale, const float* bias,
                                                           const void* residual, void* out,
                                                           moe_w4a16_stream_t stream) {
  const char* op = "linear";
  if (!cfg) return blk::reject(op, "cfg is NULL");
  const moe_w4a16_linear_config c = *cfg;
  const bool f8 = c.in_dtype == MOE_W4A16_E4M3;
  if (c.in_dtype != MOE_W4A16_F16 && c.in_dtype != MOE_W4A16_BF16 && !f8)
    return blk::reject(op, "in_dtype must be F16, BF16 or E4M3");
  if (c.out_dtype != MOE_W4A16_F16 && c.out_dtype != MOE_W4A16_BF16 && c.out_dtype != MOE_W4A16_F32)
    return blk::reject(op, "out_dtype must be F16, BF16 or F32");
  if (c.act < MOE_W4A16_ACT_NONE || c.act > MOE_W4A16_ACT_SWIGLU) return blk::reject(op, "unknown activation");
  if (c.reserved) return blk::reject(op, "reserved must be 0");
  if (c.n < 1 || c.n > (1 << 29) || c.k < 1 || c.k > (1 << 30))
    return blk::reject(op, "n outside [1, 2^29] or k outside [1, 2^30]");
  if (T < 0 || T > (1 << 30)) return blk::reject(op, "T outside [0, 2^30]");
  const int es = elem_size(c.in_dtype), os = elem_size(c.out_dtype);
  const int64_t ld_x = c.ld_x ? c.ld_x : c.k, ld_w = c.ld_w ? c.ld_w : c.k;
  const int64_t ld_out = c.ld_out ? c.ld_out : c.n, ld_res = c.ld_residual ? c.ld_residual : c.n;
  if (ld_x < c.k || ld_w < c.k || ld_out < c.n || ld_res < c.n)
    return blk::reject(op, "a row stride is below the row length");
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
  p.num_sms = current_sms();
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
  // FP32 accumulator; operand formats: kind::f16 0 = FP16, 1 = BF16; kind::f8f6f4 0 = E4M3; M = 128
  const uint32_t fmt = c.in_dtype == MOE_W4A16_BF16 ? 1u : 0u;
  p.a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 4) << 24);
  const size_t vb = 4 * (size_t)os;
  p.a.vec = blk::aligned(out, vb) && ld_out % 4 == 0 && (!residual || (blk::aligned(residual, vb) && ld_res % 4 == 0)) ? 4 : 1;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = f8 ? launch_linear<true>(p, st) : launch_linear<false>(p, st);
  return e == cudaSuccess ? MOE_W4A16_OK : blk::launch_failed(op, e);
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
