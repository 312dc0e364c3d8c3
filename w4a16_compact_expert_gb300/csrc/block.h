// Declarations shared by the block operators (norm.cu, score.cu, linear.cu):
// element types, conversions and argument errors.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdio.h>

#include <atomic>

#include "moe_w4a16.h"
#include "internal.h"

namespace blk {

DEV_INLINE float to_float(__half v) { return __half2float(v); }
DEV_INLINE float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
DEV_INLINE float to_float(float v) { return v; }
template <typename E>
DEV_INLINE E from_float(float v);
template <>
DEV_INLINE __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
DEV_INLINE __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
DEV_INLINE float from_float<float>(float v) { return v; }

// One instruction each (e^x: beside the multiplication); results below 2^-126
// are 0.  2^x: 2 ulp; e^x as 2^(x log2 e): up to 1.3 |x| 2^-24 more, relative;
// 1 / x: 1 ulp, 0 where |x| passes 2^126.
DEV_INLINE float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
DEV_INLINE float fast_exp(float x) { return fast_exp2(x * 1.4426950408889634f); }
DEV_INLINE float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Packed FP32 pairs.
DEV_INLINE float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
DEV_INLINE float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
DEV_INLINE float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}

// W neighbouring elements, loaded and stored at once.
template <typename E, int W>
struct alignas(sizeof(E) * W) Pack {
  E v[W];
};

inline moe_w4a16_status reject(const char* op, const char* msg) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", op, msg);
  set_handle_free_error(buf);
  return MOE_W4A16_ERR_INVALID_ARG;
}

inline moe_w4a16_status launch_failed(const char* op, cudaError_t e) {
  cudaGetLastError();
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", op, cudaGetErrorString(e));
  set_handle_free_error(buf);
  return MOE_W4A16_ERR_CUDA;
}

// SM count of the current device, asked once per device.
inline int current_sms(int* device = nullptr) {
  static std::atomic<int> sms[64];   // racing first calls store the same
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  int n = sms[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) cudaGetLastError();
    sms[dev].store(n, std::memory_order_relaxed);
  }
  if (device) *device = dev;
  return n;
}

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace blk
