// Pieces shared by the serving operators (cache append, paged attention, prompt attention, MoE for
// a few tokens): element types, 16-byte vectors of them as fp32, and the index report.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "tl_host.h"

namespace tl {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// An index read on the device was out of range (the entry is left out): the first report of a
// context is kept, without the abort flag, since nothing waits on it.
__device__ __forceinline__ void report_index(DevStatus* st, unsigned long long info) {
  if (atomicCAS(&st->code, 0u, kStatusIndex) == 0u) st->info = info;
}

// Two elements of a 16-bit type from and to fp32 (to: round to nearest even).
template <class T>
__device__ __forceinline__ float2 to_f32x2(uint32_t v);
template <>
__device__ __forceinline__ float2 to_f32x2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 to_f32x2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <class T>
__device__ __forceinline__ uint32_t from_f32x2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t from_f32x2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t from_f32x2<__half>(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Lets a kernel use `bytes` of dynamic shared memory, once per device (a bit of `ready` each).
inline bool smem_ready(std::atomic<unsigned long long>& ready, int device, const void* kern, int bytes) {
  const unsigned long long bit = 1ull << (device & 63);
  if (device < 64 && (ready.load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  ready.fetch_or(device < 64 ? bit : 0, std::memory_order_release);
  return true;
}

inline bool esize_ok(long long stride, int esize) { return stride >= 0 && (stride * esize) % 16 == 0; }

inline bool heads_ok(int heads, int kv_heads, int d) {
  return heads >= 0 && kv_heads >= 1 && heads % kv_heads == 0 && (d == 64 || d == 128);
}

}  // namespace tl
