// Pieces shared by the serving operators (cache append, paged attention, prompt attention, MoE for
// a few tokens): element types, 16-byte vectors of them as fp32, and the index report.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

#include "tl_host.h"

namespace tl {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// An index read on the device was out of range (the entry is left out): the first report of a
// context is kept, without the abort flag, since nothing waits on it.  It never replaces a timeout, and a
// timeout replaces it (report_timeout).
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

// Softmax weights that meet V as fp16 are held times 2^7: fp16 has a step of 2^-24 below 2^-14 and nothing below
// 2^-25, and beside one dominant key the rest of a long sequence may lie there.  The maximum that weights refer to is
// stale by 2^8 at most, so they stay below 2^15.  The kernels keep m - 7 in place of m, so the factor
// costs nothing: it is in the weights, their sum and O alike.  bf16 has fp32's range and needs none.
template <class M>
constexpr float kWeightBits = std::is_same<M, __half>::value ? 7.f : 0.f;

// 16 bytes to shared memory; with bytes 0, zeros, and nothing is read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d += a b: 16 x 8 x 16, fp32 sums.
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// The first bytes of a serving operator's workspace: counters that every call leaves at zero, whatever its
// shape.  A CTA's range of work starts at most one piece that goes on in other CTAs, so the counter
// of a cut piece is that of the CTA it starts in.
constexpr int kCutCounters = 1024;         // by CTA: the largest grid
constexpr int kItemCounters = 1024;        // MoE: by item, at most 128 tokens x topk 8
constexpr int kTokenCounters = 128 * 256;  // MoE: by token and block of 256 of at most 32768 columns (twice what that takes)
constexpr size_t kCounterBytes = (kCutCounters + kItemCounters + kTokenCounters) * 4;
static_assert(kCounterBytes == TL_SERVE_COUNTER_BYTES, "header");

inline bool esize_ok(long long stride, int esize) { return stride >= 0 && (stride * esize) % 16 == 0; }

inline bool heads_ok(int heads, int kv_heads, int d) {
  return heads >= 0 && kv_heads >= 1 && heads % kv_heads == 0 && (d == 64 || d == 128);
}

}  // namespace tl
