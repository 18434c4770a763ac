// Helpers shared by the operators of a decode step around the MoE layer (rotary positions, 4-bit
// linear, tree attention, draft verification).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <exception>
#include <string>

#include "common.cuh"
#include "internal.h"

namespace gbmoe {

// The two 16-bit element types of activations and caches.
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {  // round to nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float a) { return __float2bfloat16_rn(a); }
  static __device__ __forceinline__ float to_float(__nv_bfloat16 a) { return __bfloat162float(a); }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_half2(a, b); }
  static __device__ __forceinline__ __half from_float(float a) { return __float2half_rn(a); }
  static __device__ __forceinline__ float to_float(__half a) { return __half2float(a); }
};

// D[16x8] += A[16x16] * B[16x8] with fp32 accumulation (fragments as for mma_f16_16816).
__device__ __forceinline__ void mma_16816(__half, float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  mma_f16_16816(d, a, b0, b1);
}
__device__ __forceinline__ void mma_16816(__nv_bfloat16, float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Asynchronous 16-byte copies to shared memory: through L2 only, zeros where !ok; or through L1.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_ca(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Division of 0 <= n < 2^31 by a fixed 1 <= d < 2^31: q = (n * mul) >> (32 + shift) with
// mul = ceil(2^(32 + shift) / d) and shift = ceil(log2 d) - 1, which is exact on that range
// (Granlund and Montgomery 1994, "Division by invariant integers using multiplication").
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{0, 0, d};
  if (d == 1) return f;
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  f.shift = l - 1;
  f.mul = static_cast<uint32_t>(((1ull << (32 + f.shift)) + d - 1) / d);
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return f.d == 1 ? n : __umulhi(n, f.mul) >> f.shift;
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Runs the body of a C entry point: no C++ exception leaves it.
template <typename F>
moe_status_t guarded(const char* where, F&& body) {
  try {
    return body();
  } catch (const std::exception& e) {
    try {
      return report_error(MOE_ERR_CUDA, std::string(where) + ": " + e.what());
    } catch (...) {
    }
  } catch (...) {
  }
  return MOE_ERR_CUDA;
}

inline moe_status_t launched(const char* where, cudaError_t err) {
  if (err == cudaSuccess) return MOE_OK;
  return report_error(MOE_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(err));
}

}  // namespace gbmoe
