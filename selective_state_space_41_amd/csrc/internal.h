// What the library's source files share: the last-error record, the argument checks and the
// activation types' loads and stores.  Not installed; the public interface is include/vmscan.h.
#ifndef VMSCAN_INTERNAL_H
#define VMSCAN_INTERNAL_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vmscan.h"

namespace vmscan_internal {

// Keeps a failed HIP call's error for vmscan_last_hip_error() and returns VMSCAN_ERR_HIP.
__attribute__((visibility("hidden"))) vmscan_status launch_failed(hipError_t e);

inline vmscan_status launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? VMSCAN_OK : launch_failed(e);
}

// A launch holds less than 2^32 threads along x: this many workgroups of 256.
constexpr int64_t kMaxBlocks256 = (int64_t{1} << 24) - 1;

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Eight consecutive activations as float32.  The rows of odd-length tensors start at any element:
// the hardware takes 16-byte global accesses at element alignment, and the last, partial run of a
// row goes element by element.
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {  // nearest even
  const __bf16 v = static_cast<__bf16>(f);
  uint16_t r;
  __builtin_memcpy(&r, &v, sizeof(r));
  return r;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  float4 a, b;
  __builtin_memcpy(&a, p, 16);
  __builtin_memcpy(&b, p + 4, 16);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  uint4 r;
  __builtin_memcpy(&r, p, 16);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  const float4 a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
  __builtin_memcpy(p, &a, 16);
  __builtin_memcpy(p + 4, &b, 16);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = static_cast<uint32_t>(f32_to_bf16(v[2 * k])) | (static_cast<uint32_t>(f32_to_bf16(v[2 * k + 1])) << 16);
  const uint4 r = make_uint4(w[0], w[1], w[2], w[3]);
  __builtin_memcpy(p, &r, 16);
}
// elements 0 .. n - 1 only (n may be <= 0 or >= 8); the others read as zero and are not written
template <typename T>
__device__ __forceinline__ void load_upto8(const T* p, int n, float (&v)[8]) {
  if (n >= 8) {
    load8(p, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < n ? load1(p + k) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_upto8(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    store8(p, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) store1(p + k, v[k]);
}

}  // namespace vmscan_internal

#endif
