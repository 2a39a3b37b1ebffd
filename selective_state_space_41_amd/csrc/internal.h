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

// The end of an entry point.  In a build with VMSCAN_CHECK_WAITS the call waits for its kernels and
// reads the workspace's status word, so that a wait that gave up is reported
// as VMSCAN_ERR_WAIT; otherwise the word is left for the caller to read.
inline vmscan_status finish_call(vmscan_status st, const void* workspace, hipStream_t stream) {
#ifdef VMSCAN_CHECK_WAITS
  if (st != VMSCAN_OK || !workspace) return st;
  hipError_t e = hipStreamSynchronize(stream);
  if (e != hipSuccess) return launch_failed(e);
  int word = 0;
  e = hipMemcpy(&word, workspace, sizeof(word), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return launch_failed(e);
  return word ? VMSCAN_ERR_WAIT : VMSCAN_OK;
#else
  (void)workspace;
  (void)stream;
  return st;
#endif
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
// Loads of what a call reads for the last time, and stores of what is not read soon: both leave the caches to the rest
// (large inputs that a second pass or the next kernel's reads would otherwise push out).  At element alignment.
template <typename V, int ALIGN>
struct Streamed {
  typedef V type __attribute__((aligned(ALIGN)));
};
template <typename V, typename T>
__device__ __forceinline__ V load_once(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const typename Streamed<V, sizeof(T)>::type*>(p));
}
template <typename V, typename T>
__device__ __forceinline__ void store_away(T* p, V v) {
  __builtin_nontemporal_store(v, reinterpret_cast<typename Streamed<V, sizeof(T)>::type*>(p));
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

constexpr float kFp8Max = 448.0f;         // largest finite e4m3 value
constexpr float kMinScale = 1.17549435e-38f;  // a smaller scale would have no finite reciprocal

struct Add {
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
  // keeps a NaN, so that a row that holds one gets a NaN scale
  static __device__ __forceinline__ float of(float a, float b) { return a > b || a != a ? a : b; }
};

// Over 8, 16, 32 or 64 neighbouring lanes, the result in all of them: lane-permuting operations, no LDS
// (LDS shuffles measured 5 % more on the whole of the 8-bit forward).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <typename OP, int LANES>
__device__ __forceinline__ float over_lanes(float v) {
  v = OP::of(v, dpp<0xb1>(v));   // lane ^ 1
  v = OP::of(v, dpp<0x4e>(v));   // lane ^ 2
  v = OP::of(v, dpp<0x141>(v));  // mirrored in 8
  if constexpr (LANES >= 16) v = OP::of(v, dpp<0x140>(v));  // mirrored in 16
  if constexpr (LANES >= 32) {
    const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = OP::of(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LANES >= 64) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = OP::of(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

__device__ __forceinline__ void store_fp8(uint8_t* p, int n, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int t = 0;
    t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k], v[4 * k + 1], t, false);
    t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2], v[4 * k + 3], t, true);
    w[k] = static_cast<uint32_t>(t);
  }
  if (n >= 8) {
    __builtin_memcpy(p, w, 8);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) p[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k % 4)));
}

__device__ __forceinline__ void load_fp8(const uint8_t* p, int n, float (&v)[8]) {
  uint32_t w[2] = {0, 0};
  if (n >= 8) {
    __builtin_memcpy(w, p, 8);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) w[k / 4] |= static_cast<uint32_t>(p[k]) << (8 * (k % 4));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
    v[4 * k] = lo[0], v[4 * k + 1] = lo[1], v[4 * k + 2] = hi[0], v[4 * k + 3] = hi[1];
  }
}

__device__ __forceinline__ float scale_of(float amax) {
  if (amax == 0.0f) return 1.0f;
  const float s = amax / kFp8Max;
  return s < kMinScale ? kMinScale : s;  // NaN stays
}

}  // namespace vmscan_internal

#endif
