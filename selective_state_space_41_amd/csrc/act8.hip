// Activations in 8 bits: e4m3 codes with a float32 scale for each 128 channels of a row, and back.  What is
// computed is stated in include/vmscan.h.
//
// 16 neighbouring lanes own a group of 128 channels, 8 each, so that a group's largest magnitude is a butterfly of
// four lane operations, and loads and stores are 16 or 8 bytes a lane.  Bound by HBM: 25216 x 768 bfloat16 packed in 11.5
// us (59 MB, 5.1 TB/s), 25216 x 392 unpacked in 7.6 (30 MB, 4.0 TB/s: half of it is the launch).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

constexpr int kGroup = 128;                     // channels that share a scale
constexpr int kUnits = 256 / (kGroup / 8);      // groups of a workgroup
constexpr int64_t kMaxDim = int64_t{1} << 30;

struct Act8Args {
  const void* x;
  const uint8_t* codes_in;
  const float* scale_in;
  void* out;
  float* scale;
  int64_t units, x_stride;  // units: rows * groups
  int dim, groups;
};

// The row and group of a unit.
struct Place {
  int64_t row;
  int group;
};
__device__ __forceinline__ Place place_of(int64_t unit, int groups) {
  if (groups == 1) return {unit, 0};
  const uint32_t r = static_cast<uint32_t>(unit) / static_cast<uint32_t>(groups);  // units: under 2^28
  return {r, static_cast<int>(static_cast<uint32_t>(unit) - r * static_cast<uint32_t>(groups))};
}

// v / s as far as its code shows it: the code nearest to the float32 quotient.  The product with 1 / s alone takes 4 in 10000
// bfloat16 codes across a tie.  Its remainder, times 1 / s once more, leaves an error under 2^-45 of the quotient, which
// decides a code only where the quotient lies that near to a float32 midpoint beside a tie.  A bfloat16 value's does not:
// with s an integer of 24 bits and the tie an odd T < 32 (in powers of two), v = s T + N for a whole N <= 16, s = N 2^20 + k
// with |k| <= 12 (T = 1: s = 2^24 - 1, which is no value over 448), and v has 8 bits, so k T = -N, but N < T.  Float32 values
// are divided, which costs nothing there (50176 x 768 31 us with either; bfloat16 25216 x 769 17.7 us divided, 14.4 so).
template <typename T>
__device__ __forceinline__ void over_scale(float (&v)[8], float s) {
  if (sizeof(T) == 4 || s < 0x1p-64f) {  // (a small scale's remainders would be below float32's numbers)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] /= s;
    return;
  }
  const float inv = 1.0f / s;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = v[k] * inv;
    v[k] = __builtin_fmaf(-__builtin_fmaf(q, s, -v[k]), inv, q);  // (a zero keeps its sign)
  }
}

template <typename T>
__global__ __launch_bounds__(256) void act8_pack_kernel(Act8Args a) {
  const int lane = threadIdx.x & 15;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (threadIdx.x >> 4);
  const bool live = unit < a.units;
  const Place p = place_of(live ? unit : a.units - 1, a.groups);
  const int c = p.group * kGroup + lane * 8;
  const int n = live ? a.dim - c : 0;
  float v[8];
  load_upto8(static_cast<const T*>(a.x) + p.row * a.x_stride + c, n, v);
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = Max::of(top, __builtin_fabsf(v[k]));
  top = over_lanes<Max, 16>(top);
  over_scale<T>(v, scale_of(top));
  store_fp8(static_cast<uint8_t*>(a.out) + p.row * a.dim + c, n, v);
  if (live && lane == 0) a.scale[unit] = scale_of(top);
}

template <typename T>
__global__ __launch_bounds__(256) void act8_unpack_kernel(Act8Args a) {
  const int lane = threadIdx.x & 15;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + (threadIdx.x >> 4);
  if (unit >= a.units) return;
  const Place p = place_of(unit, a.groups);
  const int c = p.group * kGroup + lane * 8, n = a.dim - c;
  if (n <= 0) return;
  float v[8];
  load_fp8(a.codes_in + p.row * a.dim + c, n, v);
  const float s = a.scale_in[unit];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= s;
  store_upto8(static_cast<T*>(a.out) + p.row * a.dim + c, n, v);
}

vmscan_status sizes_of(int64_t rows, int64_t dim, vmscan_dtype dtype, Act8Args& a) {
  if (rows < 1 || dim < 1 || dim > kMaxDim || rows >= (int64_t{1} << 40)) return VMSCAN_ERR_SHAPE;
  if (dtype != VMSCAN_F32 && dtype != VMSCAN_BF16) return VMSCAN_ERR_UNSUPPORTED;
  a.dim = static_cast<int>(dim);
  a.groups = static_cast<int>((dim + kGroup - 1) / kGroup);
  a.units = rows * a.groups;
  return a.units > kMaxBlocks256 * kUnits ? VMSCAN_ERR_SHAPE : VMSCAN_OK;
}

dim3 grid_of(const Act8Args& a) { return dim3(static_cast<unsigned>((a.units + kUnits - 1) / kUnits)); }

}  // namespace

extern "C" {

vmscan_status vmscan_act8_pack(const void* x, int64_t x_stride, void* codes, float* scale, int64_t rows, int64_t dim,
                               vmscan_dtype dtype, hipStream_t stream) {
  if (!x || !codes || !scale) return VMSCAN_ERR_NULL;
  Act8Args a{};
  const vmscan_status s = sizes_of(rows, dim, dtype, a);
  if (s != VMSCAN_OK) return s;
  if (x_stride < dim || x_stride > (int64_t{1} << 40)) return VMSCAN_ERR_SHAPE;
  if (!aligned_to(x, dtype == VMSCAN_F32 ? 4 : 2) || !aligned_to(scale, 4)) return VMSCAN_ERR_ALIGN;
  a.x = x, a.x_stride = x_stride, a.out = codes, a.scale = scale;
  if (dtype == VMSCAN_F32)
    hipLaunchKernelGGL((act8_pack_kernel<float>), grid_of(a), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((act8_pack_kernel<uint16_t>), grid_of(a), dim3(256), 0, stream, a);
  return launched();
}

vmscan_status vmscan_act8_unpack(const void* codes, const float* scale, void* x, int64_t rows, int64_t dim,
                                 vmscan_dtype dtype, hipStream_t stream) {
  if (!codes || !scale || !x) return VMSCAN_ERR_NULL;
  Act8Args a{};
  const vmscan_status s = sizes_of(rows, dim, dtype, a);
  if (s != VMSCAN_OK) return s;
  if (!aligned_to(x, dtype == VMSCAN_F32 ? 4 : 2) || !aligned_to(scale, 4)) return VMSCAN_ERR_ALIGN;
  a.codes_in = static_cast<const uint8_t*>(codes), a.scale_in = scale, a.out = x;
  if (dtype == VMSCAN_F32)
    hipLaunchKernelGGL((act8_unpack_kernel<float>), grid_of(a), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((act8_unpack_kernel<uint16_t>), grid_of(a), dim3(256), 0, stream, a);
  return launched();
}

}  // extern "C"
