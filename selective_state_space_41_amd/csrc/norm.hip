// Root-mean-square norm with the residual's addition: forward (activations or 8 bits out) and
// gradient.  What is computed is stated in include/vmscan.h.
//
// A row belongs to LPR lanes of one wave (short rows share a wave) or to all W waves of a
// workgroup; a lane keeps its E runs of 8 consecutive elements in registers from the load to the
// store, so x and the residual are read once and nothing but the outputs is written (but for the gradient of rows over
// 8192 channels, which spills some 50 registers of a lane).  The sum of
// squares, the scale's maximum and the gradient's dot product are float32 butterflies over the
// row's lanes.  Bound by HBM: the arithmetic is about 6 (forward) or 12 (gradient) operations for
// 8 or more bytes.  Measured: 48680 x 768 bfloat16 with residual to 8 bits, 262 MB in 62 us, 4.2 TB/s;
// gradient of 25216 x 384 bfloat16 with a float32 residual, 155 MB in 28 us, and 4 us for dw's partial rows.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

constexpr float kFp8Max = 448.0f;         // largest finite e4m3 value
constexpr float kMinScale = 1.17549435e-38f;  // a smaller scale would have no finite reciprocal
constexpr int kGroupLanes = 16;           // a group of 128 channels: 16 lanes' runs of 8
constexpr int kMaxDim = 16 * 64 * 4 * 8;  // 16 waves, 4 runs of 8 per lane
// Forward: a workgroup per rows, 60 us on 48680 x 768 (a fixed grid that goes round over the rows: 68); only past this many
// do they go round.
constexpr int kFwdBlocks = 1 << 20;
// Gradient: workgroups that go round over the rows, each with a partial row of the weight's gradient (2048 of
// them measured 50 us instead of 38 on 25216 x 384).
constexpr int kBwdBlocks = 1024;

struct NormArgs {
  const void *x, *res;
  const float* w;
  void *y, *res_out;
  float *scale, *rstd;
  int64_t rows, x_stride;
  int dim, group;  // group 0: one scale per row
  float eps;
};

struct NormBwdArgs {
  const void *dy, *r, *dres;
  const float *w, *rstd;
  void *dx, *dres_out;
  float* part;
  int64_t rows, r_stride;
  int dim;
};

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
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
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

// Over the lanes of the row: LPR lanes of a wave, or all lanes of W waves.  `slot` holds W floats
// of LDS that no other reduction of the same row uses.
template <typename OP, int LPR, int W>
__device__ __forceinline__ float over_row(float v, float* slot) {
  v = over_lanes<OP, LPR>(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = OP::of(v, slot[i]);
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

__device__ __forceinline__ float scale_of(float amax) {
  if (amax == 0.0f) return 1.0f;
  const float s = amax / kFp8Max;
  return s < kMinScale ? kMinScale : s;  // NaN stays
}

template <typename T, typename R, bool FP8, int LPR, int W, int E>
__global__ __launch_bounds__(W > 1 ? 64 * W : 256) void rmsnorm_fwd_kernel(NormArgs a) {
  constexpr int kRows = W > 1 ? 1 : 256 / LPR;  // rows per workgroup
  __shared__ float slots[2][2][W];              // [which reduction][row parity][wave]
  const int lane = W > 1 ? threadIdx.x : threadIdx.x % LPR;
  const int sub = W > 1 ? 0 : threadIdx.x / LPR;
  constexpr int kLanes = W > 1 ? 64 * W : LPR;
  const int dim = a.dim;
  float w[E][8];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (e * kLanes + lane) * 8;
    load_upto8(a.w + c, dim - c, w[e]);
  }
  const float inv_dim = 1.0f / static_cast<float>(dim);
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < a.rows;
       row0 += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;  // W > 1: uniform and true
    const int n = live ? dim : 0;
    const T* xp = static_cast<const T*>(a.x) + row * a.x_stride;
    const R* rp = static_cast<const R*>(a.res) + row * dim;
    float r[E][8];
    float sq = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * kLanes + lane) * 8;
      load_upto8(xp + c, n - c, r[e]);
    }
    if (a.res) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * kLanes + lane) * 8;
        float t[8];
        load_upto8(rp + c, n - c, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[e][k] += t[k];
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) sq = __builtin_fmaf(r[e][k], r[e][k], sq);
    if (a.res_out) {
      R* op = static_cast<R*>(a.res_out) + row * dim;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * kLanes + lane) * 8;
        store_upto8(op + c, n - c, r[e]);
      }
    }
    sq = over_row<Add, LPR, W>(sq, slots[0][turn]);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sq, inv_dim, a.eps));
    if (a.rstd && lane == 0 && live) a.rstd[row] = rstd;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) r[e][k] = r[e][k] * rstd * w[e][k];
    if constexpr (!FP8) {
      T* yp = static_cast<T*>(a.y) + row * dim;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * kLanes + lane) * 8;
        store_upto8(yp + c, n - c, r[e]);
      }
    } else {
      uint8_t* yp = static_cast<uint8_t*>(a.y) + row * dim;
      float top[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        top[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) top[e] = Max::of(top[e], __builtin_fabsf(r[e][k]));
      }
      if (a.group == 0) {
        float t = top[0];
#pragma unroll
        for (int e = 1; e < E; ++e) t = Max::of(t, top[e]);
        t = over_row<Max, LPR, W>(t, slots[1][turn]);
#pragma unroll
        for (int e = 0; e < E; ++e) top[e] = t;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) top[e] = over_lanes<Max, LPR < kGroupLanes ? LPR : kGroupLanes>(top[e]);
      }
      const int groups = a.group ? (dim + a.group - 1) / a.group : 1;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * kLanes + lane) * 8;
        const float s = scale_of(top[e]);
        // The code is the value nearest to y times the scale's reciprocal: within one unit in the
        // last place of y / scale in float32, against the 2^-4 step of the codes.
        const float inv = 1.0f / s;
#pragma unroll
        for (int k = 0; k < 8; ++k) r[e][k] *= inv;
        store_fp8(yp + c, n - c, r[e]);
        if (a.group ? (lane % kGroupLanes == 0 && c < n) : (e == 0 && lane == 0 && live))
          a.scale[row * groups + (a.group ? c / a.group : 0)] = s;
      }
    }
  }
}

// Floats from one partial row to the next: whole groups of the 32 columns that the sum takes at a time.
__host__ __device__ constexpr int64_t part_stride(int64_t dim) { return (dim + 31) / 32 * 32; }

template <typename T, typename R, int LPR, int W, int E>
__global__ __launch_bounds__(W > 1 ? 64 * W : 256) void rmsnorm_bwd_kernel(NormBwdArgs a) {
  constexpr int kRows = W > 1 ? 1 : 256 / LPR;
  constexpr int kLanes = W > 1 ? 64 * W : LPR;
  constexpr bool kSplit = !std::is_same<T, R>::value;  // dx and the residual's gradient differ in type
  __shared__ float slots[2][W];
  __shared__ __align__(16) float rowsum[W > 1 ? 1 : 256 * E * 8];
  const int lane = W > 1 ? threadIdx.x : threadIdx.x % LPR;
  const int sub = W > 1 ? 0 : threadIdx.x / LPR;
  const int dim = a.dim;
  // 16 waves have 128 registers each, which r, dy and the weight's gradient nearly fill: they read the weight again for each
  // row, and the gradient of the residual where it is added.  4000 x 16384, us, so / all kept, in scratch: bfloat16 with a
  // float32 residual 616 / 922, float32 518 / 823; a second read of the whole row instead 774 and 736.
  constexpr bool kKeep = W * E < 64;
  float w[kKeep ? E : 1][8], dw[E][8];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (e * kLanes + lane) * 8;
    if constexpr (kKeep) load_upto8(a.w + c, dim - c, w[e]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[e][k] = 0.0f;
  }
  const float inv_dim = 1.0f / static_cast<float>(dim);
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < a.rows;
       row0 += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
    const int64_t row = row0 + sub;
    int here = lane;
    if constexpr (!kKeep) asm volatile("" : "+v"(here));  // places are made where they are used, not kept for all rows
    const bool live = row < a.rows;
    const int n = live ? dim : 0;
    const int64_t at = row * dim;
    const float rstd = live ? a.rstd[row] : 0.0f;
    float r[E][8], g[E][8], d[kKeep ? E : 1][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * kLanes + here) * 8;
      load_upto8(static_cast<const R*>(a.r) + row * a.r_stride + c, n - c, r[e]);
      load_upto8(static_cast<const T*>(a.dy) + at + c, n - c, g[e]);
      if constexpr (kKeep)
        if (a.dres) load_upto8(static_cast<const R*>(a.dres) + at + c, n - c, d[e]);
    }
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float (&we)[8] = w[kKeep ? e : 0];
      if constexpr (!kKeep) {
        __builtin_amdgcn_sched_barrier(0);
        load_upto8(a.w + (e * kLanes + here) * 8, dim - (e * kLanes + here) * 8, we);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[e][k] *= rstd;
        dw[e][k] = __builtin_fmaf(g[e][k], r[e][k], dw[e][k]);
        g[e][k] *= we[k];
        dot = __builtin_fmaf(r[e][k], g[e][k], dot);
      }
    }
    dot = over_row<Add, LPR, W>(dot, slots[turn]) * inv_dim;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * kLanes + here) * 8;
      float (&de)[8] = d[kKeep ? e : 0];
      if constexpr (!kKeep) {
        __builtin_amdgcn_sched_barrier(0);
        if (a.dres) load_upto8(static_cast<const R*>(a.dres) + at + c, n - c, de);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = rstd * __builtin_fmaf(-r[e][k], dot, g[e][k]);
        g[e][k] = a.dres ? v + de[k] : v;
      }
      store_upto8(static_cast<T*>(a.dx) + at + c, n - c, g[e]);
      if constexpr (kSplit)
        if (a.dres_out) store_upto8(static_cast<R*>(a.dres_out) + at + c, n - c, g[e]);
    }
  }
  // this workgroup's share of dw: its rows' sums, in a fixed order
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * part_stride(dim);
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * kLanes + lane) * 8;
      store_upto8(part + c, dim - c, dw[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) rowsum[sub * (LPR * E * 8) + (e * LPR + lane) * 8 + k] = dw[e][k];
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += 256) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) t += rowsum[i * (LPR * E * 8) + c];
      part[c] = t;
    }
  }
}

// dw[c] = the sum of `n` partial rows: a workgroup takes 32 columns, 8 lanes of 4 columns and 128 shares of the
// rows, whose sums meet in LDS in a fixed order.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                          int n, int dim) {
  __shared__ __align__(16) float4 s[128][8];
  const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
  const int64_t stride = part_stride(dim);
  const float* p = part + blockIdx.x * 32 + cx * 4;
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = ry; i < n; i += 128) {
    const float4 v = *reinterpret_cast<const float4*>(p + i * stride);
    t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
  }
  s[ry][cx] = t;
#pragma unroll
  for (int m = 64; m >= 1; m >>= 1) {
    __syncthreads();
    if (ry < m) {
      const float4 v = s[ry + m][cx];
      t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
      s[ry][cx] = t;
    }
  }
  const int c = blockIdx.x * 32 + cx * 4;
  if (ry == 0) {
    const float v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < dim) dw[c + k] = v[k];
  }
}

// Calls f with the row layout for `dim`: the fewest lanes that hold the row, 8 elements each, then
// more runs per lane, then more waves.
template <typename F>
void with_layout(int dim, F&& f) {
  using std::integral_constant;
#define VMSCAN_LAYOUT(LPR, W, E) \
  f(integral_constant<int, LPR>{}, integral_constant<int, W>{}, integral_constant<int, E>{})
  if (dim <= 64) VMSCAN_LAYOUT(8, 1, 1);
  else if (dim <= 128) VMSCAN_LAYOUT(16, 1, 1);
  else if (dim <= 256) VMSCAN_LAYOUT(32, 1, 1);
  else if (dim <= 512) VMSCAN_LAYOUT(64, 1, 1);
  else if (dim <= 1024) VMSCAN_LAYOUT(64, 1, 2);
  else if (dim <= 2048) VMSCAN_LAYOUT(64, 1, 4);
  else if (dim <= 8192) VMSCAN_LAYOUT(64, 4, 4);
  else VMSCAN_LAYOUT(64, 16, 4);
#undef VMSCAN_LAYOUT
}

int rows_per_block(int64_t dim) { return dim > 2048 ? 1 : dim > 256 ? 4 : dim > 128 ? 8 : dim > 64 ? 16 : 32; }

unsigned blocks_for(int64_t rows, int64_t dim, int64_t most) {
  const int64_t b = (rows + rows_per_block(dim) - 1) / rows_per_block(dim);
  return static_cast<unsigned>(b < most ? b : most);
}

template <typename T, typename R>
void launch_fwd(const NormArgs& a, bool fp8, hipStream_t stream) {
  const dim3 grid(blocks_for(a.rows, a.dim, kFwdBlocks));
  with_layout(a.dim, [&](auto lpr, auto wv, auto ev) {
    constexpr int LPR = decltype(lpr)::value, W = decltype(wv)::value, E = decltype(ev)::value;
    const dim3 block(W > 1 ? 64 * W : 256);
    if (fp8)
      hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, R, true, LPR, W, E>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((rmsnorm_fwd_kernel<T, R, false, LPR, W, E>), grid, block, 0, stream, a);
  });
}

template <typename T, typename R>
void launch_bwd(const NormBwdArgs& a, unsigned blocks, hipStream_t stream) {
  with_layout(a.dim, [&](auto lpr, auto wv, auto ev) {
    constexpr int LPR = decltype(lpr)::value, W = decltype(wv)::value, E = decltype(ev)::value;
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, R, LPR, W, E>), dim3(blocks), dim3(W > 1 ? 64 * W : 256), 0, stream, a);
  });
}

bool norm_shape_ok(int64_t rows, int64_t dim) {
  return rows >= 1 && dim >= 1 && dim <= kMaxDim && rows < (int64_t{1} << 40);
}

bool dtypes_ok(vmscan_dtype dtype, vmscan_dtype res_dtype) {
  return (dtype == VMSCAN_F32 && res_dtype == VMSCAN_F32) ||
         (dtype == VMSCAN_BF16 && (res_dtype == VMSCAN_F32 || res_dtype == VMSCAN_BF16));
}

}  // namespace

extern "C" {

vmscan_status vmscan_rmsnorm_fwd(const void* x, int64_t x_stride, const void* residual, const float* weight, void* y,
                                 float* scale, void* residual_out, float* rstd, int64_t rows, int64_t dim, float eps,
                                 vmscan_dtype dtype, vmscan_dtype residual_dtype, int out_fp8, int group,
                                 hipStream_t stream) {
  if (!x || !weight || !y) return VMSCAN_ERR_NULL;
  if ((residual == nullptr) != (residual_out == nullptr)) return VMSCAN_ERR_NULL;  // the sum and its place
  if ((out_fp8 != 0) != (scale != nullptr)) return VMSCAN_ERR_NULL;
  if (!norm_shape_ok(rows, dim) || x_stride < dim || x_stride > (int64_t{1} << 40) || !(eps >= 0.0f))
    return VMSCAN_ERR_SHAPE;
  if (!dtypes_ok(dtype, residual_dtype) || (out_fp8 != 0 && out_fp8 != 1) || (group != 0 && group != 128) ||
      (group && !out_fp8))
    return VMSCAN_ERR_UNSUPPORTED;
  const void* ptrs[] = {x, residual, weight, y, scale, residual_out, rstd};
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return VMSCAN_ERR_ALIGN;
  const NormArgs a{x, residual, weight, y, residual_out, scale, rstd, rows, x_stride, static_cast<int>(dim), group, eps};
  if (dtype == VMSCAN_F32)
    launch_fwd<float, float>(a, out_fp8 != 0, stream);
  else if (residual_dtype == VMSCAN_F32)
    launch_fwd<uint16_t, float>(a, out_fp8 != 0, stream);
  else
    launch_fwd<uint16_t, uint16_t>(a, out_fp8 != 0, stream);
  return launched();
}

size_t vmscan_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  if (!norm_shape_ok(rows, dim)) return 0;
  return static_cast<size_t>(blocks_for(rows, dim, kBwdBlocks)) * part_stride(dim) * sizeof(float);
}

vmscan_status vmscan_rmsnorm_bwd(const void* dy, const void* r, const float* weight, const float* rstd,
                                 const void* dresidual_out, void* dx, void* dresidual, float* dweight, int64_t rows,
                                 int64_t dim, vmscan_dtype dtype, vmscan_dtype residual_dtype, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  return vmscan_rmsnorm_bwd_ex(dy, r, dim, weight, rstd, dresidual_out, dx, dresidual, dweight, rows, dim, dtype,
                               residual_dtype, workspace, workspace_bytes, stream);
}

vmscan_status vmscan_rmsnorm_bwd_ex(const void* dy, const void* r, int64_t r_stride, const float* weight,
                                    const float* rstd, const void* dresidual_out, void* dx, void* dresidual,
                                    float* dweight, int64_t rows, int64_t dim, vmscan_dtype dtype,
                                    vmscan_dtype residual_dtype, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream) {
  if (!dy || !r || !weight || !rstd || !dx || !dweight) return VMSCAN_ERR_NULL;
  if (!norm_shape_ok(rows, dim) || r_stride < dim || r_stride > (int64_t{1} << 40)) return VMSCAN_ERR_SHAPE;
  // with one type for both, dx is the residual's gradient too
  if (!dtypes_ok(dtype, residual_dtype) || (dresidual && dtype == residual_dtype)) return VMSCAN_ERR_UNSUPPORTED;
  const void* ptrs[] = {dy, r, weight, rstd, dresidual_out, dx, dresidual, dweight, workspace};
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return VMSCAN_ERR_ALIGN;
  if (!workspace || workspace_bytes < vmscan_rmsnorm_bwd_workspace_bytes(rows, dim)) return VMSCAN_ERR_WORKSPACE;
  const unsigned blocks = blocks_for(rows, dim, kBwdBlocks);
  float* part = static_cast<float*>(workspace);
  const NormBwdArgs a{dy, r, dresidual_out, weight, rstd, dx, dresidual, part, rows, r_stride, static_cast<int>(dim)};
  if (dtype == VMSCAN_F32)
    launch_bwd<float, float>(a, blocks, stream);
  else if (residual_dtype == VMSCAN_F32)
    launch_bwd<uint16_t, float>(a, blocks, stream);
  else
    launch_bwd<uint16_t, uint16_t>(a, blocks, stream);
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3(static_cast<unsigned>((dim + 31) / 32)), dim3(1024), 0, stream, part,
                     dweight, static_cast<int>(blocks), static_cast<int>(dim));
  return launched();
}

}  // extern "C"
