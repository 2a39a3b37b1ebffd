// Group norm with an optional SiLU on channels-last tokens: forward and gradient.  What is computed is stated in
// include/vmscan.h.
//
// A workgroup takes a run of one batch row's tokens, whole rows of channels: a thread owns 8 neighbouring channels
// (one 16-byte access in bfloat16) and steps over the tokens, so all accesses are dense whatever the groups' width.
// Forward: one launch leaves each run's mean and sum of squared deviations per group, the next joins a row's runs
// and normalises.  The gradient needs two sums per group and per channel of what it then reads again.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

constexpr int kMaxDim = 4096;     // 512 threads of 8 channels
constexpr int kMaxSplits = 64;    // runs of a batch row
constexpr int kGroupLanes = 16;   // 8-bit copies: lanes whose channels share a scale

struct GnArgs {
  const void *x, *dy;
  const uint8_t* codes;        // the gradient's x in 8 bits
  const float* codes_scale;
  const float *w, *b;
  const int32_t* lengths;
  void* y;
  uint8_t* keep;               // the forward's x in 8 bits
  float* keep_scale;
  float *mean, *rstd;          // [batch, groups]
  float* part;                 // per batch row and run: groups' pairs
  float* chan;                 // gradient: per batch row and run, channels' two sums
  float *dw, *db;
  int64_t x_batch, x_token, dy_batch, dy_token;
  int64_t batch, seqlen;
  int dim, groups, width;      // width: channels of a group
  int lanes, rows;             // threads per row of channels, rows of a step
  int splits, run;             // runs of a batch row, tokens of a run
  float eps;
  int act;
};

__device__ __forceinline__ int64_t tokens_of(const GnArgs& a, int64_t b) {
  if (!a.lengths) return a.seqlen;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : n > a.seqlen ? a.seqlen : n;
}

// What a thread does: its channels and its row of a step.
struct Lane {
  int c, n, row;  // first channel, how many of 8 exist (<= 0: none), row of the step
  __device__ __forceinline__ explicit Lane(const GnArgs& a) {
    row = threadIdx.x / a.lanes;
    c = (threadIdx.x - row * a.lanes) * 8;
    n = row < a.rows ? a.dim - c : 0;
  }
};

__device__ __forceinline__ float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504f));
}

// Sums of two values per (row of a step, channel), left in LDS as [rows][dim], to sums per group: TPG neighbouring
// lanes share a group, in a fixed order.  f gets the group and the sums, in one lane each.
template <typename LOAD, typename F>
__device__ __forceinline__ void over_groups(const GnArgs& a, LOAD&& load, F&& f) {
  int tpg = 1;
  while (tpg < 64 && tpg < a.width && 2 * tpg * a.groups <= static_cast<int>(blockDim.x)) tpg *= 2;
  const int per = blockDim.x / tpg, sub = threadIdx.x % tpg;
  for (int g0 = 0; g0 < a.groups; g0 += per) {
    const int g = g0 + threadIdx.x / tpg;
    float s = 0.0f, q = 0.0f;
    if (g < a.groups)
      for (int r = 0; r < a.rows; ++r)
        for (int c = sub; c < a.width; c += tpg) load(g, r, g * a.width + c, s, q);
    for (int m = 1; m < tpg; m *= 2) {
      s += __shfl_xor(s, m);
      q += __shfl_xor(q, m);
    }
    if (g < a.groups && sub == 0) f(g, s, q);
  }
}

// Tokens that a row of the step saw of a run of `n`.
__device__ __forceinline__ int seen(int n, int row, int rows) { return n > row ? (n - row + rows - 1) / rows : 0; }

// Mean and sum of squared deviations of each group over a run.  A thread's sums are of differences to its first
// token, so that a large mean costs nothing; sums of different threads are joined by their means (each term's
// deviation is taken from the joint mean, nothing is subtracted from a sum of squares).
template <typename T>
__global__ __launch_bounds__(512) void groupnorm_stats_kernel(GnArgs a) {
  extern __shared__ float lds[];  // [2][rows][dim] and the groups' means
  const int64_t b = blockIdx.y;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.run, all = tokens_of(a, b);
  const int n = static_cast<int>(all - first < a.run ? (all > first ? all - first : 0) : a.run);
  const Lane l(a);
  const int dim = a.dim, rows = a.rows;
  float *lm = lds, *lq = lds + rows * dim, *gm = lq + rows * dim;
  float k0[8], s[8], q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = q[k] = k0[k] = 0.0f;
  const T* p = static_cast<const T*>(a.x) + b * a.x_batch + first * a.x_token + l.c;
  if (l.n > 0 && l.row < n) {
    load_upto8(p + l.row * a.x_token, l.n, k0);
#pragma unroll 4
    for (int t = l.row + rows; t < n; t += rows) {
      float v[8];
      load_upto8(p + t * a.x_token, l.n, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = v[k] - k0[k];
        s[k] += d;
        q[k] = __builtin_fmaf(d, d, q[k]);
      }
    }
  }
  if (l.row < rows) {
    const int m = seen(n, l.row, rows);
    const float inv = m ? 1.0f / static_cast<float>(m) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < l.n) {
        const float d = s[k] * inv;
        lm[l.row * dim + l.c + k] = k0[k] + d;
        const float m2 = __builtin_fmaf(-s[k], d, q[k]);
        lq[l.row * dim + l.c + k] = m2 < 0.0f ? 0.0f : m2;  // a NaN stays
      }
  }
  __syncthreads();
  const float inv = n ? 1.0f / (static_cast<float>(n) * a.width) : 0.0f;
  over_groups(
      a, [&](int, int r, int c, float& t, float&) { t += seen(n, r, rows) * lm[r * dim + c]; },
      [&](int g, float t, float) { gm[g] = t * inv; });
  __syncthreads();
  over_groups(
      a,
      [&](int g, int r, int c, float& t, float&) {
        const float d = lm[r * dim + c] - gm[g];
        const int m = seen(n, r, rows);
        if (m) t += __builtin_fmaf(m * d, d, lq[r * dim + c]);
      },
      [&](int g, float t, float) {
        float* out = a.part + ((b * a.splits + blockIdx.x) * a.groups + g) * 2;
        out[0] = gm[g], out[1] = t;
      });
}

// The groups' mean and reciprocal deviation of a batch row from its runs, into LDS.
__device__ __forceinline__ void join_runs(const GnArgs& a, int64_t b, int64_t all, float* mean, float* rstd) {
  for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
    const float* p = a.part + (b * a.splits * a.groups + g) * 2;
    float m = 0.0f, q = 0.0f;
    const float inv = all ? 1.0f / static_cast<float>(all) : 0.0f;
    for (int s = 0; s < a.splits; ++s) {
      const int64_t left = all - static_cast<int64_t>(s) * a.run;
      if (left <= 0) break;
      m += static_cast<float>(left < a.run ? left : a.run) * inv * p[static_cast<int64_t>(s) * a.groups * 2];
    }
    for (int s = 0; s < a.splits; ++s) {
      const int64_t left = all - static_cast<int64_t>(s) * a.run;
      if (left <= 0) break;
      const float d = p[static_cast<int64_t>(s) * a.groups * 2] - m;
      q += __builtin_fmaf(static_cast<float>(left < a.run ? left : a.run) * a.width * d, d,
                          p[static_cast<int64_t>(s) * a.groups * 2 + 1]);
    }
    mean[g] = m;
    rstd[g] = 1.0f / __builtin_sqrtf(__builtin_fmaf(q, inv / a.width, a.eps));
  }
}

template <typename T, bool KEEP>
__global__ __launch_bounds__(512) void groupnorm_apply_kernel(GnArgs a) {
  extern __shared__ float lds[];  // the groups' means and deviations
  const int64_t b = blockIdx.y, all = tokens_of(a, b);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.run;
  const int n = static_cast<int>(a.seqlen - first < a.run ? a.seqlen - first : a.run);  // tokens written
  const int live = static_cast<int>(all - first < 0 ? 0 : all - first < n ? all - first : n);
  const Lane l(a);
  join_runs(a, b, all, lds, lds + a.groups);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
      a.mean[b * a.groups + g] = lds[g];
      a.rstd[b * a.groups + g] = lds[a.groups + g];
    }
  if (l.row >= a.rows) return;
  float mean[8], scale[8], bias[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const bool has = k < l.n;
    const int g = has ? (l.c + k) / a.width : 0;
    mean[k] = lds[g];
    scale[k] = has ? lds[a.groups + g] * a.w[l.c + k] : 0.0f;
    bias[k] = has ? a.b[l.c + k] : 0.0f;
  }
  const T* p = static_cast<const T*>(a.x) + b * a.x_batch + first * a.x_token + l.c;
  T* out = static_cast<T*>(a.y) + (b * a.seqlen + first) * a.dim + l.c;
#pragma unroll 2
  for (int t = l.row; t < n; t += a.rows) {
    float v[8], u[8];
    load_upto8(p + t * a.x_token, t < live ? l.n : 0, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      u[k] = __builtin_fmaf(v[k] - mean[k], scale[k], bias[k]);
      if (a.act) u[k] *= sigmoid(u[k]);
      if (t >= live) u[k] = 0.0f;
    }
    store_upto8(out + static_cast<int64_t>(t) * a.dim, l.n, u);
    if constexpr (KEEP) {
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = Max::of(top, __builtin_fabsf(v[k]));
      top = over_lanes<Max, kGroupLanes>(top);
      const float sc = scale_of(top), inv = 1.0f / sc;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= inv;
      const int64_t at = b * a.seqlen + first + t;
      store_fp8(a.keep + at * a.dim + l.c, l.n, v);
      if (l.n > 0 && l.c % 128 == 0) a.keep_scale[at * ((a.dim + 127) / 128) + l.c / 128] = sc;
    }
  }
}

// The gradient's x, activations or 8-bit codes.
template <typename T, bool CODES>
__device__ __forceinline__ void load_x(const GnArgs& a, int64_t b, int64_t t, const Lane& l, float (&v)[8]) {
  if constexpr (CODES) {
    const int64_t at = b * a.seqlen + t;
    load_fp8(a.codes + at * a.dim + l.c, l.n, v);
    const float s = l.n > 0 ? a.codes_scale[at * ((a.dim + 127) / 128) + l.c / 128] : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= s;
  } else {
    load_upto8(static_cast<const T*>(a.x) + b * a.x_batch + t * a.x_token + l.c, l.n, v);
  }
}

// x -> its normal form, dy -> the gradient before the activation.
struct Grad {
  float mean[8], rstd[8], w[8], b[8];
  __device__ __forceinline__ Grad(const GnArgs& a, int64_t row, const Lane& l) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool has = k < l.n;
      const int64_t g = row * a.groups + (has ? (l.c + k) / a.width : 0);
      mean[k] = a.mean[g], rstd[k] = a.rstd[g];
      w[k] = has ? a.w[l.c + k] : 0.0f;
      b[k] = has ? a.b[l.c + k] : 0.0f;
    }
  }
  __device__ __forceinline__ void of(int act, float (&x)[8], float (&dy)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = (x[k] - mean[k]) * rstd[k];
      if (act) {
        const float u = __builtin_fmaf(x[k], w[k], b[k]), s = sigmoid(u);
        dy[k] *= s * __builtin_fmaf(u, 1.0f - s, 1.0f);
      }
    }
  }
};

template <typename T, bool CODES>
__global__ __launch_bounds__(512) void groupnorm_sums_kernel(GnArgs a) {
  extern __shared__ float lds[];  // [2][rows][dim]
  const int64_t b = blockIdx.y;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.run, all = tokens_of(a, b);
  const int n = static_cast<int>(all - first < a.run ? (all > first ? all - first : 0) : a.run);
  const Lane l(a);
  const int dim = a.dim, rows = a.rows;
  float *l1 = lds, *l2 = lds + rows * dim;
  if (l.row < rows) {
    const Grad grad(a, b, l);
    float s1[8], s2[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s1[k] = s2[k] = 0.0f;
    const T* p = static_cast<const T*>(a.dy) + b * a.dy_batch + first * a.dy_token + l.c;
#pragma unroll 2
    for (int t = l.row; t < n; t += rows) {
      float x[8], dy[8];
      load_x<T, CODES>(a, b, first + t, l, x);
      load_upto8(p + t * a.dy_token, l.n, dy);
      grad.of(a.act, x, dy);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s1[k] += dy[k];
        s2[k] = __builtin_fmaf(dy[k], x[k], s2[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < l.n) l1[l.row * dim + l.c + k] = s1[k], l2[l.row * dim + l.c + k] = s2[k];
  }
  __syncthreads();
  const int64_t at = b * a.splits + blockIdx.x;
  for (int c = threadIdx.x; c < dim; c += blockDim.x) {
    float t1 = 0.0f, t2 = 0.0f;
    for (int r = 0; r < rows; ++r) t1 += l1[r * dim + c], t2 += l2[r * dim + c];
    a.chan[at * 2 * dim + c] = t1;
    a.chan[(at * 2 + 1) * dim + c] = t2;
  }
  over_groups(
      a, [&](int, int r, int c, float& t1, float& t2) { t1 += a.w[c] * l1[r * dim + c], t2 += a.w[c] * l2[r * dim + c]; },
      [&](int g, float t1, float t2) {
        float* out = a.part + (at * a.groups + g) * 2;
        out[0] = t1, out[1] = t2;
      });
}

// dw and db: sums over the batch rows' runs.  32 columns of one of the two, 32 shares of the runs, joined in LDS.
__device__ __forceinline__ void sum_runs(const GnArgs& a, int block, float* lds) {
  const int per = (a.dim + 31) / 32, which = block / per, c = (block % per) * 32 + (threadIdx.x & 31);
  const int share = threadIdx.x >> 5, shares = blockDim.x >> 5;
  const int64_t runs = a.batch * a.splits;
  float t = 0.0f;
  if (c < a.dim)
#pragma unroll 4
    for (int64_t i = share; i < runs; i += shares) t += a.chan[(i * 2 + which) * a.dim + c];
  lds[threadIdx.x] = t;
  __syncthreads();
  if (share == 0 && c < a.dim) {
    for (int i = 1; i < shares; ++i) t += lds[i * 32 + (threadIdx.x & 31)];
    (which ? a.dw : a.db)[c] = t;
  }
}

// dx; the workgroups past the rows' runs sum dw and db.
template <typename T, bool CODES>
__global__ __launch_bounds__(512) void groupnorm_dx_kernel(GnArgs a) {
  extern __shared__ float lds[];  // the groups' two means, or sum_runs' shares
  const int64_t runs = a.batch * a.splits;
  if (blockIdx.x >= runs) {
    sum_runs(a, static_cast<int>(blockIdx.x - runs), lds);
    return;
  }
  const int64_t b = blockIdx.x / a.splits, all = tokens_of(a, b);
  const int64_t first = static_cast<int64_t>(blockIdx.x - b * a.splits) * a.run;
  const int n = static_cast<int>(a.seqlen - first < a.run ? a.seqlen - first : a.run);
  const int live = static_cast<int>(all - first < 0 ? 0 : all - first < n ? all - first : n);
  const Lane l(a);
  const float inv = all ? 1.0f / (static_cast<float>(all) * a.width) : 0.0f;
  for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
    const float* p = a.part + (b * a.splits * a.groups + g) * 2;
    float t1 = 0.0f, t2 = 0.0f;
    for (int s = 0; s < a.splits; ++s) t1 += p[static_cast<int64_t>(s) * a.groups * 2], t2 += p[static_cast<int64_t>(s) * a.groups * 2 + 1];
    lds[g] = t1 * inv, lds[a.groups + g] = t2 * inv;
  }
  __syncthreads();
  if (l.row >= a.rows) return;
  const Grad grad(a, b, l);
  float m1[8], m2[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int g = k < l.n ? (l.c + k) / a.width : 0;
    m1[k] = lds[g], m2[k] = lds[a.groups + g];
  }
  const T* p = static_cast<const T*>(a.dy) + b * a.dy_batch + first * a.dy_token + l.c;
  T* out = static_cast<T*>(a.y) + (b * a.seqlen + first) * a.dim + l.c;
#pragma unroll 2
  for (int t = l.row; t < n; t += a.rows) {
    float x[8], dy[8];
    if (t < live) {
      load_x<T, CODES>(a, b, first + t, l, x);
      load_upto8(p + t * a.dy_token, l.n, dy);
      grad.of(a.act, x, dy);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dy[k] = grad.rstd[k] * (__builtin_fmaf(dy[k], grad.w[k], -m1[k]) - x[k] * m2[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) dy[k] = 0.0f;
    }
    store_upto8(out + static_cast<int64_t>(t) * a.dim, l.n, dy);
  }
}

// Threads of a workgroup and rows of a step: of 256 to 512 threads the count that leaves
// the fewest idle.
int threads_for(GnArgs& a, bool keep) {
  a.lanes = (a.dim + 7) / 8;
  if (keep) a.lanes = (a.lanes + kGroupLanes - 1) / kGroupLanes * kGroupLanes;
  int best = 0;
  float share = 0.0f;
  for (int nt = 256; nt <= 512; nt += 64) {
    const int rows = nt / a.lanes;
    const float f = static_cast<float>(rows * a.lanes) / nt;
    if (rows && f > share + 1e-3f) best = nt, share = f;
  }
  a.rows = best / a.lanes;
  return best;
}

// Runs: enough workgroups for the chip, each of 16 steps at least.
void split(GnArgs& a) {
  const int64_t steps = (a.seqlen + a.rows - 1) / a.rows;
  int64_t splits = (1024 + a.batch - 1) / a.batch;
  if (splits > (steps + 15) / 16) splits = (steps + 15) / 16;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1) splits = 1;
  a.run = static_cast<int>((steps + splits - 1) / splits * a.rows);
  a.splits = static_cast<int>((a.seqlen + a.run - 1) / a.run);
}

bool shape_ok(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups) {
  return batch >= 1 && seqlen >= 1 && dim >= 1 && dim <= kMaxDim && groups >= 1 && groups <= dim && dim % groups == 0 &&
         batch < 65536 && seqlen < (int64_t{1} << 30);
}

bool strides_ok(const int64_t* s, int64_t dim) {
  return s[0] >= 0 && s[1] >= 0 && s[0] <= (int64_t{1} << 40) && s[1] < (int64_t{1} << 32) && dim >= 1;
}

GnArgs sizes(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups) {
  GnArgs a{};
  a.batch = batch, a.seqlen = seqlen, a.dim = static_cast<int>(dim), a.groups = static_cast<int>(groups);
  a.width = a.dim / a.groups;
  return a;
}

size_t stats_bytes(const GnArgs& a) { return static_cast<size_t>(a.batch) * a.splits * a.groups * 2 * sizeof(float); }
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

template <typename T>
void launch_fwd(GnArgs& a, int threads, hipStream_t stream) {
  const dim3 grid(a.splits, static_cast<unsigned>(a.batch)), block(threads);
  const size_t lds = (2 * static_cast<size_t>(a.rows) * a.dim + a.groups) * sizeof(float);
  hipLaunchKernelGGL((groupnorm_stats_kernel<T>), grid, block, lds, stream, a);
  if (a.keep)
    hipLaunchKernelGGL((groupnorm_apply_kernel<T, true>), grid, block, 2 * a.groups * sizeof(float), stream, a);
  else
    hipLaunchKernelGGL((groupnorm_apply_kernel<T, false>), grid, block, 2 * a.groups * sizeof(float), stream, a);
}

template <typename T, bool CODES>
void launch_bwd(GnArgs& a, int threads, hipStream_t stream) {
  const size_t lds = 2 * static_cast<size_t>(a.rows) * a.dim * sizeof(float);
  hipLaunchKernelGGL((groupnorm_sums_kernel<T, CODES>), dim3(a.splits, static_cast<unsigned>(a.batch)), dim3(threads), lds,
                     stream, a);
  const size_t groups = 2 * static_cast<size_t>(a.groups) * sizeof(float), shares = threads * sizeof(float);
  const int64_t sums = 2 * ((a.dim + 31) / 32);
  hipLaunchKernelGGL((groupnorm_dx_kernel<T, CODES>), dim3(static_cast<unsigned>(a.batch * a.splits + sums)), dim3(threads),
                     groups > shares ? groups : shares, stream, a);
}

}  // namespace

extern "C" {

size_t vmscan_groupnorm_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int keep) {
  if (!shape_ok(batch, seqlen, dim, groups)) return 0;
  GnArgs a = sizes(batch, seqlen, dim, groups);
  threads_for(a, keep != 0);
  split(a);
  return stats_bytes(a);
}

vmscan_status vmscan_groupnorm_fwd(const void* x, const int64_t* x_strides, const float* weight, const float* bias,
                                   const int32_t* lengths, void* y, float* mean, float* rstd, void* keep_codes,
                                   float* keep_scale, int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, float eps,
                                   int act, vmscan_dtype dtype, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  if (!x || !x_strides || !weight || !bias || !y || !mean || !rstd) return VMSCAN_ERR_NULL;
  if ((keep_codes == nullptr) != (keep_scale == nullptr)) return VMSCAN_ERR_NULL;
  if (!shape_ok(batch, seqlen, dim, groups) || !strides_ok(x_strides, dim) || !(eps >= 0.0f)) return VMSCAN_ERR_SHAPE;
  if ((dtype != VMSCAN_F32 && dtype != VMSCAN_BF16) || (act != 0 && act != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  if (!aligned_to(x, e) || !aligned_to(y, 16) || !aligned_to(workspace, 16)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(lengths),
                        static_cast<const void*>(mean), static_cast<const void*>(rstd), static_cast<const void*>(keep_scale)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  GnArgs a = sizes(batch, seqlen, dim, groups);
  const int threads = threads_for(a, keep_codes != nullptr);
  split(a);
  if (!workspace || workspace_bytes < stats_bytes(a)) return VMSCAN_ERR_WORKSPACE;
  a.x = x, a.w = weight, a.b = bias, a.lengths = lengths, a.y = y, a.mean = mean, a.rstd = rstd;
  a.keep = static_cast<uint8_t*>(keep_codes), a.keep_scale = keep_scale, a.part = static_cast<float*>(workspace);
  a.x_batch = x_strides[0], a.x_token = x_strides[1], a.eps = eps, a.act = act;
  if (dtype == VMSCAN_F32)
    launch_fwd<float>(a, threads, stream);
  else
    launch_fwd<uint16_t>(a, threads, stream);
  return launched();
}

size_t vmscan_groupnorm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups) {
  if (!shape_ok(batch, seqlen, dim, groups)) return 0;
  GnArgs a = sizes(batch, seqlen, dim, groups);
  threads_for(a, false);
  split(a);
  return round16(stats_bytes(a)) + static_cast<size_t>(a.batch) * a.splits * 2 * a.dim * sizeof(float);
}

vmscan_status vmscan_groupnorm_bwd(const void* dy, const int64_t* dy_strides, const void* x, const int64_t* x_strides,
                                   const void* codes, const float* codes_scale, const float* weight, const float* bias,
                                   const float* mean, const float* rstd, const int32_t* lengths, void* dx, float* dweight,
                                   float* dbias, int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int act,
                                   vmscan_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!dy || !dy_strides || !weight || !bias || !mean || !rstd || !dx || !dweight || !dbias) return VMSCAN_ERR_NULL;
  if ((x == nullptr) == (codes == nullptr) || (x && !x_strides) || (codes == nullptr) != (codes_scale == nullptr))
    return VMSCAN_ERR_NULL;
  if (!shape_ok(batch, seqlen, dim, groups) || !strides_ok(dy_strides, dim) || (x && !strides_ok(x_strides, dim)))
    return VMSCAN_ERR_SHAPE;
  if ((dtype != VMSCAN_F32 && dtype != VMSCAN_BF16) || (act != 0 && act != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, 16) || !aligned_to(workspace, 16)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(lengths),
                        static_cast<const void*>(mean), static_cast<const void*>(rstd),
                        static_cast<const void*>(codes_scale), static_cast<const void*>(dweight),
                        static_cast<const void*>(dbias)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  if (!workspace || workspace_bytes < vmscan_groupnorm_bwd_workspace_bytes(batch, seqlen, dim, groups))
    return VMSCAN_ERR_WORKSPACE;
  GnArgs a = sizes(batch, seqlen, dim, groups);
  const int threads = threads_for(a, false);
  split(a);
  a.x = x, a.dy = dy, a.codes = static_cast<const uint8_t*>(codes), a.codes_scale = codes_scale;
  a.w = weight, a.b = bias, a.lengths = lengths, a.y = dx, a.dw = dweight, a.db = dbias, a.act = act;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.part = static_cast<float*>(workspace);
  a.chan = reinterpret_cast<float*>(static_cast<char*>(workspace) + round16(stats_bytes(a)));
  a.dy_batch = dy_strides[0], a.dy_token = dy_strides[1];
  if (x) a.x_batch = x_strides[0], a.x_token = x_strides[1];
  if (dtype == VMSCAN_F32)
    codes ? launch_bwd<float, true>(a, threads, stream) : launch_bwd<float, false>(a, threads, stream);
  else
    codes ? launch_bwd<uint16_t, true>(a, threads, stream) : launch_bwd<uint16_t, false>(a, threads, stream);
  return launched();
}

}  // extern "C"
