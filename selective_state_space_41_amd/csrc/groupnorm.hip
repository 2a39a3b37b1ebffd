// Group norm with an optional SiLU on channels-last tokens: forward and gradient.  What is computed is stated in
// include/vmscan.h.
//
// A thread owns 8 neighbouring channels (one 16-byte access in bfloat16) and steps over the tokens.
// Where a batch row's slab of whole groups fits a workgroup's registers it is read once: the workgroup keeps it from
// the statistics to the output.  Larger rows are cut into runs of tokens, whole rows of channels, so that accesses
// are dense whatever the groups' width: one launch leaves each run's mean and sum of squared deviations per group (the
// gradient: two sums per group and channel), the next joins a row's runs and reads the tokens again (from memory or the
// last-level cache: the counters do not tell).
//
// Measured (whole calls): 32 x 3136 x 512 bfloat16 kept in 8 bits 75 us (first launch 25, second 50) for 257 MB, 51 us at
// a copy's rate, or 360 MB with the second read; its gradient from 8 bits 79 (38 and 47, the second's sums from the cache
// in part).  One float32 image 197 x 384 in one launch of 8 us, under a call of 11.  A single pass over large rows too,
// runs held in registers and each waiting for the others of its row, took 79 to 100 us: loads, wait and stores of a
// workgroup come one after the other, and two workgroups a CU do not cover that.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

constexpr int kMaxDim = 4096;     // 512 threads of 8 channels
constexpr int kMaxSplits = 128;   // runs of a batch row
constexpr int kGroupLanes = 16;   // 8-bit copies: lanes whose channels share a scale
// Tokens that a thread loads at once: 4, and 2 in the gradient, whose registers leave room for more waves then (32 x 3136 x
// 512 from 8 bits 82 us instead of 89, with 1024 workgroups; the forward takes the same time with either).
constexpr int kAhead = 4, kAheadBack = 2;
constexpr int kRecentre = 8;  // tokens of a thread after which the statistics' sums move to the mean so far
static_assert(kRecentre % kAhead == 0, "whole turns");

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
  int scales;                  // scales of a token of the 8-bit form
  int slab, slabs;             // channels of a workgroup and how many such slabs; runs: all, 1
  int lanes, rows;             // threads per row of channels, rows of a step
  int splits, run;             // runs of a batch row, tokens of a run
  float eps;
  int act;
};

__device__ __forceinline__ int tokens_of(const GnArgs& a, int64_t b) {
  const int all = static_cast<int>(a.seqlen);
  if (!a.lengths) return all;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > all ? all : n;
}

// What a thread does: its row of a step, its channels from c on, of which n of 8 exist in the slab (<= 0: none).
struct Lane {
  int row, c, n;
  __device__ __forceinline__ Lane(const GnArgs& a, int slab) {
    row = threadIdx.x / a.lanes;
    const int at = (threadIdx.x - row * a.lanes) * 8;
    c = slab * a.slab + at;
    const int end = (slab + 1) * a.slab < a.dim ? (slab + 1) * a.slab : a.dim;
    n = row < a.rows ? end - c : 0;
  }
};

// Without the tail of u * log2(e), for float32 too: u is a rounded result here, off by up to 2^-24 of itself (and of its
// terms), which already costs e^-u as much.
__device__ __forceinline__ float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504f));
}

// Eight channels as loaded.  W8: the groups' width is a multiple of 8, so a thread's channels exist all or none and
// share a group; bfloat16 ones then stay packed until they are used.
// ONCE: there are too many tokens for the last-level cache to hold them beside the outputs; their loads leave it alone.
template <typename V, bool ONCE, typename T>
__device__ __forceinline__ V load_as(const T* p) {
  if constexpr (ONCE) return load_once<V>(p);
  V v;
  __builtin_memcpy(&v, p, sizeof(v));
  return v;
}
template <typename T, bool W8>
struct Vec {
  float v[8];
  template <bool ONCE = false>
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (W8) {  // float32
      const f32x4 a = load_as<f32x4, ONCE>(p), b = load_as<f32x4, ONCE>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      load_upto8(p, n, v);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
  }
  __device__ __forceinline__ void get(float (&to)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) to[k] = v[k];
  }
  // The largest magnitude as an unsigned number, whose order is the same and in which a NaN is the largest.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t m = __float_as_uint(v[k]) & 0x7fffffffu;
      t = m > t ? m : t;
    }
    return t;
  }
};
template <>
struct Vec<uint16_t, true> {
  uint32_t w[4];
  template <bool ONCE = false>
  __device__ __forceinline__ void load(const uint16_t* p, int) {
    const u32x4 r = load_as<u32x4, ONCE>(p);
    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ void get(float (&to)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) to[2 * k] = __uint_as_float(w[k] << 16), to[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  __device__ __forceinline__ uint32_t top() const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 t = __builtin_bit_cast(u16x2, w[0] & 0x7fff7fffu);
#pragma unroll
    for (int k = 1; k < 4; ++k) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, w[k] & 0x7fff7fffu));
    return static_cast<uint32_t>(t.x > t.y ? t.x : t.y) << 16;
  }
};
// Eight channels in 8 bits with their scale.
struct Codes {
  uint32_t w[2];
  float scale;
  template <bool W8, bool ONCE>
  __device__ __forceinline__ void load(const uint8_t* p, int n, const float* s) {
    w[0] = w[1] = 0;
    if (W8 || n >= 8) {
      const u32x2 r = load_as<u32x2, ONCE>(p);
      w[0] = r.x, w[1] = r.y;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) w[k / 4] |= static_cast<uint32_t>(p[k]) << (8 * (k % 4));
    }
    scale = n > 0 ? *s : 0.0f;
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = 0, scale = 0.0f; }
  // the codes; `scale` is still to be multiplied
  __device__ __forceinline__ void get(float (&to)[8]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
      to[4 * k] = lo[0], to[4 * k + 1] = lo[1], to[4 * k + 2] = hi[0], to[4 * k + 3] = hi[1];
    }
  }
};

template <typename T, bool W8>
__device__ __forceinline__ void store_vec(T* p, int n, const float (&v)[8]) {
  if constexpr (W8 && sizeof(T) == 2) {  // nearest even, two at once
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    const bf16x8 w = __builtin_convertvector((f32x8{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}), bf16x8);
    __builtin_memcpy(p, &w, 16);
  } else if constexpr (W8) {
    store8(p, v);
  } else {
    store_upto8(p, n, v);
  }
}

// The places of a thread's tokens, one after another: a row of the step apart.
template <typename T>
struct Steps {
  T* p;
  int64_t step;
  // base: of the first row; stride: from token to token; the thread starts at token `row`
  __device__ __forceinline__ Steps(T* base, int64_t stride, const GnArgs& a, int row) : p(base + row * stride), step(a.rows * stride) {}
  __device__ __forceinline__ T* next() {
    T* q = p;
    p += step;
    return q;
  }
};

// A thread's tokens row, row + rows, ... below n: `load(slot)` for AHEAD of them one after another, then `use(slot)` in
// the same order and, where all AHEAD were there, `turn(tokens so far)`.
struct NoTurn {
  __device__ __forceinline__ void operator()(int) const {}
};
template <int AHEAD, typename LOAD, typename USE, typename TURN = NoTurn>
__device__ __forceinline__ void over_tokens(int row, int rows, int n, LOAD&& load, USE&& use, TURN&& turn = {}) {
  const int turns = n / (AHEAD * rows);  // the same number for all
  for (int i = 0; i < turns; ++i) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) load(k);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) use(k);
    turn((i + 1) * AHEAD);
  }
  const int t = row + turns * AHEAD * rows;
  if (t < n) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (t + k * rows < n) load(k);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (t + k * rows < n) use(k);
  }
}

// Sums of `terms` values of each of `groups` groups, by up to 64 neighbouring lanes each, in a fixed order: load adds a
// term to two sums, f gets the group and the sums in one lane.
template <typename LOAD, typename F>
__device__ __forceinline__ void over_groups(int groups, int terms, LOAD&& load, F&& f) {
  int tpg = 1;
  while (tpg < 64 && tpg < terms && 2 * tpg * groups <= static_cast<int>(blockDim.x)) tpg *= 2;
  const int per = blockDim.x / tpg, sub = threadIdx.x % tpg;
  for (int g0 = 0; g0 < groups; g0 += per) {
    const int g = g0 + threadIdx.x / tpg;
    float s = 0.0f, q = 0.0f;
    if (g < groups) {
#pragma unroll 4
      for (int i = sub; i < terms; i += tpg) load(g, i, s, q);
    }
    for (int m = 1; m < tpg; m *= 2) {
      s += __shfl_xor(s, m);
      q += __shfl_xor(q, m);
    }
    if (g < groups && sub == 0) f(g, s, q);
  }
}

// Sums of each channel's `rows` values, in a fixed order: term gives one, done gets a channel's sum.  `scratch`: a float
// per thread.
template <typename TERM, typename DONE>
__device__ __forceinline__ void over_rows(int rows, int channels, float* scratch, TERM&& term, DONE&& done) {
  const int nt = blockDim.x;
  if (channels >= nt) {
    for (int c = threadIdx.x; c < channels; c += nt) {
      float t = 0.0f;
      for (int r = 0; r < rows; ++r) t += term(r, c);
      done(c, t);
    }
    return;
  }
  const int shares = nt / channels < rows ? nt / channels : rows, share = threadIdx.x / channels;
  const int c = threadIdx.x - share * channels;
  if (share < shares) {
    float t = 0.0f;
#pragma unroll 4
    for (int r = share; r < rows; r += shares) t += term(r, c);
    scratch[threadIdx.x] = t;
  }
  __syncthreads();
  if (share == 0) {
    float t = scratch[c];
    for (int i = 1; i < shares; ++i) t += scratch[i * channels + c];
    done(c, t);
  }
  __syncthreads();  // scratch may be written again
}

// Tokens that a row of the step saw of a run of `n`.
__device__ __forceinline__ int seen(int n, int row, int rows) { return n > row ? (n - row + rows - 1) / rows : 0; }

// Mean and sum of squared deviations of each group over a run.  A thread's sums are of differences to a centre, its first
// token at first; every eight tokens the centre moves to the mean so far, and the sums are moved with it exactly, by the
// distance between the two float32 centres.  So neither a large mean nor tokens far from the others, the first ones among
// them, are subtracted from a sum of squares that they dominate (a centre left at a first token 100 times the others cost
// the variance 4e-4 of itself over 784 tokens; moving it costs nothing, every four tokens 2 % of the call).  Sums of
// different threads are joined by their means in the same sense.
template <typename T, bool W8, bool ONCE>
__global__ __launch_bounds__(512) void groupnorm_stats_kernel(GnArgs a) {
  extern __shared__ float lds[];  // [2][rows][dim], the channels' and the groups' means, a float per thread
  const int64_t b = blockIdx.y;
  const int first = blockIdx.x * a.run, left = tokens_of(a, b) - first;
  const int n = left < a.run ? (left > 0 ? left : 0) : a.run;
  const Lane l(a, 0);
  const int dim = a.dim, rows = a.rows;
  float *lm = lds, *lq = lds + rows * dim, *cm = lq + rows * dim, *gm = cm + dim, *scratch = gm + a.groups;
  if (l.n > 0) {
    float k0[8], s[8], q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = q[k] = k0[k] = 0.0f;
    Steps<const T> p(static_cast<const T*>(a.x) + b * a.x_batch + first * a.x_token + l.c, a.x_token, a, l.row);
    Vec<T, W8> x[kAhead];
    if (l.row < n) x[0].load(p.p, l.n), x[0].get(k0);
    over_tokens<kAhead>(
        l.row, rows, n, [&](int k) { x[k].template load<ONCE>(p.next(), l.n); },
        [&](int k) {
          float v[8];
          x[k].get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = v[e] - k0[e];
            s[e] += d;
            q[e] = __builtin_fmaf(d, d, q[e]);
          }
        },
        [&](int m) {
          if (m % kRecentre) return;
          const float tokens = static_cast<float>(m), inv = __builtin_amdgcn_rcpf(tokens);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float k1 = __builtin_fmaf(s[e], inv, k0[e]), by = k1 - k0[e], t = __builtin_fmaf(-tokens, by, s[e]);
            q[e] = __builtin_fmaf(-by, s[e] + t, q[e]);
            s[e] = t, k0[e] = k1;
          }
        });
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
  // the channels' means and squares from their rows', then the groups' from the channels', which saw as many tokens each
  const float inv = n ? 1.0f / static_cast<float>(n) : 0.0f;
  over_rows(rows, dim, scratch, [&](int r, int c) { return seen(n, r, rows) * lm[r * dim + c]; },
            [&](int c, float t) { cm[c] = t * inv; });
  __syncthreads();
  over_rows(
      rows, dim, scratch,
      [&](int r, int c) {
        const float d = lm[r * dim + c] - cm[c];
        const int m = seen(n, r, rows);
        return m ? __builtin_fmaf(m * d, d, lq[r * dim + c]) : 0.0f;
      },
      [&](int c, float t) { lq[c] = t; });
  __syncthreads();
  over_groups(
      a.groups, a.width, [&](int g, int i, float& t, float&) { t += cm[g * a.width + i]; },
      [&](int g, float t, float) { gm[g] = t / a.width; });
  __syncthreads();
  over_groups(
      a.groups, a.width,
      [&](int g, int i, float& t, float&) {
        const float d = cm[g * a.width + i] - gm[g];
        t += __builtin_fmaf(n * d, d, lq[g * a.width + i]);
      },
      [&](int g, float t, float) {
        float* out = a.part + ((b * a.splits + blockIdx.x) * a.groups + g) * 2;
        out[0] = gm[g], out[1] = t;
      });
}

// The groups' mean and reciprocal deviation of a batch row from its runs, into LDS.
__device__ __forceinline__ void join_runs(const GnArgs& a, int64_t b, int all, float* mean, float* rstd) {
  const float inv = all ? 1.0f / static_cast<float>(all) : 0.0f;
  const float* p = a.part + b * a.splits * a.groups * 2;
  const auto tokens = [&](int s) {
    const int left = all - s * a.run;
    return static_cast<float>(left < 0 ? 0 : left < a.run ? left : a.run);
  };
  const auto at = [&](int g, int s) { return p + (static_cast<int64_t>(s) * a.groups + g) * 2; };
  over_groups(
      a.groups, a.splits, [&](int g, int s, float& t, float&) { t += tokens(s) * inv * at(g, s)[0]; },
      [&](int g, float t, float) { mean[g] = t; });
  __syncthreads();
  over_groups(
      a.groups, a.splits,
      [&](int g, int s, float& t, float&) {
        const float d = at(g, s)[0] - mean[g];
        t += __builtin_fmaf(tokens(s) * a.width * d, d, at(g, s)[1]);
      },
      [&](int g, float t, float) { rstd[g] = 1.0f / __builtin_sqrtf(__builtin_fmaf(t, inv / a.width, a.eps)); });
}

// A thread's channels' parameters.
template <bool W8>
struct Channels {
  float mean[W8 ? 1 : 8], scale[8], bias[8];  // scale: rstd * weight
  // mean, rstd: of the groups from `first` on
  __device__ __forceinline__ Channels(const GnArgs& a, const Lane& l, const float* means, const float* rstds, int first) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool has = W8 ? l.n > 0 : k < l.n;
      const int g = has ? (l.c + (W8 ? 0 : k)) / a.width - first : 0;
      if (!W8 || k == 0) mean[k] = means[g];
      scale[k] = has ? rstds[g] * a.w[l.c + k] : 0.0f;
      bias[k] = has ? a.b[l.c + k] : 0.0f;
    }
  }
  __device__ __forceinline__ float of(int k) const { return mean[W8 ? 0 : k]; }
};

// Where a thread's outputs go, token after token.
template <typename T, bool KEEP>
struct Outputs {
  Steps<T> y;
  Steps<uint8_t> keep;
  Steps<float> scale;
  // from token `at` of all the batch rows' on
  __device__ __forceinline__ Outputs(const GnArgs& a, const Lane& l, int64_t at, int row)
      : y(static_cast<T*>(a.y) + at * a.dim + l.c, a.dim, a, row),
        keep(a.keep + (KEEP ? at * a.dim + l.c : 0), a.dim, a, row),
        scale(a.keep_scale + (KEEP ? at * a.scales + l.c / 128 : 0), a.scales, a, row) {}
};

// x -> y, and the 8-bit copy; a token that is not live gives zeros.
template <typename T, bool W8, bool KEEP>
__device__ __forceinline__ void put_token(const GnArgs& a, const Lane& l, const Channels<W8>& ch, Outputs<T, KEEP>& out, bool live,
                                          const Vec<T, W8>& x) {
  float v[8], u[8];
  x.get(v);
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = __builtin_fmaf(v[k] - ch.of(k), ch.scale[k], ch.bias[k]);
  if (a.act) {
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] *= sigmoid(u[k]);
  }
  if (!live) {
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = 0.0f;
  }
  T* y = out.y.next();
  if (!KEEP || l.n > 0) store_vec<T, W8>(y, l.n, u);
  if constexpr (KEEP) {
    // the largest magnitude of 16 lanes
    const auto with = [](uint32_t m, float other) {
      const uint32_t o = __float_as_uint(other);
      return m > o ? m : o;
    };
    uint32_t top = x.top();
    top = with(top, dpp<0xb1>(__uint_as_float(top)));
    top = with(top, dpp<0x4e>(__uint_as_float(top)));
    top = with(top, dpp<0x141>(__uint_as_float(top)));
    top = with(top, dpp<0x140>(__uint_as_float(top)));
    // as scale_of and its reciprocal, by products (one unit in the last place)
    const float big = __uint_as_float(top), s = big * (1.0f / kFp8Max);
    const float sc = big == 0.0f ? 1.0f : s < kMinScale ? kMinScale : s, inv = __builtin_amdgcn_rcpf(sc);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= inv;
    uint8_t* codes = out.keep.next();
    float* scale = out.scale.next();
    if (l.n > 0) {
      store_fp8(codes, W8 ? 8 : l.n, v);
      if (l.c % 128 == 0) *scale = sc;
    }
  }
}

template <typename T, bool W8, bool KEEP, bool ONCE>
__global__ __launch_bounds__(512) void groupnorm_apply_kernel(GnArgs a) {
  extern __shared__ float lds[];  // the groups' means and deviations
  const int64_t b = blockIdx.y;
  const int first = blockIdx.x * a.run, all = tokens_of(a, b), rest = static_cast<int>(a.seqlen) - first;
  const int n = rest < a.run ? rest : a.run;  // tokens written
  const int live = all - first < 0 ? 0 : all - first < n ? all - first : n;
  const Lane l(a, 0);
  join_runs(a, b, all, lds, lds + a.groups);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
      a.mean[b * a.groups + g] = lds[g];
      a.rstd[b * a.groups + g] = lds[a.groups + g];
    }
  if (l.row >= a.rows || (!KEEP && l.n <= 0)) return;
  const Channels<W8> ch(a, l, lds, lds + a.groups, 0);
  Steps<const T> p(static_cast<const T*>(a.x) + b * a.x_batch + first * a.x_token + l.c, a.x_token, a, l.row);
  Outputs<T, KEEP> out(a, l, b * a.seqlen + first, l.row);
  Vec<T, W8> x[kAhead];
  over_tokens<kAhead>(
      l.row, a.rows, live,
      [&](int k) {
        const T* q = p.next();
        if (!KEEP || l.n > 0)
          x[k].template load<ONCE>(q, l.n);
        else
          x[k].clear();
      },
      [&](int k) { put_token<T, W8, KEEP>(a, l, ch, out, true, x[k]); });
  x[0].clear();
  for (int t = l.row + seen(live, l.row, a.rows) * a.rows; t < n; t += a.rows) put_token<T, W8, KEEP>(a, l, ch, out, false, x[0]);
}

// The slab of a batch row in a workgroup's registers: NI tokens of every thread, a.rows * NI >= seqlen.  128 x 197 x 384
// bfloat16: 14 us a call, 39 MB.
template <typename T, bool W8, int NI, bool KEEP>
__global__ __launch_bounds__(1024) void groupnorm_slab_kernel(GnArgs a) {
  extern __shared__ float lds[];  // [rows][slab's entries], the groups' means and deviations
  const int64_t b = blockIdx.x / a.slabs;
  const int slab = static_cast<int>(blockIdx.x - b * a.slabs), n = tokens_of(a, b);
  const Lane l(a, slab);
  const int here = a.dim - slab * a.slab < a.slab ? a.dim - slab * a.slab : a.slab;
  const int groups = here / a.width, g0 = slab * a.slab / a.width;
  // W8: an entry of a row is a thread's eight channels
  const int entries = W8 ? a.slab / 8 : a.slab, per = W8 ? a.width / 8 : a.width, mine = W8 ? (l.c - slab * a.slab) / 8 : l.c - slab * a.slab;
  float *means = lds + a.rows * entries, *rstds = means + a.slab / a.width;
  Vec<T, W8> x[NI];
  Steps<const T> p(static_cast<const T*>(a.x) + b * a.x_batch + l.c, a.x_token, a, l.row);
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const T* q = p.next();
    if (l.n > 0 && l.row + k * a.rows < n)
      x[k].load(q, l.n);
    else
      x[k].clear();
  }
  const float inv = n ? 1.0f / (static_cast<float>(n) * a.width) : 0.0f;
  // both passes: each row's sums to LDS, then the groups'
  const auto reduce = [&](auto&& term, float* to, auto&& finish) {
    float s[8] = {};
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (l.row + k * a.rows >= n) continue;
      float v[8];
      x[k].get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += term(v[e], e);
    }
    if (l.n > 0) {
      if constexpr (W8) {
        lds[l.row * entries + mine] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < l.n) lds[l.row * entries + mine + e] = s[e];
      }
    }
    __syncthreads();
    over_groups(
        groups, a.rows * per, [&](int g, int i, float& t, float&) { t += lds[i / per * entries + g * per + i % per]; },
        [&](int g, float t, float) { to[g] = finish(t); });
    __syncthreads();
  };
  reduce([](float v, int) { return v; }, means, [&](float t) { return t * inv; });
  float mean[W8 ? 1 : 8];
#pragma unroll
  for (int e = 0; e < (W8 ? 1 : 8); ++e) mean[e] = means[e < l.n ? (l.c + e) / a.width - g0 : 0];
  reduce(
      [&](float v, int e) {
        const float d = v - mean[W8 ? 0 : e];
        return d * d;
      },
      rstds, [&](float t) { return 1.0f / __builtin_sqrtf(__builtin_fmaf(t, inv, a.eps)); });
  for (int g = threadIdx.x; g < groups; g += blockDim.x) {
    a.mean[b * a.groups + g0 + g] = means[g];
    a.rstd[b * a.groups + g0 + g] = rstds[g];
  }
  if (l.row >= a.rows || (!KEEP && l.n <= 0)) return;
  const Channels<W8> ch(a, l, means, rstds, g0);
  Outputs<T, KEEP> out(a, l, b * a.seqlen, l.row);
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int t = l.row + k * a.rows;
    if (t >= a.seqlen) break;
    put_token<T, W8, KEEP>(a, l, ch, out, t < n, x[k]);
  }
}

// The gradient's x, activations or 8-bit codes, token after token.
template <typename T, bool W8, bool CODES>
struct Input : Vec<T, W8> {
  using Place = Steps<const T>;
  static __device__ __forceinline__ Place place(const GnArgs& a, const Lane& l, int64_t b, int first) {
    return Place(static_cast<const T*>(a.x) + b * a.x_batch + first * a.x_token + l.c, a.x_token, a, l.row);
  }
  template <bool ONCE = false>
  __device__ __forceinline__ void take(const Lane& l, Place& p, bool live = true) {
    const T* q = p.next();
    if (live)
      this->template load<ONCE>(q, l.n);
    else
      this->clear();
  }
  __device__ __forceinline__ void centred(const float (&v)[8], int k, float mean, float& to) const { to = v[k] - mean; }
};
template <typename T, bool W8>
struct Input<T, W8, true> : Codes {
  struct Place {
    Steps<const uint8_t> codes;
    Steps<const float> scale;
  };
  static __device__ __forceinline__ Place place(const GnArgs& a, const Lane& l, int64_t b, int first) {
    const int64_t at = b * a.seqlen + first;
    return {Steps<const uint8_t>(a.codes + at * a.dim + l.c, a.dim, a, l.row),
            Steps<const float>(a.codes_scale + at * a.scales + l.c / 128, a.scales, a, l.row)};
  }
  template <bool ONCE = false>
  __device__ __forceinline__ void take(const Lane& l, Place& p, bool live = true) {
    const uint8_t* q = p.codes.next();
    const float* s = p.scale.next();
    if (live)
      this->template load<W8, ONCE>(q, l.n, s);
    else
      this->clear();
  }
  __device__ __forceinline__ void centred(const float (&v)[8], int k, float mean, float& to) const { to = __builtin_fmaf(v[k], scale, -mean); }
};

// x -> x - mean, dy -> the gradient before the activation.
template <typename T, bool W8, bool CODES>
__device__ __forceinline__ void before_act(const GnArgs& a, const Channels<W8>& ch, const Input<T, W8, CODES>& x,
                                           const Vec<T, W8>& dy, float (&d)[8], float (&g)[8]) {
  float v[8];
  x.get(v);
  dy.get(g);
#pragma unroll
  for (int k = 0; k < 8; ++k) x.centred(v, k, ch.of(k), d[k]);
  if (a.act) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float u = __builtin_fmaf(d[k], ch.scale[k], ch.bias[k]), s = sigmoid(u);
      g[k] *= s * __builtin_fmaf(u, 1.0f - s, 1.0f);
    }
  }
}

// The rows' two sums of each channel, l1 and l2 [rows][slab], joined over the rows of the step, to `chan`, and the groups'
// sums weighted by the channels' weights, to `to`.  `scratch`: a float per thread.
template <typename TO>
__device__ __forceinline__ void join_rows(const GnArgs& a, float* l1, float* l2, float* scratch, int c0, int channels,
                                          float* chan, TO&& to) {
  over_rows(a.rows, channels, scratch, [&](int r, int c) { return l1[r * a.slab + c]; }, [&](int c, float t) { l1[c] = chan[c0 + c] = t; });
  over_rows(a.rows, channels, scratch, [&](int r, int c) { return l2[r * a.slab + c]; },
            [&](int c, float t) { l2[c] = chan[a.dim + c0 + c] = t; });
  __syncthreads();
  over_groups(
      channels / a.width, a.width,
      [&](int g, int i, float& t1, float& t2) {
        const int c = g * a.width + i;
        const float w = a.w[c0 + c];
        t1 += w * l1[c], t2 += w * l2[c];
      },
      to);
}

template <typename T, bool W8, bool CODES, bool ONCE>
__global__ __launch_bounds__(512) void groupnorm_sums_kernel(GnArgs a) {
  extern __shared__ float lds[];  // [2][rows][dim] and a float per thread
  const int64_t b = blockIdx.y;
  const int first = blockIdx.x * a.run, left = tokens_of(a, b) - first;
  const int n = left < a.run ? (left > 0 ? left : 0) : a.run;
  const Lane l(a, 0);
  float *l1 = lds, *l2 = lds + a.rows * a.dim;
  if (l.n > 0) {
    const float* rstds = a.rstd + b * a.groups;
    const Channels<W8> ch(a, l, a.mean + b * a.groups, rstds, 0);
    float s1[8], s2[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s1[k] = s2[k] = 0.0f;
    Steps<const T> p(static_cast<const T*>(a.dy) + b * a.dy_batch + first * a.dy_token + l.c, a.dy_token, a, l.row);
    auto px = Input<T, W8, CODES>::place(a, l, b, first);
    Input<T, W8, CODES> x[kAheadBack];
    Vec<T, W8> dy[kAheadBack];
    over_tokens<kAheadBack>(
        l.row, a.rows, n,
        [&](int k) {
          x[k].template take<ONCE>(l, px);
          dy[k].template load<ONCE>(p.next(), l.n);
        },
        [&](int k) {
          float xv[8], g[8];
          before_act<T, W8, CODES>(a, ch, x[k], dy[k], xv, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s1[e] += g[e];
            s2[e] = __builtin_fmaf(g[e], xv[e], s2[e]);
          }
        });
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < l.n) {
        l1[l.row * a.dim + l.c + k] = s1[k];
        l2[l.row * a.dim + l.c + k] = n ? s2[k] * rstds[(l.c + k) / a.width] : 0.0f;  // (infinite where eps is 0)
      }
  }
  __syncthreads();
  const int64_t at = b * a.splits + blockIdx.x;
  join_rows(a, l1, l2, l2 + a.rows * a.dim, 0, a.dim, a.chan + at * 2 * a.dim, [&](int g, float t1, float t2) {
    float* out = a.part + (at * a.groups + g) * 2;
    out[0] = t1, out[1] = t2;
  });
}

// dw and db: sums over the batch rows' runs.  32 columns of one of the two, shares of the runs, joined in LDS.
__device__ __forceinline__ void sum_runs(const GnArgs& a, int block, float* lds) {
  const int per = (a.dim + 31) / 32, which = block / per, c = (block % per) * 32 + (threadIdx.x & 31);
  const int share = threadIdx.x >> 5, shares = blockDim.x >> 5;
  const int64_t runs = a.batch * a.splits;
  float t = 0.0f;
  if (c < a.dim) {
#pragma unroll 8
    for (int64_t i = share; i < runs; i += shares) t += a.chan[(i * 2 + which) * a.dim + c];
  }
  lds[threadIdx.x] = t;
  __syncthreads();
  if (share == 0 && c < a.dim) {
    for (int i = 1; i < shares; ++i) t += lds[i * 32 + (threadIdx.x & 31)];
    (which ? a.dw : a.db)[c] = t;
  }
}

__global__ __launch_bounds__(1024) void groupnorm_dw_kernel(GnArgs a) {
  __shared__ float lds[1024];
  sum_runs(a, blockIdx.x, lds);
}

// The part of dx that a thread's channels share: dx = scale g - first - (x - mean) second.
template <bool W8>
struct Means {
  float first[W8 ? 1 : 8], second[W8 ? 1 : 8];
  // m1, m2: the groups' means of weight g and weight g n, from group g0 on
  __device__ __forceinline__ Means(const GnArgs& a, const Lane& l, int64_t b, const float* m1, const float* m2, int g0) {
#pragma unroll
    for (int k = 0; k < (W8 ? 1 : 8); ++k) {
      const int g = k < l.n ? (l.c + k) / a.width : g0;
      const float r = a.rstd[b * a.groups + g];
      first[k] = r * m1[g - g0], second[k] = r * r * m2[g - g0];
    }
  }
};
template <typename T, bool W8, bool CODES>
__device__ __forceinline__ void put_dx(const GnArgs& a, const Lane& l, const Channels<W8>& ch, const Means<W8>& m, T* to,
                                       const Input<T, W8, CODES>& x, const Vec<T, W8>& dy) {
  float d[8], g[8];
  before_act<T, W8, CODES>(a, ch, x, dy, d, g);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    g[k] = __builtin_fmaf(-d[k], m.second[W8 ? 0 : k], __builtin_fmaf(g[k], ch.scale[k], -m.first[W8 ? 0 : k]));
  store_vec<T, W8>(to, l.n, g);
}

// dx; the workgroups past the rows' runs sum dw and db.
template <typename T, bool W8, bool CODES, bool ONCE>
__global__ __launch_bounds__(512) void groupnorm_dx_kernel(GnArgs a) {
  extern __shared__ float lds[];  // the groups' two means, or sum_runs' shares
  const int64_t runs = a.batch * a.splits;
  if (blockIdx.x >= runs) {
    sum_runs(a, static_cast<int>(blockIdx.x - runs), lds);
    return;
  }
  const int64_t b = blockIdx.x / a.splits;
  const int all = tokens_of(a, b), first = static_cast<int>(blockIdx.x - b * a.splits) * a.run;
  const int rest = static_cast<int>(a.seqlen) - first, n = rest < a.run ? rest : a.run;
  const int live = all - first < 0 ? 0 : all - first < n ? all - first : n;
  const Lane l(a, 0);
  const float inv = all ? 1.0f / (static_cast<float>(all) * a.width) : 0.0f;
  over_groups(
      a.groups, a.splits,
      [&](int g, int s, float& t1, float& t2) {
        const float* p = a.part + ((b * a.splits + s) * a.groups + g) * 2;
        t1 += p[0], t2 += p[1];
      },
      [&](int g, float t1, float t2) { lds[g] = t1 * inv, lds[a.groups + g] = t2 * inv; });
  __syncthreads();
  if (l.n <= 0) return;
  const Channels<W8> ch(a, l, a.mean + b * a.groups, a.rstd + b * a.groups, 0);
  const Means<W8> m(a, l, b, lds, lds + a.groups, 0);
  Steps<const T> p(static_cast<const T*>(a.dy) + b * a.dy_batch + first * a.dy_token + l.c, a.dy_token, a, l.row);
  Steps<T> out(static_cast<T*>(a.y) + (b * a.seqlen + first) * a.dim + l.c, a.dim, a, l.row);
  auto px = Input<T, W8, CODES>::place(a, l, b, first);
  Input<T, W8, CODES> x[kAheadBack];
  Vec<T, W8> dy[kAheadBack];
  over_tokens<kAheadBack>(
      l.row, a.rows, live,
      [&](int k) {
        x[k].template take<ONCE>(l, px);
        dy[k].template load<ONCE>(p.next(), l.n);
      },
      [&](int k) { put_dx<T, W8, CODES>(a, l, ch, m, out.next(), x[k], dy[k]); });
  const float zero[8] = {};
  for (int t = l.row + seen(live, l.row, a.rows) * a.rows; t < n; t += a.rows) store_vec<T, W8>(out.next(), l.n, zero);
}

// The gradient of a slab in registers.
template <typename T, bool W8, int NI, bool CODES>
__global__ __launch_bounds__(512, W8 ? 4 : 2) void groupnorm_slab_bwd_kernel(GnArgs a) {
  extern __shared__ float lds[];  // [2][rows][slab], the groups' two means and a float per thread
  const int64_t b = blockIdx.x / a.slabs;
  const int slab = static_cast<int>(blockIdx.x - b * a.slabs), n = tokens_of(a, b);
  const Lane l(a, slab);
  const int here = a.dim - slab * a.slab < a.slab ? a.dim - slab * a.slab : a.slab, g0 = slab * a.slab / a.width;
  float *l1 = lds, *l2 = l1 + a.rows * a.slab, *m1 = l2 + a.rows * a.slab, *m2 = m1 + a.slab / a.width;
  const float inv = n ? 1.0f / (static_cast<float>(n) * a.width) : 0.0f;
  Input<T, W8, CODES> x[NI];
  Vec<T, W8> dy[NI];
  Steps<const T> p(static_cast<const T*>(a.dy) + b * a.dy_batch + l.c, a.dy_token, a, l.row);
  auto px = Input<T, W8, CODES>::place(a, l, b, 0);
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const bool live = l.n > 0 && l.row + k * a.rows < n;
    x[k].take(l, px, live);
    const T* q = p.next();
    if (live)
      dy[k].load(q, l.n);
    else
      dy[k].clear();
  }
  const Channels<W8> ch(a, l, a.mean + b * a.groups, a.rstd + b * a.groups, 0);
  if (l.n > 0) {
    float s1[8], s2[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s1[e] = s2[e] = 0.0f;
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (l.row + k * a.rows >= n) continue;
      float xv[8], g[8];
      before_act<T, W8, CODES>(a, ch, x[k], dy[k], xv, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1[e] += g[e];
        s2[e] = __builtin_fmaf(g[e], xv[e], s2[e]);
      }
    }
    const int at = l.row * a.slab + l.c - slab * a.slab;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < l.n) l1[at + e] = s1[e], l2[at + e] = n ? s2[e] * a.rstd[b * a.groups + (l.c + e) / a.width] : 0.0f;
  }
  __syncthreads();
  join_rows(a, l1, l2, m2 + a.slab / a.width, slab * a.slab, here, a.chan + b * 2 * a.dim,
            [&](int g, float t1, float t2) { m1[g] = t1 * inv, m2[g] = t2 * inv; });
  __syncthreads();
  if (l.n <= 0) return;
  const Means<W8> m(a, l, b, m1, m2, g0);
  Steps<T> out(static_cast<T*>(a.y) + b * a.seqlen * a.dim + l.c, a.dim, a, l.row);
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int t = l.row + k * a.rows;
    if (t >= a.seqlen) break;
    T* to = out.next();
    if (t < n) {
      put_dx<T, W8, CODES>(a, l, ch, m, to, x[k], dy[k]);
    } else {
      const float zero[8] = {};
      store_vec<T, W8>(to, l.n, zero);
    }
  }
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// How a call is done.
struct Plan {
  GnArgs a{};
  int threads = 0, tokens = 0;  // tokens: of a thread that keeps a slab; 0: runs
  bool w8 = false, once = false;

  // Threads of a workgroup and rows of a step: of the counts from 256 to 512 the one that leaves the fewest idle, or with
  // `many` the largest that leaves few.
  int threads_for(bool many) {
    int best = 0;
    float share = 0.0f;
    for (int i = 0; i <= 4; ++i) {
      const int nt = many ? 512 - 64 * i : 256 + 64 * i, rows = nt / a.lanes;
      const float f = static_cast<float>(rows * a.lanes) / nt;
      if (rows && f > share + (many && best ? 0.1f : 1e-3f)) best = nt, share = f;
    }
    a.rows = best ? best / a.lanes : 0;
    return best;
  }
  void lanes_for(int channels, bool keep) {
    a.lanes = (channels + 7) / 8;
    if (keep) a.lanes = (a.lanes + kGroupLanes - 1) / kGroupLanes * kGroupLanes;
  }

  Plan(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, vmscan_dtype dtype, bool gradient, bool keep, bool codes) {
    a.batch = batch, a.seqlen = seqlen, a.dim = static_cast<int>(dim), a.groups = static_cast<int>(groups);
    a.width = a.dim / a.groups;
    a.scales = (a.dim + 127) / 128;
    w8 = a.width % 8 == 0;
    if (slab_fits(dtype == VMSCAN_BF16, gradient, keep, codes)) return;
    tokens = 0;
    a.slab = a.dim, a.slabs = 1;
    lanes_for(a.dim, keep);
    // (the bfloat16 gradient with 512 threads rather than 256: 32 x 3136 x 512 from 8 bits 79 us instead of 83, 8 x 12544 x 384
    // 65 for 71; forwards and float32 are up to 10 % slower that way)
    threads = threads_for(gradient && dtype == VMSCAN_BF16);
    // Inputs and outputs past this fill the 256 MB last-level cache: streamed loads leave it to the outputs on their way
    // to memory.  32 x 3136 x 512 takes 74 us instead of 91 (gradient from 8 bits 79 for 91), a half of that 47 for 43.
    const int64_t bytes = batch * seqlen * dim * ((dtype == VMSCAN_BF16 ? 2 : 4) * (gradient && !codes ? 3 : 2) + (keep || codes));
    once = bytes > (int64_t{160} << 20);
    // Runs: two workgroups a CU, not one more (64 x 3136 x 192, gradient: 512 workgroups 100 us, 1024 141; 24 images of 512
    // channels: 504 workgroups 61 us, 528 70), or one where two would have less than 16 steps each.
    const int64_t steps = (seqlen + a.rows - 1) / a.rows;
    int64_t splits = 512 / batch;
    if (splits * 16 > steps) splits = 256 / batch;
    if (splits > steps) splits = steps;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits < 1) splits = 1;
    a.run = static_cast<int>((steps + splits - 1) / splits * a.rows);
    a.splits = static_cast<int>((seqlen + a.run - 1) / a.run);
  }

  // A slab: the fewest whole groups of 128 bytes of a token, or of all channels; with 8-bit copies a multiple of 128
  // channels.  The fewest threads that hold it.
  bool slab_fits(bool bf16, bool gradient, bool keep, bool codes) {
    // registers that a thread keeps for 8 channels of a token
    const int regs = w8 && bf16 ? (gradient ? (codes ? 7 : 8) : 4) : (gradient ? (codes ? 11 : 16) : 8);
    const int least = bf16 ? 64 : 32;
    int channels = (least + a.width - 1) / a.width * a.width;
    if (keep)
      while (channels % 128 && channels < a.dim) channels += a.width;
    if (channels > a.dim) channels = a.dim;
    if (!w8 && channels % 8 && channels < a.dim) {  // whole vectors but at the end
      while (channels % 8 && channels < a.dim) channels += a.width;
      if (channels > a.dim) channels = a.dim;
    }
    if (keep && channels % 128 && channels < a.dim) return false;
    lanes_for(channels, keep);
    const int most = regs <= 4 ? 16 : regs <= 8 ? 8 : 4;
    const int widest = gradient ? 512 : 1024;
    for (int nt = 256; nt <= widest; nt *= 2) {
      a.rows = nt / a.lanes;
      if (!a.rows) continue;
      const int64_t each = (a.seqlen + a.rows - 1) / a.rows;
      if (each > most) continue;
      threads = nt;
      tokens = each <= 4 ? 4 : each <= 8 ? 8 : 16;
      a.slab = channels, a.slabs = (a.dim + channels - 1) / channels, a.splits = 1, a.run = static_cast<int>(a.seqlen);
      return true;
    }
    return false;
  }
  size_t stats_bytes() const {
    return tokens ? 0 : static_cast<size_t>(a.batch) * a.splits * a.groups * 2 * sizeof(float);
  }
  size_t chan_bytes() const { return static_cast<size_t>(a.batch) * a.splits * 2 * a.dim * sizeof(float); }
};

template <typename T, bool W8, bool KEEP, bool ONCE>
void launch_runs(const Plan& p, hipStream_t stream) {
  const GnArgs& a = p.a;
  const dim3 grid(a.splits, static_cast<unsigned>(a.batch)), block(p.threads);
  const size_t lds = (2 * static_cast<size_t>(a.rows) * a.dim + a.dim + a.groups + p.threads) * sizeof(float);
  hipLaunchKernelGGL((groupnorm_stats_kernel<T, W8, ONCE>), grid, block, lds, stream, a);
  hipLaunchKernelGGL((groupnorm_apply_kernel<T, W8, KEEP, ONCE>), grid, block, 2 * a.groups * sizeof(float), stream, a);
}
template <typename T, bool W8, bool CODES, bool ONCE>
void launch_bwd_runs(const Plan& p, unsigned sums, hipStream_t stream) {
  const GnArgs& a = p.a;
  const dim3 block(p.threads);
  const size_t lds = (2 * static_cast<size_t>(a.rows) * a.dim + p.threads) * sizeof(float);
  hipLaunchKernelGGL((groupnorm_sums_kernel<T, W8, CODES, ONCE>), dim3(a.splits, static_cast<unsigned>(a.batch)), block, lds,
                     stream, a);
  const size_t groups = 2 * static_cast<size_t>(a.groups) * sizeof(float), shares = p.threads * sizeof(float);
  hipLaunchKernelGGL((groupnorm_dx_kernel<T, W8, CODES, ONCE>), dim3(static_cast<unsigned>(a.batch * a.splits) + sums), block,
                     groups > shares ? groups : shares, stream, a);
}

template <typename T, bool W8, bool KEEP>
void launch_fwd(const Plan& p, hipStream_t stream) {
  const GnArgs& a = p.a;
  if (p.tokens) {
    const dim3 grid(static_cast<unsigned>(a.batch * a.slabs)), block(p.threads);
    const size_t lds = (static_cast<size_t>(a.rows) * (W8 ? a.slab / 8 : a.slab) + 2 * (a.slab / a.width)) * sizeof(float);
    if (p.tokens == 4)
      hipLaunchKernelGGL((groupnorm_slab_kernel<T, W8, 4, KEEP>), grid, block, lds, stream, a);
    else if (p.tokens == 8)
      hipLaunchKernelGGL((groupnorm_slab_kernel<T, W8, 8, KEEP>), grid, block, lds, stream, a);
    else if constexpr (W8 && sizeof(T) == 2)
      hipLaunchKernelGGL((groupnorm_slab_kernel<T, W8, 16, KEEP>), grid, block, lds, stream, a);
    return;
  }
  p.once ? launch_runs<T, W8, KEEP, true>(p, stream) : launch_runs<T, W8, KEEP, false>(p, stream);
}

template <typename T, bool W8, bool CODES>
void launch_bwd(const Plan& p, hipStream_t stream) {
  const GnArgs& a = p.a;
  const unsigned sums = 2 * static_cast<unsigned>((a.dim + 31) / 32);
  if (p.tokens) {
    const dim3 grid(static_cast<unsigned>(a.batch * a.slabs)), block(p.threads);
    const size_t lds = (2 * static_cast<size_t>(a.rows) * a.slab + 2 * (a.slab / a.width) + p.threads) * sizeof(float);
    if (p.tokens == 4)
      hipLaunchKernelGGL((groupnorm_slab_bwd_kernel<T, W8, 4, CODES>), grid, block, lds, stream, a);
    else if constexpr (W8 && sizeof(T) == 2)
      hipLaunchKernelGGL((groupnorm_slab_bwd_kernel<T, W8, 8, CODES>), grid, block, lds, stream, a);
    hipLaunchKernelGGL(groupnorm_dw_kernel, dim3(sums), dim3(1024), 0, stream, a);
    return;
  }
  p.once ? launch_bwd_runs<T, W8, CODES, true>(p, sums, stream) : launch_bwd_runs<T, W8, CODES, false>(p, sums, stream);
}

template <typename T>
void dispatch_fwd(const Plan& p, hipStream_t stream) {
  if (p.w8)
    p.a.keep ? launch_fwd<T, true, true>(p, stream) : launch_fwd<T, true, false>(p, stream);
  else
    p.a.keep ? launch_fwd<T, false, true>(p, stream) : launch_fwd<T, false, false>(p, stream);
}
template <typename T>
void dispatch_bwd(const Plan& p, hipStream_t stream) {
  if (p.w8)
    p.a.codes ? launch_bwd<T, true, true>(p, stream) : launch_bwd<T, true, false>(p, stream);
  else
    p.a.codes ? launch_bwd<T, false, true>(p, stream) : launch_bwd<T, false, false>(p, stream);
}

bool shape_ok(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups) {
  return batch >= 1 && seqlen >= 1 && dim >= 1 && dim <= kMaxDim && groups >= 1 && groups <= dim && dim % groups == 0 &&
         batch < 65536 && seqlen < (int64_t{1} << 30);
}

bool strides_ok(const int64_t* s) {
  return s[0] >= 0 && s[1] >= 0 && s[0] <= (int64_t{1} << 40) && s[1] < (int64_t{1} << 32);
}

}  // namespace

extern "C" {

size_t vmscan_groupnorm_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int keep) {
  if (!shape_ok(batch, seqlen, dim, groups)) return 0;
  const size_t f = Plan(batch, seqlen, dim, groups, VMSCAN_F32, false, keep != 0, false).stats_bytes();
  const size_t b = Plan(batch, seqlen, dim, groups, VMSCAN_BF16, false, keep != 0, false).stats_bytes();
  return f > b ? f : b;
}

vmscan_status vmscan_groupnorm_fwd(const void* x, const int64_t* x_strides, const float* weight, const float* bias,
                                   const int32_t* lengths, void* y, float* mean, float* rstd, void* keep_codes,
                                   float* keep_scale, int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, float eps,
                                   int act, vmscan_dtype dtype, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  if (!x || !x_strides || !weight || !bias || !y || !mean || !rstd) return VMSCAN_ERR_NULL;
  if ((keep_codes == nullptr) != (keep_scale == nullptr)) return VMSCAN_ERR_NULL;
  if (!shape_ok(batch, seqlen, dim, groups) || !strides_ok(x_strides) || !(eps >= 0.0f)) return VMSCAN_ERR_SHAPE;
  if ((dtype != VMSCAN_F32 && dtype != VMSCAN_BF16) || (act != 0 && act != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  if (!aligned_to(x, e) || !aligned_to(y, 16) || !aligned_to(workspace, 16)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(lengths),
                        static_cast<const void*>(mean), static_cast<const void*>(rstd), static_cast<const void*>(keep_scale)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  Plan plan(batch, seqlen, dim, groups, dtype, false, keep_codes != nullptr, false);
  const size_t need = vmscan_groupnorm_fwd_workspace_bytes(batch, seqlen, dim, groups, keep_codes != nullptr);
  if (need && (!workspace || workspace_bytes < need)) return VMSCAN_ERR_WORKSPACE;
  GnArgs& a = plan.a;
  a.x = x, a.w = weight, a.b = bias, a.lengths = lengths, a.y = y, a.mean = mean, a.rstd = rstd;
  a.keep = static_cast<uint8_t*>(keep_codes), a.keep_scale = keep_scale, a.part = static_cast<float*>(workspace);
  a.x_batch = x_strides[0], a.x_token = x_strides[1], a.eps = eps, a.act = act;
  if (dtype == VMSCAN_F32)
    dispatch_fwd<float>(plan, stream);
  else
    dispatch_fwd<uint16_t>(plan, stream);
  return launched();
}

size_t vmscan_groupnorm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t groups) {
  if (!shape_ok(batch, seqlen, dim, groups)) return 0;
  size_t most = 0;
  for (const vmscan_dtype dtype : {VMSCAN_F32, VMSCAN_BF16})
    for (const bool codes : {false, true}) {
      const Plan p(batch, seqlen, dim, groups, dtype, true, false, codes);
      const size_t n = round16(p.stats_bytes()) + p.chan_bytes();
      most = n > most ? n : most;
    }
  return most;
}

vmscan_status vmscan_groupnorm_bwd(const void* dy, const int64_t* dy_strides, const void* x, const int64_t* x_strides,
                                   const void* codes, const float* codes_scale, const float* weight, const float* bias,
                                   const float* mean, const float* rstd, const int32_t* lengths, void* dx, float* dweight,
                                   float* dbias, int64_t batch, int64_t seqlen, int64_t dim, int64_t groups, int act,
                                   vmscan_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!dy || !dy_strides || !weight || !bias || !mean || !rstd || !dx || !dweight || !dbias) return VMSCAN_ERR_NULL;
  if ((x == nullptr) == (codes == nullptr) || (x && !x_strides) || (codes == nullptr) != (codes_scale == nullptr))
    return VMSCAN_ERR_NULL;
  if (!shape_ok(batch, seqlen, dim, groups) || !strides_ok(dy_strides) || (x && !strides_ok(x_strides)))
    return VMSCAN_ERR_SHAPE;
  if ((dtype != VMSCAN_F32 && dtype != VMSCAN_BF16) || (act != 0 && act != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, 16) || !aligned_to(workspace, 16)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(weight), static_cast<const void*>(bias), static_cast<const void*>(lengths),
                        static_cast<const void*>(mean), static_cast<const void*>(rstd),
                        static_cast<const void*>(codes_scale), static_cast<const void*>(dweight),
                        static_cast<const void*>(dbias)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  Plan plan(batch, seqlen, dim, groups, dtype, true, false, codes != nullptr);
  if (!workspace || workspace_bytes < vmscan_groupnorm_bwd_workspace_bytes(batch, seqlen, dim, groups))
    return VMSCAN_ERR_WORKSPACE;
  GnArgs& a = plan.a;
  a.x = x, a.dy = dy, a.codes = static_cast<const uint8_t*>(codes), a.codes_scale = codes_scale;
  a.w = weight, a.b = bias, a.lengths = lengths, a.y = dx, a.dw = dweight, a.db = dbias, a.act = act;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.part = static_cast<float*>(workspace);
  a.chan = reinterpret_cast<float*>(static_cast<char*>(workspace) + round16(plan.stats_bytes()));
  a.dy_batch = dy_strides[0], a.dy_token = dy_strides[1];
  if (x) a.x_batch = x_strides[0], a.x_token = x_strides[1];
  if (dtype == VMSCAN_F32)
    dispatch_bwd<float>(plan, stream);
  else
    dispatch_bwd<uint16_t>(plan, stream);
  return launched();
}

}  // extern "C"
