// Rotary positions with several axes for queries and keys.  What is computed is stated in
// include/vmscan.h.
//
// Bound by HBM: every element is read and written once.  A thread owns one unit of channels of one
// token (V channels of each half, or V channels in neighbouring pairs), computes the unit's sines
// and cosines once and applies them to its share of the token's query and key heads; the trigonometry
// is thus paid once per token and pair, not per head.  Measured: 128 x 197 tokens, 6 + 6 heads of 64, bfloat16,
// 77 MB in 16.2 us (partly from the 256 MB cache); 12544 tokens, 12 + 4 heads of 128, float32, 205 MB in 43 us, 4.8 TB/s.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

struct RopeTensor {
  const void* in;
  void* out;
  int64_t ib, it, ih, ob, ot, oh;  // strides in elements: batch, token, head
  int heads;
};

struct RopeArgs {
  RopeTensor q, k;  // k.heads 0 when there is none
  const float *pos, *inv_freq;
  const int* axis;
  int64_t pos_stride;  // between batches; 0: one grid for all
  int64_t first, tokens;  // of batch * seqlen, the launch's first one and how far it goes
  int64_t seqlen;
  int dim, rot, axes;
  int units, pass_units;  // units of rotated channels; of channels that only pass through
  int shares;             // threads a token's heads are shared out over, per unit
  int inverse;
};

// cos and sin of p * f radians.  The product is taken as a head and a tail (their sum is exact)
// and turned into revolutions with 1 / (2 pi) in two parts, so that the part of a revolution that
// is left after taking out whole ones is good to about 2^-24 whatever p: a plain float32 product
// is off by 2^-25 |p f| radians, which is visible for positions in the thousands.
__device__ __forceinline__ void cos_sin(float p, float f, float& c, float& s) {
#pragma clang fp contract(off)  // t has to be the rounded product wherever it is used
  constexpr float kHi = 0.15915494309189535f;
  constexpr float kLo = static_cast<float>(0.15915494309189535 - static_cast<double>(kHi));
  const float head = p * f, tail = __builtin_fmaf(p, f, -head);
  const float t = head * kHi;
  const float rest = __builtin_fmaf(head, kHi, -t) + __builtin_fmaf(head, kLo, tail * kHi);
  const float part = (t - __builtin_rintf(t)) + rest;
  sincospif(2.0f * part, &s, &c);
}

// V consecutive channels: one 16-byte access, or one by one.
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V * sizeof(T) == 16 && V == 8) {
    load8(p, v);
  } else if constexpr (V * sizeof(T) == 16) {
    __builtin_memcpy(v, p, 16);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = load1(p + k);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V * sizeof(T) == 16 && V == 8) {
    store8(p, v);
  } else if constexpr (V * sizeof(T) == 16) {
    __builtin_memcpy(p, v, 16);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) store1(p + k, v[k]);
  }
}

template <typename T, int V, bool INTERLEAVED>
__device__ __forceinline__ void rope_heads(const RopeTensor& x, int64_t b, int64_t t, int first, int step, int at,
                                           int half, const float* c, const float* s) {
  const T* in = static_cast<const T*>(x.in) + b * x.ib + t * x.it + at;
  T* out = static_cast<T*>(x.out) + b * x.ob + t * x.ot + at;
#pragma unroll 2
  for (int h = first; h < x.heads; h += step) {
    float u[V], w[V];
    load_v<T, V>(in + h * x.ih, u);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        w[2 * k] = __builtin_fmaf(u[2 * k], c[k], -(u[2 * k + 1] * s[k]));
        w[2 * k + 1] = __builtin_fmaf(u[2 * k], s[k], u[2 * k + 1] * c[k]);
      }
      store_v<T, V>(out + h * x.oh, w);
    } else {
      load_v<T, V>(in + h * x.ih + half, w);
      float y[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        y[k] = __builtin_fmaf(u[k], c[k], -(w[k] * s[k]));
        w[k] = __builtin_fmaf(u[k], s[k], w[k] * c[k]);
      }
      store_v<T, V>(out + h * x.oh, y);
      store_v<T, V>(out + h * x.oh + half, w);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void pass_heads(const RopeTensor& x, int64_t b, int64_t t, int first, int step, int at,
                                           int n) {
  const T* in = static_cast<const T*>(x.in) + b * x.ib + t * x.it + at;
  T* out = static_cast<T*>(x.out) + b * x.ob + t * x.ot + at;
  if (in == out && x.ih == x.oh) return;  // in place
  for (int h = first; h < x.heads; h += step) {
    if (n >= V) {
      float u[V];
      load_v<T, V>(in + h * x.ih, u);
      store_v<T, V>(out + h * x.oh, u);
    } else {
      for (int k = 0; k < n; ++k) out[h * x.oh + k] = in[h * x.ih + k];
    }
  }
}

template <typename T, int V, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  constexpr int kPairs = INTERLEAVED ? V / 2 : V;  // pairs per unit
  const int per_token = (a.units + a.pass_units) * a.shares;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t in_launch = id / per_token, token = a.first + in_launch;
  if (token >= a.tokens) return;
  const int rest = static_cast<int>(id - in_launch * per_token);
  const int share = rest / (a.units + a.pass_units), unit = rest % (a.units + a.pass_units);
  const int64_t b = token / a.seqlen, t = token - b * a.seqlen;
  if (unit >= a.units) {
    const int at = a.rot + (unit - a.units) * V;
    pass_heads<T, V>(a.q, b, t, share, a.shares, at, a.dim - at);
    if (a.k.heads) pass_heads<T, V>(a.k, b, t, share, a.shares, at, a.dim - at);
    return;
  }
  const float* pos = a.pos + b * a.pos_stride + t * a.axes;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int pair = unit * kPairs + i, ax = a.axis[pair];
    c[i] = 1.0f, s[i] = 0.0f;
    if (ax >= 0 && ax < a.axes) cos_sin(pos[ax], a.inv_freq[pair], c[i], s[i]);
    if (a.inverse) s[i] = -s[i];
  }
  const int at = unit * V, half = a.rot / 2;
  rope_heads<T, V, INTERLEAVED>(a.q, b, t, share, a.shares, at, half, c, s);
  if (a.k.heads) rope_heads<T, V, INTERLEAVED>(a.k, b, t, share, a.shares, at, half, c, s);
}

// Threads wanted before a token's heads stay with one thread: about 8 waves on every SIMD.  Measured on those two
// shapes, us: 128 K threads 17.4 and 43.6, 300 K 18.0 and 40.5, 512 K 17.6 and 42.8, 2 M 19.2 and 62.
constexpr int64_t kWantThreads = 256 * 4 * 8 * 64;

template <typename T, int V, bool INTERLEAVED>
vmscan_status launch_rope(RopeArgs a, hipStream_t stream) {
  a.units = INTERLEAVED ? (a.rot + V - 1) / V : (a.rot / 2 + V - 1) / V;
  a.pass_units = (a.dim - a.rot + V - 1) / V;
  const int per = a.units + a.pass_units;
  const int heads = a.q.heads > a.k.heads ? a.q.heads : a.k.heads;
  a.shares = 1;
  while (a.shares < heads && a.tokens * per * a.shares < kWantThreads) a.shares *= 2;
  if (a.shares > heads) a.shares = heads;
  const int64_t tokens = a.tokens, most = kMaxBlocks256 * 256 / (per * a.shares);  // tokens of a launch
  for (a.first = 0; a.first < tokens; a.first += most) {
    a.tokens = tokens - a.first < most ? tokens : a.first + most;
    const int64_t blocks = ((a.tokens - a.first) * per * a.shares + 255) / 256;
    hipLaunchKernelGGL((rope_kernel<T, V, INTERLEAVED>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, a);
    const vmscan_status st = launched();
    if (st != VMSCAN_OK) return st;
  }
  return VMSCAN_OK;
}

bool runs_aligned(const RopeTensor& x, int64_t n) {
  return aligned_to(x.in, 16) && aligned_to(x.out, 16) && x.ib % n == 0 && x.it % n == 0 && x.ih % n == 0 &&
         x.ob % n == 0 && x.ot % n == 0 && x.oh % n == 0;
}

// The unit of channels: 16 bytes when every run of that size starts on a 16-byte boundary and the rotated
// channels and the rest are whole runs, else one pair (the 205 MB of float32 above: 43 us, 58 in 32-byte units).
template <typename T>
vmscan_status run_rope(const RopeArgs& a, int interleaved, hipStream_t stream) {
  constexpr int kRun = 16 / sizeof(T);
  const bool wide = runs_aligned(a.q, kRun) && (!a.k.heads || runs_aligned(a.k, kRun)) && a.dim % kRun == 0 &&
                    (interleaved ? a.rot % kRun == 0 : (a.rot / 2) % kRun == 0);
  if (interleaved) return wide ? launch_rope<T, kRun, true>(a, stream) : launch_rope<T, 2, true>(a, stream);
  return wide ? launch_rope<T, kRun, false>(a, stream) : launch_rope<T, 1, false>(a, stream);
}

// Whether no two elements of [batch][token][head][dim] with these strides are one: every stride covers what lies
// inside it.
bool distinct(const int64_t* strides, int64_t batch, int64_t seqlen, int64_t heads, int64_t dim) {
  int64_t st[3] = {0, 0, 0}, n[3] = {batch, seqlen, heads};
  for (int i = 0; i < 3; ++i) st[i] = strides[i] < 0 ? -strides[i] : strides[i];
  for (int i = 0; i < 2; ++i)  // by stride
    for (int j = 0; j + 1 < 3 - i; ++j)
      if (st[j] > st[j + 1]) std::swap(st[j], st[j + 1]), std::swap(n[j], n[j + 1]);
  int64_t inside = dim;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1) {
      if (st[i] < inside) return false;
      inside += st[i] * (n[i] - 1);
    }
  return true;
}

}  // namespace

extern "C" {

vmscan_status vmscan_rope_axes(const void* q, const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                               const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                               const float* positions, int64_t positions_stride, const float* inv_freq,
                               const int32_t* axis, int64_t batch, int64_t seqlen, int heads, int kheads, int dim,
                               int rot, int axes, int interleaved, int inverse, vmscan_dtype dtype,
                               hipStream_t stream) {
  if (!q || !q_strides || !q_out || !q_out_strides || !positions || !inv_freq || !axis) return VMSCAN_ERR_NULL;
  if (kheads != 0 && (!k || !k_strides || !k_out || !k_out_strides)) return VMSCAN_ERR_NULL;
  if (batch < 1 || seqlen < 1 || heads < 1 || kheads < 0 || dim < 2 || rot < 2 || rot > dim || rot % 2 != 0 ||
      axes < 1 || positions_stride < 0)
    return VMSCAN_ERR_SHAPE;
  if (seqlen >= (int64_t{1} << 31) || batch >= (int64_t{1} << 31) || heads > 65536 || kheads > 65536 || dim > 65536 ||
      batch * seqlen >= (int64_t{1} << 40))
    return VMSCAN_ERR_SHAPE;
  if ((dtype != VMSCAN_F32 && dtype != VMSCAN_BF16) || (interleaved != 0 && interleaved != 1) ||
      (inverse != 0 && inverse != 1))
    return VMSCAN_ERR_UNSUPPORTED;
  const size_t elem = dtype == VMSCAN_F32 ? 4 : 2;
  const void* heads_at[] = {q, q_out, kheads ? k : nullptr, kheads ? k_out : nullptr};
  for (const void* p : heads_at)
    if (!aligned_to(p, elem)) return VMSCAN_ERR_ALIGN;
  if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(axis, 4)) return VMSCAN_ERR_ALIGN;
  if (!distinct(q_out_strides, batch, seqlen, heads, dim) ||
      (kheads && !distinct(k_out_strides, batch, seqlen, kheads, dim)))
    return VMSCAN_ERR_SHAPE;
  RopeArgs a{};
  a.q = RopeTensor{q, q_out, q_strides[0], q_strides[1], q_strides[2], q_out_strides[0], q_out_strides[1],
                   q_out_strides[2], heads};
  if (kheads)
    a.k = RopeTensor{k, k_out, k_strides[0], k_strides[1], k_strides[2], k_out_strides[0], k_out_strides[1],
                     k_out_strides[2], kheads};
  a.pos = positions, a.pos_stride = positions_stride, a.inv_freq = inv_freq, a.axis = axis;
  a.tokens = batch * seqlen, a.seqlen = seqlen, a.dim = dim, a.rot = rot, a.axes = axes, a.inverse = inverse;
  return dtype == VMSCAN_F32 ? run_rope<float>(a, interleaved, stream) : run_rope<uint16_t>(a, interleaved, stream);
}

}  // extern "C"
