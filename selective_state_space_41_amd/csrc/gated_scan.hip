// Gated linear recurrence with one state per channel: forward, gradient and single tokens.  What is computed is
// stated in include/vmscan.h.
//
// A workgroup owns 2 * CL neighbouring channels of one sequence, two to a lane, and walks the sequence in blocks of
// R runs of S tokens.  A run's S tokens stay in registers: their (decay, input) pairs are joined to one pair, the R
// pairs of a block meet in LDS, and every run then walks its tokens from the state that enters it.  Inputs are read
// once and the outputs written once.  Where there are too few sequences and channels for the chip a sequence is cut
// into segments, whose own pairs a first launch makes.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.925963033500e-8f, kLn2 = 0.69314718055994531f;
constexpr int kGroup = 128;  // channels that share a scale of the 8-bit copies

struct ScanArgs {
  const void *x, *r, *i, *h, *dout;
  const uint8_t* codes;          // the gradient's x, r, i, h in 8 bits: four planes
  const float* codes_scale;
  const float* A_log;
  const float *first, *last;     // the state at the start; the gradient of the one at the end
  const int32_t* lengths;
  void *out, *dx, *dr, *di;
  uint8_t* keep;
  float* keep_scale;
  float *end, *dA_log;           // the state at the end (gradient: of the one at the start)
  float2* pairs;                 // per sequence and segment: channels' pairs
  float* part;                   // gradient: per sequence and segment, channels' sums for A_log
  int64_t x_batch, x_token, r_batch, r_token, i_batch, i_token, dout_batch, dout_token;
  int64_t batch, seqlen, plane;  // plane: tokens of a plane of the 8-bit copies
  int dim, groups, tiles;
  int segments, seg_len;
  int reverse;
};

// Two neighbouring channels.
struct Two {
  float a, b;
};
// `p` is the row's place of this lane's first channel; ODD: the second may be missing (d1 = 0 reads the first again).
template <bool ODD>
__device__ __forceinline__ Two load2(const uint16_t* p, int d1) {
  if constexpr (ODD) return {bf16_to_f32(p[0]), bf16_to_f32(p[d1])};
  uint32_t w;
  __builtin_memcpy(&w, p, 4);
  return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
}
template <bool ODD>
__device__ __forceinline__ Two load2(const float* p, int d1) {
  if constexpr (ODD) return {p[0], p[d1]};
  float2 v;
  __builtin_memcpy(&v, p, 8);
  return {v.x, v.y};
}
template <bool ODD>
__device__ __forceinline__ Two load2(const uint8_t* p, int d1) {
  uint32_t w;
  if constexpr (ODD) {
    w = p[0] | static_cast<uint32_t>(p[d1]) << 8;
  } else {
    uint16_t h;
    __builtin_memcpy(&h, p, 2);
    w = h;
  }
  const auto v = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
  return {v[0], v[1]};
}
template <bool ODD>
__device__ __forceinline__ void store2(uint16_t* p, int n, Two v) {
  if (ODD && n == 1) {
    store1(p, v.a);
  } else if (n > 0) {
    const uint32_t w = static_cast<uint32_t>(f32_to_bf16(v.a)) | static_cast<uint32_t>(f32_to_bf16(v.b)) << 16;
    __builtin_memcpy(p, &w, 4);
  }
}
template <bool ODD>
__device__ __forceinline__ void store2(float* p, int n, Two v) {
  if (ODD && n == 1) {
    *p = v.a;
  } else if (n > 0) {
    const float2 w = make_float2(v.a, v.b);
    __builtin_memcpy(p, &w, 8);
  }
}

// 1 / (1 + e^-x).  The product x * log2(e) is kept as head and tail for float32 activations, whose sigmoid is then
// good to float32; bfloat16 ones do not show the tail.
template <bool TAIL>
__device__ __forceinline__ float sigmoid(float x) {
  const float t = x * -kLog2e;
  float e = __builtin_amdgcn_exp2f(t);
  if constexpr (TAIL) {
    float low = __builtin_fmaf(x, -kLog2e, -t);
    low = __builtin_fmaf(x, -kLog2eLow, low);
    e = __builtin_fabsf(t) < 126.0f ? __builtin_fmaf(e, low * kLn2, e) : e;
  }
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// A token's decay from rate = e^A_log and the gate's sigmoid: a = e^-y and w = 1 - a^2 for y = rate * sigmoid(r) >= 0.
// Below v = 2 y = 1/4 the difference is the series of 1 - e^-v (the next term is under 2^-24 of it); above, one
// fused multiply-add.
struct Decay {
  float a, w, y;
};
__device__ __forceinline__ Decay decay_of(float rate, float p) {
  Decay d;
  d.y = rate * p;
  d.a = __builtin_amdgcn_exp2f(d.y * -kLog2e);
  const float v = d.y + d.y;
  float s = __builtin_fmaf(v, -1.0f / 720.0f, 1.0f / 120.0f);
  s = __builtin_fmaf(v, s, -1.0f / 24.0f);
  s = __builtin_fmaf(v, s, 1.0f / 6.0f);
  s = __builtin_fmaf(v, s, -0.5f);
  s = __builtin_fmaf(v, s, 1.0f);
  d.w = v < 0.25f ? v * s : __builtin_fmaf(-d.a, d.a, 1.0f);
  return d;
}

template <typename T>
constexpr bool kTail = sizeof(T) == 4;

__device__ __forceinline__ int64_t tokens_of(const ScanArgs& a, int64_t b) {
  if (!a.lengths) return a.seqlen;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : n > a.seqlen ? a.seqlen : n;
}

// What a workgroup and a lane work on.  Tokens are counted along the walk; `back` walks turn the count around within
// the row's n tokens, and what lies past them keeps its place.
template <int CL, bool ODD>
struct Where {
  int64_t b, n;
  int seg, tile, run, c, cc, d1, have;  // c: first channel, cc: one that exists, have: channels that exist
  bool back;
  __device__ __forceinline__ Where(const ScanArgs& a, bool turn) {
    const int64_t u = blockIdx.x;
    tile = static_cast<int>(u % a.tiles);
    const int64_t s = u / a.tiles;
    seg = static_cast<int>(s % a.segments);
    b = s / a.segments;
    n = tokens_of(a, b);
    run = threadIdx.x / CL;
    c = (tile * CL + threadIdx.x % CL) * 2;
    have = a.dim - c;
    const int top = ODD ? a.dim - 1 : a.dim - 2;
    cc = c < top ? c : top;
    d1 = !ODD || cc + 1 < a.dim ? 1 : 0;
    back = (a.reverse != 0) != turn;
  }
  // The place of the walk's token t < n; of any other, t itself.
  __device__ __forceinline__ int64_t at(int64_t t) const { return back && t < n ? n - 1 - t : t; }
  __device__ __forceinline__ int64_t in(int64_t t) const { return at(t < n ? t : n - 1); }  // n > 0
};

__device__ __forceinline__ float rate_of(const float* A_log, int c) { return __builtin_amdgcn_exp2f(A_log[c] * kLog2e); }

// (decay, input) pairs after one another: h -> A h + H.
struct Pairs {
  float A0, H0, A1, H1;
};
__device__ __forceinline__ void then(Pairs& p, float a0, float h0, float a1, float h1) {
  p.H0 = __builtin_fmaf(a0, p.H0, h0), p.A0 *= a0;
  p.H1 = __builtin_fmaf(a1, p.H1, h1), p.A1 *= a1;
}

// The state that enters this thread's run, from the one that enters the block (c0, c1), which becomes the one after it.
template <int CL, int R>
__device__ __forceinline__ Two enter(const float4 (&part)[R][CL], int run, float& c0, float& c1) {
  Two in{c0, c1};
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j == run) in = {c0, c1};
    const float4 q = part[j][threadIdx.x % CL];
    c0 = __builtin_fmaf(q.x, c0, q.y);
    c1 = __builtin_fmaf(q.z, c1, q.w);
  }
  return in;
}

// The state that enters a segment: the given one through the pairs of the segments before.  Of several segments each
// takes the given one from its copy in the last segment's place, so that the state at the end may be written over it.
template <typename W>
__device__ __forceinline__ Two enter_segment(const ScanArgs& a, const W& w, const float* first) {
  Two h{0.0f, 0.0f};
  if (a.segments > 1) {
    const float2* p = a.pairs + (w.b * a.segments + a.segments - 1) * a.dim + w.cc;
    h = {p[0].y, p[w.d1].y};
  } else if (first) {
    h = {first[w.b * a.dim + w.cc], first[w.b * a.dim + w.cc + w.d1]};
  }
  for (int s = 0; s < w.seg; ++s) {
    const float2* p = a.pairs + (w.b * a.segments + s) * a.dim + w.cc;
    const float2 p0 = p[0], p1 = p[w.d1];
    h.a = __builtin_fmaf(p0.x, h.a, p0.y);
    h.b = __builtin_fmaf(p1.x, h.b, p1.y);
  }
  return h;
}

template <typename W>
__device__ __forceinline__ void put(float* to, const ScanArgs& a, const W& w, float v0, float v1) {
  if (w.have > 0) to[w.b * a.dim + w.c] = v0;
  if (w.have > 1) to[w.b * a.dim + w.c + 1] = v1;
}

// A token's (a, beta, sigmoid(i) x) of both channels -> (a, b).
template <typename T>
__device__ __forceinline__ void forward_of(Two x, Two r, Two i, Two rate, bool live, Two& a, Two& b) {
  const Decay d0 = decay_of(rate.a, sigmoid<kTail<T>>(r.a)), d1 = decay_of(rate.b, sigmoid<kTail<T>>(r.b));
  const float q0 = sigmoid<kTail<T>>(i.a), q1 = sigmoid<kTail<T>>(i.b);
  a = live ? Two{d0.a, d1.a} : Two{1.0f, 1.0f};
  b = live ? Two{__builtin_amdgcn_sqrtf(d0.w) * q0 * x.a, __builtin_amdgcn_sqrtf(d1.w) * q1 * x.b} : Two{0.0f, 0.0f};
}

// The 8-bit copy of a token's 128 channels, two to a lane of the wave.
template <bool ODD>
__device__ __forceinline__ void keep2(const ScanArgs& a, int plane, int64_t row, int c, int have, Two v) {
  float top = Max::of(have > 0 ? __builtin_fabsf(v.a) : 0.0f, have > 1 ? __builtin_fabsf(v.b) : 0.0f);
  top = over_lanes<Max, 64>(top);
  const float s = scale_of(top), inv = 1.0f / s;
  const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(v.a * inv, v.b * inv, 0, false);
  const int64_t at = plane * a.plane + row;
  uint8_t* p = a.keep + at * a.dim + c;
  if (have > 1) {
    const uint16_t h = static_cast<uint16_t>(w);
    __builtin_memcpy(p, &h, 2);
  } else if (ODD && have == 1) {
    *p = static_cast<uint8_t>(w);
  }
  if (threadIdx.x % 64 == 0) a.keep_scale[at * a.groups + c / kGroup] = s;
}

template <typename T, int CL, int R, int S, bool ODD, bool KEEP>
__global__ __launch_bounds__(CL * R) void gated_scan_fwd_kernel(ScanArgs a) {
  static_assert(!KEEP || CL == 64, "a scale's 128 channels are one wave's");
  __shared__ float4 part[2][R][CL];
  const Where<CL, ODD> w(a, false);
  const Two rate{rate_of(a.A_log, w.cc), rate_of(a.A_log, w.cc + w.d1)};
  Two carry = enter_segment(a, w, a.first);
  const int64_t begin = static_cast<int64_t>(w.seg) * a.seg_len;
  const int64_t end = begin + a.seg_len < a.seqlen ? begin + a.seg_len : a.seqlen;
  const T* x = static_cast<const T*>(a.x) + w.b * a.x_batch + w.cc;
  const T* r = static_cast<const T*>(a.r) + w.b * a.r_batch + w.cc;
  const T* i = static_cast<const T*>(a.i) + w.b * a.i_batch + w.cc;
  T* out = static_cast<T*>(a.out) + w.b * a.seqlen * a.dim + w.c;
  int turn = 0;
  for (int64_t t0 = begin; t0 < end; t0 += R * S, turn ^= 1) {
    const int64_t mine = t0 + w.run * S;
    Two av[S], bv[S];
    Pairs p{1.0f, 0.0f, 1.0f, 0.0f};
    if (t0 < w.n) {
      Two xv[S], rv[S], iv[S];
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const int64_t t = w.in(mine + k);
        xv[k] = load2<ODD>(x + t * a.x_token, w.d1);
        rv[k] = load2<ODD>(r + t * a.r_token, w.d1);
        iv[k] = load2<ODD>(i + t * a.i_token, w.d1);
      }
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const bool live = mine + k < w.n;
        forward_of<T>(xv[k], rv[k], iv[k], rate, live, av[k], bv[k]);
        then(p, av[k].a, bv[k].a, av[k].b, bv[k].b);
        if constexpr (KEEP)
          if (mine + k < end) {
            const int64_t row = w.b * a.seqlen + w.at(mine + k);
            const Two zero{0.0f, 0.0f};
            keep2<ODD>(a, 0, row, w.c, w.have, live ? xv[k] : zero);
            keep2<ODD>(a, 1, row, w.c, w.have, live ? rv[k] : zero);
            keep2<ODD>(a, 2, row, w.c, w.have, live ? iv[k] : zero);
          }
      }
    } else {
#pragma unroll
      for (int k = 0; k < S; ++k) av[k] = {1.0f, 1.0f}, bv[k] = {0.0f, 0.0f};
      if constexpr (KEEP)
        for (int k = 0; k < S; ++k)
          if (mine + k < end)
            for (int plane = 0; plane < 3; ++plane)
              keep2<ODD>(a, plane, w.b * a.seqlen + mine + k, w.c, w.have, Two{0.0f, 0.0f});
    }
    part[turn][w.run][threadIdx.x % CL] = make_float4(p.A0, p.H0, p.A1, p.H1);
    __syncthreads();
    Two h = enter<CL, R>(part[turn], w.run, carry.a, carry.b);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      h = {__builtin_fmaf(av[k].a, h.a, bv[k].a), __builtin_fmaf(av[k].b, h.b, bv[k].b)};
      const int64_t t = mine + k;
      if (t < end) {
        const Two y = t < w.n ? h : Two{0.0f, 0.0f};
        store2<ODD>(out + w.at(t) * a.dim, w.have, y);
        if constexpr (KEEP) keep2<ODD>(a, 3, w.b * a.seqlen + w.at(t), w.c, w.have, y);
      }
    }
  }
  if (a.end && w.seg == a.segments - 1 && w.run == 0) put(a.end, a, w, carry.a, carry.b);
}

// The last segment's pair, which nothing follows, holds the state given at the start.
template <typename W>
__device__ __forceinline__ void copy_first(const ScanArgs& a, const W& w, const float* first) {
  if (w.run != 0) return;
  float2* p = a.pairs + (w.b * a.segments + w.seg) * a.dim + w.c;
  const float* f = first + w.b * a.dim + w.c;
  if (w.have > 0) p[0] = make_float2(0.0f, first ? f[0] : 0.0f);
  if (w.have > 1) p[1] = make_float2(0.0f, first ? f[1] : 0.0f);
}

// The pairs of the segments but the last.  A run takes a contiguous share of the segment, and
// the shares are joined at the end.
template <typename T, int CL, int R, bool ODD>
__global__ __launch_bounds__(CL * R) void gated_scan_pairs_kernel(ScanArgs a) {
  __shared__ float4 part[R][CL];
  const Where<CL, ODD> w(a, false);
  if (w.seg == a.segments - 1) {
    copy_first(a, w, a.first);
    return;
  }
  const Two rate{rate_of(a.A_log, w.cc), rate_of(a.A_log, w.cc + w.d1)};
  const int64_t begin = static_cast<int64_t>(w.seg) * a.seg_len;
  const int share = (a.seg_len + R - 1) / R;
  const int64_t from = begin + w.run * share;
  int64_t to = from + share;
  if (to > begin + a.seg_len) to = begin + a.seg_len;
  if (to > w.n) to = w.n;
  const T* x = static_cast<const T*>(a.x) + w.b * a.x_batch + w.cc;
  const T* r = static_cast<const T*>(a.r) + w.b * a.r_batch + w.cc;
  const T* i = static_cast<const T*>(a.i) + w.b * a.i_batch + w.cc;
  Pairs p{1.0f, 0.0f, 1.0f, 0.0f};
#pragma unroll 8
  for (int64_t t = from; t < to; ++t) {
    const int64_t at = w.at(t);
    Two av, bv;
    forward_of<T>(load2<ODD>(x + at * a.x_token, w.d1), load2<ODD>(r + at * a.r_token, w.d1),
                  load2<ODD>(i + at * a.i_token, w.d1), rate, true, av, bv);
    then(p, av.a, bv.a, av.b, bv.b);
  }
  part[w.run][threadIdx.x % CL] = make_float4(p.A0, p.H0, p.A1, p.H1);
  __syncthreads();
  if (w.run != 0) return;
  for (int j = 1; j < R; ++j) {
    const float4 q = part[j][threadIdx.x % CL];
    then(p, q.x, q.y, q.z, q.w);
  }
  float2* to_pairs = a.pairs + (w.b * a.segments + w.seg) * a.dim + w.c;
  if (w.have > 0) to_pairs[0] = make_float2(p.A0, p.H0);
  if (w.have > 1) to_pairs[1] = make_float2(p.A1, p.H1);
}

// The gradient's reads of one token.
template <typename T, bool ODD, bool CODES>
struct Reads {
  const T *x, *r, *i, *h, *d;
  template <typename W>
  __device__ __forceinline__ Reads(const ScanArgs& a, const W& w) {
    x = static_cast<const T*>(a.x) + w.b * a.x_batch + w.cc;
    r = static_cast<const T*>(a.r) + w.b * a.r_batch + w.cc;
    i = static_cast<const T*>(a.i) + w.b * a.i_batch + w.cc;
    h = static_cast<const T*>(a.h) + w.b * a.seqlen * a.dim + w.cc;
    d = static_cast<const T*>(a.dout) + w.b * a.dout_batch + w.cc;
  }
  template <typename W>
  __device__ __forceinline__ Two code(const ScanArgs& a, const W& w, int plane, int64_t t) const {
    const int64_t at = plane * a.plane + w.b * a.seqlen + t;
    const float s = a.codes_scale[at * a.groups + w.cc / kGroup];
    const Two v = load2<ODD>(a.codes + at * a.dim + w.cc, w.d1);
    return {v.a * s, v.b * s};
  }
  template <typename W>
  __device__ __forceinline__ Two rv(const ScanArgs& a, const W& w, int64_t t) const {
    if constexpr (CODES) return code(a, w, 1, t);
    return load2<ODD>(r + t * a.r_token, w.d1);
  }
  template <typename W>
  __device__ __forceinline__ Two xv(const ScanArgs& a, const W& w, int64_t t) const {
    if constexpr (CODES) return code(a, w, 0, t);
    return load2<ODD>(x + t * a.x_token, w.d1);
  }
  template <typename W>
  __device__ __forceinline__ Two iv(const ScanArgs& a, const W& w, int64_t t) const {
    if constexpr (CODES) return code(a, w, 2, t);
    return load2<ODD>(i + t * a.i_token, w.d1);
  }
  // the state before the walk-back's token t: the next one's output, or the state at the start
  template <typename W>
  __device__ __forceinline__ Two before(const ScanArgs& a, const W& w, int64_t t, Two first) const {
    if (t + 1 >= w.n) return first;
    const int64_t at = w.at(t + 1);
    if constexpr (CODES) return code(a, w, 3, at);
    return load2<ODD>(h + at * a.dim, w.d1);
  }
  __device__ __forceinline__ Two dv(const ScanArgs& a, int d1, int64_t t) const { return load2<ODD>(d + t * a.dout_token, d1); }
};

// One channel of a token of the gradient: G is the gradient of its state.
struct TokenGrad {
  float dx, dr, di, dA;
};
template <bool TAIL>
__device__ __forceinline__ TokenGrad gradient_of(float G, const Decay& d, float p, float x, float i, float before) {
  const float q = sigmoid<TAIL>(i);
  // Below the normal numbers w counts as 2^-126: beta, under 2^-63, is then off by less than that, and its limit 0 is met.
  const float rs = __builtin_amdgcn_rsqf(__builtin_fmaxf(d.w, 1.17549435e-38f));
  const float beta = d.w * rs;
  const float gb = G * beta;
  TokenGrad g;
  g.dx = gb * q;
  g.di = g.dx * x * (1.0f - q);
  // d/d(log a), times log a = -y; log a / beta has the limit 0 at a = 1
  g.dA = G * d.a * d.y * __builtin_fmaf(q * x * d.a, rs, -before);
  // log a / beta = -y rs
  g.dr = g.dA * (1.0f - p);
  return g;
}

template <typename T, int CL, int R, int S, bool ODD, bool CODES>
__global__ __launch_bounds__(CL * R) void gated_scan_bwd_kernel(ScanArgs a) {
  __shared__ float4 part[2][R][CL];
  const Where<CL, ODD> w(a, true);
  const Two rate{rate_of(a.A_log, w.cc), rate_of(a.A_log, w.cc + w.d1)};
  Two carry = enter_segment(a, w, a.last);
  Two first{0.0f, 0.0f};
  if (a.first) first = {a.first[w.b * a.dim + w.cc], a.first[w.b * a.dim + w.cc + w.d1]};
  const int64_t begin = static_cast<int64_t>(w.seg) * a.seg_len;
  const int64_t end = begin + a.seg_len < a.seqlen ? begin + a.seg_len : a.seqlen;
  const Reads<T, ODD, CODES> reads(a, w);
  const int64_t row0 = w.b * a.seqlen;
  T* dx = static_cast<T*>(a.dx) + row0 * a.dim + w.c;
  T* dr = static_cast<T*>(a.dr) + row0 * a.dim + w.c;
  T* di = static_cast<T*>(a.di) + row0 * a.dim + w.c;
  Two dA{0.0f, 0.0f};
  int turn = 0;
  for (int64_t t0 = begin; t0 < end; t0 += R * S, turn ^= 1) {
    const int64_t mine = t0 + w.run * S;
    Two pv[S], dv[S], xv[S], iv[S], hv[S];
    Pairs p{1.0f, 0.0f, 1.0f, 0.0f};
    if (t0 < w.n) {
      Two rv[S];
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const int64_t t = w.in(mine + k);
        rv[k] = reads.rv(a, w, t);
        dv[k] = reads.dv(a, w.d1, t);
        xv[k] = reads.xv(a, w, t);
        iv[k] = reads.iv(a, w, t);
        hv[k] = reads.before(a, w, mine + k, first);
      }
#pragma unroll
      for (int k = 0; k < S; ++k) {
        pv[k] = {sigmoid<kTail<T>>(rv[k].a), sigmoid<kTail<T>>(rv[k].b)};
        const Decay d0 = decay_of(rate.a, pv[k].a), d1 = decay_of(rate.b, pv[k].b);
        if (mine + k < w.n) then(p, d0.a, d0.a * dv[k].a, d1.a, d1.a * dv[k].b);
      }
    }
    part[turn][w.run][threadIdx.x % CL] = make_float4(p.A0, p.H0, p.A1, p.H1);
    __syncthreads();
    Two c = enter<CL, R>(part[turn], w.run, carry.a, carry.b);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int64_t t = mine + k;
      if (t >= end) break;
      Two gx{0.0f, 0.0f}, gr{0.0f, 0.0f}, gi{0.0f, 0.0f};
      if (t < w.n) {
        const Decay d0 = decay_of(rate.a, pv[k].a), d1 = decay_of(rate.b, pv[k].b);
        const float G0 = dv[k].a + c.a, G1 = dv[k].b + c.b;
        const TokenGrad g0 = gradient_of<kTail<T>>(G0, d0, pv[k].a, xv[k].a, iv[k].a, hv[k].a);
        const TokenGrad g1 = gradient_of<kTail<T>>(G1, d1, pv[k].b, xv[k].b, iv[k].b, hv[k].b);
        gx = {g0.dx, g1.dx}, gr = {g0.dr, g1.dr}, gi = {g0.di, g1.di};
        dA.a += g0.dA, dA.b += g1.dA;
        c = {d0.a * G0, d1.a * G1};
      }
      const int64_t at = w.at(t) * a.dim;
      store2<ODD>(dx + at, w.have, gx);
      store2<ODD>(dr + at, w.have, gr);
      store2<ODD>(di + at, w.have, gi);
    }
  }
  if (a.end && w.seg == a.segments - 1 && w.run == 0) put(a.end, a, w, carry.a, carry.b);
  // this segment's share of A_log's gradient, its runs in a fixed order
  __syncthreads();
  part[0][w.run][threadIdx.x % CL] = make_float4(dA.a, dA.b, 0.0f, 0.0f);
  __syncthreads();
  if (w.run != 0) return;
  for (int j = 1; j < R; ++j) dA.a += part[0][j][threadIdx.x].x, dA.b += part[0][j][threadIdx.x].y;
  float* to = a.part + (w.b * a.segments + w.seg) * a.dim + w.c;
  if (w.have > 0) to[0] = dA.a;
  if (w.have > 1) to[1] = dA.b;
}

template <typename T, int CL, int R, bool ODD, bool CODES>
__global__ __launch_bounds__(CL * R) void gated_scan_bwd_pairs_kernel(ScanArgs a) {
  __shared__ float4 part[R][CL];
  const Where<CL, ODD> w(a, true);
  if (w.seg == a.segments - 1) {
    copy_first(a, w, a.last);
    return;
  }
  const Two rate{rate_of(a.A_log, w.cc), rate_of(a.A_log, w.cc + w.d1)};
  const int64_t begin = static_cast<int64_t>(w.seg) * a.seg_len;
  const int share = (a.seg_len + R - 1) / R;
  const int64_t from = begin + w.run * share;
  int64_t to = from + share;
  if (to > begin + a.seg_len) to = begin + a.seg_len;
  if (to > w.n) to = w.n;
  const Reads<T, ODD, CODES> reads(a, w);
  Pairs p{1.0f, 0.0f, 1.0f, 0.0f};
#pragma unroll 8
  for (int64_t t = from; t < to; ++t) {
    const int64_t at = w.at(t);
    const Two r = reads.rv(a, w, at), d = reads.dv(a, w.d1, at);
    const Decay d0 = decay_of(rate.a, sigmoid<kTail<T>>(r.a)), d1 = decay_of(rate.b, sigmoid<kTail<T>>(r.b));
    then(p, d0.a, d0.a * d.a, d1.a, d1.a * d.b);
  }
  part[w.run][threadIdx.x % CL] = make_float4(p.A0, p.H0, p.A1, p.H1);
  __syncthreads();
  if (w.run != 0) return;
  for (int j = 1; j < R; ++j) {
    const float4 q = part[j][threadIdx.x % CL];
    then(p, q.x, q.y, q.z, q.w);
  }
  float2* to_pairs = a.pairs + (w.b * a.segments + w.seg) * a.dim + w.c;
  if (w.have > 0) to_pairs[0] = make_float2(p.A0, p.H0);
  if (w.have > 1) to_pairs[1] = make_float2(p.A1, p.H1);
}

// dA_log: 32 channels of a workgroup, 8 shares of the partial rows, joined in LDS in a fixed order.
__global__ __launch_bounds__(256) void gated_scan_rate_kernel(const float* __restrict__ part, float* __restrict__ to,
                                                              int64_t rows, int dim) {
  __shared__ float s[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), share = threadIdx.x >> 5;
  float t = 0.0f;
  if (c < dim)
#pragma unroll 4
    for (int64_t i = share; i < rows; i += 8) t += part[i * dim + c];
  s[share][threadIdx.x & 31] = t;
  __syncthreads();
  if (share == 0 && c < dim) {
    for (int i = 1; i < 8; ++i) t += s[i][threadIdx.x];
    to[c] = t;
  }
}

struct StepArgs {
  const void *x, *r, *i;
  const float* A_log;
  float* state;
  const int32_t* slots;
  void* out;
  int64_t x_batch, r_batch, i_batch, batch, pool;
  int dim;
};

template <typename T>
__global__ __launch_bounds__(64) void gated_scan_step_kernel(StepArgs a) {
  const int64_t b = blockIdx.y;
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= a.dim) return;
  const int64_t slot = a.slots ? a.slots[b] : b;
  T* out = static_cast<T*>(a.out) + b * a.dim + c;
  if (slot < 0 || slot >= a.pool) {
    store1(out, 0.0f);
    return;
  }
  const float x = load1(static_cast<const T*>(a.x) + b * a.x_batch + c);
  const float p = sigmoid<kTail<T>>(load1(static_cast<const T*>(a.r) + b * a.r_batch + c));
  const float q = sigmoid<kTail<T>>(load1(static_cast<const T*>(a.i) + b * a.i_batch + c));
  const Decay d = decay_of(rate_of(a.A_log, c), p);
  float* h = a.state + slot * a.dim + c;
  const float v = __builtin_fmaf(d.a, *h, __builtin_amdgcn_sqrtf(d.w) * q * x);
  *h = v;
  store1(out, v);
}

// How a call is cut: tiles of channels, and segments where the sequences' tiles are too few for the chip.
constexpr int kRuns = 8, kTokens = 16, kGradTokens = 8;
void cut(ScanArgs& a, int channels, int tokens) {
  a.tiles = (a.dim + channels - 1) / channels;
  const int block = kRuns * tokens;
  const int64_t blocks = (a.seqlen + block - 1) / block, walks = a.batch * a.tiles;
  int64_t segments = (1024 + walks - 1) / walks;
  if (segments > (blocks + 1) / 2) segments = (blocks + 1) / 2;
  if (segments < 1) segments = 1;
  a.seg_len = static_cast<int>((blocks + segments - 1) / segments * block);
  a.segments = static_cast<int>((a.seqlen + a.seg_len - 1) / a.seg_len);
}

bool shape_ok(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch >= 1 && seqlen >= 1 && dim >= 1 && batch < (int64_t{1} << 24) && seqlen < (int64_t{1} << 30) &&
         dim < (int64_t{1} << 20) && batch * seqlen < (int64_t{1} << 40) / dim;
}

bool strides_ok(const int64_t* s) { return s[0] >= 0 && s[1] >= 0 && s[0] <= (int64_t{1} << 40) && s[1] < (int64_t{1} << 24); }

bool dtype_ok(vmscan_dtype d) { return d == VMSCAN_F32 || d == VMSCAN_BF16; }

ScanArgs sizes(int64_t batch, int64_t seqlen, int64_t dim, int channels, int tokens) {
  ScanArgs a{};
  a.batch = batch, a.seqlen = seqlen, a.dim = static_cast<int>(dim), a.plane = batch * seqlen;
  a.groups = static_cast<int>((dim + kGroup - 1) / kGroup);
  cut(a, channels, tokens);
  return a;
}

// States may be updated in place (one buffer) and must not overlap otherwise.
bool states_ok(const ScanArgs& a, const float* to, const float* from, bool same) {
  if (!to || !from) return true;
  const uintptr_t t = reinterpret_cast<uintptr_t>(to), f = reinterpret_cast<uintptr_t>(from);
  const uintptr_t n = static_cast<uintptr_t>(a.batch) * a.dim * sizeof(float);
  return t == f ? same : t + n <= f || f + n <= t;
}

size_t pairs_bytes(const ScanArgs& a) {
  return a.segments > 1 ? static_cast<size_t>(a.batch) * a.segments * a.dim * sizeof(float2) : 0;
}
size_t part_bytes(const ScanArgs& a) { return static_cast<size_t>(a.batch) * a.segments * a.dim * sizeof(float); }
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

template <typename T, bool ODD>
void launch_fwd(const ScanArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.batch * a.segments * a.tiles)), block(64 * kRuns);
  if (a.segments > 1) hipLaunchKernelGGL((gated_scan_pairs_kernel<T, 64, kRuns, ODD>), grid, block, 0, stream, a);
  if (a.keep)
    hipLaunchKernelGGL((gated_scan_fwd_kernel<T, 64, kRuns, kTokens, ODD, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((gated_scan_fwd_kernel<T, 64, kRuns, kTokens, ODD, false>), grid, block, 0, stream, a);
}

template <typename T, bool ODD, bool CODES>
void launch_bwd(const ScanArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.batch * a.segments * a.tiles)), block(64 * kRuns);
  if (a.segments > 1)
    hipLaunchKernelGGL((gated_scan_bwd_pairs_kernel<T, 64, kRuns, ODD, CODES>), grid, block, 0, stream, a);
  hipLaunchKernelGGL((gated_scan_bwd_kernel<T, 64, kRuns, kGradTokens, ODD, CODES>), grid, block, 0, stream, a);
  hipLaunchKernelGGL(gated_scan_rate_kernel, dim3(static_cast<unsigned>((a.dim + 31) / 32)), dim3(256), 0, stream, a.part,
                     a.dA_log, a.batch * a.segments, a.dim);
}

}  // namespace

extern "C" {

size_t vmscan_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  if (!shape_ok(batch, seqlen, dim)) return 0;
  return pairs_bytes(sizes(batch, seqlen, dim, 2 * 64, kTokens));
}

vmscan_status vmscan_gated_scan_fwd(const void* x, const int64_t* x_strides, const void* r, const int64_t* r_strides,
                                    const void* i, const int64_t* i_strides, const float* A_log,
                                    const float* initial_state, const int32_t* lengths, int reverse, void* out,
                                    float* final_state, void* keep_codes, float* keep_scale, int64_t batch,
                                    int64_t seqlen, int64_t dim, vmscan_dtype dtype, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  if (!x || !x_strides || !r || !r_strides || !i || !i_strides || !A_log || !out) return VMSCAN_ERR_NULL;
  if ((keep_codes == nullptr) != (keep_scale == nullptr)) return VMSCAN_ERR_NULL;
  if (!shape_ok(batch, seqlen, dim) || !strides_ok(x_strides) || !strides_ok(r_strides) || !strides_ok(i_strides))
    return VMSCAN_ERR_SHAPE;
  if (!dtype_ok(dtype) || (reverse != 0 && reverse != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  for (const void* p : {x, r, i})
    if (!aligned_to(p, e)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(A_log), static_cast<const void*>(initial_state),
                        static_cast<const void*>(lengths), static_cast<const void*>(final_state),
                        static_cast<const void*>(keep_scale)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  if (!aligned_to(out, 16) || !aligned_to(workspace, 16) || !aligned_to(keep_codes, 16)) return VMSCAN_ERR_ALIGN;
  ScanArgs a = sizes(batch, seqlen, dim, 2 * 64, kTokens);
  if (batch * a.segments * a.tiles >= (int64_t{1} << 23)) return VMSCAN_ERR_SHAPE;
  if (!states_ok(a, final_state, initial_state, true)) return VMSCAN_ERR_UNSUPPORTED;
  if (pairs_bytes(a) && (!workspace || workspace_bytes < pairs_bytes(a))) return VMSCAN_ERR_WORKSPACE;
  a.x = x, a.r = r, a.i = i, a.A_log = A_log, a.first = initial_state, a.lengths = lengths, a.out = out;
  a.end = final_state, a.keep = static_cast<uint8_t*>(keep_codes), a.keep_scale = keep_scale, a.reverse = reverse;
  a.pairs = static_cast<float2*>(workspace);
  a.x_batch = x_strides[0], a.x_token = x_strides[1], a.r_batch = r_strides[0], a.r_token = r_strides[1];
  a.i_batch = i_strides[0], a.i_token = i_strides[1];
  const bool odd = a.dim % 2 != 0;
  if (dtype == VMSCAN_F32)
    odd ? launch_fwd<float, true>(a, stream) : launch_fwd<float, false>(a, stream);
  else
    odd ? launch_fwd<uint16_t, true>(a, stream) : launch_fwd<uint16_t, false>(a, stream);
  return launched();
}

size_t vmscan_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  if (!shape_ok(batch, seqlen, dim)) return 0;
  const ScanArgs a = sizes(batch, seqlen, dim, 2 * 64, kGradTokens);
  return round16(pairs_bytes(a)) + part_bytes(a);
}

vmscan_status vmscan_gated_scan_bwd(const void* x, const int64_t* x_strides, const void* r, const int64_t* r_strides,
                                    const void* i, const int64_t* i_strides, const void* h, const void* codes,
                                    const float* codes_scale, const float* A_log, const float* initial_state,
                                    const int32_t* lengths, int reverse, const void* dout, const int64_t* dout_strides,
                                    const float* dfinal_state, void* dx, void* dr, void* di, float* dA_log,
                                    float* dinitial_state, int64_t batch, int64_t seqlen, int64_t dim,
                                    vmscan_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!A_log || !dout || !dout_strides || !dx || !dr || !di || !dA_log) return VMSCAN_ERR_NULL;
  if ((codes == nullptr) != (codes_scale == nullptr)) return VMSCAN_ERR_NULL;
  if (!codes && (!x || !x_strides || !r || !r_strides || !i || !i_strides || !h)) return VMSCAN_ERR_NULL;
  if (codes && (x || r || i || h)) return VMSCAN_ERR_UNSUPPORTED;  // one of the two forms
  if (!shape_ok(batch, seqlen, dim) || !strides_ok(dout_strides)) return VMSCAN_ERR_SHAPE;
  if (!codes && (!strides_ok(x_strides) || !strides_ok(r_strides) || !strides_ok(i_strides))) return VMSCAN_ERR_SHAPE;
  if (!dtype_ok(dtype) || (reverse != 0 && reverse != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  for (const void* p : {x, r, i, h, dout})
    if (!aligned_to(p, e)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(A_log), static_cast<const void*>(initial_state),
                        static_cast<const void*>(lengths), static_cast<const void*>(dfinal_state),
                        static_cast<const void*>(dA_log), static_cast<const void*>(dinitial_state),
                        static_cast<const void*>(codes_scale)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(dx), static_cast<const void*>(dr), static_cast<const void*>(di),
                        static_cast<const void*>(workspace)})
    if (!aligned_to(p, 16)) return VMSCAN_ERR_ALIGN;
  ScanArgs a = sizes(batch, seqlen, dim, 2 * 64, kGradTokens);
  if (batch * a.segments * a.tiles >= (int64_t{1} << 23)) return VMSCAN_ERR_SHAPE;
  if (!states_ok(a, dinitial_state, dfinal_state, true) || !states_ok(a, dinitial_state, initial_state, false))
    return VMSCAN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < vmscan_gated_scan_bwd_workspace_bytes(batch, seqlen, dim)) return VMSCAN_ERR_WORKSPACE;
  a.x = x, a.r = r, a.i = i, a.h = h, a.codes = static_cast<const uint8_t*>(codes), a.codes_scale = codes_scale;
  a.A_log = A_log, a.first = initial_state, a.last = dfinal_state, a.lengths = lengths, a.reverse = reverse;
  a.dout = dout, a.dx = dx, a.dr = dr, a.di = di, a.dA_log = dA_log, a.end = dinitial_state;
  a.pairs = static_cast<float2*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + round16(pairs_bytes(a)));
  if (!codes) {
    a.x_batch = x_strides[0], a.x_token = x_strides[1], a.r_batch = r_strides[0], a.r_token = r_strides[1];
    a.i_batch = i_strides[0], a.i_token = i_strides[1];
  }
  a.dout_batch = dout_strides[0], a.dout_token = dout_strides[1];
  const bool odd = a.dim % 2 != 0;
  if (dtype == VMSCAN_F32) {
    if (codes)
      odd ? launch_bwd<float, true, true>(a, stream) : launch_bwd<float, false, true>(a, stream);
    else
      odd ? launch_bwd<float, true, false>(a, stream) : launch_bwd<float, false, false>(a, stream);
  } else {
    if (codes)
      odd ? launch_bwd<uint16_t, true, true>(a, stream) : launch_bwd<uint16_t, false, true>(a, stream);
    else
      odd ? launch_bwd<uint16_t, true, false>(a, stream) : launch_bwd<uint16_t, false, false>(a, stream);
  }
  return launched();
}

vmscan_status vmscan_gated_scan_step(const void* x, int64_t x_stride, const void* r, int64_t r_stride, const void* i,
                                     int64_t i_stride, const float* A_log, float* state, const int32_t* slots, void* out,
                                     int64_t batch, int64_t pool, int64_t dim, vmscan_dtype dtype, hipStream_t stream) {
  if (!x || !r || !i || !A_log || !state || !out) return VMSCAN_ERR_NULL;
  if (batch < 1 || batch > 65535 || pool < 1 || pool >= (int64_t{1} << 40) || dim < 1 || dim >= (int64_t{1} << 20) ||
      (!slots && pool != batch))
    return VMSCAN_ERR_SHAPE;
  for (int64_t s : {x_stride, r_stride, i_stride})
    if (s < 0 || s > (int64_t{1} << 40)) return VMSCAN_ERR_SHAPE;
  if (!dtype_ok(dtype)) return VMSCAN_ERR_UNSUPPORTED;
  const size_t e = dtype == VMSCAN_F32 ? 4 : 2;
  for (const void* p : {x, r, i, static_cast<const void*>(out)})
    if (!aligned_to(p, e)) return VMSCAN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(A_log), static_cast<const void*>(state), static_cast<const void*>(slots)})
    if (!aligned_to(p, 4)) return VMSCAN_ERR_ALIGN;
  const StepArgs a{x, r, i, A_log, state, slots, out, x_stride, r_stride, i_stride, batch, pool, static_cast<int>(dim)};
  const dim3 grid(static_cast<unsigned>((dim + 63) / 64), static_cast<unsigned>(batch));
  if (dtype == VMSCAN_F32)
    hipLaunchKernelGGL((gated_scan_step_kernel<float>), grid, dim3(64), 0, stream, a);
  else
    hipLaunchKernelGGL((gated_scan_step_kernel<uint16_t>), grid, dim3(64), 0, stream, a);
  return launched();
}

}  // extern "C"
