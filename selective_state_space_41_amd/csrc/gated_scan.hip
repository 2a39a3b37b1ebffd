// Gated linear recurrence with one state per channel: forward, gradient and single tokens.  What is computed is
// stated in include/vmscan.h.
//
// A workgroup owns 128 neighbouring channels, two to a lane, of a chunk of R * S tokens; a wave owns a run of S of
// them, whose (decay, input) pairs stay in its registers.  The pairs of a run are joined to one pair, the R pairs of a
// chunk meet in LDS and become the chunk's pair, which is published for the chunks after it; the state that enters
// the chunk comes from those before it in the same way, and every run then walks its tokens from the state that
// enters it.  So inputs are read once and outputs written once however long the sequence is.
//
// Between chunks: a chunk waits for the published pairs of the chunks before it in its group of 4 R and for the state
// that the last chunk of the group before published.  The order of the joins is fixed, whatever arrives first.  Workgroups take their chunks in the order in which they start (a counter), chunks of all sequences by their
// place, so a chunk only waits for chunks that running workgroups hold: every wait ends.  A published value is one
// 64-bit word that is written at once; a first launch sets all of them to a value that no result has.
//
// Measured (whole calls): 128 x 197 x 384 bfloat16 kept in 8 bits 41 us for 118 MB, without the copies 26; 8 x 6085 x 768
// ragged, from a state, 65 us, where a copy of the live inputs and all outputs takes 48; gradient of 32 x 3136 x 512 from 8
// bits 162 us for 623 MB, of which the scan's launch takes 150; gradient of 20001 x 195 float32 61 us for 125 MB.  Bound by HBM and, where a
// call has few workgroups (the last case: 626 for 512 places), by a chunk's chain of load, join, wait and store.  Vector
// instructions take 70 % of the large gradient's cycles, yet 7 % fewer of them changed nothing.  Runs and tokens: 8 x 16
// and 8 x 8 leave four waves a SIMD; the forward with 4 x 16, 16 x 8, 8 x 8 took 79, 76, 78 us instead of 64 on the second
// case, the gradient with 4 x 8, 7 x 8, 16 x 8 193, 190, 195 instead of 162.  Persistent workgroups that take their next
// chunk early were slower (the chunks after them wait longer), a second level of groups gained nothing.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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
  uint32_t* status;              // the wait status word and, behind it, the counter of started workgroups
  uint64_t* pairs;               // per chain and chunk: 128 channels' pairs
  uint64_t* states;              // per chain and group of chunks: the states after it
  float* part;                   // gradient: per sequence and chunk, channels' sums for A_log
  int64_t x_batch, x_token, r_batch, r_token, i_batch, i_token, dout_batch, dout_token;
  int64_t batch, seqlen, plane;  // plane: tokens of a plane of the 8-bit copies
  int dim, groups, tiles;
  int chains, chunks;            // chains: sequences' tiles of 128 channels; chunks of a sequence
  int reverse;
};

constexpr int kTile = 128;          // channels of a workgroup
// Chunks whose pairs are joined one by one, four by each of a workgroup's R waves.
__host__ __device__ constexpr int groups_of(int chunks, int R) { return (chunks + 4 * R - 1) / (4 * R); }
constexpr uint64_t kNothing = ~uint64_t{0};
constexpr int kPatience = 1 << 22;  // polls of a wait that should have ended long ago

// Two neighbouring channels.
struct Two {
  float a, b;
};
// How a row's channels lie in the lanes' pairs.
enum Layout {
  kPairs,   // an even number of channels (of those kept in 8 bits: a multiple of 4)
  kShifted, // any number over 1: a lane whose second channel would be past the end loads the pair before
  kSingle   // one channel
};
// As loaded: a bfloat16 or 8-bit pair stays one register until it is used.
struct RawB {
  uint32_t w;
};
struct Raw8 {
  uint32_t w;
};
// `shift`: the lane's first channel (or, past the last one, what stands for it) is the second of the pair that it loaded.
template <Layout L>
__device__ __forceinline__ RawB shifted(RawB r, bool shift) {
  if (L == kShifted && shift) r.w = r.w >> 16 | (r.w & 0xffff0000u);
  return r;
}
template <Layout L>
__device__ __forceinline__ Two shifted(Two r, bool shift) {
  if (L == kShifted && shift) r.a = r.b;
  return r;
}
template <Layout L>
__device__ __forceinline__ Two values(RawB r, bool shift) {
  r = shifted<L>(r, shift);
  return {__uint_as_float(r.w << 16), __uint_as_float(r.w & 0xffff0000u)};
}
template <Layout L>
__device__ __forceinline__ Two values(Two r, bool shift) {
  return shifted<L>(r, shift);
}
template <Layout L>
__device__ __forceinline__ Two values(Raw8 r, bool shift) {
  if constexpr (L == kShifted) r.w = shift ? r.w >> 8 : r.w;
  const auto v = __builtin_amdgcn_cvt_pk_f32_fp8(r.w, false);
  return {v[0], v[1]};
}
// ONCE: what is read is not needed again (the gradient's inputs: 32 x 3136 x 512 from 8 bits takes 164 us instead of
// 171, 16 x 3136 x 256 in float32 102 instead of 113; the forward gains nothing).
template <Layout L, bool ONCE = false>
__device__ __forceinline__ RawB load2(const uint16_t* p) {
  if constexpr (L == kSingle) return {p[0] * 0x10001u};
  if constexpr (ONCE) return {load_once<uint32_t>(p)};
  uint32_t w;
  __builtin_memcpy(&w, p, 4);
  return {w};
}
template <Layout L, bool ONCE = false>
__device__ __forceinline__ Two load2(const float* p) {
  if constexpr (L == kSingle) return {p[0], p[0]};
  f32x2 v;
  if constexpr (ONCE)
    v = load_once<f32x2>(p);
  else
    __builtin_memcpy(&v, p, 8);
  return {v.x, v.y};
}
template <Layout L, bool ONCE = true>
__device__ __forceinline__ Raw8 load2(const uint8_t* p) {
  if constexpr (L == kSingle) return {p[0] * 0x101u};
  return {load_once<uint16_t>(p)};
}
template <typename T, Layout L>
using Raw = decltype(load2<L>(static_cast<const T*>(nullptr)));
// n: channels that exist, 1 at least.
template <Layout L>
__device__ __forceinline__ void store2(uint16_t* p, int n, Two v) {
  if (L != kPairs && n == 1) {
    store1(p, v.a);
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 w = __builtin_convertvector((f32x2{v.a, v.b}), bf16x2);  // nearest even, both at once
    __builtin_memcpy(p, &w, 4);
  }
}
template <Layout L>
__device__ __forceinline__ void store2(float* p, int n, Two v) {
  if (L != kPairs && n == 1) {
    *p = v.a;
  } else {
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

// 1 / (1 + 2^t)
__device__ __forceinline__ float sigmoid_of(float t) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t)); }

// A channel's rate e^A_log, as the factor of the decay's exponent and of v below.  A rate over 2^125 counts as that, which
// leaves both factors finite: its decay is 0 under any gate sigmoid(r) over 2^-118 already, and an infinite rate times a zero
// decay or gate would be a NaN.
constexpr float kMaxRate = 0x1p125f;
struct Rate {
  float e, v;  // -rate log2(e), 2 rate
};
__device__ __forceinline__ Rate rate_of(const float* A_log, int c) {
  const float all = __builtin_amdgcn_exp2f(A_log[c] * kLog2e), r = all > kMaxRate ? kMaxRate : all;  // a NaN stays
  return {r * -kLog2e, r + r};
}
__device__ __forceinline__ float decay_of(Rate rate, float p) { return __builtin_amdgcn_exp2f(rate.e * p); }

// w = 1 - a^2 = 1 - e^-v for v = 2 rate sigmoid(r) >= 0 and a = e^(-v/2).  Below v = 1/4 by v times a polynomial for
// (1 - e^-v) / v, interpolated at Chebyshev points with the value 1 at 0 (within 0.2 * 2^-24 of it; the first four
// terms of the series would leave 23); above, one fused multiply-add.
__device__ __forceinline__ float gain_of(float a, float v) {
  float s = __builtin_fmaf(v, 0x1.f6c6ecp-8f, -0x1.547fd4p-5f);
  s = __builtin_fmaf(v, s, 0x1.5552aep-3f);
  s = __builtin_fmaf(v, s, -0x1.fffffep-2f);
  s = __builtin_fmaf(v, s, 1.0f);
  s *= v;
  asm volatile("" : "+v"(s));  // both are computed: the compiler would branch around the polynomial
  return v < 0.25f ? s : __builtin_fmaf(-a, a, 1.0f);
}

template <typename T>
constexpr bool kTail = sizeof(T) == 4;

__device__ __forceinline__ int tokens_of(const ScanArgs& a, int64_t b) {
  const int all = static_cast<int>(a.seqlen);
  if (!a.lengths) return all;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > all ? all : n;
}

// What a workgroup and a wave work on.  Tokens are counted along the walk; `back` walks turn the count around within
// the row's n tokens, and what lies past them keeps its place.
template <int R, int S, Layout L>
struct Where {
  int64_t b;
  int n, mine, left, rest;  // the sequence's tokens, the wave's first; live and written ones from there on (any sign)
  int chain, chunk, run, tile, lane;
  int c, have;              // first channel, channels that exist
  int cc, c0, c1;           // where the lane loads, and the channels that its values belong to (ones that exist)
  bool back, shift;
  __device__ __forceinline__ Where(const ScanArgs& a, uint32_t unit, bool turn) {
    chunk = __builtin_amdgcn_readfirstlane(unit / static_cast<uint32_t>(a.chains));
    chain = static_cast<int>(unit - static_cast<uint32_t>(chunk) * static_cast<uint32_t>(a.chains));
    const int row = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(chain) / static_cast<uint32_t>(a.tiles));
    tile = chain - row * a.tiles;
    b = row;
    n = __builtin_amdgcn_readfirstlane(tokens_of(a, b));
    run = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    lane = threadIdx.x % 64;
    mine = chunk * (R * S) + run * S;
    left = n - mine;
    rest = static_cast<int>(a.seqlen) - mine;
    c = tile * kTile + lane * 2;
    have = a.dim - c;
    const int top = L == kSingle ? 0 : a.dim - 2;
    cc = c < top ? c : top;
    shift = L == kShifted && c >= a.dim - 1;
    c1 = L == kSingle ? 0 : cc + 1;
    c0 = shift ? c1 : cc;
    back = (a.reverse != 0) != turn;
  }
  __device__ __forceinline__ int begin() const { return chunk * (R * S); }
  // The chunk that holds the walk's last token (the first one of a row without tokens).
  __device__ __forceinline__ bool last() const { return begin() + R * S >= n; }
  // The place of the wave's token k, live or not.
  __device__ __forceinline__ int at(int k) const { return back && k < left ? n - 1 - mine - k : mine + k; }
};

// A lane's channels in a uniform row: a scalar base and a 32-bit offset.
template <typename T>
__device__ __forceinline__ T* in_row(T* row, int c) {
  using Byte = typename std::conditional<std::is_const<T>::value, const char, char>::type;
  using Global = Byte __attribute__((address_space(1)));
  const uint64_t at = reinterpret_cast<uint64_t>(row);
  const uint32_t low = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));  // (an int: not to be widened as one)
  const uint32_t high = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
  Global* base = (Global*)reinterpret_cast<Byte*>(static_cast<uint64_t>(high) << 32 | low);
  asm("" : "+s"(base));  // the sum is the load's or store's own, not a 64-bit addition in every lane
  return reinterpret_cast<T*>((Byte*)(base + static_cast<uint32_t>(c) * static_cast<uint32_t>(sizeof(T))));
}

// The rows of the wave's live tokens, one after another along the walk.
template <typename T>
struct Rows {
  T* row;
  int64_t step;
  template <typename W>
  __device__ __forceinline__ Rows(T* tokens, int64_t token, const W& w, int from = 0)
      : row(tokens + (w.back ? w.n - 1 - w.mine - from : w.mine + from) * token), step(w.back ? -token : token) {}
  __device__ __forceinline__ T* next(int c) {
    T* p = in_row(row, c);
    row += step;
    return p;
  }
};

// (decay, input) pairs after one another: h -> A h + H.
struct Pairs {
  float A0, H0, A1, H1;
};
__device__ __forceinline__ void then(Pairs& p, float a0, float h0, float a1, float h1) {
  p.H0 = __builtin_fmaf(a0, p.H0, h0), p.A0 *= a0;
  p.H1 = __builtin_fmaf(a1, p.H1, h1), p.A1 *= a1;
}
__device__ __forceinline__ Two through(const Pairs& p, Two h) {
  return {__builtin_fmaf(p.A0, h.a, p.H0), __builtin_fmaf(p.A1, h.b, p.H1)};
}

// Published words.  A NaN is published as the usual one, so that no result is kNothing.
__device__ __forceinline__ uint32_t word_of(float v) { return v == v ? __float_as_uint(v) : 0x7fc00000u; }
__device__ __forceinline__ void publish(uint64_t* at, float lo, float hi) {
  __hip_atomic_store(at, static_cast<uint64_t>(word_of(hi)) << 32 | word_of(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 await(const uint64_t* at, uint64_t v, uint32_t* status) {
  for (int i = 0; v == kNothing && i < kPatience; ++i) {
    __builtin_amdgcn_s_sleep(1);
    v = peek(at);
  }
  if (v == kNothing) *status = 1;
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// What a workgroup's waves share.
template <int R>
struct Shared {
  float4 part[R][64];    // the runs' pairs
  float4 before[R][64];  // the pairs of the chunks before, four by four
  float2 base[64];       // the state before those
};

// The workgroup's unit of work, of chains times chunks: where chunks wait for others, by the order of their start.
__device__ __forceinline__ uint32_t unit_of(const ScanArgs& a) {
  __shared__ uint32_t ticket;
  if (a.chunks == 1) return blockIdx.x;
  if (threadIdx.x == 0) ticket = __hip_atomic_fetch_add(a.status + 1, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(ticket);
}

// The state that enters this wave's run, from its pair p.  `first` is the state at the sequence's start; `after` gets the
// state after the sequence's last token.  Each wave joins four of the chunks before, and all of them the waves' pairs.
template <int R, int S, Layout L>
__device__ __forceinline__ Two enter(const ScanArgs& a, const Where<R, S, L>& w, const Pairs& p, Shared<R>& s,
                                     const float* first, float* after) {
  constexpr int kEach = 4, kGroupChunks = kEach * R;
  const int lane = w.lane, group = w.chunk / kGroupChunks, begin = group * kGroupChunks;
  uint64_t* mine = a.pairs + (static_cast<int64_t>(w.chain) * a.chunks + w.chunk) * kTile + lane;
  uint64_t* state = a.states + (static_cast<int64_t>(w.chain) * groups_of(a.chunks, R) + group) * 64 + lane;
  const bool last = w.last();
  // what the chunks before have published by now; the others are waited for below
  const int from = begin + w.run * kEach, many = w.chunk - from < kEach ? w.chunk - from : kEach;
  const uint64_t* theirs = mine - static_cast<int64_t>(w.chunk - from) * kTile;
  uint64_t v[kEach][2], base = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (k < many) v[k][0] = peek(theirs + k * kTile), v[k][1] = peek(theirs + k * kTile + 64);
  if (w.run == R - 1 && group > 0) base = peek(state - 64);
  s.part[w.run][lane] = make_float4(p.A0, p.H0, p.A1, p.H1);
  __syncthreads();
  Pairs all{1.0f, 0.0f, 1.0f, 0.0f};
  if (w.run == 0) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float4 q = s.part[j][lane];
      then(all, q.x, q.y, q.z, q.w);
    }
    if (group == 0) {
      Two h{0.0f, 0.0f};
      if (w.chunk == 0 && first) h = {first[w.b * a.dim + w.c0], first[w.b * a.dim + w.c1]};
      s.base[lane] = make_float2(h.a, h.b);
      if (w.chunk == 0) {  // the state after it, whatever enters: no other chunk reads the state at the start
        const Two end = through(all, h);
        all = {0.0f, end.a, 0.0f, end.b};
      }
    }
    if (!last) {
      publish(mine, all.A0, all.H0);
      publish(mine + 64, all.A1, all.H1);
    }
  }
  Pairs q{1.0f, 0.0f, 1.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (k < many) {
      const float2 p0 = await(theirs + k * kTile, v[k][0], a.status), p1 = await(theirs + k * kTile + 64, v[k][1], a.status);
      then(q, p0.x, p0.y, p1.x, p1.y);
    }
  if (many > 0) s.before[w.run][lane] = make_float4(q.A0, q.H0, q.A1, q.H1);
  if (w.run == R - 1 && group > 0) s.base[lane] = await(state - 64, base, a.status);
  __syncthreads();
  const float2 b = s.base[lane];
  Two h{b.x, b.y};
#pragma unroll
  for (int j = 0; j < R; ++j)
    if (begin + j * kEach < w.chunk) {
      const float4 t = s.before[j][lane];
      h = {__builtin_fmaf(t.x, h.a, t.y), __builtin_fmaf(t.z, h.b, t.w)};
    }
  if (w.run == 0) {
    const Two end = through(all, h);
    if (!last && w.chunk == begin + kGroupChunks - 1) publish(state, end.a, end.b);
    if (last && after) {
      if (w.have > 0) after[w.b * a.dim + w.c] = end.a;
      if (w.have > 1) after[w.b * a.dim + w.c + 1] = end.b;
    }
  }
  for (int j = 0; j < w.run; ++j) {
    const float4 t = s.part[j][lane];
    h = {__builtin_fmaf(t.x, h.a, t.y), __builtin_fmaf(t.z, h.b, t.w)};
  }
  return h;
}

// Two tokens' pairs of 8-bit codes in a register, the first's in its lower half, become four neighbouring channels of
// one token (the first in even lanes, the second in odd ones): half the stores, of 4 bytes.  (The gradient's loads gain
// nothing that way: 167 us instead of 161 on 32 x 3136 x 512.)
__device__ __forceinline__ uint32_t trade(uint32_t w, uint32_t selector) {
  const uint32_t other = __float_as_uint(dpp<0xb1>(__uint_as_float(w)));
  return __builtin_amdgcn_perm(other, w, selector);
}
__device__ __forceinline__ uint32_t trade_selector(int lane) { return lane & 1 ? 0x03020706u : 0x05040100u; }
// A lane's place in the rows of two tokens: four channels of its token's row, from the lower of the two.
__device__ __forceinline__ int trade_place(int lane, int c, bool back, int dim) {
  return (c & ~3) + (((lane & 1) != 0) != back ? dim : 0);
}

// The largest magnitudes of four tokens' 128 channels, two to a lane, as unsigned numbers, whose order is that of the
// magnitudes and in which a NaN is the largest.  They are found together: each exchange of half the lanes leaves one
// register for two, so that a row of 16 lanes ends up with one token: 0, 2, 1, 3.  (A lane past the last channel holds
// channels that exist.)
__device__ __forceinline__ uint32_t larger(uint32_t x, uint32_t y) { return x > y ? x : y; }
template <typename MAX>
__device__ __forceinline__ uint32_t by_rows(const uint32_t (&m)[4], MAX&& max) {
  u32x2 r = __builtin_amdgcn_permlane32_swap(m[0], m[1], false, false);
  const uint32_t m01 = max(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(m[2], m[3], false, false);
  const uint32_t m23 = max(r[0], r[1]);
  r = __builtin_amdgcn_permlane16_swap(m01, m23, false, false);
  return max(r[0], r[1]);
}
__device__ __forceinline__ uint32_t in_row16(uint32_t t) {
  t = larger(t, __float_as_uint(dpp<0xb1>(__uint_as_float(t))));
  t = larger(t, __float_as_uint(dpp<0x4e>(__uint_as_float(t))));
  t = larger(t, __float_as_uint(dpp<0x141>(__uint_as_float(t))));
  return larger(t, __float_as_uint(dpp<0x140>(__uint_as_float(t))));
}
__device__ __forceinline__ uint32_t tops(RawB a, RawB b, RawB c, RawB d) {  // both channels at once, as 16-bit numbers
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const uint32_t m[4] = {a.w & 0x7fff7fffu, b.w & 0x7fff7fffu, c.w & 0x7fff7fffu, d.w & 0x7fff7fffu};
  const uint32_t t = by_rows(m, [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x), __builtin_bit_cast(u16x2, y)));
  });
  return in_row16(larger(t & 0xffff0000u, t << 16));
}
__device__ __forceinline__ uint32_t tops(Two a, Two b, Two c, Two d) {
  const auto one = [](Two v) { return larger(__float_as_uint(v.a) & 0x7fffffffu, __float_as_uint(v.b) & 0x7fffffffu); };
  const uint32_t m[4] = {one(a), one(b), one(c), one(d)};
  return in_row16(by_rows(m, larger));
}

// Where the 8-bit copies of a plane go, four tokens after four.
template <Layout L>
struct Kept {
  uint8_t* codes;
  float* scale;
  template <typename W>
  __device__ __forceinline__ Kept(const ScanArgs& a, const W& w, int plane) {
    const int64_t first = plane * a.plane + w.b * a.seqlen;
    codes = a.keep + first * a.dim, scale = a.keep_scale + first * a.groups + w.tile;
  }
  // FULL: the run's tokens k to k + 3 are live; else `many` of them are written, live or not.
  template <bool FULL, typename W>
  __device__ __forceinline__ void put(const ScanArgs& a, const W& w, int k, int many, uint32_t top, const Two (&v)[4]) const {
    // as scale_of and its reciprocal, by products (one unit in the last place)
    const float big = __uint_as_float(top), q = big * (1.0f / kFp8Max);
    const float s = big == 0.0f ? 1.0f : q < kMinScale ? kMinScale : q, inv = __builtin_amdgcn_rcpf(s);
    constexpr int kRow[4] = {0, 32, 16, 48};
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), kRow[j]));
    const int token = ((w.lane >> 5) & 1) | ((w.lane >> 3) & 2);
    if constexpr (FULL) {
      const int low = w.back ? w.at(k + 3) : w.at(k);
      float* row = in_row(scale + static_cast<int64_t>(low) * a.groups, (w.back ? 3 - token : token) * a.groups);
      if (w.lane % 16 == 0) *row = s;
    } else {
      if (w.lane % 16 == 0 && token < many) scale[static_cast<int64_t>(w.at(k + token)) * a.groups] = s;
    }
    if constexpr (FULL && L == kPairs) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(v[j].a * f[j], v[j].b * f[j], 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(v[j + 1].a * f[j + 1], v[j + 1].b * f[j + 1], c, true);
        c = trade(c, trade_selector(w.lane));
        const int low = w.back ? w.at(k + j + 1) : w.at(k + j);
        uint8_t* to = in_row(codes + static_cast<int64_t>(low) * a.dim, trade_place(w.lane, w.c, w.back, a.dim));
        if (w.have > 0) store_away(to, c);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!FULL && j >= many) break;
        const uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(v[j].a * f[j], v[j].b * f[j], 0, false);
        uint8_t* to = in_row(codes + static_cast<int64_t>(w.at(k + j)) * a.dim, w.c);
        if (L != kPairs && w.have == 1)
          *to = static_cast<uint8_t>(c);
        else if (w.have > 0)
          store_away(to, static_cast<uint16_t>(c));
      }
    }
  }
};

// Before the chunk's entering state is known: a run's decays and inputs, joined to a pair, and its 8-bit copies.  FULL:
// all S tokens are live.
template <bool FULL, typename T, int R, int S, Layout L, bool KEEP>
__device__ __forceinline__ Pairs take_run(const ScanArgs& a, const Where<R, S, L>& w, Two (&av)[S], Two (&bv)[S]) {
  const Rate rate0 = rate_of(a.A_log, w.c0), rate1 = rate_of(a.A_log, w.c1);
  Rows<const T> x(static_cast<const T*>(a.x) + w.b * a.x_batch, a.x_token, w);
  Rows<const T> r(static_cast<const T*>(a.r) + w.b * a.r_batch, a.r_token, w);
  Rows<const T> i(static_cast<const T*>(a.i) + w.b * a.i_batch, a.i_token, w);
  Raw<T, L> raw[3][S];
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if (FULL || k < w.left) {
      raw[0][k] = load2<L>(x.next(w.cc));
      raw[1][k] = load2<L>(r.next(w.cc));
      raw[2][k] = load2<L>(i.next(w.cc));
    } else {
      raw[0][k] = raw[1][k] = raw[2][k] = {};
    }
  }
  if constexpr (KEEP) {
#pragma unroll
    for (int k = 0; k < S; k += 4) {
#pragma unroll
      for (int plane = 0; plane < 3; ++plane) {
        Raw<T, L>* in = raw[plane] + k;
        if (FULL || k < w.rest)
          Kept<L>(a, w, plane).template put<FULL>(a, w, k, w.rest - k,
                                                  tops(shifted<L>(in[0], w.shift), shifted<L>(in[1], w.shift),
                                                       shifted<L>(in[2], w.shift), shifted<L>(in[3], w.shift)),
                                                  {values<L>(in[0], w.shift), values<L>(in[1], w.shift),
                                                   values<L>(in[2], w.shift), values<L>(in[3], w.shift)});
        __builtin_amdgcn_sched_barrier(0);  // one after another: registers
      }
    }
  }
  Pairs p{1.0f, 0.0f, 1.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if (FULL || k < w.left) {
      const Two x = values<L>(raw[0][k], w.shift), r = values<L>(raw[1][k], w.shift), i = values<L>(raw[2][k], w.shift);
      const float p0 = sigmoid<kTail<T>>(r.a), p1 = sigmoid<kTail<T>>(r.b);
      av[k] = {decay_of(rate0, p0), decay_of(rate1, p1)};
      bv[k] = {__builtin_amdgcn_sqrtf(gain_of(av[k].a, rate0.v * p0)) * sigmoid<kTail<T>>(i.a) * x.a,
               __builtin_amdgcn_sqrtf(gain_of(av[k].b, rate1.v * p1)) * sigmoid<kTail<T>>(i.b) * x.b};
      then(p, av[k].a, bv[k].a, av[k].b, bv[k].b);
    } else {
      av[k] = {1.0f, 1.0f}, bv[k] = {0.0f, 0.0f};
    }
  }
  return p;
}

// A run's states from the one that enters it.
template <bool FULL, typename T, int R, int S, Layout L, bool KEEP>
__device__ __forceinline__ void walk_run(const ScanArgs& a, const Where<R, S, L>& w, const Two (&av)[S], const Two (&bv)[S],
                                         Two h) {
  const int64_t row0 = w.b * a.seqlen;
  T* out = static_cast<T*>(a.out) + row0 * a.dim;
  Rows<T> rows(out, a.dim, w);
  if (!KEEP && w.have <= 0) return;  // 8-bit copies take all lanes
#pragma unroll
  for (int k = 0; k < S; k += 4) {
    Two y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h = {__builtin_fmaf(av[k + j].a, h.a, bv[k + j].a), __builtin_fmaf(av[k + j].b, h.b, bv[k + j].b)};
      y[j] = FULL || k + j < w.left ? h : Two{0.0f, 0.0f};
      if (FULL || k + j < w.rest) {
        T* to = FULL ? rows.next(w.c) : in_row(out + static_cast<int64_t>(w.at(k + j)) * a.dim, w.c);
        if (!KEEP || w.have > 0) store2<L>(to, w.have, y[j]);
      }
    }
    if constexpr (KEEP) {
      if (FULL || k < w.rest) Kept<L>(a, w, 3).template put<FULL>(a, w, k, w.rest - k, tops(y[0], y[1], y[2], y[3]), y);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <typename T, int R, int S, Layout L, bool KEEP>
__global__ __launch_bounds__(64 * R, 4) void gated_scan_fwd_kernel(ScanArgs a) {
  static_assert(S % 4 == 0, "8-bit copies are made four tokens at a time");
  __shared__ Shared<R> shared;
  const Where<R, S, L> w(a, unit_of(a), false);
  Two av[S], bv[S], h{0.0f, 0.0f};
  const Pairs p = w.left >= S ? take_run<true, T, R, S, L, KEEP>(a, w, av, bv) : take_run<false, T, R, S, L, KEEP>(a, w, av, bv);
  if (w.chunk == 0 || w.begin() < w.n) h = enter<R, S, L>(a, w, p, shared, a.first, a.end);
  if (w.left >= S)
    walk_run<true, T, R, S, L, KEEP>(a, w, av, bv, h);
  else
    walk_run<false, T, R, S, L, KEEP>(a, w, av, bv, h);
}

// A uniform load through the scalar cache, of what no kernel that runs writes.
__device__ __forceinline__ float scalar_load(const float* p) {
  return *reinterpret_cast<const float __attribute__((address_space(4)))*>(reinterpret_cast<uintptr_t>(p));
}

// One channel of a token of the gradient: G is the gradient of its state, p and q the gates' sigmoids, a its decay.
struct TokenGrad {
  float dx, dr, di, dA, c;  // dr and dA: half of dA; c: what reaches the state before
};
__device__ __forceinline__ TokenGrad gradient_of(float G, Rate rate, float p, float a, float x, float q, float before) {
  const float v = rate.v * p, w = gain_of(a, v);
  // Below the normal numbers w counts as 2^-126: beta, under 2^-63, is then off by less than that, and its limit 0 is met.
  const float rs = __builtin_amdgcn_rsqf(__builtin_fmaxf(w, 1.17549435e-38f));
  const float gb = G * (w * rs), u = q * x;
  TokenGrad g;
  g.c = a * G;
  g.dx = gb * q;
  g.di = gb * u * (1.0f - q);
  // d/d(log a), times log a = -v / 2; log a / beta = -v rs / 2 has the limit 0 at a = 1
  g.dA = g.c * v * __builtin_fmaf(u * a, rs, -before);
  g.dr = g.dA * __builtin_fmaf(p, -0.5f, 0.5f);
  return g;
}

// What the gradient reads of a wave's tokens.
template <typename T, int S, Layout L, bool CODES>
struct Taken {
  Raw<typename std::conditional<CODES, uint8_t, T>::type, L> in[4][S];  // x, r, i, h
  Raw<T, L> d[S];
  Two p[S];                       // sigmoid(r)
  float scale[CODES ? 4 : 1][S];  // of the 8-bit forms, uniform
  bool shift;
  __device__ __forceinline__ Two of(int plane, int k) const {
    const Two v = values<L>(in[plane][k], shift);
    if constexpr (CODES) return Two{v.a * scale[plane][k], v.b * scale[plane][k]};
    return v;
  }
  __device__ __forceinline__ Two gate(int plane, int k) const {
    const Two v = values<L>(in[plane][k], shift);
    if constexpr (CODES) {  // the scale and log2(e) in one factor: what that rounds is far under a code's 2^-4
      const float f = scale[plane][k] * -kLog2e;
      return {sigmoid_of(v.a * f), sigmoid_of(v.b * f)};
    }
    return {sigmoid<kTail<T>>(v.a), sigmoid<kTail<T>>(v.b)};
  }
};

template <bool FULL, typename T, int R, int S, Layout L, bool CODES>
__device__ __forceinline__ Pairs take_back(const ScanArgs& a, const Where<R, S, L>& w, Rate rate0, Rate rate1,
                                           Taken<T, S, L, CODES>& v) {
  const int64_t row0 = w.b * a.seqlen;
  Rows<const T> d(static_cast<const T*>(a.dout) + w.b * a.dout_batch, a.dout_token, w);
  v.shift = w.shift;
  // the state before a token is the output of the walk-back's next one; the very last's is the state given
  const auto there = [&](int plane, int k) { return (FULL && (plane < 3 || k < S - 1)) || k + (plane == 3) < w.left; };
  const auto scales = [&](int plane) {
    return Rows<const float>(a.codes_scale + (plane * a.plane + row0) * a.groups + w.tile, a.groups, w, plane == 3);
  };
  const auto codes = [&](int plane) { return Rows<const uint8_t>(a.codes + (plane * a.plane + row0) * a.dim, a.dim, w, plane == 3); };
  if constexpr (CODES) {
    Rows<const uint8_t> c[4] = {codes(0), codes(1), codes(2), codes(3)};
    Rows<const float> scale[4] = {scales(0), scales(1), scales(2), scales(3)};
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (FULL || k < w.left) v.d[k] = load2<L, true>(d.next(w.cc));
#pragma unroll
      for (int plane = 0; plane < 4; ++plane)
        if (there(plane, k)) {
          v.in[plane][k] = load2<L>(c[plane].next(w.cc));
          // the scales' loads between the codes': all of them first cost 10 us of 160, all of them last 20
          v.scale[plane][k] = scalar_load(scale[plane].next(0));
        }
    }
  } else {
    Rows<const T> in[4] = {Rows<const T>(static_cast<const T*>(a.x) + w.b * a.x_batch, a.x_token, w),
                           Rows<const T>(static_cast<const T*>(a.r) + w.b * a.r_batch, a.r_token, w),
                           Rows<const T>(static_cast<const T*>(a.i) + w.b * a.i_batch, a.i_token, w),
                           Rows<const T>(static_cast<const T*>(a.h) + row0 * a.dim, a.dim, w, 1)};
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (FULL || k < w.left) v.d[k] = load2<L, true>(d.next(w.cc));
#pragma unroll
      for (int plane = 0; plane < 4; ++plane)
        if (there(plane, k)) v.in[plane][k] = load2<L, true>(in[plane].next(w.cc));
    }
  }
  Pairs p{1.0f, 0.0f, 1.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if (FULL || k < w.left) {
      const Two d = values<L>(v.d[k], w.shift);
      v.p[k] = v.gate(1, k);
      const float a0 = decay_of(rate0, v.p[k].a), a1 = decay_of(rate1, v.p[k].b);
      then(p, a0, a0 * d.a, a1, a1 * d.b);
    }
  }
  return p;
}

// A run's gradients from c, the gradient that the walk-back brings; returns the run's sums for A_log.
template <bool FULL, typename T, int R, int S, Layout L, bool CODES>
__device__ __forceinline__ Two walk_back(const ScanArgs& a, const Where<R, S, L>& w, Rate rate0, Rate rate1,
                                         const Taken<T, S, L, CODES>& v, Two c) {
  const int64_t row0 = w.b * a.seqlen;
  T *dx = static_cast<T*>(a.dx) + row0 * a.dim, *dr = static_cast<T*>(a.dr) + row0 * a.dim,
    *di = static_cast<T*>(a.di) + row0 * a.dim;
  Rows<T> px(dx, a.dim, w), pr(dr, a.dim, w), pi(di, a.dim, w);
  Two dA{0.0f, 0.0f}, first{0.0f, 0.0f};
  if (w.have <= 0) return dA;
  if (w.left <= S && a.first) first = {a.first[w.b * a.dim + w.c0], a.first[w.b * a.dim + w.c1]};
#pragma unroll
  for (int k = 0; k < S; ++k) {
    Two gx{0.0f, 0.0f}, gr{0.0f, 0.0f}, gi{0.0f, 0.0f};
    if (FULL || k < w.left) {
      const Two d = values<L>(v.d[k], w.shift), x = v.of(0, k), q = v.gate(2, k), p = v.p[k];
      const Two h = (FULL && k < S - 1) || k + 1 < w.left ? v.of(3, k) : first;
      const TokenGrad g0 = gradient_of(d.a + c.a, rate0, p.a, decay_of(rate0, p.a), x.a, q.a, h.a);
      const TokenGrad g1 = gradient_of(d.b + c.b, rate1, p.b, decay_of(rate1, p.b), x.b, q.b, h.b);
      gx = {g0.dx, g1.dx}, gr = {g0.dr, g1.dr}, gi = {g0.di, g1.di};
      dA.a += g0.dA, dA.b += g1.dA;
      c = {g0.c, g1.c};
    }
    if (FULL) {
      store2<L>(px.next(w.c), w.have, gx);
      store2<L>(pr.next(w.c), w.have, gr);
      store2<L>(pi.next(w.c), w.have, gi);
    } else if (k < w.rest) {
      const int64_t at = static_cast<int64_t>(w.at(k)) * a.dim;
      store2<L>(in_row(dx + at, w.c), w.have, gx);
      store2<L>(in_row(dr + at, w.c), w.have, gr);
      store2<L>(in_row(di + at, w.c), w.have, gi);
    }
  }
  return {0.5f * dA.a, 0.5f * dA.b};
}

template <typename T, int R, int S, Layout L, bool CODES>
__global__ __launch_bounds__(64 * R, 4) void gated_scan_bwd_kernel(ScanArgs a) {
  __shared__ Shared<R> shared;
  const Where<R, S, L> w(a, unit_of(a), true);
  const Rate rate0 = rate_of(a.A_log, w.c0), rate1 = rate_of(a.A_log, w.c1);
  Taken<T, S, L, CODES> v;
  const Pairs p = w.left >= S ? take_back<true, T, R, S, L, CODES>(a, w, rate0, rate1, v)
                              : take_back<false, T, R, S, L, CODES>(a, w, rate0, rate1, v);
  Two c{0.0f, 0.0f};
  if (w.chunk == 0 || w.begin() < w.n) c = enter<R, S, L>(a, w, p, shared, a.last, a.end);
  Two dA = w.left >= S ? walk_back<true, T, R, S, L, CODES>(a, w, rate0, rate1, v, c)
                       : walk_back<false, T, R, S, L, CODES>(a, w, rate0, rate1, v, c);
  // this chunk's share of A_log's gradient, its runs in a fixed order
  __syncthreads();
  shared.part[w.run][w.lane] = make_float4(dA.a, dA.b, 0.0f, 0.0f);
  __syncthreads();
  if (w.run != 0) return;
  for (int j = 1; j < R; ++j) dA.a += shared.part[j][w.lane].x, dA.b += shared.part[j][w.lane].y;
  float2* to = reinterpret_cast<float2*>(a.part + (w.b * a.chunks + w.chunk) * (a.tiles * kTile) + w.c);
  *to = make_float2(dA.a, dA.b);  // channels past the last are not summed
}

// Sets the published words to kNothing and the two words before them to 0: 1.3 to 7.6 us, 4.9 in the mean of the profiled calls.
__global__ __launch_bounds__(256) void gated_scan_clear_kernel(uint32_t* status, uint64_t* words, int64_t n) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 2;
  if (i == 0) status[0] = status[1] = 0;
  if (i < n) *reinterpret_cast<ulonglong2*>(words + i) = make_ulonglong2(kNothing, kNothing);
}

// dA_log: the sum of `rows` partial rows, tiles * 128 channels each: a workgroup takes 4 * COLS channels, COLS lanes of 4 and
// 1024 / COLS shares of the rows; a wave's shares are joined by exchanges, the waves' in LDS, in a fixed order.
constexpr int kRateCols = 2;  // 1 to 8 within 1 us of each other
__global__ __launch_bounds__(1024) void gated_scan_rate_kernel(const float* __restrict__ part, float* __restrict__ to,
                                                               int64_t rows, int64_t stride, int dim) {
  __shared__ __align__(16) float4 s[16][kRateCols];
  const int cx = threadIdx.x % kRateCols, share = threadIdx.x / kRateCols;
  const float* p = part + blockIdx.x * (4 * kRateCols) + cx * 4;
  float v[4] = {};
#pragma unroll 4
  for (int64_t i = share; i < rows; i += 1024 / kRateCols) {
    const float4 t = *reinterpret_cast<const float4*>(p + i * stride);
    v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
  }
#pragma unroll
  for (int m = kRateCols; m < 64; m *= 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += __shfl_xor(v[k], m);
  }
  if (threadIdx.x % 64 < kRateCols) s[threadIdx.x / 64][cx] = make_float4(v[0], v[1], v[2], v[3]);
  __syncthreads();
  if (threadIdx.x < 4 * kRateCols) {
    const int c = blockIdx.x * (4 * kRateCols) + threadIdx.x;
    const float* f = reinterpret_cast<const float*>(s) + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += f[w * 4 * kRateCols];
    if (c < dim) to[c] = t;
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

// One token of each sequence: a lane a channel, 64 channels a workgroup, so that a few sequences reach many CUs.  Latency:
// 2.5 us for 1 x 384, 4 for 256 x 1536 (5 MB), under calls of 8.7.
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
  const Rate rate = rate_of(a.A_log, c);
  const float decay = decay_of(rate, p);
  float* h = a.state + slot * a.dim + c;
  const float v = __builtin_fmaf(decay, *h, __builtin_amdgcn_sqrtf(gain_of(decay, rate.v * p)) * q * x);
  *h = v;
  store1(out, v);
}

// Waves of a workgroup and tokens of a wave's run.
constexpr int kRuns = 8;
constexpr int kTokens = 16, kGradTokens = 8;

bool shape_ok(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch >= 1 && seqlen >= 1 && dim >= 1 && batch < (int64_t{1} << 24) && seqlen < (int64_t{1} << 30) &&
         dim < (int64_t{1} << 20) && batch * seqlen < (int64_t{1} << 40) / dim;
}

bool strides_ok(const int64_t* s) { return s[0] >= 0 && s[1] >= 0 && s[0] <= (int64_t{1} << 40) && s[1] < (int64_t{1} << 24); }

bool dtype_ok(vmscan_dtype d) { return d == VMSCAN_F32 || d == VMSCAN_BF16; }

// A call's sizes and where its workspace's parts begin: the status words, the published words, the gradient's rows.
struct Plan {
  ScanArgs a{};
  bool ok = false;
  int64_t words = 0;
  size_t bytes = 0, part_at = 0;
  Plan(int64_t batch, int64_t seqlen, int64_t dim, bool gradient) {
    if (!shape_ok(batch, seqlen, dim)) return;
    const int tokens = gradient ? kGradTokens : kTokens;
    a.batch = batch, a.seqlen = seqlen, a.dim = static_cast<int>(dim), a.plane = batch * seqlen;
    a.groups = a.tiles = static_cast<int>((dim + kTile - 1) / kTile);
    static_assert(kGroup == kTile, "a tile's channels share a scale");
    const int64_t chains = batch * a.tiles, chunks = (seqlen + kRuns * tokens - 1) / (kRuns * tokens);
    if (chains * chunks >= (int64_t{1} << 23)) return;  // a launch holds less than 2^32 threads
    a.chains = static_cast<int>(chains), a.chunks = static_cast<int>(chunks);
    if (chunks > 1) {
      words = chains * (chunks * kTile + groups_of(static_cast<int>(chunks), kRuns) * 64);
      bytes = 16 + static_cast<size_t>(words) * sizeof(uint64_t);
    }
    if (gradient) {
      part_at = bytes;
      bytes += static_cast<size_t>(batch) * chunks * a.tiles * kTile * sizeof(float);
    }
    ok = true;
  }
  void place(void* workspace) {
    char* p = static_cast<char*>(workspace);
    a.status = reinterpret_cast<uint32_t*>(p);
    a.pairs = reinterpret_cast<uint64_t*>(p + 16);
    a.states = a.pairs + static_cast<int64_t>(a.chains) * a.chunks * kTile;
    a.part = reinterpret_cast<float*>(p + part_at);
  }
  // The word that a wait sets when it gives up; a call of one chunk waits for nothing and has none.
  const void* status() const { return words ? a.status : nullptr; }
  void clear(hipStream_t stream) const {
    if (words)
      hipLaunchKernelGGL(gated_scan_clear_kernel, dim3(static_cast<unsigned>((words + 511) / 512)), dim3(256), 0, stream,
                         a.status, a.pairs, words);
  }
  dim3 grid() const { return dim3(static_cast<unsigned>(a.chains * a.chunks)); }
};

// States may be updated in place (one buffer) and must not overlap otherwise.
bool states_ok(const ScanArgs& a, const float* to, const float* from, bool same) {
  if (!to || !from) return true;
  const uintptr_t t = reinterpret_cast<uintptr_t>(to), f = reinterpret_cast<uintptr_t>(from);
  const uintptr_t n = static_cast<uintptr_t>(a.batch) * a.dim * sizeof(float);
  return t == f ? same : t + n <= f || f + n <= t;
}

template <typename T, Layout L>
void launch_fwd(const Plan& p, hipStream_t stream) {
  p.clear(stream);
  if (p.a.keep)
    hipLaunchKernelGGL((gated_scan_fwd_kernel<T, kRuns, kTokens, L, true>), p.grid(), dim3(64 * kRuns), 0, stream, p.a);
  else
    hipLaunchKernelGGL((gated_scan_fwd_kernel<T, kRuns, kTokens, L, false>), p.grid(), dim3(64 * kRuns), 0, stream, p.a);
}

template <typename T, Layout L, bool CODES>
void launch_bwd(const Plan& p, hipStream_t stream) {
  p.clear(stream);
  hipLaunchKernelGGL((gated_scan_bwd_kernel<T, kRuns, kGradTokens, L, CODES>), p.grid(), dim3(64 * kRuns), 0, stream, p.a);
  hipLaunchKernelGGL(gated_scan_rate_kernel, dim3(static_cast<unsigned>((p.a.dim + 4 * kRateCols - 1) / (4 * kRateCols))), dim3(1024), 0, stream, p.a.part,
                     p.a.dA_log, p.a.batch * p.a.chunks, static_cast<int64_t>(p.a.tiles) * kTile, p.a.dim);
}

// keep: 8-bit copies are stored four channels at once
Layout layout_of(int dim, bool keep) { return dim == 1 ? kSingle : dim % (keep ? 4 : 2) ? kShifted : kPairs; }

template <typename T>
void dispatch_fwd(const Plan& p, hipStream_t stream) {
  switch (layout_of(p.a.dim, p.a.keep != nullptr)) {
    case kPairs: return launch_fwd<T, kPairs>(p, stream);
    case kShifted: return launch_fwd<T, kShifted>(p, stream);
    case kSingle: return launch_fwd<T, kSingle>(p, stream);
  }
}
template <typename T, bool CODES>
void dispatch_bwd(const Plan& p, hipStream_t stream) {
  switch (layout_of(p.a.dim, false)) {
    case kPairs: return launch_bwd<T, kPairs, CODES>(p, stream);
    case kShifted: return launch_bwd<T, kShifted, CODES>(p, stream);
    case kSingle: return launch_bwd<T, kSingle, CODES>(p, stream);
  }
}

}  // namespace

extern "C" {

size_t vmscan_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  return Plan(batch, seqlen, dim, false).bytes;
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
  Plan plan(batch, seqlen, dim, false);
  if (!plan.ok) return VMSCAN_ERR_SHAPE;
  ScanArgs& a = plan.a;
  if (!states_ok(a, final_state, initial_state, true)) return VMSCAN_ERR_UNSUPPORTED;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return VMSCAN_ERR_WORKSPACE;
  plan.place(workspace);
  a.x = x, a.r = r, a.i = i, a.A_log = A_log, a.first = initial_state, a.lengths = lengths, a.out = out;
  a.end = final_state, a.keep = static_cast<uint8_t*>(keep_codes), a.keep_scale = keep_scale, a.reverse = reverse;
  a.x_batch = x_strides[0], a.x_token = x_strides[1], a.r_batch = r_strides[0], a.r_token = r_strides[1];
  a.i_batch = i_strides[0], a.i_token = i_strides[1];
  if (dtype == VMSCAN_F32)
    dispatch_fwd<float>(plan, stream);
  else
    dispatch_fwd<uint16_t>(plan, stream);
  return finish_call(launched(), plan.status(), stream);
}

size_t vmscan_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  return Plan(batch, seqlen, dim, true).bytes;
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
  Plan plan(batch, seqlen, dim, true);
  if (!plan.ok) return VMSCAN_ERR_SHAPE;
  ScanArgs& a = plan.a;
  if (!states_ok(a, dinitial_state, dfinal_state, true) || !states_ok(a, dinitial_state, initial_state, false))
    return VMSCAN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < plan.bytes) return VMSCAN_ERR_WORKSPACE;
  plan.place(workspace);
  a.x = x, a.r = r, a.i = i, a.h = h, a.codes = static_cast<const uint8_t*>(codes), a.codes_scale = codes_scale;
  a.A_log = A_log, a.first = initial_state, a.last = dfinal_state, a.lengths = lengths, a.reverse = reverse;
  a.dout = dout, a.dx = dx, a.dr = dr, a.di = di, a.dA_log = dA_log, a.end = dinitial_state;
  if (!codes) {
    a.x_batch = x_strides[0], a.x_token = x_strides[1], a.r_batch = r_strides[0], a.r_token = r_strides[1];
    a.i_batch = i_strides[0], a.i_token = i_strides[1];
  }
  a.dout_batch = dout_strides[0], a.dout_token = dout_strides[1];
  if (dtype == VMSCAN_F32)
    codes ? dispatch_bwd<float, true>(plan, stream) : dispatch_bwd<float, false>(plan, stream);
  else
    codes ? dispatch_bwd<uint16_t, true>(plan, stream) : dispatch_bwd<uint16_t, false>(plan, stream);
  return finish_call(launched(), plan.status(), stream);
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
