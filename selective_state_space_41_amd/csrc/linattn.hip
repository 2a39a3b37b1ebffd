// Linear attention with a decay for each head: forward over sequences, gradient, single tokens.
// What is computed is stated in include/vmscan.h.
//
// Per head the state is a matrix S [dk, dv] and token t does S = e^{g_t} S + k_t v_t^T, o_t = scale
// S^T q_t.  Over a block of C tokens with G_i = g_1 + .. + g_i and the state S entering it, that is
//   o_i  = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j),
//   S'   = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T:
// four matrix products per block, on the matrix cores, with float32 accumulators.  Every exponent
// is a sum of logarithms over the tokens between two positions, so nothing overflows for decays
// however strong; the running sums are taken in float64 and kept as a head and a tail in float32,
// because a difference of two of them is a small number between large ones.
//
// A workgroup walks the blocks of one sequence and head, or of a segment of it when there are too few
// (sequence, head) pairs to fill the chip: then a first pass sums each segment's own state, a small
// prefix kernel makes the state entering each, and the walk starts from there.
//
// Layouts.  All products use the 16 x 16 (x 32) matrix instructions, whose operands hold 8 elements
// of the contracted index per lane and whose results hold 4 consecutive rows of one column.  The
// contracted index may be taken in any order as long as both operands agree, so a result (a tile of
// the masked scores) becomes an operand of the next product in the register it is in, in the order
// 16 t + 4 (lane / 16) + r; the other operand, whose contracted index is the token, is read from
// the row-major tile with the transposing LDS read, which gives that order.  Tiles in LDS: K, V (in
// the gradient also Q, dO) [token][channel], the state [dk][dv]; the forward's queries, which only one
// wave reads, go from global memory straight to operands.  The float32 path has the same structure with
// the 16 x 16 x 4 float32 instruction, eight per product, and plain LDS reads.
//
// Rounding for bfloat16 activations.  Everything is float32 until an output's one rounding.  An operand that is
// not a plain activation (the state and its gradient, the scores and theirs, weighted keys and queries) enters the bfloat16
// products as three bfloat16 numbers, which hold all of its 24 bits.  With two (16 bits, up to 2^-18 of a term) an
// output whose terms cancel to 2^-12 of themselves was off by 1 % instead of its rounding's 0.2 %, and the decays'
// gradient by 2.6e-6 of its largest value instead of under 5e-7.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "vmscan.h"

namespace {

using namespace vmscan_internal;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog = -1e4f;  // e^-1e4 is 0 in float32; keeps sums of -inf finite

struct Frag32 {
  float v[8];
};
template <typename T>
struct FragOf {
  using type = bf16x8;
};
template <>
struct FragOf<float> {
  using type = Frag32;
};
template <typename T>
using Frag = typename FragOf<T>::type;

__device__ __forceinline__ f32x4 mma(const bf16x8& a, const bf16x8& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag32& a, const Frag32& b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
  return c;
}

// LDS tiles are [rows][D] without padding; the 16-byte runs of a row lie in an order that depends on the
// row, so that the products' accesses meet no bank twice (the padded tiles that this replaced lost 40 % of
// their LDS cycles to conflicts; the 8-byte writes of states and scores still lose 16 to 18 % in the kernels that
// have them).  256 bytes are served at a time, one word from each of 64 banks: 16 rows of
// one run (row operands), and 8 rows of two neighbouring runs, rows 0 .. 7 or 0 .. 3 and 8 .. 11 (column
// operands).  256 / row bytes rows (at least 1) lie side by side; row r's run c is at place c ^ m, m from the
// bits k of r above those: all k differ in m, and the k of such 8 rows differ in m / 2.  (Float32 columns are
// read word by word, rows r, 4 + r, 8 + r, 12 + r of four runs: there m = k.)
template <typename T, int D>
__device__ __forceinline__ int run_mask(int r) {
  constexpr int kRuns = D * static_cast<int>(sizeof(T)) / 16;  // 4 .. 32
  constexpr int kSide = kRuns < 16 ? 16 / kRuns : 1;
  constexpr int kBits = kRuns == 4 ? 2 : kRuns == 8 ? 3 : 4;
  constexpr int kTop = kBits - 1;
  const int k = (r / kSide) & ((1 << kBits) - 1);
  if constexpr (sizeof(T) == 4) return k;
  else return (((k & ((1 << kTop) - 1)) ^ ((k >> kTop) << (kTop - 1))) << 1) | (k >> kTop);
}
template <typename T, int D>
__device__ __forceinline__ int place(int r, int col) {  // in bytes, r < 32
  constexpr int kPer = 16 / sizeof(T);
  return r * D * static_cast<int>(sizeof(T)) + ((col / kPer) ^ run_mask<T, D>(r)) * 16 + col % kPer * static_cast<int>(sizeof(T));
}
// A lane's places in a tile of rows of D.  The mask is linear in the bits of the row (over exclusive or), and what
// a product adds to the lane's row and column has other bits than those, so any place is one of these four with
// constants taken in by one exclusive or and the instruction's offset.
template <typename T, int D>
struct Places {
  int row;      // row i, elements 8 g ..
  int perm;     // row i, elements 4 g ..
  int col;      // row 4 g + .., the column operands' first rows
  int col_row;  // row 8 g + ..
  __device__ __forceinline__ Places() {
    const int l = threadIdx.x & 63, i = l & 15, g = l >> 4;
    row = place<T, D>(i, 8 * g);
    perm = place<T, D>(i, 4 * g);
    if constexpr (sizeof(T) == 2) {  // the transposing read: 4 rows of 16 lanes, 4 elements each
      col = place<T, D>(4 * g + (i >> 2), (l & 3) * 4);
      col_row = place<T, D>(8 * g + (i >> 2), (l & 3) * 4);
    } else {
      col = place<T, D>(4 * g, i);
      col_row = place<T, D>(8 * g, i);
    }
  }
  // Called at the top of a loop: the places with their constants are then made in the loop, where they are
  // used, and do not take its registers (the constants' many combinations would).  Only for those that it uses: each
  // takes a register all the way.
  template <bool ROW = true, bool PERM = true, bool COL = true, bool COL_ROW = true>
  __device__ __forceinline__ void here() {
    if constexpr (ROW) asm volatile("" : "+v"(row));
    if constexpr (PERM) asm volatile("" : "+v"(perm));
    if constexpr (COL) asm volatile("" : "+v"(col));
    if constexpr (COL_ROW) asm volatile("" : "+v"(col_row));
  }
};
// base with `r` more rows and `col` more elements; the tile's rows start at row0, a multiple of 16.
template <typename T, int D>
__device__ __forceinline__ T* at(T* tile, int row0, int base, int r, int col) {
  using E = typename std::remove_const<T>::type;
  constexpr int kRow = D * static_cast<int>(sizeof(T));
  const int off = (base ^ (run_mask<E, D>(r) * 16) ^ (col * static_cast<int>(sizeof(T)))) + r * kRow;
  using Byte = typename std::conditional<std::is_const<T>::value, const char, char>::type;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(tile + row0 * D) + off);
}

// Operand whose contracted index runs along the LDS row: lane (i, g) holds row row0 + i, elements
// col + 8 g .. + 7 of the 32.
template <int D>
__device__ __forceinline__ bf16x8 frag_row(const Places<uint16_t, D>& w, const uint16_t* tile, int row0, int col) {
  return *reinterpret_cast<const bf16x8*>(at<const uint16_t, D>(tile, row0, w.row, 0, col));
}
template <int D>
__device__ __forceinline__ Frag32 frag_row(const Places<float, D>& w, const float* tile, int row0, int col) {
  Frag32 f;
  __builtin_memcpy(f.v, __builtin_assume_aligned(at<const float, D>(tile, row0, w.row, 0, col), 16), 16);
  __builtin_memcpy(f.v + 4, __builtin_assume_aligned(at<const float, D>(tile, row0, w.row, 0, col + 4), 16), 16);
  return f;
}

// The same with the elements in the order of frag_col: 16 t + 4 g + r.
template <int D>
__device__ __forceinline__ bf16x8 frag_row_perm(const Places<uint16_t, D>& w, const uint16_t* tile, int row0, int col) {
  const uint2 a = *reinterpret_cast<const uint2*>(at<const uint16_t, D>(tile, row0, w.perm, 0, col));
  const uint2 b = *reinterpret_cast<const uint2*>(at<const uint16_t, D>(tile, row0, w.perm, 0, col + 16));
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}
template <int D>
__device__ __forceinline__ Frag32 frag_row_perm(const Places<float, D>& w, const float* tile, int row0, int col) {
  Frag32 f;
  __builtin_memcpy(f.v, __builtin_assume_aligned(at<const float, D>(tile, row0, w.perm, 0, col), 16), 16);
  __builtin_memcpy(f.v + 4, __builtin_assume_aligned(at<const float, D>(tile, row0, w.perm, 0, col + 16), 16), 16);
  return f;
}

// An operand in that order back into a row-major tile, to be read by its columns.
template <int D>
__device__ __forceinline__ void put_row_perm(const Places<uint16_t, D>& w, uint16_t* tile, int row0, int col, const bf16x8& f) {
  const uint4 u = __builtin_bit_cast(uint4, f);
  *reinterpret_cast<uint2*>(at<uint16_t, D>(tile, row0, w.perm, 0, col)) = make_uint2(u.x, u.y);
  *reinterpret_cast<uint2*>(at<uint16_t, D>(tile, row0, w.perm, 0, col + 16)) = make_uint2(u.z, u.w);
}
template <int D>
__device__ __forceinline__ void put_row_perm(const Places<float, D>& w, float* tile, int row0, int col, const Frag32& f) {
  __builtin_memcpy(__builtin_assume_aligned(at<float, D>(tile, row0, w.perm, 0, col), 16), f.v, 16);
  __builtin_memcpy(__builtin_assume_aligned(at<float, D>(tile, row0, w.perm, 0, col + 16), 16), f.v + 4, 16);
}

// Operand whose contracted index runs down the LDS column: lane (i, g) holds column col + i, rows
// row0 + 16 t + 4 g + r (t 0..1, r 0..3) of the 32.
__device__ __forceinline__ bf16x8 read_transposed(const uint16_t* a, const uint16_t* b) {
  union {
    i16x4 h[2];
    bf16x8 f;
  } u;
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(a));
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(b));
  return u.f;
}
template <int D>
__device__ __forceinline__ bf16x8 frag_col(const Places<uint16_t, D>& w, const uint16_t* tile, int row0, int col) {
  const uint16_t* p = at<const uint16_t, D>(tile, row0, w.col, 0, col);
  return read_transposed(p, p + 16 * D);
}
template <int D>
__device__ __forceinline__ Frag32 frag_col(const Places<float, D>& w, const float* tile, int row0, int col) {
  Frag32 f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float* p = at<const float, D>(tile, row0, w.col, r, col);
    f.v[r] = p[0];
    f.v[4 + r] = p[16 * D];
  }
  return f;
}

// The same in frag_row's order, rows 8 g .. 8 g + 7.
template <int D>
__device__ __forceinline__ bf16x8 frag_col_row(const Places<uint16_t, D>& w, const uint16_t* tile, int row0, int col) {
  return read_transposed(at<const uint16_t, D>(tile, row0, w.col_row, 0, col),
                         at<const uint16_t, D>(tile, row0, w.col_row, 4, col));
}
template <int D>
__device__ __forceinline__ Frag32 frag_col_row(const Places<float, D>& w, const float* tile, int row0, int col) {
  Frag32 f;
#pragma unroll
  for (int r = 0; r < 8; ++r) f.v[r] = *at<const float, D>(tile, row0, w.col_row, r, col);
  return f;
}

// The column operands of all of a row's tiles: read once and kept (for several products, where registers allow: 4
// for one bfloat16 operand, 8 for a float32 one) or read at each use.
template <typename T, int D, bool KEEP = sizeof(T) == 2>
struct Cols {
  const Places<T, D>& w;
  const T* p;
  int row0;
  Frag<T> f[KEEP ? D / 16 : 1];
  __device__ __forceinline__ Cols(const Places<T, D>& places, const T* tile, int row) : w(places), p(tile), row0(row) {
    if constexpr (KEEP) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n) f[n] = frag_col<D>(w, p, row0, n * 16);
    }
  }
  __device__ __forceinline__ Frag<T> operator[](int n) const {
    if constexpr (KEEP) return f[n];
    else return frag_col<D>(w, p, row0, n * 16);
  }
};

// two roundings to nearest, one instruction
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ float elem(const bf16x8& f, int e) { return static_cast<float>(f[e]); }
__device__ __forceinline__ float elem(const Frag32& f, int e) { return f.v[e]; }

// Eight float32 numbers as the sum of three operands of bfloat16 numbers: each piece is the leading 8
// bits of what the ones before left, so the three hold all 24.
__device__ __forceinline__ void split(const float (&x)[8], bf16x8 (&f)[3]) {
  float rest[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = x[e];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)  // the upper halves of two numbers
      w[e] = __builtin_amdgcn_perm(__float_as_uint(rest[2 * e + 1]), __float_as_uint(rest[2 * e]), 0x07060302u);
    f[i] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
    if (i < 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) rest[e] -= __uint_as_float(__float_as_uint(rest[e]) & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void split(const float (&x)[8], Frag32 (&f)[1]) { __builtin_memcpy(f[0].v, x, sizeof(x)); }
template <typename T>
constexpr int kPieces = sizeof(T) == 2 ? 3 : 1;

// Sums and scans over the 16 lanes of a row with lane-rotating adds, over the 4 rows (g) of a wave
// with row swaps: no LDS round trips.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf, 0xf, true);
  return __hiloint2double(hi, lo);
}
constexpr int kRor = 0x120, kShr = 0x110, kShl = 0x100;  // by n lanes of the row; shifts bring in 0
__device__ __forceinline__ float row_sum(float v) {  // in every lane of the row
  v += dpp<kRor + 8>(v);
  v += dpp<kRor + 4>(v);
  v += dpp<kRor + 2>(v);
  return v + dpp<kRor + 1>(v);
}
template <typename F>
__device__ __forceinline__ F row_prefix(F v) {  // inclusive
  v += dpp<kShr + 1>(v);
  v += dpp<kShr + 2>(v);
  v += dpp<kShr + 4>(v);
  return v + dpp<kShr + 8>(v);
}
__device__ __forceinline__ float row_suffix(float v) {
  v += dpp<kShl + 1>(v);
  v += dpp<kShl + 2>(v);
  v += dpp<kShl + 4>(v);
  return v + dpp<kShl + 8>(v);
}
// the four rows' values, each in every lane (of the same place in its row)
__device__ __forceinline__ void rows_of(float v, float (&r)[4]) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const unsigned x = __float_as_uint(v);
  const u32x2 half = __builtin_amdgcn_permlane32_swap(x, x, false, false);  // rows (0, 1), rows (2, 3)
  const u32x2 lo = __builtin_amdgcn_permlane16_swap(half[0], half[0], false, false);
  const u32x2 hi = __builtin_amdgcn_permlane16_swap(half[1], half[1], false, false);
  r[0] = __uint_as_float(lo[0]), r[1] = __uint_as_float(lo[1]);
  r[2] = __uint_as_float(hi[0]), r[3] = __uint_as_float(hi[1]);
}
__device__ __forceinline__ float sum_rows(float v) {
  float r[4];
  rows_of(v, r);
  return (r[0] + r[1]) + (r[2] + r[3]);
}
// the sum over the rows after / before this one
__device__ __forceinline__ float sum_after(const float (&r)[4], int g) {
  return (g < 1 ? r[1] : 0.0f) + (g < 2 ? r[2] : 0.0f) + (g < 3 ? r[3] : 0.0f);
}
__device__ __forceinline__ float sum_before(const float (&r)[4], int g) {
  return (g > 0 ? r[0] : 0.0f) + (g > 1 ? r[1] : 0.0f) + (g > 2 ? r[2] : 0.0f);
}

// ---------------------------------------------------------------------------------------------
// arguments

struct View {  // [batch, seqlen, heads, dim], innermost contiguous; strides in elements
  const void* p;
  int64_t b, t, h;
};

struct LinArgs {
  View q, k, v, dout;
  const float* g;          // log decay
  int64_t gb, gt, gh;      // its strides (0: broadcast)
  const float *s0, *dsT;   // initial state; gradient of the final state
  const int* lengths;
  void* out;               // [batch, seqlen, heads, dv]
  float* sT;               // final state
  float *ds0;              // gradient of the initial state
  void *dq, *dk_out;       // [batch, seqlen, heads, dk]: activations, or float32 where heads share q and k
  void* dv_out;            // [batch, seqlen, heads, dv]
  float* dg;               // [batch, seqlen, heads]
  float *seg_s, *seg_ds;   // [batch * heads][segment][DK][ld]
  float *seg_g, *seg_dg;   // [batch * heads][segment]: the segment's log2 decay, as each walk found it
  float* states;           // [batch * heads][block][DK][DV]: a segment's own state before each block
  float* block_g;          // [batch * heads][block]: the segment's log2 decay before each block
  int64_t batch;
  int seqlen, heads, share, dk, dvd;  // share: heads per query/key head
  int blocks, segments, per_segment;  // blocks of C tokens; segments; blocks per segment
  int slices, ld;                     // slices of the value channels; a segment state's row
  int subs, parts, per_part;          // the gradient's passes: parts of a segment, all of them, blocks of one
  bool chain;                         // few segments: each walk joins the states before it itself
  float scale;
};

// Tokens per block and waves: a wave owns 16 tokens of a block.  64 tokens, but 32 where the gradient's float32
// tiles of 128 channels would not fit LDS (all kernels of a call use the same blocks).
constexpr int waves_of(size_t elem, int dk, int dv) { return elem == 4 && dk == 128 && dv == 128 ? 2 : 4; }
template <int W>
struct Block {
  static constexpr int kWaves = W;
  static constexpr int kC = 16 * kWaves;
  static constexpr int kThreads = 64 * kWaves;
};
template <typename T, int DK, int DV>
using BlockOf = Block<waves_of(sizeof(T), DK, DV)>;

// Whether the gradient's walk reads the state that enters a part of a segment again for each block instead of keeping it:
// where R alone takes 64 registers (float32: 128) of a wave.  Call, us, read again / kept: bfloat16 4 x 2048 tokens, 8 heads of
// 128 x 128 174 / 202, float32 4 x 1024 183 / 270; heads of 64 x 64 have registers for both.
constexpr bool rereads(int dk, int dv) { return dk == 128 && dv == 128; }

// Waves per SIMD that a kernel's registers must leave room for, where LDS does too: bfloat16 heads; the others need
// their registers.
constexpr int waves_for(size_t elem, int dk, int dv, int narrow) {
  return elem != 2 || dk + dv > 192 ? 1 : dk + dv > 128 ? (narrow > 2 ? 2 : 1) : narrow;
}
// The gradient's walk: two workgroups of 8 waves on a CU where LDS holds both, else one.
constexpr int grad_waves_for(size_t elem, int dk, int dv) { return elem == 2 && dk + dv <= 128 ? 4 : waves_of(elem, dk, dv) / 2; }
#define VMSCAN_WAVES(N) __attribute__((amdgpu_waves_per_eu(waves_for(sizeof(T), DK, DV, N))))

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The lane, in a loop that shall make what depends on it where it is used, as Places::here().
__device__ __forceinline__ int lane_here() {
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));
  return l;
}

// Accesses off a base that all lanes share, at 32-bit byte offsets: one register per address, and no branch where
// something is left out, which an offset of kNowhere, past the buffer's end, says (a load then gives zeros, a store
// does nothing).  The forward of 128 x 197 tokens and the gradient's passes measured 5 % less time than with branches.
constexpr uint32_t kNowhere = 0xffff0000u;  // more than 63 tokens of the largest stride
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
constexpr int kRaw = 0x00027000;  // the resource's last word: plain 32-bit data
struct Buffer {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ explicit Buffer(const void* base)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(kNowhere), kRaw)) {}
  // At at + more (less than 64 KB).  Stores have the sum in the address and not `more` in the instruction's scalar
  // offset: the compiler then takes a 16-byte store's registers as free at once, and a few lanes' values written to
  // them by the next instruction were stored instead (float32 outputs of the forward, when stores had to queue).
  __device__ __forceinline__ u32x4 load16(uint32_t at, int more = 0) const {
    return __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(at), more, 0);
  }
  __device__ __forceinline__ void store(const float*, f32x4 v, uint32_t at, int more) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, static_cast<int>(at + more), 0, 0);
  }
  __device__ __forceinline__ void store(const uint16_t*, f32x4 v, uint32_t at, int more) const {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])}, r, static_cast<int>(at + more), 0, 0);
  }
};

// A tile of C tokens on its way from global memory to LDS.  Tokens from `rows` on and channels from
// `dim` on are not read: they enter as zeros, whatever the memory holds.
template <typename T, int D, typename B>
struct Tile {
  static constexpr int kPer = 16 / sizeof(T);
  static constexpr int kRow = D / kPer;
  static constexpr int kRuns = B::kC * kRow;
  static constexpr int kN = (kRuns + B::kThreads - 1) / B::kThreads;
  // fewer runs than threads: the last waves have none
  __device__ __forceinline__ static bool mine() { return kRuns >= B::kThreads || threadIdx.x < kRuns; }
  u32x4 r[kN];
  // base: the block's first token; offsets in it fit 32 bits (the caller checked the stride)
  __device__ __forceinline__ void load(const T* base, uint32_t st, int rows, int dim) {
    const Buffer p(base);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t id = i * B::kThreads + threadIdx.x, row = id / kRow, col = (id % kRow) * kPer;
      const bool in = mine() && static_cast<int>(row) < rows && static_cast<int>(col) < dim;
      r[i] = p.load16(in ? (row * st + col) * static_cast<uint32_t>(sizeof(T)) : kNowhere);
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
    if (!mine()) return;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int id = i * B::kThreads + threadIdx.x, row = id / kRow, col = (id % kRow) * kPer;
      *reinterpret_cast<u32x4*>(reinterpret_cast<char*>(lds + (row & ~15) * D) + place<T, D>(row & 15, col)) = r[i];
    }
  }
};

// A wave's 16 rows of a block straight from global memory as row operands, for a tensor no other wave reads.
template <typename T, int D>
struct OwnRows {
  Frag<T> f[D / 32];
  __device__ __forceinline__ void load(const T* base, uint32_t st, int row0, int rows, int dim) {
    const int l = threadIdx.x & 63, row = row0 + (l & 15), col = (l >> 4) * 8;
    const Buffer p(base);
    const uint32_t at = (row * st + col) * static_cast<uint32_t>(sizeof(T));
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      u32x4 w[sizeof(T) / 2];
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        w[i] = p.load16(row < rows && col + kk * 32 < dim ? at : kNowhere, (kk * 32 + i * 4) * static_cast<int>(sizeof(T)));
      __builtin_memcpy(&f[kk], w, sizeof(w));
    }
  }
};

// A tensor of one (sequence, head), block by block.
template <typename T, int D, typename B>
struct Stream {
  const T* p;  // the block's first token
  int st;      // token stride
  Tile<T, D, B> tile;
  __device__ __forceinline__ Stream(const View& v, int64_t b, int h, int n0)
      : p(static_cast<const T*>(v.p) + b * v.b + h * v.h + n0), st(static_cast<int>(v.t)) {}
  __device__ __forceinline__ void skip(int blocks) { p += static_cast<int64_t>(blocks) * (B::kC * st); }
  __device__ __forceinline__ void load(int rows, int dim) { tile.load(p, st, rows, dim); }
};

// A block's decays.  With G the running log2 decay, E(t) the last token of t's 16 and F(t) the last one
// before t's 16 (G = 0 before the block):
template <int C>
struct Decays {
  float hi[C], lo[C];  // G, head and tail
  float from0[C];      // 2^G_t
  float toC[C];        // 2^(G_C - G_t)
  float toE[C];        // 2^(G_E(t) - G_t)
  float fromF[C];      // 2^(G_t - G_F(t))
  // 2^(G_i - G_j) for j <= i
  __device__ __forceinline__ float between(float hi_i, float lo_i, int j) const {
    return __builtin_amdgcn_exp2f((hi_i - hi[j]) + (lo_i - lo[j]));
  }
};
// By one wave, lane t for token t0 + t: load, then scan.
template <int C>
__device__ __forceinline__ float load_g(const LinArgs& a, const float* g, int t0, int live) {
  const int l = threadIdx.x & 63;
  float x = 0.0f;
  if (l < C && t0 + l < live) {
    x = g[(t0 + l) * a.gt];
    x = x < kMinLog ? kMinLog : x;  // NaN stays
  }
  return x;
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}
template <int C>
__device__ __forceinline__ void scan_g(float x, Decays<C>& d) {
  const int l = threadIdx.x & 63;
  double s = row_prefix(static_cast<double>(x) * 1.4426950408889634);
  double before = 0.0;  // at the end of the rows of 16 before this one
  double end = 0.0, all = 0.0;
#pragma unroll
  for (int g = 0; g < C / 16; ++g) {
    if ((l >> 4) == g) before = all;
    all += lane_of(s, 16 * g + 15);
    if ((l >> 4) == g) end = all;
  }
  const double own = s;
  s += before;
  if (l < C) {
    const float h = static_cast<float>(s);
    d.hi[l] = h;
    d.lo[l] = static_cast<float>(s - static_cast<double>(h));
    d.from0[l] = __builtin_amdgcn_exp2f(h);
    d.toC[l] = __builtin_amdgcn_exp2f(static_cast<float>(all - s));
    d.toE[l] = __builtin_amdgcn_exp2f(static_cast<float>(end - s));
    d.fromF[l] = __builtin_amdgcn_exp2f(static_cast<float>(own));
  }
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }

// Results in the accumulators' layout (4 consecutive channels of one token per lane) to memory.
__device__ __forceinline__ void store_acc(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store_acc(uint16_t* p, f32x4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}

// N tiles of 16 channels of one token, of which `dim` exist, if it is there at all.  block: the block's place in the
// tensor, the same for all lanes; at: the lane's offset in it.
template <typename O, int N>
__device__ __forceinline__ void store_tiles(O* block, uint32_t at, int dim, bool there, const f32x4 (&acc)[N]) {
  const int g4 = ((threadIdx.x & 63) >> 4) * 4;
  const Buffer p(block);
#pragma unroll
  for (int n = 0; n < N; ++n)
    p.store(block, acc[n], there && n * 16 + g4 < dim ? at * static_cast<uint32_t>(sizeof(O)) : kNowhere,
            n * 16 * static_cast<int>(sizeof(O)));
}

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
               __uint_as_float(w.y & 0xffff0000u)};
}

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return __builtin_fmaf(a[3], b[3], __builtin_fmaf(a[2], b[2], __builtin_fmaf(a[1], b[1], a[0] * b[0])));
}

// The state, transposed in the accumulators: wave w holds columns d of its own tiles (tile index
// w * DT + t), rows n = 16 nt + 4 g + r.
template <typename T, int DK, int DV>
struct State {
  using B = BlockOf<T, DK, DV>;
  static constexpr int kDT = DK / 16 < B::kWaves ? 1 : DK / 16 / B::kWaves;
  static constexpr int kNT = DV / 16;
  // DK 32: two waves hold the state, the others have none of it
  __device__ __forceinline__ static bool mine() { return DK / 16 >= B::kWaves || wave_id() < DK / 16; }
  f32x4 s[kDT][kNT];

  __device__ __forceinline__ static int d_of(int t) { return (wave_id() * kDT + t) * 16 + (threadIdx.x & 15); }
  __device__ __forceinline__ static int n_of(int nt) { return nt * 16 + ((threadIdx.x & 63) >> 4) * 4; }

  // rows of `ld` floats, of which d < dk and n < dv exist
  __device__ __forceinline__ static uint32_t place_of(int ld) {  // of [0][0], in bytes
    return (static_cast<uint32_t>(d_of(0)) * ld + n_of(0)) * 4;
  }
  // tiles nt0 .. nt1 - 1 of each row of them
  __device__ __forceinline__ void load(const float* p, int dk, int dv, int ld, int nt0 = 0, int nt1 = kNT) {
    const Buffer from(p);
#pragma unroll
    for (int t = 0; t < kDT; ++t)
#pragma unroll
      for (int nt = nt0; nt < nt1; ++nt)
        s[t][nt] = __builtin_bit_cast(
            f32x4, from.load16(p && d_of(t) < dk && n_of(nt) < dv ? place_of(ld) : kNowhere, (t * 16 * ld + nt * 16) * 4));
  }
  __device__ __forceinline__ void store(float* p, int dk, int dv, int ld) const {
    const Buffer to(p);
#pragma unroll
    for (int t = 0; t < kDT; ++t)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        to.store(p, s[t][nt], d_of(t) < dk && n_of(nt) < dv ? place_of(ld) : kNowhere, (t * 16 * ld + nt * 16) * 4);
  }
  // What enters after segments from, from + dir, .. (n of them) that each add their own state, on top of what is
  // here: s = s 2^g + own, AHEAD segments on their way at a time.
  template <int AHEAD = 4>
  __device__ __forceinline__ void join(const float* own, const float* g, int from, int dir, int n, int ld) {
    const int64_t step = static_cast<int64_t>(DK) * ld;
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
      State x[AHEAD];
      float m[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i0 + i < n) {
          const int at = from + dir * (i0 + i);
          x[i].load(own + at * step, DK, DV, ld);
          m[i] = g[at];
        }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i0 + i < n) {
          const float e = __builtin_amdgcn_exp2f(m[i]);
#pragma unroll
          for (int t = 0; t < kDT; ++t)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) s[t][nt] = s[t][nt] * e + x[i].s[t][nt];
        }
    }
  }
  // into LDS as an operand, [d][n]: for bfloat16 three planes, each the rounded rest of those before.  Planes
  // FROM .. TO - 1, one after the other from p.
  static constexpr int kPlane = DK * DV;
  static constexpr int kPlanes = kPieces<T>;
  template <int FROM = 0, int TO = kPlanes>
  __device__ __forceinline__ void publish(const Places<T, DV>& wv, T* p) const {
    if (!mine()) return;
#pragma unroll
    for (int t = 0; t < kDT; ++t)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        T* to = at<T, DV>(p, (wave_id() * kDT + t) * 16, wv.perm, 0, nt * 16);
        if constexpr (kPlanes == 1) {
          store_acc(to, s[t][nt]);
        } else {
          f32x4 rest = s[t][nt];
          if constexpr (FROM > 0) asm volatile("" : "+v"(rest));  // the rests are made again, not kept since the planes before
#pragma unroll
          for (int pl = 0; pl < TO; ++pl) {
            const uint32_t lo = pack2(rest[0], rest[1]), hi = pack2(rest[2], rest[3]);
            if (pl >= FROM) *reinterpret_cast<uint2*>(to + (pl - FROM) * kPlane) = make_uint2(lo, hi);
            rest[0] -= __uint_as_float(lo << 16), rest[1] -= __uint_as_float(lo & 0xffff0000u);
            rest[2] -= __uint_as_float(hi << 16), rest[3] -= __uint_as_float(hi & 0xffff0000u);
          }
        }
      }
  }
  // Rows d of this wave's tile t as operands, n in frag_col's order, 32 from n0.
  __device__ __forceinline__ void rows(int t, int n0, Frag<T> (&piece)[kPieces<T>]) const {
    float x[8];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = s[t][n0 / 16][r], x[4 + r] = s[t][n0 / 16 + 1][r];
    split(x, piece);
  }
  __device__ __forceinline__ void decay(float e) {
#pragma unroll
    for (int t = 0; t < kDT; ++t)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) s[t][nt] *= e;
  }
  // s += sum_j w_j y_j x_j^T over the 32 tokens from row0 of y (the tile [token][d]); xa: the operand of x,
  // w: the weights, both in frag_col's order.
  template <bool KEEP>
  __device__ __forceinline__ void add(const Places<T, DK>& wk, const T* y, int row0, const Cols<T, DV, KEEP>& xa,
                                      const float (&w)[8]) {
    if (!mine()) return;
#pragma unroll
    for (int t = 0; t < kDT; ++t) {
      const Frag<T> f = frag_col<DK>(wk, y, row0, (wave_id() * kDT + t) * 16);
      float m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = elem(f, e) * w[e];
      Frag<T> piece[kPieces<T>];
      split(m, piece);
      if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const Frag<T> x = xa[nt];
#pragma unroll
        for (int i = 0; i < kPieces<T>; ++i) s[t][nt] = mma(x, piece[i], s[t][nt]);
      }
    }
  }
};

// Eight values of a table in frag_col's order, for the 32 tokens from p.
__device__ __forceinline__ void eight(const float* p, float (&w)[8]) {
  const int g4 = ((threadIdx.x & 63) >> 4) * 4;
  const f32x4 a = load4(p + g4), b = load4(p + 16 + g4);
#pragma unroll
  for (int r = 0; r < 4; ++r) w[r] = a[r], w[4 + r] = b[r];
}

struct Where {  // this workgroup's place
  int64_t bh, b;
  int h, seg, n0, live, c0, c1, end;  // n0: first value channel; c0 .. c1: blocks with tokens, .. end: all
};
// Workgroup i runs on XCD i % 8.  An XCD takes consecutive places: the slices of the value channels and the
// heads that share q and k, which then find them in its L2, then a sequence's segments.
template <typename B>
__device__ __forceinline__ Where where(const LinArgs& a, int width, uint32_t id0, uint32_t n) {
  constexpr int C = B::kC;
  const uint32_t q = n >> 3, r = n & 7, xcd = id0 & 7, local = id0 >> 3;
  uint32_t id = (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + local;
  Where w;
  w.n0 = static_cast<int>(id % a.slices) * width;
  id /= a.slices;
  const int in = static_cast<int>(id % a.share);
  id /= a.share;
  w.seg = static_cast<int>(id % a.segments);
  id /= a.segments;
  const int kheads = a.heads / a.share;
  w.b = id / kheads;
  w.h = static_cast<int>(id % kheads) * a.share + in;
  w.bh = w.b * a.heads + w.h;
  int len = a.seqlen;
  if (a.lengths) {
    len = a.lengths[w.b];
    len = len < 0 ? 0 : len > a.seqlen ? a.seqlen : len;
  }
  w.live = __builtin_amdgcn_readfirstlane(len);
  w.c0 = w.seg * a.per_segment;
  w.end = w.c0 + a.per_segment < a.blocks ? w.c0 + a.per_segment : a.blocks;
  const int live_blocks = (w.live + C - 1) / C;
  w.c1 = w.end < live_blocks ? w.end : live_blocks;
  return w;
}

// Zeros for this place's tokens past the row's length, in a tensor with token stride `st`, `dim` (a multiple
// of 4) channels.
template <typename B, typename O>
__device__ __forceinline__ void zero_rest(const LinArgs& a, const Where& w, O* p, int64_t st, int dim) {
  constexpr int C = B::kC;
  const int t1 = w.end * C < a.seqlen ? w.end * C : a.seqlen;
  const int t0 = w.live > w.c0 * C ? w.live : w.c0 * C;
  const int runs = dim / 4;
  for (int64_t id = threadIdx.x; id < static_cast<int64_t>(t1 - t0) * runs; id += B::kThreads) {
    const int64_t t = id / runs;
    store_acc(p + (t0 + t) * st + (id - t * runs) * 4, zero4());
  }
}

// ---------------------------------------------------------------------------------------------
// A segment's own state from a zero start: forward (k, v) or, BACK, the state's gradient (q, dout)
// from a zero end.  KEEP also writes the state before each block.
// Bound by a block's chain (its loads, its decays, then the state's update), not by HBM: 8 x 6085 tokens (three quarters of them
// live), 6 heads of 128 x 64, 2 key heads, bfloat16: 31 us, 60 MB at 1.9 TB/s.

template <typename T, int DK, int DV, bool BACK, bool KEEP, int C = BlockOf<T, DK, DV>::kC>
__device__ __forceinline__ void segment_walk(const LinArgs& a, uint32_t id, uint32_t n_ids, T* ys, T* xs,
                                             Decays<C>* decays) {
  using B = BlockOf<T, DK, DV>;
  using S = State<T, DK, DV>;
  const Where w = where<B>(a, DV, id, n_ids);
  if (BACK ? w.seg < a.subs : !KEEP && w.seg == a.segments - 1) return;  // no segment lies past it
  Stream<T, DK, B> y(BACK ? a.q : a.k, w.b, w.h / a.share, 0);
  Stream<T, DV, B> x(BACK ? a.dout : a.v, w.b, w.h, w.n0);
  const int dv = a.dvd - w.n0;
  const float* g = a.g + w.b * a.gb + w.h * a.gh;
  const int wave = wave_id();
  Places<T, DK> wk;
  Places<T, DV> wv;
  S st;
  st.load(nullptr, 0, 0, 0);
  float total = 0.0f;
  const int n = w.c1 - w.c0;
  float gx = 0.0f;
  auto at = [&](int i) { return (BACK ? w.c1 - 1 - i : w.c0 + i) * C; };
  if (n > 0) {
    y.skip(BACK ? w.c1 - 1 : w.c0);
    x.skip(BACK ? w.c1 - 1 : w.c0);
    y.load(w.live - at(0), a.dk);
    x.load(w.live - at(0), dv);
    if (wave == 0) scan_g(load_g<C>(a, g, at(0), w.live), decays[0]);
    if (n > 1) gx = load_g<C>(a, g, at(1), w.live);
  }
  for (int i = 0; i < n; ++i) {
    const Decays<C>& d = decays[i & 1];
    wk.here();
    wv.here();
    y.tile.store(ys);
    x.tile.store(xs);
    if constexpr (KEEP) {
      const int64_t block = w.bh * a.blocks + (w.c0 + i);
      st.store(a.states + block * (DK * DV), DK, DV, DV);
      if (threadIdx.x == 0) a.block_g[block] = total;
    }
    __syncthreads();
    if (i + 1 < n) {
      y.skip(BACK ? -1 : 1);
      x.skip(BACK ? -1 : 1);
      y.load(w.live - at(i + 1), a.dk);
      x.load(w.live - at(i + 1), dv);
      if (wave == i % B::kWaves) scan_g(gx, decays[(i + 1) & 1]);
      if (i + 2 < n) gx = load_g<C>(a, g, at(i + 2), w.live);
    }
    total += d.hi[C - 1] + d.lo[C - 1];
    st.decay(d.from0[C - 1]);
#pragma unroll
    for (int kk = 0; kk < C / 32; ++kk) {
      float m[8];
      eight((BACK ? d.from0 : d.toC) + kk * 32, m);
      if (BACK) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] *= a.scale;
      }
      const Cols<T, DV> xa(wv, xs, kk * 32);
      st.add(wk, ys, kk * 32, xa, m);
    }
    __syncthreads();
  }
  if (a.segments == 1) return;
  st.store((BACK ? a.seg_ds : a.seg_s) + (w.bh * a.segments + w.seg) * (DK * a.ld) + w.n0, DK, DV, a.ld);
  if (w.n0 == 0 && threadIdx.x == 0) (BACK ? a.seg_dg : a.seg_g)[w.bh * a.segments + w.seg] = total;
}

template <typename T, int DK, int DV, bool BACK, bool KEEP>
__global__ __launch_bounds__((BlockOf<T, DK, DV>::kThreads)) VMSCAN_WAVES(4) void linattn_segment_kernel(LinArgs a) {
  constexpr int C = BlockOf<T, DK, DV>::kC;
  __shared__ __align__(16) T ys[C * DK];
  __shared__ __align__(16) T xs[C * DV];
  __shared__ __align__(16) Decays<C> decays[2];
  segment_walk<T, DK, DV, BACK, KEEP>(a, blockIdx.x, gridDim.x, ys, xs, decays);
}

// The gradient's two passes, which do not depend on each other, in one launch: the first half of the
// workgroups walks from the end, and only the parts that a later segment's walk needs.  Bound by HBM: 32 x 3136 tokens, 8
// heads of 64 x 64, bfloat16, read 309 MB (k and v, half of q and dout) and write 232 MB (206 of them states) in 123 us, 4.4 TB/s.
template <typename T, int DK, int DV>
__global__ __launch_bounds__((BlockOf<T, DK, DV>::kThreads)) VMSCAN_WAVES(4) void linattn_passes_kernel(LinArgs a) {
  constexpr int C = BlockOf<T, DK, DV>::kC;
  __shared__ __align__(16) T ys[C * DK];
  __shared__ __align__(16) T xs[C * DV];
  __shared__ __align__(16) Decays<C> decays[2];
  const uint32_t half = gridDim.x / 2;
  if (blockIdx.x < half)
    segment_walk<T, DK, DV, true, false>(a, blockIdx.x, half, ys, xs, decays);
  else
    segment_walk<T, DK, DV, false, true>(a, blockIdx.x - half, half, ys, xs, decays);
}

// In place: each segment's own state becomes the state that enters it (BACK: the gradient at its
// end).  A thread owns 4 elements of one (sequence, head) and has 8 segments on their way at a time.
// Latency bound: 10 segments of 48 states of 128 x 64, 8 us.
template <bool BACK>
__global__ __launch_bounds__(256) void linattn_prefix_kernel(LinArgs a, int DK) {
  const int per = DK * a.ld / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t bh = id / per;
  if (bh >= a.batch * a.heads) return;
  const int e = static_cast<int>(id - bh * per) * 4, d = e / a.ld, n = e % a.ld;
  f32x4 run = zero4();
  const float* first = BACK ? a.dsT : a.s0;
  if (first && d < a.dk && n < a.dvd) run = load4(first + (bh * a.dk + d) * a.dvd + n);
  const int64_t step = static_cast<int64_t>(DK) * a.ld;
  float* p = (BACK ? a.seg_ds : a.seg_s) + bh * a.segments * step + e;
  const float* g = (BACK ? a.seg_dg : a.seg_g) + bh * a.segments;
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < a.segments; i0 += kAhead) {
    f32x4 own[kAhead];
    float m[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < a.segments) {
        const int s = BACK ? a.segments - 1 - i0 - i : i0 + i;
        own[i] = zero4();
        m[i] = 0.0f;
        if (BACK ? s >= a.subs : s + 1 < a.segments) {  // what the last one adds enters nothing
          own[i] = load4(p + s * step);
          m[i] = __builtin_amdgcn_exp2f(g[s]);
        }
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < a.segments) {
        const int s = BACK ? a.segments - 1 - i0 - i : i0 + i;
        store_acc(p + s * step, run);
        run = run * m[i] + own[i];
      }
  }
}

// ---------------------------------------------------------------------------------------------
// forward
//
// A wave owns 16 queries of a block and a part of the state's rows.  Keys and values come one block ahead through
// registers; a deeper prefetch or both of them in LDS twice would cost a workgroup per CU.  Bound by the chain of
// dependent products of a block and by LDS: 128 x 197 tokens, 6 heads of 64 x 64, bfloat16: 29.8 us, 3.0 TB/s (vector
// instructions 44 % of the cycles, LDS 25 %, the matrix cores 20 %); 8 x 6085, 6 heads of 128 x 64: 77 us, 1.5 TB/s, after the
// segments' 31 and the prefix's 8; float32 1 x 197: 9 us after 5.

template <typename T, int DK, int DV>
__global__ __launch_bounds__((BlockOf<T, DK, DV>::kThreads)) VMSCAN_WAVES(3) void linattn_fwd_kernel(LinArgs a) {
  using B = BlockOf<T, DK, DV>;
  using S = State<T, DK, DV>;
  constexpr int C = B::kC, NT = DV / 16;
  __shared__ __align__(16) T ks[C * DK];
  __shared__ __align__(16) T vs[C * DV];
  __shared__ __align__(16) T ss[S::kPlanes * S::kPlane];
  __shared__ __align__(16) Decays<C> decays[2];
  const Where w = where<B>(a, DV, blockIdx.x, gridDim.x);
  Stream<T, DK, B> q(a.q, w.b, w.h / a.share, 0), k(a.k, w.b, w.h / a.share, 0);
  Stream<T, DV, B> v(a.v, w.b, w.h, w.n0);
  const int dv = a.dvd - w.n0;
  const float* g = a.g + w.b * a.gb + w.h * a.gh;
  T* out = static_cast<T*>(a.out) + (w.b * a.seqlen * a.heads + w.h) * a.dvd + w.n0;
  const int64_t ot = static_cast<int64_t>(a.heads) * a.dvd;
  const int wave = wave_id(), l = threadIdx.x & 63, li = l & 15, g4 = (l >> 4) * 4;
  Places<T, DK> wk;
  Places<T, DV> wv;
  // The last 16 queries of a block have four times the first ones' scores.  Workgroups that share a CU give
  // them to different waves, so that no SIMD gets all of them.
  const int qt = (blockIdx.x >> 8) & 1 ? B::kWaves - 1 - wave : wave;

  S st;
  if (a.segments > 1 && !a.chain) {
    st.load(a.seg_s + (w.bh * a.segments + w.seg) * (DK * a.ld) + w.n0, DK, DV, a.ld);
  } else {
    st.load(a.s0 ? a.s0 + w.bh * a.dk * a.dvd + w.n0 : nullptr, a.dk, dv, a.dvd);
    if (w.seg > 0)
      st.join(a.seg_s + w.bh * a.segments * (DK * a.ld) + w.n0, a.seg_g + w.bh * a.segments, 0, 1, w.seg, a.ld);
  }

  OwnRows<T, DK> qn;  // the next block's queries
  auto load = [&](int t0) {
    qn.load(q.p, q.st, qt * 16, w.live - t0, a.dk);
    k.load(w.live - t0, a.dk);
    v.load(w.live - t0, dv);
  };
  float gx = 0.0f;
  if (w.c0 < w.c1) {
    q.skip(w.c0);
    k.skip(w.c0);
    v.skip(w.c0);
    load(w.c0 * C);
    if (wave == 0) scan_g(load_g<C>(a, g, w.c0 * C, w.live), decays[w.c0 & 1]);
    gx = load_g<C>(a, g, w.c0 * C + C, w.live);
  }
  for (int c = w.c0; c < w.c1; ++c) {
    const int t0 = c * C;
    const Decays<C>& d = decays[c & 1];
    wk.here();
    wv.here();
    const OwnRows<T, DK> qf = qn;
    k.tile.store(ks);
    v.tile.store(vs);
    st.publish(wv, ss);
    __syncthreads();
    if (c + 1 < w.c1) {
      q.skip(1);
      k.skip(1);
      v.skip(1);
      load(t0 + C);
      // the next block's decays, by one wave; the others' products run meanwhile
      if (wave == c % B::kWaves) scan_g(gx, decays[(c + 1) & 1]);
      gx = load_g<C>(a, g, t0 + 2 * C, w.live);
    }
    // this wave's 16 queries: column i of every result tile
    const int i0 = qt * 16, i = i0 + li;
    const bool own = t0 + i0 < w.live;
    const float gh = d.hi[i], gl = d.lo[i];
    f32x4 acc[NT];
    if (own) {
      // e^{G_i} S^T q_i
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt] = zero4();
#pragma unroll
      for (int kk = 0; kk < DK / 32; ++kk) {
#pragma unroll
        for (int pl = 0; pl < S::kPlanes; ++pl)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            acc[nt] = mma(frag_col_row<DV>(wv, ss + pl * S::kPlane, kk * 32, nt * 16), qf.f[kk], acc[nt]);
      }
      const float e = d.from0[i];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt] *= e;
    }
    st.decay(d.from0[C - 1]);
#pragma unroll
    for (int kk = 0; kk < C / 32; ++kk) {
      if (t0 + kk * 32 >= w.live) break;
      const Cols<T, DV> xa(wv, vs, kk * 32);
      if (own && kk <= qt / 2) {
        // the masked scores of 32 keys, then their product with the values
        float p[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int j0 = kk * 32 + t * 16;
          if (j0 <= i0) {
            f32x4 sc = zero4();
#pragma unroll
            for (int n = 0; n < DK / 32; ++n) sc = mma(frag_row<DK>(wk, ks, j0, n * 32), qf.f[n], sc);
            if (j0 < i0) {  // through the last of the 16 keys: both factors are powers of the decays between
              const f32x4 e = load4(d.toE + j0 + g4);
              const float from = d.between(gh, gl, j0 + 15);
#pragma unroll
              for (int r = 0; r < 4; ++r) p[t * 4 + r] = sc[r] * (e[r] * from);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                p[t * 4 + r] = g4 + r <= li ? sc[r] * d.between(gh, gl, j0 + g4 + r) : 0.0f;
            }
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) p[t * 4 + r] = 0.0f;
          }
        }
        Frag<T> pf[kPieces<T>];
        split(p, pf);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const Frag<T> x = xa[nt];
#pragma unroll
          for (int i = 0; i < kPieces<T>; ++i) acc[nt] = mma(x, pf[i], acc[nt]);
        }
      }
      float m[8];
      eight(d.toC + kk * 32, m);
      st.add(wk, ks, kk * 32, xa, m);
    }
    if (own) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt] *= a.scale;
      store_tiles(out + t0 * ot, static_cast<uint32_t>(i * ot) + g4, dv, t0 + i < w.live, acc);
    }
    __syncthreads();
  }
  zero_rest<B>(a, w, out, ot, dv < DV ? dv : DV);
  if (a.sT && w.seg == a.segments - 1) st.store(a.sT + w.bh * a.dk * a.dvd + w.n0, a.dk, dv, a.dvd);
}

// ---------------------------------------------------------------------------------------------
// gradient
//
// With R the gradient of the state leaving a block (it includes every later token) and X_ij =
// scale e^{G_i - G_j} (do_i . v_j), P_ij = scale e^{G_i - G_j} (q_i . k_j) for j <= i:
//   dq_i = e^{G_i} scale S do_i + sum_j X_ij k_j
//   dk_j = e^{G_C - G_j} R v_j  + sum_i X_ij q_i
//   dv_j = e^{G_C - G_j} R^T k_j + sum_i P_ij do_i
//   R'   = e^{G_C} R + sum_i e^{G_i} scale q_i do_i^T.
// The decay of token t multiplies every contribution from a token before t to one at or after it,
// so its logarithm's gradient is the sum of those contributions, here split by where the two lie:
// both in the block (M_ij = scale e^{G_i - G_j} (q_i . k_j)(do_i . v_j)), before and in it (a_i = q_i .
// the first term of dq_i), in and after it (b_j = k_j . the first term of dk_j), before and after it
// (Y = e^{G_C} <S, R>):
//   dg_t = sum_{j < t <= i} M_ij + sum_{i >= t} a_i + sum_{j < t} b_j + Y.
// Summing q . dq - k . dk over all later tokens would give the same with two dot products, but as a
// small difference of sums over the whole sequence; here only terms that belong are added.

//
// A first walk forwards (the segment kernel) leaves each block's entering state, counted from its segment's
// start; this kernel walks backwards and does the rest, reading q, k, v and dout once.

//
// Twice the waves of the other kernels: one half (the state waves) carries R, makes dq and the sums a and b, the
// other (the key waves) dk, dv, the in-block part of dg and dg itself.  A key wave owns 16 tokens, a state wave the
// rows d of S and R that it holds.  With one wave doing both, 2 waves per SIMD were all that the registers left, and they waited
// 57 % of the time.  a and b are dot products with the first terms of dq and dk, which the accumulators hold.
//
// Six planes of states (S and R in three bfloat16 pieces each) do not fit LDS beside the tiles of 64 x 64 heads for two
// workgroups on a CU.  So only R is published.  S never leaves its registers: a state wave multiplies its rows with all of the
// block's dO, which leaves its channels of every query's dq, and X, which that needs whole, comes from the key waves, which
// make it for dk, through LDS.  (With S's and R's last planes in one place, exchanged within a block, the call took 519 us
// instead of 424: 32 x 3136 tokens, 8 heads of 64 x 64.)  That walk takes 332 us (318 to 347) and is bound by instruction issue:
// of its cycles vector instructions take 51 %, LDS 31 %, the matrix cores 22 %.
// Float32, 2 x 1001 tokens, 8 heads of 32 x 128: 36 us, bound by a block's chain of float32 products, whose rate is
// a ninth of bfloat16's.

// The gradient's workgroup: a block's tokens as in B, twice the waves.
template <typename B>
struct Pairs {
  static constexpr int kWaves = B::kWaves;
  static constexpr int kC = B::kC;
  static constexpr int kThreads = 2 * B::kThreads;
};

template <typename T, int DK, int DV>
struct GradLds {
  using B = BlockOf<T, DK, DV>;
  using S = State<T, DK, DV>;
  static constexpr int kSmall = 6 * 1024;  // the tables below
  // R's planes: all of them, or for bfloat16 heads of 128 x 128 two, and the third when they have been read
  // (X: blocks of 32 keys and 32 queries [key][query], those with a query at or after a key)
  static constexpr int kHalves = B::kC / 32;
  static constexpr int kX = kHalves * (kHalves + 1) / 2 * 1024;
  static constexpr size_t kAll =
      (2 * B::kC * (DK + DV) + S::kPlanes * S::kPlane + kPieces<T> * kX) * sizeof(T) + kSmall;
  static constexpr int kPlanes = S::kPlanes == 3 && kAll > 160 * 1024 ? 2 : S::kPlanes;
  __align__(16) T qs[B::kC * DK];
  __align__(16) T ks[B::kC * DK];
  __align__(16) T vs[B::kC * DV];
  __align__(16) T os[B::kC * DV];
  __align__(16) T rs[kPlanes * S::kPlane];
  __align__(16) T xs[kPieces<T> * kX];
  __align__(16) Decays<B::kC> decays[2];
  float rows[B::kWaves][B::kC], into[B::kWaves][B::kC], after[B::kC];
  float across[B::kWaves];
  __device__ __forceinline__ T* x(int keys, int queries, int piece) { return xs + piece * kX + (keys + queries) * 1024; }
};

// q, k, v and dout of a block on their way to LDS.
template <typename T, int DK, int DV>
struct GradTiles {
  using G = Pairs<BlockOf<T, DK, DV>>;
  Stream<T, DK, G> q, k;
  Stream<T, DV, G> v, o;
  const Where& w;
  int dk, dv;
  __device__ __forceinline__ GradTiles(const LinArgs& a, const Where& where)
      : q(a.q, where.b, where.h / a.share, 0), k(a.k, where.b, where.h / a.share, 0), v(a.v, where.b, where.h, 0),
        o(a.dout, where.b, where.h, 0), w(where), dk(a.dk), dv(a.dvd) {}
  __device__ __forceinline__ void skip(int blocks) {
    q.skip(blocks);
    k.skip(blocks);
    v.skip(blocks);
    o.skip(blocks);
  }
  __device__ __forceinline__ void load(int t0) {
    q.load(w.live - t0, dk);
    k.load(w.live - t0, dk);
    v.load(w.live - t0, dv);
    o.load(w.live - t0, dv);
  }
  __device__ __forceinline__ void store(GradLds<T, DK, DV>& lds) const {
    q.tile.store(lds.qs);
    k.tile.store(lds.ks);
    v.tile.store(lds.vs);
    o.tile.store(lds.os);
  }
};

// The two halves pass the same barriers: one when a block's tiles and R's planes are in LDS, one when X is, one when the
// block is done; where LDS holds two of R's three planes, two more around the exchange for the third.
template <typename T, int DK, int DV>
__device__ __forceinline__ void grad_states(const LinArgs& a, const Where& w, GradLds<T, DK, DV>& lds) {
  using B = BlockOf<T, DK, DV>;
  using S = State<T, DK, DV>;
  constexpr int C = B::kC;
  constexpr int NT = DV / 16, kTiles = C / 16;
  constexpr int kPlanes = GradLds<T, DK, DV>::kPlanes;
  const int wave = wave_id();
  const int kt = a.heads * a.dk;
  const int64_t kbase = (w.b * a.seqlen * a.heads + w.h) * a.dk;
  GradTiles<T, DK, DV> tiles(a, w);
  Places<T, DK> wk;
  Places<T, DV> wv;
  Places<T, 32> wx;
  S st;  // R
  // The state that enters the part of the segment: kept, or read again for each block (never with a chain, which would have
  // to sum it up each time).
  constexpr bool kReload = rereads(DK, DV);
  S first;
  const float* first_at = nullptr;
  int first_dk = DK, first_dv = DV;
  const int end = (w.seg + 1) * a.subs < a.parts ? (w.seg + 1) * a.subs : a.parts;
  const int64_t part0 = w.bh * a.parts;
  const bool summed = a.parts > 1 && (kReload || !a.chain);  // by the prefix kernels
  if (summed) {
    st.load(a.seg_ds + (part0 + end - 1) * (DK * DV), DK, DV, DV);
  } else {
    st.load(a.dsT ? a.dsT + w.bh * a.dk * a.dvd : nullptr, a.dk, a.dvd, a.dvd);
    if constexpr (!kReload) {
      if (end < a.parts) st.join(a.seg_ds + part0 * (DK * DV), a.seg_dg + part0, a.parts - 1, -1, a.parts - end, DV);
    }
  }
  auto enter = [&](int part, auto ahead) {
    if (summed) {
      first_at = a.seg_s + (part0 + part) * (DK * DV);
    } else {
      first_at = a.s0 ? a.s0 + w.bh * a.dk * a.dvd : nullptr;
      first_dk = a.dk, first_dv = a.dvd;
    }
    if constexpr (!kReload) {
      first.load(first_at, first_dk, first_dv, first_dv);
      if (!summed && part > 0)
        first.template join<decltype(ahead)::value>(a.seg_s + part0 * (DK * DV), a.seg_g + part0, 0, 1, part, DV);
    }
  };
  if (w.c0 < w.c1) {
    enter((w.c1 - 1) / a.per_part, std::integral_constant<int, 4>{});
    tiles.skip(w.c1 - 1);
    tiles.load((w.c1 - 1) * C);
  }
  for (int c = w.c1 - 1; c >= w.c0; --c) {
    const int t0 = c * C;
    const Decays<C>& d = lds.decays[c & 1];
    wk.template here<false, true, true, false>();
    wv.template here<false, true, true, false>();
    wx.template here<false, false, true, false>();
    const int l = lane_here(), li = l & 15, g4 = (l >> 4) * 4;
    const int64_t block = w.bh * a.blocks + c;
    if (a.subs > 1 && (c + 1) % a.per_part == 0 && c + 1 < w.c1)
      enter(c / a.per_part, std::integral_constant<int, 1>{});  // few registers
    // The state that enters the block, put together 32 value channels at a time where they are used, kAhead of them on
    // their way.
    S old;
    constexpr int kAhead = kReload ? 1 : DV / 32;
    const float* kept = a.states + block * (DK * DV);
#pragma unroll
    for (int kk = 0; kk < kAhead; ++kk) {
      old.load(kept, DK, DV, DV, 2 * kk, 2 * kk + 2);
      if constexpr (kReload) first.load(first_at, first_dk, first_dv, first_dv, 2 * kk, 2 * kk + 2);
    }
    const float since = __builtin_amdgcn_exp2f(a.block_g[block]);
    float y = 0.0f;  // <S, R>, both in this wave's layout
    auto whole = [&](int kk) {
#pragma unroll
      for (int t = 0; t < S::kDT; ++t)
#pragma unroll
        for (int nt = 2 * kk; nt < 2 * kk + 2; ++nt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            old.s[t][nt][r] = __builtin_fmaf(first.s[t][nt][r], since, old.s[t][nt][r]);
            y = __builtin_fmaf(old.s[t][nt][r], st.s[t][nt][r], y);
          }
    };
    tiles.store(lds);
    st.template publish<0, kPlanes>(wv, lds.rs);
    __syncthreads();
    // dq of all of the block's queries in this wave's channels: column li of tile it is query 16 it + li.  First the states'
    // part, whose product with q is the decays' sum a.
    f32x4 acc[S::kDT][kTiles];
    float part[kTiles];
#pragma unroll
    for (int it = 0; it < kTiles; ++it) {
      part[it] = 0.0f;
#pragma unroll
      for (int t = 0; t < S::kDT; ++t) acc[t][it] = zero4();
    }
    if (S::mine()) {
#pragma unroll
      for (int kk = 0; kk < DV / 32; ++kk) {
        if (kk + kAhead < DV / 32) {
          old.load(kept, DK, DV, DV, 2 * (kk + kAhead), 2 * (kk + kAhead) + 2);
          if constexpr (kReload) first.load(first_at, first_dk, first_dv, first_dv, 2 * (kk + kAhead), 2 * (kk + kAhead) + 2);
        }
        whole(kk);
        Frag<T> piece[S::kDT][kPieces<T>];
#pragma unroll
        for (int t = 0; t < S::kDT; ++t) old.rows(t, kk * 32, piece[t]);
#pragma unroll
        for (int it = 0; it < kTiles; ++it) {
          const Frag<T> o = frag_row_perm<DV>(wv, lds.os, it * 16, kk * 32);
#pragma unroll
          for (int pl = 0; pl < kPieces<T>; ++pl)
#pragma unroll
            for (int t = 0; t < S::kDT; ++t) acc[t][it] = mma(piece[t][pl], o, acc[t][it]);
        }
      }
#pragma unroll
      for (int it = 0; it < kTiles; ++it) {
        const float e0 = d.from0[it * 16 + li] * a.scale;
#pragma unroll
        for (int t = 0; t < S::kDT; ++t) {
          part[it] += dot4(acc[t][it], load4(at<T, DK>(lds.qs, it * 16, wk.perm, 0, (wave * S::kDT + t) * 16)));
          acc[t][it] *= e0;
        }
      }
    }
    y = sum_rows(row_sum(y));
    if (l == 0) lds.across[wave] = y;
#pragma unroll
    for (int it = 0; it < kTiles; ++it) {
      const float into = sum_rows(part[it]);
      if (l < 16) lds.into[wave][it * 16 + l] = into;
    }
    if (c > w.c0) {
      tiles.skip(-1);
      tiles.load(t0 - C);
    }
    auto next = [&]() {  // R before the block
      st.decay(d.from0[C - 1]);
#pragma unroll
      for (int kk = C / 32 - 1; kk >= 0; --kk) {
        if (t0 + kk * 32 >= w.live) continue;
        const Cols<T, DV, (S::kDT > 1 && sizeof(T) == 2)> xa(wv, lds.os, kk * 32);
        float m[8];
        eight(d.from0 + kk * 32, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] *= a.scale;
        st.add(wk, lds.qs, kk * 32, xa, m);
      }
    };
    if constexpr (kPlanes == S::kPlanes) next();
    __syncthreads();
    if (S::mine()) {
      // then X's: sum_j X_ij k_j
#pragma unroll
      for (int jj = 0; jj < C / 32; ++jj) {
        if (t0 + jj * 32 >= w.live) break;
        Frag<T> kf[S::kDT];
#pragma unroll
        for (int t = 0; t < S::kDT; ++t) kf[t] = frag_col<DK>(wk, lds.ks, jj * 32, (wave * S::kDT + t) * 16);
#pragma unroll
        for (int it = jj * 2; it < kTiles; ++it) {
          if (t0 + it * 16 >= w.live) break;
#pragma unroll
          for (int pl = 0; pl < kPieces<T>; ++pl) {
            const Frag<T> x = frag_col<32>(wx, lds.x(jj, it / 2, pl), 0, it % 2 * 16);
#pragma unroll
            for (int t = 0; t < S::kDT; ++t) acc[t][it] = mma(kf[t], x, acc[t][it]);
          }
        }
      }
      const uint32_t at = static_cast<uint32_t>(li) * kt + g4;
      auto put = [&](auto* out) {
        const Buffer to(out);
#pragma unroll
        for (int it = 0; it < kTiles; ++it)
#pragma unroll
          for (int t = 0; t < S::kDT; ++t) {
            const int ch = (wave * S::kDT + t) * 16;
            to.store(out, acc[t][it], t0 + it * 16 + li < w.live && ch + g4 < a.dk
                         ? (at + static_cast<uint32_t>(it * 16) * kt + ch) * static_cast<uint32_t>(sizeof(*out)) : kNowhere, 0);
          }
      };
      const int64_t first_query = kbase + static_cast<int64_t>(t0) * kt;
      if (a.share == 1) put(static_cast<T*>(a.dq) + first_query);
      else put(static_cast<float*>(a.dq) + first_query);
    }
    if constexpr (kPlanes < S::kPlanes) {
      __syncthreads();
      st.template publish<2, 3>(wv, lds.rs);
      __syncthreads();
      next();
    }
    __syncthreads();
  }
  if (a.ds0 && w.seg == 0) st.store(a.ds0 + w.bh * a.dk * a.dvd, a.dk, a.dvd, a.dvd);
}

template <typename T, int DK, int DV>
__device__ __forceinline__ void grad_keys(const LinArgs& a, const Where& w, GradLds<T, DK, DV>& lds) {
  using B = BlockOf<T, DK, DV>;
  using S = State<T, DK, DV>;
  constexpr int C = B::kC;
  constexpr int DT = DK / 16, NT = DV / 16;
  constexpr int kPlanes = GradLds<T, DK, DV>::kPlanes;
  const int wave = wave_id() - B::kWaves;
  const float* g = a.g + w.b * a.gb + w.h * a.gh;
  const int kt = a.heads * a.dk;
  const int64_t kbase = (w.b * a.seqlen * a.heads + w.h) * a.dk;
  const int vt = a.heads * a.dvd;
  const int64_t vbase = (w.b * a.seqlen * a.heads + w.h) * a.dvd;
  float* dg = a.dg + w.b * a.seqlen * a.heads + w.h;
  GradTiles<T, DK, DV> tiles(a, w);
  Places<T, DK> wk;
  Places<T, DV> wv;
  Places<T, 32> wx;
  float gx = 0.0f;
  if (w.c0 < w.c1) {
    tiles.skip(w.c1 - 1);
    tiles.load((w.c1 - 1) * C);
    if (wave == 0) scan_g(load_g<C>(a, g, (w.c1 - 1) * C, w.live), lds.decays[(w.c1 - 1) & 1]);
    if (w.c1 - 1 > w.c0) gx = load_g<C>(a, g, (w.c1 - 2) * C, w.live);
  }
  for (int c = w.c1 - 1; c >= w.c0; --c) {
    const int t0 = c * C;
    const Decays<C>& d = lds.decays[c & 1];
    wk.template here<true, true, true, false>();
    wv.template here<true, false, true, true>();
    wx.template here<false, true, false, false>();
    const int l = lane_here(), li = l & 15, g4 = (l >> 4) * 4;
    tiles.store(lds);
    __syncthreads();
    if (c > w.c0) {
      if (wave == c % B::kWaves) scan_g(gx, lds.decays[(c - 1) & 1]);
      if (c - 1 > w.c0) gx = load_g<C>(a, g, t0 - 2 * C, w.live);
    }
    // dk and dv of this wave's 16 keys: column j of every result tile
    const int j0 = wave * 16, j = j0 + li;
    const float gh = d.hi[j], gl = d.lo[j], toC = d.toC[j];
    Frag<T> kf[DK / 32], vf[DV / 32];
#pragma unroll
    for (int kk = 0; kk < DK / 32; ++kk) kf[kk] = frag_row<DK>(wk, lds.ks, j0, kk * 32);
#pragma unroll
    for (int kk = 0; kk < DV / 32; ++kk) vf[kk] = frag_row<DV>(wv, lds.vs, j0, kk * 32);
    f32x4 ak[DT], av[NT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) ak[dt] = zero4();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) av[nt] = zero4();
    float after = 0.0f;
    auto states = [&](auto from, auto to) {  // the products with planes from .. to - 1 of R
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        f32x4 s = zero4();
#pragma unroll
        for (int pl = decltype(from)::value; pl < decltype(to)::value; ++pl)
#pragma unroll
          for (int kk = 0; kk < DV / 32; ++kk)
            s = mma(frag_row<DV>(wv, lds.rs + (pl - decltype(from)::value) * S::kPlane, dt * 16, kk * 32), vf[kk], s);
        after += dot4(s, load4(at<T, DK>(lds.ks, j0, wk.perm, 0, dt * 16)));
        ak[dt] += s * toC;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 s = zero4();
#pragma unroll
        for (int pl = decltype(from)::value; pl < decltype(to)::value; ++pl)
#pragma unroll
          for (int kk = 0; kk < DK / 32; ++kk) 
            s = mma(frag_col_row<DV>(wv, lds.rs + (pl - decltype(from)::value) * S::kPlane, kk * 32, nt * 16), kf[kk], s);
        av[nt] += s * toC;
      }
    };
    // Queries from the last 32 down.  Beside the products, M_ij summed over the queries from t on (in
    // this lane's column; `later`: the tiles done) and then over the keys before t.
    float later = 0.0f;
#pragma unroll
    for (int kk = C / 32 - 1; kk >= 0; --kk) {
      if (kk < wave / 2) break;
      if (t0 + kk * 32 >= w.live) {  // no tokens; the table of rows has to be whole
        if (l < 32 && kk * 32 + l >= j0) lds.rows[wave][kk * 32 + l] = 0.0f;
        continue;
      }
      float p[8], x[8];
#pragma unroll
      for (int t = 1; t >= 0; --t) {
        const int i0 = kk * 32 + t * 16;
        if (i0 >= j0) {
          f32x4 sc = zero4(), dp = zero4();
#pragma unroll
          for (int n = 0; n < DK / 32; ++n) sc = mma(frag_row<DK>(wk, lds.qs, i0, n * 32), kf[n], sc);
#pragma unroll
          for (int n = 0; n < DV / 32; ++n) dp = mma(frag_row<DV>(wv, lds.os, i0, n * 32), vf[n], dp);
          float u[4];
          if (i0 > j0) {  // through the last token before the 16 queries
            const f32x4 e = load4(d.fromF + i0 + g4);
            const float to = __builtin_amdgcn_exp2f((d.hi[i0 - 1] - gh) + (d.lo[i0 - 1] - gl)) * a.scale;
#pragma unroll
            for (int r = 3; r >= 0; --r) {
              const float f = e[r] * to;
              p[t * 4 + r] = sc[r] * f;
              x[t * 4 + r] = dp[r] * f;
              u[r] = sc[r] * x[t * 4 + r] + (r < 3 ? u[r + 1] : 0.0f);
            }
          } else {
#pragma unroll
            for (int r = 3; r >= 0; --r) {
              const int i = i0 + g4 + r;
              const float f = __builtin_amdgcn_exp2f((d.hi[i] - gh) + (d.lo[i] - gl)) * a.scale;
              p[t * 4 + r] = i >= j ? sc[r] * f : 0.0f;
              x[t * 4 + r] = i >= j ? dp[r] * f : 0.0f;
              u[r] = (i > j ? sc[r] * x[t * 4 + r] : 0.0f) + (r < 3 ? u[r + 1] : 0.0f);
            }
          }
          float quads[4];  // this lane's rows of the tile, and the other lanes' of the column
          rows_of(u[0], quads);
          const float below = sum_after(quads, g4 / 4) + later;
          later += (quads[0] + quads[1]) + (quads[2] + quads[3]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = i0 + g4 + r;
            const float m = row_sum(j < i ? u[r] + below : 0.0f);
            if (li == 0) lds.rows[wave][i] = m;
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) p[t * 4 + r] = x[t * 4 + r] = 0.0f;
        }
      }
      Frag<T> piece[kPieces<T>];
      split(p, piece);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Frag<T> f = frag_col<DV>(wv, lds.os, kk * 32, nt * 16);
#pragma unroll
        for (int i = 0; i < kPieces<T>; ++i) av[nt] = mma(f, piece[i], av[nt]);
      }
      split(x, piece);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const Frag<T> f = frag_col<DK>(wk, lds.qs, kk * 32, dt * 16);
#pragma unroll
        for (int i = 0; i < kPieces<T>; ++i) ak[dt] = mma(f, piece[i], ak[dt]);
      }
#pragma unroll
      for (int i = 0; i < kPieces<T>; ++i) put_row_perm<32>(wx, lds.x(wave / 2, kk, i), wave % 2 * 16, 0, piece[i]);
    }
    if (c > w.c0) {
      tiles.skip(-1);
      tiles.load(t0 - C);
    }
    __syncthreads();
    states(std::integral_constant<int, 0>{}, std::integral_constant<int, kPlanes>{});
    if constexpr (kPlanes < S::kPlanes) {
      __syncthreads();
      __syncthreads();
      states(std::integral_constant<int, 2>{}, std::integral_constant<int, 3>{});
    }
    after = sum_rows(after);
    if (l < 16) lds.after[j] = after;
    const bool there = t0 + j < w.live;
    const uint32_t at = static_cast<uint32_t>(j) * kt + g4;
    if (a.share == 1)
      store_tiles(static_cast<T*>(a.dk_out) + (kbase + static_cast<int64_t>(t0) * kt), at, a.dk, there, ak);
    else
      store_tiles(static_cast<float*>(a.dk_out) + (kbase + static_cast<int64_t>(t0) * kt), at, a.dk, there, ak);
    store_tiles(static_cast<T*>(a.dv_out) + (vbase + static_cast<int64_t>(t0) * vt), static_cast<uint32_t>(j) * vt + g4,
                a.dvd, there, av);
    __syncthreads();
    if (wave == c % B::kWaves) {
      // lane t: token t0 + t.  The other waves write these arrays again only past the next barrier.
      const bool mine = l < C && t0 + l < w.live;
      float from = 0.0f, before = 0.0f, y = 0.0f;
      if (mine) {
#pragma unroll
        for (int i = 0; i < B::kWaves; ++i) from += lds.into[i][l];
        before = lds.after[l];
        from *= a.scale * d.from0[l];
        before *= d.toC[l];
#pragma unroll
        for (int i = 0; i < B::kWaves; ++i) y += lds.across[i];
        y *= d.from0[C - 1];
        for (int i = 0; i <= l / 16; ++i) y += lds.rows[i][l];
      }
      float r[4];
      rows_of(row_sum(from), r);
      from = row_suffix(from) + sum_after(r, l >> 4);
      rows_of(row_sum(before), r);
      before = dpp<kShr + 1>(row_prefix(before)) + sum_before(r, l >> 4);
      if (mine) dg[static_cast<int64_t>(t0 + l) * a.heads] = from + before + y;
    }
  }
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__((Pairs<BlockOf<T, DK, DV>>::kThreads)) __attribute__((amdgpu_waves_per_eu(
    grad_waves_for(sizeof(T), DK, DV)))) void linattn_grad_kernel(LinArgs a) {
  using B = BlockOf<T, DK, DV>;
  using G = Pairs<B>;
  constexpr int C = B::kC;
  __shared__ GradLds<T, DK, DV> lds;
  const Where w = where<B>(a, DV, blockIdx.x, gridDim.x);
  if (wave_id() < B::kWaves)
    grad_states<T, DK, DV>(a, w, lds);
  else
    grad_keys<T, DK, DV>(a, w, lds);
  const int64_t kt = static_cast<int64_t>(a.heads) * a.dk, kbase = (w.b * a.seqlen * a.heads + w.h) * a.dk;
  const int64_t vt = static_cast<int64_t>(a.heads) * a.dvd, vbase = (w.b * a.seqlen * a.heads + w.h) * a.dvd;
  if (a.share == 1) {
    zero_rest<G>(a, w, static_cast<T*>(a.dq) + kbase, kt, a.dk);
    zero_rest<G>(a, w, static_cast<T*>(a.dk_out) + kbase, kt, a.dk);
  } else {
    zero_rest<G>(a, w, static_cast<float*>(a.dq) + kbase, kt, a.dk);
    zero_rest<G>(a, w, static_cast<float*>(a.dk_out) + kbase, kt, a.dk);
  }
  zero_rest<G>(a, w, static_cast<T*>(a.dv_out) + vbase, vt, a.dvd);
  float* dg = a.dg + w.b * a.seqlen * a.heads + w.h;
  const int t_end = w.end * C < a.seqlen ? w.end * C : a.seqlen;
  for (int64_t t = (w.live > w.c0 * C ? w.live : w.c0 * C) + static_cast<int>(threadIdx.x); t < t_end; t += G::kThreads)
    dg[t * a.heads] = 0.0f;
}

// dq and dk of a shared head: the sum over the heads that read it, rounded once.  `in` is [tokens]
// [heads][dim] float32, `out` [tokens][heads / share][dim]; a thread takes 4 channels.  2002 tokens, 8 heads of 32
// on 2: 4.8 us for 5 MB, mostly the launch.
template <typename T>
__global__ __launch_bounds__(256) void linattn_share_kernel(const float* __restrict__ in_q, T* __restrict__ out_q,
                                                            const float* __restrict__ in_k, T* __restrict__ out_k,
                                                            int64_t tokens, int heads, int share, int dim) {
  const float* in = blockIdx.y ? in_k : in_q;
  T* out = blockIdx.y ? out_k : out_q;
  const int runs = dim / 4, per = heads / share * runs;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = id / per;
  if (t >= tokens) return;
  const int rest = static_cast<int>(id - t * per), hk = rest / runs, c = rest % runs * 4;
  const float* p = in + (t * heads + static_cast<int64_t>(hk) * share) * dim + c;
  f32x4 s = *reinterpret_cast<const f32x4*>(p);
  for (int i = 1; i < share; ++i) s += *reinterpret_cast<const f32x4*>(p + i * dim);
  store_acc(out + t * (heads / share) * dim + hk * dim + c, s);
}

// The gradient of a decay that all tokens of a head share: kDecayParts partial sums of dg, then
// their sum, each in a fixed order; few tokens in one go (2002 tokens, 8 heads: 4 us, one launch less).
constexpr int kDecayParts = 64;
constexpr int64_t kDecayTokens = 4096;  // up to here one launch sums them
__global__ __launch_bounds__(256) void linattn_decay_kernel(const float* __restrict__ in, float* __restrict__ out,
                                                            int64_t n, int heads) {
  __shared__ float s[256];
  const int h = blockIdx.x, parts = gridDim.y;
  float t = 0.0f;
  for (int64_t i = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(parts) * 256)
    t += in[i * heads + h];
  s[threadIdx.x] = t;
  __syncthreads();
#pragma unroll
  for (int m = 128; m >= 1; m >>= 1) {
    if (threadIdx.x < m) s[threadIdx.x] += s[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[static_cast<int64_t>(blockIdx.y) * heads + h] = s[0];
}

// ---------------------------------------------------------------------------------------------
// single tokens

struct StepArgs {
  View q, k, v;  // t stride unused
  const float* g;
  int64_t gb, gh;
  float* state;
  const int* slots;
  void* out;
  int64_t batch, pool;
  int heads, share, dk, dv;
  float scale;
};

// One workgroup per (sequence, head, 64 columns): 16 lanes hold 4 columns each, 16 rows at a time, all ROWS /
// 16 of them on their way at once.  The state is read once and written once in 16-byte accesses, which is all
// the time there is to it; the products are float32.  256 sequences, 12 heads of 64 x 64: 18 us a call for 101 MB,
// 5.5 TB/s (a part of the states is still in the 256 MB cache).
template <typename T, int ROWS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(6))) void linattn_step_kernel(StepArgs a) {
  constexpr int kN = ROWS / 16;
  __shared__ float qs[ROWS], ks[ROWS];
  __shared__ __align__(16) float red[4][64];
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / a.heads;
  const int h = static_cast<int>(bh - b * a.heads);
  const int n = blockIdx.y * 64 + (threadIdx.x & 15) * 4, row = threadIdx.x >> 4;
  const int64_t slot = a.slots ? a.slots[b] : b;
  T* out = static_cast<T*>(a.out) + bh * a.dv;
  if (slot < 0 || slot >= a.pool) {  // no state: the row is skipped
    if (threadIdx.x < 16 && n < a.dv) store_acc(out + n, zero4());
    return;
  }
  float* s = a.state + (slot * a.heads + h) * static_cast<int64_t>(a.dk) * a.dv;
  const bool mine = n < a.dv;
  const uint32_t off = row * a.dv + n, step = 16 * a.dv;
  f32x4 st[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    st[i] = zero4();
    if (mine && i * 16 + row < a.dk) st[i] = load4(s + (off + i * step));
  }
  const int hk = h / a.share;
  if (threadIdx.x < a.dk) {
    qs[threadIdx.x] = load1(static_cast<const T*>(a.q.p) + b * a.q.b + hk * a.q.h + threadIdx.x);
    ks[threadIdx.x] = load1(static_cast<const T*>(a.k.p) + b * a.k.b + hk * a.k.h + threadIdx.x);
  }
  f32x4 v = zero4();
  if (mine) {
    const T* vp = static_cast<const T*>(a.v.p) + b * a.v.b + h * a.v.h + n;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = load1(vp + r);
  }
  const float decay = __builtin_amdgcn_exp2f(a.g[b * a.gb + h * a.gh] * kLog2e);
  __syncthreads();
  f32x4 o = zero4();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int d = i * 16 + row;
    if (mine && d < a.dk) {
      const f32x4 u = st[i] * decay + v * ks[d];
      store_acc(s + (off + i * step), u);
      o += u * qs[d];
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = sum_rows(o[r]);
  if ((threadIdx.x & 63) < 16) store_acc(&red[threadIdx.x >> 6][(threadIdx.x & 15) * 4], o);
  __syncthreads();
  if (threadIdx.x < 16 && mine) {
    f32x4 t = zero4();
#pragma unroll
    for (int i = 0; i < 4; ++i) t += load4(&red[i][threadIdx.x * 4]);
    store_acc(out + n, t * a.scale);
  }
}

// ---------------------------------------------------------------------------------------------
// host side

constexpr int kMaxHeadDim = 128;
constexpr int64_t kMaxTokenStride = int64_t{1} << 24;  // a block's offsets fit 32 bits in bytes
// Estimates of plan(), us: the segments' pass as a share of the walk and its launches by [gradient]; the join, by a
// launch and per segment, or per MB read.
constexpr double kPassShare[2] = {0.4, 0.15}, kPassUs[2] = {7.0, 5.0}, kJoinUs = 3.0, kSegmentUs = 0.2, kMbUs = 0.1;
// Calls measured, us, joined by the walks / by a launch: 12 MB 17 / 20 (1 x 1000 tokens, 6 heads of 64 x 64, 16
// segments), 29 MB 38 / 40 (4 x 2048, 16 heads, 8 segments), 77 MB 108 / 104 (8 x 6085, 6 of 128 x 64, 10 segments).
constexpr double kChainMb = 64.0;
constexpr int64_t kPassWalks = 1024;    // workgroups wanted in each of the gradient's passes ..
constexpr int kMaxParts = 12;           // .. as long as no more than so many parts have to be joined
constexpr int kMaxSegments = 64;
constexpr int kSlice = 32;              // value channels of the narrowest workgroup

int pad_key(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }
int pad_value(int d) { return d <= 64 ? 64 : 128; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Plan {
  int blocks, segments, per, width, slices;
  int subs, parts;
  bool chain;
};
// A walk's workgroups by [gradient][float32][padded key channels 32, 64, 128][value channels of a workgroup 32, 64, 128]:
// how many of them a CU holds at a time, which is what the compiler's report of registers and LDS leaves room for (the build
// checks the report against this table), and the time of a block, us, where one has a CU for itself and where all places are
// taken (16 blocks of 64 tokens, 32 for float32 128 x 128; the gradient with its passes).  {}: no such kernel.  The gradient
// needs all value channels; in the forward 128 of them in one workgroup lose to two halves (us for 128: bfloat16 128 x 128
// 10.2 and 8.0, float32 64 x 128 12.1 and 11.6, 128 x 128 45 and 25).
struct Walk {
  int per_cu;
  double alone, full;
};
constexpr Walk kWalks[2][2][3][3] = {
    {{{{4, 2.5, 5.1}, {3, 3.1, 5.2}, {2, 4.6, 6.7}},
      {{4, 3.0, 6.3}, {3, 4.0, 7.1}, {2, 5.5, 8.1}},
      {{2, 4.1, 5.6}, {2, 6.0, 8.0}, {}}},
     {{{4, 4.0, 9.6}, {2, 5.1, 9.0}, {1, 8.7, 8.7}},
      {{3, 5.8, 11.2}, {2, 7.7, 11.6}, {}},
      {{2, 9.6, 13.0}, {1, 12.6, 12.6}, {}}}},
    {{{{}, {2, 7.5, 10.5}, {1, 10.4, 10.4}}, {{}, {2, 9.2, 14.8}, {1, 13.8, 13.8}}, {{}, {1, 14.1, 14.1}, {1, 30.4, 30.4}}},
     {{{}, {1, 13.1, 13.1}, {1, 21.4, 21.4}}, {{}, {1, 16.9, 16.9}, {1, 26.2, 26.2}}, {{}, {1, 31.1, 31.1}, {1, 35.7, 35.7}}}}};
constexpr int size_class(int channels) { return channels == 32 ? 0 : channels == 64 ? 1 : 2; }
template <typename T, int DK, int DV, bool BACK>
constexpr bool kHasWalk = kWalks[BACK][sizeof(T) == 4][size_class(DK)][size_class(DV)].per_cu > 0;
// A block's time in `n` workgroups: whole rounds of them over the chip, and a last one that leaves places free.
double block_time(const Walk& w, int64_t n) {
  const int64_t places = 256 * w.per_cu, rest = n % places;
  double us = static_cast<double>(n / places) * w.full;
  if (rest) {
    const int64_t on_cu = (rest + 255) / 256;
    us += w.per_cu > 1 ? w.alone + (w.full - w.alone) * static_cast<double>(on_cu - 1) / (w.per_cu - 1) : w.full;
  }
  return us;
}
// How a call is cut up.  The forward's value channels are independent, so several workgroups can share them (each
// repeats the scores), and a sequence can be cut into segments (a pass over the keys and values more, and
// a prefix over the segments).  Of all cuts the one with the least estimated time is taken: rounds of workgroups
// times blocks, a block's time as kWalks has it.  Calls measured, us, cut as taken / otherwise: bfloat16, 8 x 6085 tokens, 6
// heads of 128 x 64: 107 (10 segments) / 500 whole, 113 in 16; 1 x 6085, 6 of 64 x 64: 30 (20, halves of the channels) / 317
// whole, 31 in 32; 1 x 197, 6 of 64 x 64: 16 (whole, halves) / 17 not halved, 20 in 4; 128 x 197, 6 of 64 x 64: 30 (whole) / 45
// in 2, 36 in halves.  Float32 64 x 64: 8 x 6085, 6 heads: 151 (10) / 166 (8, halves); 16 x 3136, 12: 280 (5) / 326 (2, halves);
// 1 x 197, 6: 20 (4, halves) / 24 whole.
// The gradient needs all channels of a token together and is only cut into segments: bfloat16 64 x 64, 32 x 3136, 8 heads:
// 408 (2) / 481 whole; 2 x 3136, 8: 54 (13) / 62 (25); float32, 32 x 3136, 8 of 64 x 64: 830 (whole) / 913 in 2; 2 x 1001, 8 of 32
// x 128: 52 (16) / 329 whole.
Plan plan(int64_t batch, int64_t seqlen, int heads, int dk, int dv, vmscan_dtype dtype, bool back) {
  Plan best{};
  double least = 0.0;
  const bool f32 = dtype == VMSCAN_F32;
  for (int width = pad_value(dv); width >= (back ? pad_value(dv) : kSlice); width /= 2) {
    const int C = 16 * waves_of(f32 ? 4 : 2, pad_key(dk), width);
    const int blocks = static_cast<int>((seqlen + C - 1) / C);
    const int slices = (dv + width - 1) / width;
    const int64_t walks = batch * heads * slices;
    const Walk walk = kWalks[back][f32][size_class(pad_key(dk))][size_class(width)];
    if (walk.per_cu == 0) continue;
    for (int seg = 1; seg <= blocks && seg <= kMaxSegments; ++seg) {
      const int per = (blocks + seg - 1) / seg;
      if ((blocks + per - 1) / per != seg) continue;
      // Each round takes a block's time more to start and end; the gradient's, which is latency, even on a full CU.
      const double block = block_time(walk, walks * seg);
      const double rounds = static_cast<double>((walks * seg + 256 * walk.per_cu - 1) / (256 * walk.per_cu));
      double time = per * block + (back ? rounds * walk.alone : block);
      // Joining the segments' states: each walk reads those before it, or one more launch makes the sums.
      const double mb = 0.5e-6 * walks * seg * (seg - 1) * pad_key(dk) * width * 4;
      const bool chain = seg > 1 && mb < kChainMb && !(back && rereads(pad_key(dk), width));
      if (seg > 1) time += kPassShare[back] * time + kPassUs[back] + (back ? 2 : 1) * (chain ? kMbUs * mb : kJoinUs + kSegmentUs * seg);
      if (best.blocks == 0 || time < least) {
        least = time;
        best = Plan{blocks, seg, per, width, slices, 1, seg, chain};
      }
    }
  }
  // The gradient's passes are light and need more workgroups than its walk to fill the chip: they cut each
  // segment into parts.
  if (back && best.segments > 1) {
    const int64_t walks = batch * heads * best.segments;
    int64_t subs = (kPassWalks + walks - 1) / walks;
    if (subs > kMaxParts / best.segments) subs = kMaxParts / best.segments;
    if (subs > best.per) subs = best.per;
    if (subs < 1) subs = 1;
    const int part = static_cast<int>((best.per + subs - 1) / subs);
    best.subs = (best.per + part - 1) / part;
    best.per = best.subs * part;
    best.segments = (best.blocks + best.per - 1) / best.per;
    best.parts = (best.blocks + part - 1) / part;
    if (best.segments == 1) best.subs = best.parts = 1;
  }
  return best;
}

bool sizes_ok(int64_t batch, int64_t seqlen, int heads, int kheads, int dk, int dv) {
  if (batch < 1 || seqlen < 1 || heads < 1 || kheads < 1 || dk < 1 || dv < 1) return false;
  if (batch >= (int64_t{1} << 31) || seqlen >= (int64_t{1} << 30) || heads > 65536 || kheads > heads) return false;
  return batch * heads < (int64_t{1} << 31);
}
bool options_ok(int heads, int kheads, int dk, int dv, vmscan_dtype dtype) {
  return heads % kheads == 0 && dk % 8 == 0 && dv % 8 == 0 && dk <= kMaxHeadDim && dv <= kMaxHeadDim &&
         (dtype == VMSCAN_F32 || dtype == VMSCAN_BF16);
}

struct Layout {
  Plan p;
  size_t seg_s, seg_ds, seg_g, seg_dg, states, block_g, dq, dk, dg, parts, total;
};
Layout layout(int64_t batch, int64_t seqlen, int heads, int kheads, int dk, int dv, bool per_head, vmscan_dtype dtype,
              bool back) {
  Layout y{};
  y.p = plan(batch, seqlen, heads, dk, dv, dtype, back);
  const size_t bh = static_cast<size_t>(batch) * heads;
  const size_t state = static_cast<size_t>(pad_key(dk)) * y.p.slices * y.p.width * 4;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += round256(n);
    return was;
  };
  if (y.p.segments > 1) {
    y.seg_s = take(bh * y.p.parts * state);
    y.seg_g = take(bh * y.p.parts * 4);
    if (back) {
      y.seg_ds = take(bh * y.p.parts * state);
      y.seg_dg = take(bh * y.p.parts * 4);
    }
  }
  if (back) {
    y.states = take(bh * y.p.blocks * state);
    y.block_g = take(bh * y.p.blocks * 4);
    if (kheads != heads) {
      y.dq = take(bh * seqlen * dk * 4);
      y.dk = take(bh * seqlen * dk * 4);
    }
    if (per_head) {
      y.dg = take(bh * seqlen * 4);
      y.parts = take(static_cast<size_t>(kDecayParts) * heads * 4);
    }
  }
  y.total = at;
  return y;
}

// The pointers and strides of one [batch, seqlen, heads, dim] argument: 16-byte aligned.
vmscan_status view(View& v, const void* p, const int64_t* strides, vmscan_dtype dtype) {
  const int64_t run = dtype == VMSCAN_F32 ? 4 : 8;
  if (!aligned_to(p, 16)) return VMSCAN_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || (i == 1 && strides[i] >= kMaxTokenStride)) return VMSCAN_ERR_SHAPE;
    if (strides[i] % run) return VMSCAN_ERR_ALIGN;
  }
  v = View{p, strides[0], strides[1], strides[2]};
  return VMSCAN_OK;
}

// Calls f with the padded dk and the width of a workgroup's value channels.
template <typename F>
void with_dims(int dk, int width, F&& f) {
  using std::integral_constant;
  integral_constant<int, 32> t;
  integral_constant<int, 64> s;
  integral_constant<int, 128> b;
  if (dk <= 32) width == 32 ? f(t, t) : width == 64 ? f(t, s) : f(t, b);
  else if (dk <= 64) width == 32 ? f(s, t) : width == 64 ? f(s, s) : f(s, b);
  else width == 32 ? f(b, t) : width == 64 ? f(b, s) : f(b, b);
}

dim3 walks(const LinArgs& a) { return dim3(static_cast<unsigned>(a.batch * a.heads * a.segments * a.slices)); }

// The sums over the segments, where the walks do not make them themselves.
template <bool BACK>
void launch_prefix(const LinArgs& a, int dk, hipStream_t stream) {
  if (a.segments == 1 || a.chain) return;
  const int64_t n = a.batch * a.heads * (dk * a.ld / 4);
  hipLaunchKernelGGL((linattn_prefix_kernel<BACK>), dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, a,
                     dk);
}

template <typename T>
vmscan_status run_fwd(const LinArgs& a, int width, hipStream_t stream) {
  with_dims(a.dk, width, [&](auto dk, auto dv) {
    constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
    if constexpr (kHasWalk<T, DK, DV, false>) {
      const dim3 block(BlockOf<T, DK, DV>::kThreads);
      if (a.segments > 1)
        hipLaunchKernelGGL((linattn_segment_kernel<T, DK, DV, false, false>), walks(a), block, 0, stream, a);
      launch_prefix<false>(a, DK, stream);
      hipLaunchKernelGGL((linattn_fwd_kernel<T, DK, DV>), walks(a), block, 0, stream, a);
    }
  });
  return launched();
}

template <typename T>
vmscan_status run_bwd(LinArgs a, const Layout& y, unsigned char* ws, void* dq, void* dk, float* dg, bool per_head,
                      hipStream_t stream) {
  const bool shared = a.share > 1;
  a.dq = shared ? ws + y.dq : dq;
  a.dk_out = shared ? ws + y.dk : dk;
  a.dg = per_head ? reinterpret_cast<float*>(ws + y.dg) : dg;
  LinArgs b = a;  // the passes, whose segments are the parts
  b.segments = a.parts, b.per_segment = a.per_part;
  with_dims(a.dk, y.p.width, [&](auto k, auto v) {
    constexpr int DK = decltype(k)::value, DV = decltype(v)::value;
    if constexpr (kHasWalk<T, DK, DV, true>) {
      const dim3 block(BlockOf<T, DK, DV>::kThreads);
      if (a.segments > 1) {
        hipLaunchKernelGGL((linattn_passes_kernel<T, DK, DV>), dim3(2 * walks(b).x), block, 0, stream, b);
        launch_prefix<false>(b, DK, stream);
        launch_prefix<true>(b, DK, stream);
      } else {
        hipLaunchKernelGGL((linattn_segment_kernel<T, DK, DV, false, true>), walks(a), block, 0, stream, a);
      }
      hipLaunchKernelGGL((linattn_grad_kernel<T, DK, DV>), walks(a), dim3(2 * block.x), 0, stream, a);
    }
  });
  const int64_t tokens = a.batch * a.seqlen;
  if (shared) {
    const int64_t n = tokens * (a.heads / a.share) * (a.dk / 4);
    hipLaunchKernelGGL(linattn_share_kernel<T>, dim3(static_cast<unsigned>((n + 255) / 256), 2), dim3(256), 0, stream,
                       static_cast<const float*>(a.dq), static_cast<T*>(dq), static_cast<const float*>(a.dk_out),
                       static_cast<T*>(dk), tokens, a.heads, a.share, a.dk);
  }
  if (per_head && tokens <= kDecayTokens) {
    hipLaunchKernelGGL(linattn_decay_kernel, dim3(a.heads, 1), dim3(256), 0, stream, a.dg, dg, tokens, a.heads);
  } else if (per_head) {
    float* parts = reinterpret_cast<float*>(ws + y.parts);
    hipLaunchKernelGGL(linattn_decay_kernel, dim3(a.heads, kDecayParts), dim3(256), 0, stream, a.dg, parts, tokens,
                       a.heads);
    hipLaunchKernelGGL(linattn_decay_kernel, dim3(a.heads, 1), dim3(256), 0, stream, parts, dg,
                       static_cast<int64_t>(kDecayParts), a.heads);
  }
  return launched();
}

// What forward and gradient check alike; fills the shared arguments.
vmscan_status common_args(LinArgs& a, const void* q, const int64_t* qs, const void* k, const int64_t* ks,
                          const void* v, const int64_t* vs, const float* g, const int64_t* gs, const float* s0,
                          const int32_t* lengths, int64_t batch, int64_t seqlen, int heads, int kheads, int dk, int dv,
                          float scale, vmscan_dtype dtype) {
  if (!q || !qs || !k || !ks || !v || !vs || !g) return VMSCAN_ERR_NULL;
  if (!sizes_ok(batch, seqlen, heads, kheads, dk, dv)) return VMSCAN_ERR_SHAPE;
  if (!options_ok(heads, kheads, dk, dv, dtype)) return VMSCAN_ERR_UNSUPPORTED;
  vmscan_status st = view(a.q, q, qs, dtype);
  if (st == VMSCAN_OK) st = view(a.k, k, ks, dtype);
  if (st == VMSCAN_OK) st = view(a.v, v, vs, dtype);
  if (st != VMSCAN_OK) return st;
  if (!aligned_to(g, 4) || !aligned_to(s0, 16) || !aligned_to(lengths, 4)) return VMSCAN_ERR_ALIGN;
  a.g = g;
  a.gb = gs ? gs[0] : 0, a.gt = gs ? gs[1] : 0, a.gh = gs ? gs[2] : 1;
  if (a.gb < 0 || a.gt < 0 || a.gh < 0) return VMSCAN_ERR_SHAPE;
  a.s0 = s0, a.lengths = lengths;
  a.batch = batch, a.seqlen = static_cast<int>(seqlen), a.heads = heads, a.share = heads / kheads;
  a.dk = dk, a.dvd = dv, a.scale = scale;
  return VMSCAN_OK;
}

void place(LinArgs& a, const Layout& y, unsigned char* ws) {
  a.blocks = y.p.blocks, a.segments = y.p.segments, a.per_segment = y.p.per;
  a.slices = y.p.slices, a.ld = y.p.slices * y.p.width;
  a.subs = y.p.subs, a.parts = y.p.parts, a.per_part = a.per_segment / a.subs;
  a.chain = y.p.chain;
  a.seg_s = reinterpret_cast<float*>(ws + y.seg_s);
  a.seg_ds = reinterpret_cast<float*>(ws + y.seg_ds);
  a.seg_g = reinterpret_cast<float*>(ws + y.seg_g);
  a.states = reinterpret_cast<float*>(ws + y.states);
  a.block_g = reinterpret_cast<float*>(ws + y.block_g);
  a.seg_dg = reinterpret_cast<float*>(ws + y.seg_dg);
}

// Whether a state output may be written where `in` lies: not at all, or exactly there.  A walk that joins the states
// itself reads them while another one may write its output, so in place the sums are a launch of their own.
bool states_ok(const LinArgs& a, const float* out, const float* in) {
  if (!out || !in || out == in) return true;
  const uintptr_t p = reinterpret_cast<uintptr_t>(out), q = reinterpret_cast<uintptr_t>(in);
  const uintptr_t n = static_cast<uintptr_t>(a.batch) * a.heads * a.dk * a.dvd * sizeof(float);
  return p < q ? q - p >= n : p - q >= n;
}

vmscan_status need_workspace(const void* ws, size_t have, size_t need, const LinArgs& a, const Plan& p, bool back) {
  // workgroups of the largest launch: the forward's walk, the gradient's two passes (its walk has twice the threads)
  if (a.batch * a.heads * (back ? 2 * p.parts : p.segments) * p.slices > kMaxBlocks256) return VMSCAN_ERR_SHAPE;
  if (!aligned_to(ws, 16)) return VMSCAN_ERR_ALIGN;
  return need && (!ws || have < need) ? VMSCAN_ERR_WORKSPACE : VMSCAN_OK;
}

}  // namespace

extern "C" {

vmscan_status vmscan_linattn_plan(int64_t batch, int64_t seqlen, int heads, int dk, int dv, vmscan_dtype dtype,
                                  int gradient, int32_t* cut) {
  if (!cut) return VMSCAN_ERR_NULL;
  if (!sizes_ok(batch, seqlen, heads, heads, dk, dv)) return VMSCAN_ERR_SHAPE;
  if (!options_ok(heads, heads, dk, dv, dtype) || (gradient != 0 && gradient != 1)) return VMSCAN_ERR_UNSUPPORTED;
  const Plan p = plan(batch, seqlen, heads, dk, dv, dtype, gradient != 0);
  cut[0] = 16 * waves_of(dtype == VMSCAN_F32 ? 4 : 2, pad_key(dk), p.width);
  cut[1] = p.width, cut[2] = p.segments, cut[3] = p.subs;
  cut[4] = p.parts == 1 ? VMSCAN_JOIN_NONE : p.chain ? VMSCAN_JOIN_WALK : VMSCAN_JOIN_LAUNCH;
  return VMSCAN_OK;
}

size_t vmscan_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int dk, int dv,
                                          vmscan_dtype dtype) {
  if (!sizes_ok(batch, seqlen, heads, heads, dk, dv) || !options_ok(heads, heads, dk, dv, dtype)) return 0;
  return layout(batch, seqlen, heads, heads, dk, dv, false, dtype, false).total;
}

vmscan_status vmscan_linattn_fwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                                 const void* v, const int64_t* v_strides, const float* log_decay,
                                 const int64_t* decay_strides, const float* initial_state, const int32_t* lengths,
                                 void* out, float* final_state, int64_t batch, int64_t seqlen, int heads, int kheads,
                                 int dk, int dv, float scale, vmscan_dtype dtype, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  LinArgs a{};
  if (!out) return VMSCAN_ERR_NULL;
  vmscan_status st = common_args(a, q, q_strides, k, k_strides, v, v_strides, log_decay, decay_strides, initial_state,
                                 lengths, batch, seqlen, heads, kheads, dk, dv, scale, dtype);
  if (st != VMSCAN_OK) return st;
  if (!aligned_to(out, 16) || !aligned_to(final_state, 16)) return VMSCAN_ERR_ALIGN;
  const Layout y = layout(batch, seqlen, heads, kheads, dk, dv, false, dtype, false);
  st = need_workspace(workspace, workspace_bytes, y.total, a, y.p, false);
  if (st != VMSCAN_OK) return st;
  if (!states_ok(a, final_state, initial_state)) return VMSCAN_ERR_UNSUPPORTED;
  place(a, y, static_cast<unsigned char*>(workspace));
  a.out = out, a.sT = final_state;
  if (final_state && final_state == initial_state) a.chain = false;
  return dtype == VMSCAN_F32 ? run_fwd<float>(a, y.p.width, stream)
                            : run_fwd<uint16_t>(a, y.p.width, stream);
}

size_t vmscan_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int kheads, int dk, int dv,
                                          int per_head, vmscan_dtype dtype) {
  if (!sizes_ok(batch, seqlen, heads, kheads, dk, dv) || !options_ok(heads, kheads, dk, dv, dtype)) return 0;
  return layout(batch, seqlen, heads, kheads, dk, dv, per_head != 0, dtype, true).total;
}

vmscan_status vmscan_linattn_bwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                                 const void* v, const int64_t* v_strides, const float* log_decay,
                                 const int64_t* decay_strides, const float* initial_state, const int32_t* lengths,
                                 const void* dout, const int64_t* dout_strides, const float* dfinal_state, void* dq,
                                 void* dk_out, void* dv_out, float* dlog_decay, float* dinitial_state, int64_t batch,
                                 int64_t seqlen, int heads, int kheads, int dk, int dv, float scale,
                                 vmscan_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  LinArgs a{};
  if (!dout || !dout_strides || !dq || !dk_out || !dv_out || !dlog_decay) return VMSCAN_ERR_NULL;
  vmscan_status st = common_args(a, q, q_strides, k, k_strides, v, v_strides, log_decay, decay_strides, initial_state,
                                 lengths, batch, seqlen, heads, kheads, dk, dv, scale, dtype);
  if (st != VMSCAN_OK) return st;
  st = view(a.dout, dout, dout_strides, dtype);
  if (st != VMSCAN_OK) return st;
  const void* ptrs[] = {dfinal_state, dq, dk_out, dv_out, dinitial_state};
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return VMSCAN_ERR_ALIGN;
  if (!aligned_to(dlog_decay, 4)) return VMSCAN_ERR_ALIGN;
  const bool per_head = decay_strides == nullptr;
  const Layout y = layout(batch, seqlen, heads, kheads, dk, dv, per_head, dtype, true);
  st = need_workspace(workspace, workspace_bytes, y.total, a, y.p, true);
  if (st != VMSCAN_OK) return st;
  if (kheads != heads && batch * seqlen * kheads * (dk / 4) / 256 >= kMaxBlocks256) return VMSCAN_ERR_SHAPE;
  if (!states_ok(a, dinitial_state, dfinal_state) || !states_ok(a, dinitial_state, initial_state))
    return VMSCAN_ERR_UNSUPPORTED;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  place(a, y, ws);
  a.dsT = dfinal_state, a.ds0 = dinitial_state, a.dv_out = dv_out;
  if (dinitial_state && (dinitial_state == dfinal_state || dinitial_state == initial_state)) a.chain = false;
  return dtype == VMSCAN_F32 ? run_bwd<float>(a, y, ws, dq, dk_out, dlog_decay, per_head, stream)
                             : run_bwd<uint16_t>(a, y, ws, dq, dk_out, dlog_decay, per_head, stream);
}

vmscan_status vmscan_linattn_step(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                                  const void* v, const int64_t* v_strides, const float* log_decay,
                                  const int64_t* decay_strides, float* state, const int32_t* slots, void* out,
                                  int64_t batch, int64_t pool, int heads, int kheads, int dk, int dv, float scale,
                                  vmscan_dtype dtype, hipStream_t stream) {
  if (!q || !q_strides || !k || !k_strides || !v || !v_strides || !log_decay || !state || !out) return VMSCAN_ERR_NULL;
  if (!sizes_ok(batch, 1, heads, kheads, dk, dv) || pool < 1 || pool >= (int64_t{1} << 31)) return VMSCAN_ERR_SHAPE;
  if ((!slots && pool != batch) || batch * heads > kMaxBlocks256) return VMSCAN_ERR_SHAPE;
  if (!options_ok(heads, kheads, dk, dv, dtype)) return VMSCAN_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, v};
  for (const void* p : ptrs)
    if (!aligned_to(p, dtype == VMSCAN_F32 ? 4 : 2)) return VMSCAN_ERR_ALIGN;
  if (!aligned_to(state, 16) || !aligned_to(out, 16) || !aligned_to(log_decay, 4) || !aligned_to(slots, 4))
    return VMSCAN_ERR_ALIGN;
  StepArgs a{};
  a.q = View{q, q_strides[0], 0, q_strides[1]};
  a.k = View{k, k_strides[0], 0, k_strides[1]};
  a.v = View{v, v_strides[0], 0, v_strides[1]};
  a.g = log_decay;
  a.gb = decay_strides ? decay_strides[0] : 0, a.gh = decay_strides ? decay_strides[1] : 1;
  a.state = state, a.slots = slots, a.out = out, a.batch = batch, a.pool = pool;
  a.heads = heads, a.share = heads / kheads, a.dk = dk, a.dv = dv, a.scale = scale;
  const dim3 grid(static_cast<unsigned>(batch * heads), static_cast<unsigned>((dv + 63) / 64));
  auto launch = [&](auto rows) {
    constexpr int ROWS = decltype(rows)::value;
    if (dtype == VMSCAN_F32)
      hipLaunchKernelGGL((linattn_step_kernel<float, ROWS>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((linattn_step_kernel<uint16_t, ROWS>), grid, dim3(256), 0, stream, a);
  };
  if (dk <= 64) launch(std::integral_constant<int, 64>{});
  else launch(std::integral_constant<int, 128>{});
  return launched();
}

}  // extern "C"
