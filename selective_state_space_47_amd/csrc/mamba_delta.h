// mamba_delta.h -- what the gated delta rule's kernels share (mamba_delta.hip, _step.hip, _bwd.hip):
// the chunk form, matrix-core operands, launch arguments and host-side validation.
//
// Per value head, with state S (dk x dv), keys k and queries q of its key head:
//     S~_t = exp(g_t) S_{t-1},  e_t = v_t - S~_t^T k_t,  S_t = S~_t + beta_t k_t e_t^T,
//     o_t = scale S_t^T q_t
// A chunk of kC = 64 tokens with S the state before it, G_i = g_1 + .. + g_i and
// D_ij = exp(G_i - G_j) is, row by row of K, Q, V (64 x d),
//     A_ij = D_ij (k_i . k_j) beta_j  (j < i),   T = (I + A)^-1
//     Y = V - diag(exp G) K S,   E = T Y
//     P_ij = scale D_ij (q_i . k_j) beta_j  (j <= i)
//     O = scale diag(exp G) Q S + P E
//     S' = exp(G_64) S + K^T diag(c) E,   c_j = exp(G_64 - G_j) beta_j
// T and P do not depend on the state: one launch makes them for all chunks.
#pragma once
#include <cmath>

#include "mamba_common.h"

namespace mamba {
namespace delta {

constexpr int kC = 64;          // tokens per chunk
constexpr int kMaxDk = 128;
constexpr int64_t kMaxStride = (int64_t)1 << 22;  // elements between tokens: 64 tokens of fp32 stay below 2^31 bytes
constexpr int64_t kMaxDv = 1024;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Operands of the 16 x 16 matrix instructions.  Lane l (g = l / 16, r = l % 16) holds for operand A
// the row r, for operand B the column r, and of the accumulator C the column r and rows 4g .. 4g+3.
// The k values that the lanes hold may be any permutation of the depth, the same one in A and B: all
// tiles are read in the order in which accumulators hold their rows, so that the accumulators of one
// product are (converted in place) the operand of the next and nothing moves between lanes.
//   kDepth  depth of one operand: kDepth / 16 accumulator tiles
//   pack    accumulators -> operand
//   split   accumulators -> P operands that together hold the value to 8 P bits (fp32: one, whole)
//   parts   how many operands stand for a value of which P are wanted
template <typename E>
struct Mma;

template <>
struct Mma<uint16_t> {
  static constexpr int kDepth = 32;
  static constexpr int kTiles = 2;
  static constexpr int parts(int wanted) { return wanted; }
  using Frag = bf16x8;
  template <int P> struct Parts { Frag p[P]; };
  __device__ static __forceinline__ Frag join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ static __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // words of two values, so that the conversion of a pair serves the operand and the remainder
  __device__ static __forceinline__ Frag pack(const f32x4* c) {
    return __builtin_bit_cast(Frag, make_uint4(pack_bf16(make_float2(c[0][0], c[0][1])),
                                               pack_bf16(make_float2(c[0][2], c[0][3])),
                                               pack_bf16(make_float2(c[1][0], c[1][1])),
                                               pack_bf16(make_float2(c[1][2], c[1][3]))));
  }
  template <int P>
  __device__ static __forceinline__ Parts<P> split(const f32x4* c) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c[i >> 2][i & 3];
    Parts<P> s;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = pack_bf16(make_float2(v[2 * i], v[2 * i + 1]));
        const float2 f = unpack(h[i]);
        v[2 * i] -= f.x;
        v[2 * i + 1] -= f.y;
      }
      s.p[p] = __builtin_bit_cast(Frag, make_uint4(h[0], h[1], h[2], h[3]));
    }
    return s;
  }
};

template <>
struct Mma<float> {
  static constexpr int kDepth = 16;
  static constexpr int kTiles = 1;
  static constexpr int parts(int) { return 1; }
  using Frag = f32x4;
  template <int P> struct Parts { Frag p[P]; };
  // four 4-deep fp32 instructions: step j takes element j of both operands (k = 4g + j)
  __device__ static __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ Frag pack(const f32x4* c) { return c[0]; }
  template <int P>
  __device__ static __forceinline__ Parts<P> split(const f32x4* c) { return {{c[0]}}; }
};

typedef __attribute__((address_space(3))) const char* lds_ptr;

template <typename V>
__device__ __forceinline__ V lds_read(lds_ptr p) {
  return *reinterpret_cast<__attribute__((address_space(3))) const V*>(p);
}
// transposing LDS read of bf16: 16 lanes address 4 rows of 16 values, lane r the values 4 (r % 4) ..
// of row r / 4, and lane r receives the r-th value of the 4 rows
__device__ __forceinline__ bf16x4 lds_tr(lds_ptr p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// Swizzle of the 16-byte words of LDS rows.  One pass of a 16-byte read serves 8 lanes of one group and 8
// of the next: rows 0-3 and 12-15 of group g with rows 4-11 of group g + 1, or the other way round (counted:
// with the plain row number / 4 in place of this code an operand read took two passes more).  The two sets
// of rows get codes that never differ by 1, as their words do.
__device__ __forceinline__ int row_code(int t) {
  const int q = (t >> 2) & 3;  // 0 2 3 1
  return 2 * ((q ^ (q >> 1)) & 1) + (q >> 1);
}

// A 64-token tile of keys or queries in LDS: rows of kRow bytes, the 16-byte word w of row t kept at
// w ^ key(t).  With this key the rows of one pass of an operand read, and the 4 rows x 4 words of a
// transposing read (of rows of 8 or more words), lie in different banks.
template <typename E, int DK>
struct KeyTile {
  static constexpr int kRow = DK * (int)sizeof(E);
  static constexpr int kWords = kRow / 16;
  static constexpr int kBytes = kC * kRow;
  __device__ static __forceinline__ int key(int t) {
    return kWords >= 16  ? 4 * (t & 3) + row_code(t)
           : kWords == 8 ? 4 * ((t >> 1) & 1) + row_code(t)
                         : row_code(t);
  }
  // lane addresses of one tile
  int row0, tr0, g, r;
  __device__ __forceinline__ KeyTile(int lane) : g(lane >> 4), r(lane & 15) {
    row0 = r * kRow;
    tr0 = sizeof(E) == 2 ? (4 * g + (r >> 2)) * kRow : 4 * g * kRow + 4 * (r & 3);
  }
  // operand with rows = tokens 16 m + r, k = values [kDepth kb, kDepth (kb + 1)) in natural order
  __device__ __forceinline__ typename Mma<E>::Frag rows(lds_ptr t, int m, int kb) const {
    return lds_read<typename Mma<E>::Frag>(t + 16 * m * kRow + row0 + (((4 * kb + g) ^ key(r)) << 4));
  }
  // the value of the keys that row 4 g + x of accumulator tile m stands for, so that `rows` reads
  // accumulator order in whole words
  __device__ static __forceinline__ int value(int m, int g, int x) {
    return sizeof(E) == 2 ? 32 * (m >> 1) + 8 * g + 4 * (m & 1) + x : 16 * m + 4 * g + x;
  }
  // transposed operand: rows = values of accumulator tile m, k = tokens of block kb in accumulator
  // order, or (kNatural) in natural order
  template <bool kNatural = false>
  __device__ __forceinline__ typename Mma<E>::Frag cols(lds_ptr t, int m, int kb) const {
    t += Mma<E>::kDepth * kb * kRow + tr0;
    if constexpr (sizeof(E) == 2) {
      const int w = 4 * (m >> 1) + (r & 3), half = 8 * (m & 1);
      if constexpr (kNatural) {
        t += 4 * g * kRow + half;  // tokens 8 g .. instead of 4 g ..
        const int row = 8 * g + (r >> 2);
        return Mma<E>::join(lds_tr(t + ((w ^ key(row)) << 4)),
                            lds_tr(t + 4 * kRow + ((w ^ key(row + 4)) << 4)));
      }
      t += ((w ^ key(4 * g + (r >> 2))) << 4) + half;
      return Mma<E>::join(lds_tr(t), lds_tr(t + 16 * kRow));
    } else {
      typename Mma<E>::Frag f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[j] = lds_read<float>(t + j * kRow + (((4 * m + (r >> 2)) ^ key(4 * g + j)) << 4));
      return f;
    }
  }
};

// Rows of kCols values (values, output gradients), read in accumulator order, column by column.  Words are
// swizzled in pairs (bf16; fp32: in fours), a wave's 16 columns, so that the rows of one read lie in
// different banks.
template <typename E, int kCols>
struct ValueTile {
  static constexpr int kRow = kCols * (int)sizeof(E);
  static constexpr int kWords = kRow / 16;
  static constexpr int kBytes = kC * kRow;
  __device__ static __forceinline__ int key(int t) {
    return sizeof(E) == 4 ? 4 * ((t >> 2) & 3) : kWords >= 16 ? 2 * (t & 7) : 2 * ((t >> 1) & 3);
  }
  int at, g;
  // this wave's 16 columns begin at `col`
  __device__ __forceinline__ ValueTile(int lane, int col) : g(lane >> 4) {
    const int r = lane & 15, t = sizeof(E) == 2 ? 4 * g + (r >> 2) : 4 * g;
    const int byte = sizeof(E) == 2 ? 2 * col + 8 * (r & 3) : (col + r) * 4;
    at = t * kRow + (((byte >> 4) ^ key(t)) << 4) + (byte & 15);
  }
  // rows (tokens) 16 m + 4 g .. +3 of column r, in storage type
  __device__ __forceinline__ auto four(lds_ptr t, int m) const {
    t += 16 * m * kRow + at;
    if constexpr (sizeof(E) == 2)
      return lds_tr(t);
    else
      return f32x4{lds_read<float>(t), lds_read<float>(t + kRow), lds_read<float>(t + 2 * kRow),
                   lds_read<float>(t + 3 * kRow)};
  }
  __device__ __forceinline__ f32x4 tile(lds_ptr t, int m) const {
    return __builtin_convertvector(four(t, m), f32x4);
  }
  // the operand of token block kb
  __device__ __forceinline__ typename Mma<E>::Frag operand(lds_ptr t, int kb) const {
    if constexpr (sizeof(E) == 2)
      return Mma<E>::join(four(t, 2 * kb), four(t, 2 * kb + 1));
    else
      return four(t, kb);
  }
};

// Lower triangular 64 x 64 matrix in LDS and in the workspace: blocks of kDepth columns, block kb
// holding rows kDepth kb .. 63 of 64 bytes each, four words; word w of a row holds the values that
// lane group w reads in accumulator order and is kept at w ^ row_code(row).
template <typename E>
struct TriTile {
  static constexpr int kD = Mma<E>::kDepth;
  static constexpr int kBlocks = kC / kD;
  static constexpr int first_row(int kb) { return kb * kC - kD * (kb * (kb - 1) / 2) - kD * kb; }
  // byte of row t, block kb (t >= kD kb)
  __device__ static __forceinline__ int row_at(int kb, int t) { return (first_row(kb) + t) * 64; }
  static constexpr int kRows = kC * kBlocks - kD * (kBlocks * (kBlocks - 1) / 2);
  static constexpr int kBytes = kRows * 64;
  // byte of word w of row t, block kb
  __device__ static __forceinline__ int word_at(int kb, int t, int w) {
    return row_at(kb, t) + ((w ^ row_code(t)) << 4);
  }
  int row0, g, r;
  __device__ __forceinline__ TriTile(int lane) : g(lane >> 4), r(lane & 15) {
    row0 = r * 64 + ((g ^ row_code(r)) << 4);
  }
  // operand with rows 16 m + r, k = columns of block kb
  __device__ __forceinline__ typename Mma<E>::Frag rows(lds_ptr t, int m, int kb) const {
    return lds_read<typename Mma<E>::Frag>(t + row_at(kb, 16 * m) + row0);
  }
  // transposed operand: rows = columns 16 m + r, k = rows of block ib (ib >= the block of column 16 m)
  // in accumulator order
  __device__ __forceinline__ typename Mma<E>::Frag cols(lds_ptr t, int m, int ib) const {
    if constexpr (sizeof(E) == 2) {
      t += row_at(m >> 1, 32 * ib) + (4 * g + (r >> 2)) * 64 + (((r & 3) ^ row_code(4 * g)) << 4) +
           8 * (m & 1);
      return Mma<E>::join(lds_tr(t), lds_tr(t + 16 * 64));
    } else {
      t += row_at(m, 16 * ib) + 4 * g * 64 + (((r >> 2) ^ row_code(4 * g)) << 4) + 4 * (r & 3);
      return typename Mma<E>::Frag{lds_read<float>(t), lds_read<float>(t + 64),
                                   lds_read<float>(t + 128), lds_read<float>(t + 192)};
    }
  }
};

// Copies from global memory straight into LDS, 16 bytes per lane and 1 KB per wave instruction:
// lane l's word goes to lds + 16 l.  Words at or past `bytes` of the buffer read as zero.  There is
// no register to wait for; the wave waits for its copies with copies_done().
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  i32x4 d;
  d[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  d[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  d[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  d[3] = 0x00020000;
  return d;
}
__device__ __forceinline__ void copy_lds(i32x4 buf, uint32_t off, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  uint32_t saved;  // the compiler's m0
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(off), "s"(buf), "s"(lds)
      : "memory");
}
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every buffer
// Four values of one row, rounded to the storage type, to a buffer; an offset past it drops them (no
// branch around the store, so that the chunk's loop stays one block for the scheduler).
template <typename E>
__device__ __forceinline__ void store_four(__amdgpu_buffer_rsrc_t buf, uint32_t off, f32x4 v) {
  typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  if constexpr (sizeof(E) == 2)
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(make_float2(v[0], v[1])),
                                                pack_bf16(make_float2(v[2], v[3]))},
                                          buf, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), buf, off, 0, 0);
}
// every copy of this wave has landed, and every wave of the workgroup has come here
__device__ __forceinline__ void copies_done() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// Copy of R rows of a key tile layout (rows of Tile::kRow bytes, swizzled) from rows in memory by NW
// waves: instruction j fills the tile's j-th KB, wave w takes the instructions w, w + NW, ...
template <typename E, typename Tile, int R, int NW>
struct RowCopy {
  static constexpr int kI = R * Tile::kRow / 1024 / NW;
  static_assert(kI * NW * 1024 == R * Tile::kRow, "whole wave instructions");
  uint32_t off[kI];
  // `stride` elements between rows, `cols` values of a row that exist
  __device__ __forceinline__ RowCopy(int w, int lane, int64_t stride, int cols) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int at = (w + i * NW) * 64 + lane, t = at / Tile::kWords;
      const int c = ((at % Tile::kWords) ^ Tile::key(t)) * (16 / (int)sizeof(E));
      off[i] = c < cols ? (uint32_t)(t * stride + c) * (uint32_t)sizeof(E) : kOutside;
    }
  }
  __device__ __forceinline__ void operator()(i32x4 buf, uint32_t lds, int w) const {
#pragma unroll
    for (int i = 0; i < kI; ++i) copy_lds(buf, off[i], lds + (w + i * NW) * 1024);
  }
};
// rows of `cols` values, `n` of them, as a buffer
template <typename E>
__device__ __forceinline__ i32x4 rows_buffer(const E* p, int64_t n, int64_t stride, int cols) {
  return buffer_of(p, (uint32_t)(((n - 1) * stride + cols) * (int64_t)sizeof(E)));
}
// kBytes (whole KBs) as they lie
template <int kBytes, int NW>
__device__ __forceinline__ void copy_linear(const void* p, uint32_t lds, int w, int lane) {
  const i32x4 buf = buffer_of(p, kBytes);
#pragma unroll
  for (int i = 0; i < (kBytes / 1024 + NW - 1) / NW; ++i)
    if ((i + 1) * NW <= kBytes / 1024 || w + i * NW < kBytes / 1024)
      copy_lds(buf, (w + i * NW) * 1024 + lane * 16, lds + (w + i * NW) * 1024);
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}

// exp(x) for x <= 0 (and moderate x > 0)
__device__ __forceinline__ float exp_f32(float x) { return fast_exp2(x * kLog2e); }

// ------------------------------------------------------------------ launch arguments

struct Args {
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  const void* beta;
  const float* s0;         // (nseq, hv, dk, dv) or NULL: zero
  const int64_t* offsets;  // (nseq + 1) token offsets of packed sequences, or NULL
  void* out;               // (tokens, hv, dv)
  float* last;             // (nseq, hv, dk, dv) or NULL
  char* ws;                // per (chunk slot, value head): ChunkWs, ws_item bytes
  int64_t ws_item;
  char* e_img;             // backward only, per (chunk slot, value head): images of E,
  char* s_img;             // of the state before the chunk
  char* s_low;             // (bf16 storage: and what bf16 leaves of it, a byte per value)
  char* ds_img;            // of the adjoint of the state after it
  char* ds_low;            // (bf16 storage: and what bf16 leaves of it, as bf16)
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  int64_t seqlen;          // tokens per sequence (packed: of all sequences)
  int64_t nseq;
  int64_t slots;           // chunk slots
  // long sequences in segments of seg_chunks chunks (0: one segment per sequence)
  int64_t seg_chunks;
  int64_t seg_slots;
  float* seg_state;        // (segment slots, hv, dk, dv): the state before each segment
  float* seg_map;          // (segment slots, hv, dk, dk): what a segment does to the state before it
  int32_t hk, hv, rep, dk, dv;
  float scale;
};

// Tokens of chunk `c` of sequence `seq`: first (global) token and count, 0 past the end.  Offsets
// are clamped to the tokens there are, so that a wrong offset reads other tokens, never past them.
struct Span {
  int64_t first;
  int64_t len;
};
__device__ __forceinline__ Span seq_span(const Args& a, int64_t seq) {
  if (!a.offsets) return {seq * a.seqlen, a.seqlen};
  const int64_t b = min(max(a.offsets[seq], (int64_t)0), a.seqlen);
  const int64_t e = min(max(a.offsets[seq + 1], (int64_t)0), a.seqlen);
  return {b, max(e - b, (int64_t)0)};
}

// Slots of `unit` tokens (chunks, segments): sequence s owns the slots from slot_base(s) on.  For packed
// sequences offset / unit + s leaves room for a last, partial one in each, without a scan over the lengths.
__device__ __forceinline__ int64_t slot_base(const Args& a, int64_t seq, int64_t first,
                                             int64_t unit = kC) {
  return a.offsets ? first / unit + seq : seq * ((a.seqlen + unit - 1) / unit);
}

// slot -> sequence (the last one whose base is not past the slot)
__device__ __forceinline__ int64_t slot_seq(const Args& a, int64_t slot, int64_t unit = kC) {
  if (!a.offsets) return slot / ((a.seqlen + unit - 1) / unit);
  int64_t lo = 0, hi = a.nseq - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    const int64_t first = min(max(a.offsets[mid], (int64_t)0), a.seqlen);
    if (first / unit + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The sequence of a workgroup of the state passes: packed sequences (up to a wave's lanes of them) the longest
// first, so that none starts late and runs on alone.
__device__ __forceinline__ int64_t seq_by_length(const Args& a, int64_t rank) {
  if (!a.offsets || a.nseq < 2 || a.nseq > 64) return rank;
  const int lane = threadIdx.x & 63, n = (int)a.nseq;
  const int len = lane < n ? (int)min(seq_span(a, lane).len, (int64_t)0x7fffffff) : -1;
  int before = 0;  // sequences that come before this lane's
  for (int j = 0; j < n; ++j) {
    const int other = __shfl(len, j);
    before += other > len || (other == len && j < lane);
  }
  const uint64_t found = __ballot(lane < n && before == (int)rank);
  return __builtin_amdgcn_readfirstlane(__builtin_ctzll(found));
}

// Workgroups in groups of `group` that read the same keys: a group stays on one XCD (one L2), and
// consecutive groups, which are heads of one sequence and so equally long, go to different XCDs.
// (Workgroup id runs on XCD id % 8.)  A bijection of [0, n), n a multiple of `group`.
__device__ __forceinline__ int64_t spread_index(uint32_t id, uint32_t n, uint32_t group) {
  const uint32_t whole = n / group / 8 * 8 * group;
  if (id >= whole) return id;
  const uint32_t x = id & 7, l = id >> 3;
  return (int64_t)(l / group * 8 + x) * group + l % group;
}

// Parts of T that the forward uses and the workspace holds: T is unit on its diagonal and small off
// it, so that two parts leave an error of 2^-18 of the small entries.
constexpr int kTParts = 2;

// Workspace of one chunk and value head: P and T (in parts), then floats: exp(G_i) (64), c_j (64),
// exp(G_64) and 127 unused, G_i as two floats (64 + 64), beta (64), 64 unused.  P has a second part with bf16
// storage, as its rounding would weigh as much in the output and in dV as their own.
template <typename E>
struct ChunkWs {
  static constexpr int kPart = TriTile<E>::kBytes;
  static constexpr int kP = 0;                            // read where an output is made
  static constexpr int kT = Mma<E>::parts(2) * kPart;     // from here on: what every pass reads
  static constexpr int kGate = kT + Mma<E>::parts(kTParts) * kPart;
  static constexpr int kDecay = kGate + 1024;             // what only the gradients read: 1 KB
  static constexpr int kBytes = kDecay + 1024;
  static_assert(kPart % 1024 == 0, "copied in whole wave instructions");
};

inline int64_t slots_of(const mamba_delta_dims* d, bool packed, int64_t unit) {
  return packed ? d->seqlen / unit + d->batch : d->batch * ((d->seqlen + unit - 1) / unit);
}
inline int64_t chunk_slots(const mamba_delta_dims* d, bool packed) { return slots_of(d, packed, kC); }

// Whether a state pass takes workgroups of 64 columns (4 waves) instead of 128 (8 waves); `runs` sequences or
// segments per head, equally long (`even`) or not.  One workgroup runs on a CU at a time and goes through
// its chunks one after another: 128 columns share a chunk's tiles better (4.5 us a chunk of the output pass with all
// CUs busy, dk = 128, bf16), 64 are through sooner (3.6 us) and leave less idle at the end.  The weights of a round,
// 4.3 and 3.1, are those with which the rule takes the faster side in what was measured, 64 and 128 columns, bf16:
// sequences of 2048, heads of 128: forward of 120 heads 163 and 191 us, of 240 333 and 276 us; backward of 40 heads
// 248 and 317 us, of 240 1174 and 1080 us; forward of 300 heads of 192 613 and 640 us; packed, 40 heads: 8 sequences
// of 0 to 4099 285 and 338 us, 16 of 512 222 and 194 us.
inline bool narrow_pass(int64_t heads, int64_t runs, bool even, int64_t dv) {
  if (dv <= 64) return true;
  const double n = (double)heads * (double)runs, wide = n * (double)((dv + 127) / 128) / 256.0,
               slim = n * (double)((dv + 63) / 64) / 256.0;
  // lengths that differ: the longest, taken as twice the mean, or all of them spread over the CUs
  const double tw = even ? std::ceil(wide) : std::max(2.0, wide);
  const double ts = even ? std::ceil(slim) : std::max(2.0, slim);
  return ts * 3.1 < tw * 4.3;
}
inline size_t chunk_ws_bytes(const mamba_delta_dims* d) {
  return d->io_dtype == MAMBA_BF16 ? ChunkWs<uint16_t>::kBytes : ChunkWs<float>::kBytes;
}

// `packed`: seqlen counts the tokens of all `batch` sequences
inline int check_delta(const mamba_delta_dims* d, bool packed) {
  if (!d) return MAMBA_ERR_NULL;
  if (d->io_dtype != MAMBA_F32 && d->io_dtype != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (d->batch < 1 || d->seqlen < 1 || d->qk_heads < 1 || d->v_heads < 1 || d->dk < 1 || d->dv < 1)
    return MAMBA_ERR_SHAPE;
  if (d->dk % 8 || d->dk > kMaxDk || d->dv % 8 || d->dv > kMaxDv) return MAMBA_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)1 << 40;
  if (d->v_heads > 65535 || d->qk_heads > d->v_heads || d->v_heads % d->qk_heads)
    return MAMBA_ERR_SHAPE;
  if (d->batch > ((int64_t)1 << 30) || d->seqlen > lim) return MAMBA_ERR_SHAPE;
  const double tokens = (packed ? 1.0 : (double)d->batch) * (double)d->seqlen;
  if (tokens * (double)d->v_heads * (double)std::max(d->dk, d->dv) > (double)lim)
    return MAMBA_ERR_SHAPE;
  // the grids: one workgroup per chunk slot and head, and per sequence, value head and 16 columns.  (Launches that
  // could have 2^32 threads are laid out by wide_grid; for the others, which are the delta rule's chunk products and
  // gradients, the workspace would be past 300 GB by then, and its segments are not used with so many heads.)
  if ((tokens / kC + (double)d->batch) * (double)d->v_heads > 2147483647.0 ||
      (double)d->batch * (double)d->v_heads * 64.0 > 2147483647.0)
    return MAMBA_ERR_SHAPE;
  // tokens are read as 16-byte words
  const int64_t vec = d->io_dtype == MAMBA_BF16 ? 8 : 4;
  const int64_t s[3] = {d->q_stride, d->k_stride, d->v_stride};
  const int64_t w[3] = {d->qk_heads * d->dk, d->qk_heads * d->dk, d->v_heads * d->dv};
  for (int i = 0; i < 3; ++i) {
    if (w[i] > kMaxStride || s[i] > kMaxStride || (s[i] && s[i] < w[i])) return MAMBA_ERR_SHAPE;
    if (s[i] % vec) return MAMBA_ERR_ALIGN;
  }
  return MAMBA_OK;
}

inline Args make_args(const mamba_delta_dims* d, float scale, const void* q, const void* k,
                      const void* v, const void* g, const void* beta, const float* s0,
                      const int64_t* offsets) {
  Args a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.s0 = s0;
  a.offsets = offsets;
  a.q_stride = d->q_stride ? d->q_stride : d->qk_heads * d->dk;
  a.k_stride = d->k_stride ? d->k_stride : d->qk_heads * d->dk;
  a.v_stride = d->v_stride ? d->v_stride : d->v_heads * d->dv;
  a.seqlen = d->seqlen;
  a.nseq = d->batch;
  a.slots = chunk_slots(d, offsets != nullptr);
  a.seg_slots = d->batch;
  a.hk = (int32_t)d->qk_heads;
  a.hv = (int32_t)d->v_heads;
  a.rep = (int32_t)(d->v_heads / d->qk_heads);
  a.dk = (int32_t)d->dk;
  a.dv = (int32_t)d->dv;
  a.scale = scale;
  a.ws_item = (int64_t)chunk_ws_bytes(d);
  return a;
}

inline int check_delta_inputs(const mamba_delta_dims* d, const void* q, const void* k, const void* v,
                              const void* g, const void* beta, const float* s0,
                              const int64_t* offsets) {
  if (!q || !k || !v || !g || !beta) return MAMBA_ERR_NULL;
  const size_t es = d->io_dtype == MAMBA_BF16 ? 2 : 4;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, es) ||
      !aligned(beta, es) || (s0 && !aligned(s0, 16)) || (offsets && !aligned(offsets, 8)))
    return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

// What the backward keeps of one chunk and value head beside ChunkWs, as images of LDS tiles in blocks
// of kDB columns of the state (dv is padded to whole blocks): E (in parts; tokens x columns), the state
// before the chunk and the adjoint of the state after it (columns x dk).
template <typename E>
struct BwdBlock {
  static constexpr int kDB = 32;
  static constexpr int kEParts = Mma<E>::parts(2);
  static constexpr int kE = kC * kDB * (int)sizeof(E);  // bytes of one part
  static int64_t blocks(int64_t dv) { return (dv + kDB - 1) / kDB; }
};

// The byte that follows a value's bf16: the next 8 bits of its fp32 pattern, rounded.  Taken up again by
// with_low the two are the value to 2^-17.
__device__ __forceinline__ uint32_t low_byte(float v, uint32_t bf_bits_high) {
  const int d = ((int)(__float_as_uint(v) - bf_bits_high) + 0x80) >> 8;
  return (uint32_t)(d < 127 ? d : 127) & 0xffu;
}
__device__ __forceinline__ float with_low(uint32_t bf_bits_high, uint32_t low, int byte) {
  return __uint_as_float(bf_bits_high + (uint32_t)(((int)(low << (24 - 8 * byte)) >> 24) << 8));
}
// Launches the chunk products (T, P and gates of every chunk and value head) into a.ws.
__attribute__((visibility("hidden"))) int launch_chunks(const Args& a, bool bf, hipStream_t s);

}  // namespace delta
}  // namespace mamba
