// mamba_linear.h -- linear attention with a decay per head: the state through the chunks, shared by the forward
// (mamba_linear.hip) and the gradients (mamba_linear_bwd.hip).
//
// Per value head, with state S (dk x dv), keys k and queries q of its key head:
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// A chunk of kC = 64 tokens with S the state before it, G_i = g_1 + .. + g_i and D_ij = exp(G_i - G_j) is
//     O  = scale diag(exp G) Q S + (scale D o Q K^T) V        (j <= i)
//     S' = exp(G_64) S + K^T diag(exp(G_64 - G_j)) V
// and its adjoint, with dS' the adjoint of the state after it,
//     dV = diag(exp(G_64 - G_j)) K dS' + (scale D o Q K^T)^T dO
//     dS = exp(G_64) dS' + Q^T diag(scale exp G) dO
// which is the same recurrence with q and k exchanged, v = dO, backwards in time.  Read from the last token to the
// first (row x of a tile holds token 63 - x) its matrix is lower triangular again, so that one pass does both:
//     out_x = fx_x X_x S + sum_{y <= x} scale D_xy (X_x . Y_y) z_y,    S' = last S + Y^T diag(fy) Z
//
// One workgroup per sequence (or segment of one), value head and 64 columns of the state: four waves of 16 columns,
// whose state stays in accumulators from the first chunk to the last.  The accumulators of one product are the next
// one's operand, so that only the triangular matrix, which the waves share out, and the output, which is stored in whole
// rows, go through LDS.
//
// Measured (8 x 2048 tokens, 20 key and 40 value heads of 128, bf16): forward 203 us (2.5 TB/s; its bytes at a copy's
// rate 105), backwards with images 244, forwards with images and their products 208 (4.5 TB/s).  With an output a wave
// has 5.8 vector instructions of 4 cycles per product, and a product keeps the vector unit from issuing for half of its
// 16 cycles (measured), so that the best would be 110 us: the state's and the entering values' conversions to bf16 parts
// are most of it.  A chunk takes a workgroup that is alone on its CU 3.4 us.
#pragma once
#include <algorithm>
#include <cmath>

#include "mamba_delta.h"
#include "mamba_grid.h"

namespace mamba {
namespace linear {

using namespace delta;

constexpr int kWaves4 = 4;
constexpr int kCols = 16 * kWaves4;  // columns of a workgroup
// tokens between the states that the gradients keep (fp32: the gradients' tiles of more would not fit the LDS)
template <typename E>
constexpr int kUnit = sizeof(E) == 2 ? 2 * kC : kC;

struct PassArgs {
  Args f;              // q, k, v, out in the pass's roles (backwards: k, q, dout, dv); offsets, s0 and last
  const float* gate;   // (tokens, hv)
  float* seg_decay;    // (segment slots, hv): what a segment leaves of the state before it
  int32_t group;       // workgroups that stay together on an XCD
  int64_t seg_limit;   // sequences of up to so many chunks go through whole, in the place of their first segment
  float* img;          // states before (backwards: after) every kUnit tokens: see image_at
  int64_t img_item;    // floats of one unit and value head
  const float* other;  // kDots: the images of the other direction
  float* dots;         // kDots: (units, hv, column blocks, waves), parts of <state before, adjoint after> a unit
};

// floats of a state's image: fp32, so that the decays' gradients, fp32 numbers, are right to fp32
inline int64_t image_size(const mamba_delta_dims* d) { return (d->dv + 31) / 32 * 32 * (d->dk <= 64 ? 64 : 128); }

// Images lie as the accumulators do, so that a wave reads and writes whole KBs: (units, hv, dv padded to 32s / 16,
// DK / 16, 64 lanes, 4), a unit's and head's img_item floats apart.
template <int DK>
__device__ __forceinline__ int64_t image_at(int col, int m, int lane) {
  return (int64_t)(col / 16) * (16 * DK) + m * 256 + lane * 4;
}

// What a pass does: writes the output; keeps images of the states; goes backwards; starts from zero and leaves only the
// state; multiplies its images with the other direction's.
enum : int { kOutput = 1, kImages = 2, kReverse = 4, kSegmentOnly = 8, kDots = 16 };

// LDS: Y and X of a chunk once, the next chunk's wait in registers until these have been read; Z twice.  Without an
// output two stages of Y and Z, copied straight to LDS.  Three workgroups share a CU (bf16).
template <typename E, int DK, int kWhat>
struct Smem {
  static constexpr bool kO = kWhat & kOutput;
  static constexpr int kYBytes = KeyTile<E, DK>::kBytes;
  // the triangular matrix takes the place of X once that has been read
  static constexpr int kTri = Mma<E>::parts(2) * TriTile<E>::kBytes;
  static constexpr int kXBytes = kO ? (kYBytes > kTri ? kYBytes : kTri) : kYBytes;  // (no output: the second Y)
  static constexpr int kY = 0, kX = kYBytes, kZ = kX + kXBytes, kZBytes = ValueTile<E, kCols>::kBytes;
  // gates of two chunks: G as two floats, fx, fy, exp(G at the end of the token's tile - G) (64 each), last
  static constexpr int kGateFloats = 5 * kC + 4;
  static constexpr int kGate = kZ + 2 * kZBytes;
  static constexpr int kBytes = kGate + 2 * kGateFloats * 4;
  static_assert(sizeof(E) == 4 || 3 * kBytes <= 160 * 1024, "three workgroups per CU");
};

// The same value, but as a new one for the compiler: addresses made from it are made again where they are needed,
// not held in registers through a loop.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// RowCopy whose tile row x holds row 63 - x of memory where kRev, and the same by way of registers.  A lane's rows of a
// tile whose swizzle repeats between them are whole steps apart, so that it keeps one offset.
template <typename E, typename Tile, bool kRev>
struct TokenCopy {
  static constexpr int kI = kC * Tile::kRow / 1024 / kWaves4;
  static constexpr int kStep = kWaves4 * 64 / Tile::kWords;  // rows
  static constexpr bool kOne = kStep % 16 == 0;
  typedef uint32_t Word __attribute__((ext_vector_type(4)));
  uint32_t off[kOne ? 1 : kI], step;
  __device__ __forceinline__ TokenCopy(int w, int lane, int64_t stride, int cols) {
#pragma unroll
    for (int i = 0; i < (kOne ? 1 : kI); ++i) {
      const int at = (w + i * kWaves4) * 64 + lane, t = at / Tile::kWords;
      const int c = ((at % Tile::kWords) ^ Tile::key(t)) * (16 / (int)sizeof(E));
      off[i] = c < cols ? (uint32_t)((kRev ? kC - 1 - t : t) * stride + c) * (uint32_t)sizeof(E) : kOutside;
    }
    step = (uint32_t)(kStep * stride) * (uint32_t)sizeof(E);
  }
  __device__ __forceinline__ uint32_t offset(int i) const {
    if constexpr (kOne) {
      if (i == 0) return off[0];
      return off[0] == kOutside ? kOutside : kRev ? off[0] - i * step : off[0] + i * step;
    } else {
      return off[i];
    }
  }
  __device__ __forceinline__ void operator()(i32x4 buf, uint32_t lds, int w) const {
#pragma unroll
    for (int i = 0; i < kI; ++i) copy_lds(buf, offset(i), lds + (w + i * kWaves4) * 1024);
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buf, Word (&v)[kI]) const {
#pragma unroll
    for (int i = 0; i < kI; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(buf, (int)offset(i), 0, 0);
  }
  __device__ __forceinline__ static void put(char* lds, int w, int lane, const Word (&v)[kI]) {
#pragma unroll
    for (int i = 0; i < kI; ++i) *reinterpret_cast<Word*>(lds + (w + i * kWaves4) * 1024 + 16 * lane) = v[i];
  }
};

// `n` rows of `cols` values, zeros past them
template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_resource(const E* p, int64_t n, int64_t stride, int cols) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(p), 0, (int)(((n - 1) * stride + cols) * (int64_t)sizeof(E)),
                                           0x00020000);
}

template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, kRows, 0xf, false));
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const int2 x = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__builtin_amdgcn_update_dpp(0, x.x, kCtrl, kRows, 0xf, false),
                                         __builtin_amdgcn_update_dpp(0, x.y, kCtrl, kRows, 0xf, false)});
}
// sum of v over lanes 0 .. lane: within rows of 16 lanes, then the rows before
template <typename V>
__device__ __forceinline__ V prefix_sum(V v) {
  v += dpp_or_zero<0x111, 0xf>(v);  // lane - 1
  v += dpp_or_zero<0x112, 0xf>(v);
  v += dpp_or_zero<0x114, 0xf>(v);
  v += dpp_or_zero<0x118, 0xf>(v);
  v += dpp_or_zero<0x142, 0xa>(v);  // row 1 + lane 15, row 3 + lane 47
  v += dpp_or_zero<0x143, 0xc>(v);  // rows 2 and 3 + lane 31
  return v;
}
__device__ __forceinline__ double last_lane(double v) {
  const int2 x = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__builtin_amdgcn_readlane(x.x, 63), __builtin_amdgcn_readlane(x.y, 63)});
}

// The output of a chunk in LDS: rows of kCols values, 16-byte words swizzled by the row.
template <typename E>
__device__ __forceinline__ int out_word(int row, int word) {
  return word ^ (row & (kCols * (int)sizeof(E) / 16 - 1));
}
template <typename E>
__device__ __forceinline__ void put_out(char* lds, int row, int col, f32x4 v) {
  const int byte = col * (int)sizeof(E);
  char* at = lds + row * (kCols * (int)sizeof(E)) + (out_word<E>(row, byte >> 4) << 4) + (byte & 15);
  if constexpr (sizeof(E) == 2)
    *reinterpret_cast<uint2*>(at) = uint2{pack_bf16(make_float2(v[0], v[1])), pack_bf16(make_float2(v[2], v[3]))};
  else
    *reinterpret_cast<f32x4*>(at) = v;
}

// Below -200 exp is 0 in fp32; the clamp keeps -inf (a reset) out of differences and lets NaN through.
__device__ __forceinline__ float clamp_gate(float g) { return g < -200.f ? -200.f : g; }

// Which tiles (y, x) of the triangular matrix a wave makes: pairs of neighbouring y, as an operand holds them, two for
// each wave but the first, which has the gates (their 64 lines take it 2000 cycles to ask for: with a row of tiles per
// wave all waited for it).
struct WaveTiles {
  int w;
  __device__ __forceinline__ int pairs() const { return w ? 2 : 0; }
  __device__ __forceinline__ int x(int pair) const { return w == 1 ? pair : w; }
  __device__ __forceinline__ int y(int pair) const { return w == 1 ? 0 : 2 * pair; }
};

// Rounding, bf16 storage: z times its factor enters the state as three bf16 parts (24 bits); the state and the
// triangular matrix enter the output as two parts each, so that its own rounding is the only one that shows.
// A chunk: X's products, then its place is the triangular matrix's; the state, while that matrix is written; its
// product; the output.  Three workgroups share a CU, whose LDS has no room for a second stage of X and Y: they wait in
// registers, 32 of 168.  Operands are read a step ahead of their products, with barriers for the scheduler, which
// otherwise spilled, and addresses are made again in each chunk.
template <typename E, int DK, int kWhat>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 3 : 1) void linear_pass_kernel(
    PassArgs p, int32_t col_blocks, uint32_t blocks) {
  using M = Mma<E>;
  using Sm = Smem<E, DK, kWhat>;
  using KT = KeyTile<E, DK>;
  using TT = TriTile<E>;
  using VT = ValueTile<E, kCols>;
  constexpr bool kO = kWhat & kOutput, kI = kWhat & kImages, kRev = kWhat & kReverse, kSum = kWhat & kSegmentOnly,
                 kD = kWhat & kDots;
  constexpr int kPS = M::parts(2), kPP = M::parts(2), kPE = M::parts(3);
  __shared__ __align__(1024) char smem[Sm::kBytes];
  const Args& a = p.f;
  const uint32_t id = wide_index();
  if (id >= blocks) return;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wg = spread_index(id, blocks, p.group);
  const int64_t sh = wg / col_blocks;
  const int64_t seg_slot = sh / a.hv;
  const int vh = (int)(sh - seg_slot * a.hv), kh = vh / a.rep;
  const int64_t unit = a.seg_chunks * kC;
  const int64_t seq = a.seg_chunks ? slot_seq(a, seg_slot, unit) : seq_by_length(a, seg_slot);
  const Span sp = seq_span(a, seq);
  const int64_t seg = a.seg_chunks ? seg_slot - slot_base(a, seq, sp.first, unit) : 0;
  const int64_t nchunks = (sp.len + kC - 1) / kC;
  const bool cut = a.seg_chunks && nchunks > p.seg_limit;
  const int64_t first = seg * (cut ? a.seg_chunks : nchunks);
  const int64_t end = cut ? min(first + a.seg_chunks, nchunks) : nchunks;
  if (seg < 0 || (first >= end && seg > 0)) return;  // an unused slot of a packed batch
  if (kSum && (kRev ? first == 0 : end == nchunks)) return;  // no segment follows
  const int col0 = (int)(wg - sh * col_blocks) * kCols;  // this workgroup's first column
  const int col = col0 + 16 * w;                         // this wave's
  const bool has_image = col < (a.dv + 31) / 32 * 32;
  const E* yp = static_cast<const E*>(a.k) + sp.first * a.k_stride + (int64_t)kh * a.dk;
  const E* xp = static_cast<const E*>(a.q) + sp.first * a.q_stride + (int64_t)kh * a.dk;
  const E* zp = static_cast<const E*>(a.v) + sp.first * a.v_stride + (int64_t)vh * a.dv + col0;
  const float* gp = p.gate + sp.first * a.hv + vh;
  const int64_t o_stride = (int64_t)a.hv * a.dv;
  E* op = static_cast<E*>(a.out) + sp.first * o_stride + (int64_t)vh * a.dv + col0;
  const int64_t s_at = (seq * a.hv + vh) * (int64_t)a.dk * a.dv;
  const int64_t g_at = (seg_slot * a.hv + vh) * (int64_t)a.dk * a.dv;
  const float* from = kSum ? nullptr : cut ? a.seg_state + g_at : a.s0 ? a.s0 + s_at : nullptr;

  // row 4 g + x of accumulator m and column col + r of a (dk, dv) matrix, past its end if there is none
  auto state_at = [&](int l, int m, int x) {
    const int row = KT::value(m, l >> 4, x), c = col + (l & 15);
    return c < a.dv && row < a.dk ? (uint32_t)(row * a.dv + c) * 4u : kOutside;
  };
  auto state_resource = [&](const float* q) {  // (none: every load is past its end)
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(q), 0, q ? a.dk * a.dv * 4 : 0, 0x00020000);
  };
  f32x4 S[DK / 16];
  {
    const auto buf = state_resource(from);
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        S[m][x] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, (int)state_at(lane, m, x), 0, 0));
  }

  const uint32_t lds0 = lds_address(smem);
  const int vcols = min(a.dv - col0, kCols);
  const TokenCopy<E, KT, kRev> cy(w, lane, a.k_stride, a.dk), cx(w, lane, a.q_stride, a.dk);
  const TokenCopy<E, VT, kRev> cz(w, lane, a.v_stride, vcols);
  // Y and X of a chunk to registers and from there to LDS (with an output), Z, or Y and Z, straight to stage st; tokens
  // past the sequence are past the buffers and read as zero
  typename decltype(cy)::Word next_y[kO ? decltype(cy)::kI : 1], next_x[kO ? decltype(cx)::kI : 1];
  auto load_y = [&](int64_t ch) {
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    if constexpr (kO) cy.load(rows_resource(yp + t * a.k_stride, n, a.k_stride, a.dk), next_y);
  };
  auto load_x = [&](int64_t ch) {
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    if constexpr (kO) cx.load(rows_resource(xp + t * a.q_stride, n, a.q_stride, a.dk), next_x);
  };
  auto copy = [&](int64_t ch, int st) {
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    if constexpr (!kO) cy(rows_buffer(yp + t * a.k_stride, n, a.k_stride, a.dk), lds0 + st * Sm::kX, w);
    cz(rows_buffer(zp + t * a.v_stride, n, a.v_stride, vcols), lds0 + Sm::kZ + st * Sm::kZBytes, w);
  };
  // a chunk's output from stage st: each wave the KBs that it fills with the next Z, which it has read when it copies
  auto store_out = [&](int64_t ch, int st) {
    constexpr int kWords = kCols * (int)sizeof(E) / 16;  // of a row
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    const auto buf = rows_resource(op + t * o_stride, n, o_stride, vcols);
    const int l = opaque(lane);
#pragma unroll
    for (int i = 0; i < decltype(cz)::kI; ++i) {
      const int at = (w + i * kWaves4) * 64 + l, x = at / kWords, c = out_word<E>(x, at % kWords) * (16 / (int)sizeof(E));
      const auto v = *reinterpret_cast<const typename decltype(cz)::Word*>(smem + Sm::kZ + st * Sm::kZBytes + 16 * at);
      __builtin_amdgcn_raw_buffer_store_b128(
          v, buf, (int)(c < vcols ? (uint32_t)((kRev ? kC - 1 - x : x) * o_stride + c) * (uint32_t)sizeof(E) : kOutside), 0, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (the copy is not the compiler's to order)
  };
  float* const gates = reinterpret_cast<float*>(smem + Sm::kGate);
  // Wave 0: prefix sums of a chunk's log decays in fp64, kept as two floats, so that a difference of two of them is as
  // exact as its own size whatever came before in the chunk; lane = token.
  auto load_gate = [&](int64_t ch) {
    const int64_t t = ch * kC + lane;
    return t < sp.len ? clamp_gate(gp[t * a.hv]) : 0.f;
  };
  double all = 0.0;  // of the segment
  auto put_gates = [&](float v, int slot) {
    float* to = gates + slot * Sm::kGateFloats;
    const double G = prefix_sum((double)v), total = last_lane(G);
    const float hi = (float)G, lo = (float)(G - (double)hi);
    const float eg = a.scale * exp_f32(hi), c = exp_f32((float)(total - G));
    const int x = kRev ? kC - 1 - lane : lane;
    to[x] = kRev ? -hi : hi;
    to[kC + x] = kRev ? -lo : lo;
    to[2 * kC + x] = kRev ? c : eg;
    to[3 * kC + x] = kRev ? eg : c;
    const double tile_end = dpp_or_zero<kRev ? 0x150 : 0x15f, 0xf>(G);  // lane 0 or 15 of the row of 16
    to[4 * kC + x] = exp_f32((float)(kRev ? G - tile_end : tile_end - G));
    if (lane == 0) to[5 * kC] = exp_f32((float)total);
    all += total;
  };

  const WaveTiles tiles{w};
  const int64_t count = end - first;
  auto chunk_at = [&](int64_t it) { return kRev ? end - 1 - it : first + it; };
  constexpr int kPer = kUnit<E> / kC;  // chunks of a unit
  auto unit_item = [&](int64_t ch) {
    return (slot_base(a, seq, sp.first, kUnit<E>) + ch / kPer) * a.hv + vh;
  };
  f32x4 other[kD ? DK / 16 : 1];  // of the next unit
  auto load_other = [&](int64_t ch) {
    if constexpr (kD) {
      const float* img = p.other + unit_item(ch) * p.img_item;
#pragma unroll
      for (int m = 0; m < DK / 16; ++m)
        other[m] = has_image ? *reinterpret_cast<const f32x4*>(img + image_at<DK>(col, m, lane)) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };
  if (count > 0) {
    load_y(chunk_at(0));
    load_x(chunk_at(0));
    copy(chunk_at(0), 0);
    if (w == 0) put_gates(load_gate(chunk_at(0)), 0);
    load_other(chunk_at(0));
    if constexpr (kO) {
      cy.put(smem + Sm::kY, w, lane, next_y);
      cx.put(smem + Sm::kX, w, lane, next_x);
    }
  }
  for (int64_t it = 0; it < count; ++it) {
    const int64_t ch = chunk_at(it);
    // (the last chunk reads itself again: a branch would hold the registers through the whole loop)
    const int64_t next_chunk = chunk_at(min(it + 1, count - 1));
    const int st = (int)(it & 1);
    float next_gate = 0.f;
    copies_done();
    const lds_ptr sm = (lds_ptr)smem;
    const lds_ptr sy = sm + (kO ? 0 : st * Sm::kX), sz = sm + Sm::kZ + st * Sm::kZBytes;
    const float* gt = gates + st * Sm::kGateFloats;
    if (kO && it) store_out(chunk_at(it - 1), st ^ 1);
    if (it + 1 < count) {
      if (w == 0) next_gate = load_gate(chunk_at(it + 1));
      copy(chunk_at(it + 1), st ^ 1);
    }

    if constexpr (kI) {
      // the state before the unit
      if (kRev ? ch % kPer == kPer - 1 || ch == nchunks - 1 : ch % kPer == 0) {
        const int64_t item = unit_item(ch);
        float* img = p.img + item * p.img_item;
        if (has_image)
#pragma unroll
          for (int m = 0; m < DK / 16; ++m) *reinterpret_cast<f32x4*>(img + image_at<DK>(col, m, lane)) = S[m];
        if constexpr (kD) {
          f32x4 d = S[0] * other[0];
#pragma unroll
          for (int m = 1; m < DK / 16; ++m) d += S[m] * other[m];
          float sum = (d[0] + d[1]) + (d[2] + d[3]);
#pragma unroll
          for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
          if (lane == 0) p.dots[(item * col_blocks + (wg - sh * col_blocks)) * kWaves4 + w] = sum;
        }
      }
      if (kD && it + 1 < count && chunk_at(it + 1) % kPer == 0) load_other(chunk_at(it + 1));
    }
    f32x4 o[4];
    if constexpr (kO) {
      const int l = opaque(lane), g = l >> 4, r = l & 15;
      const KT kt(l);
      // pairs of tiles of (Y X^T), a lane holding 4 consecutive y of one x, times scale D
      f32x4 s[2][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j >> 1][j & 1] = o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto make_pair = [&](int j) {
        const int tx = tiles.x(j), ty = tiles.y(j);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kb = 0; kb < DK / M::kDepth; ++kb) {
          const auto f = kt.rows(sm + Sm::kX, tx, kb);
#pragma unroll
          for (int c = 0; c < 2; ++c) s[j][c] = M::mma(kt.rows(sy, ty + c, kb), f, s[j][c]);
        }
        // scale D: of a tile before x's, factors of x and y on both sides of the tile's end; of x's own one by one
        const int i = 16 * tx + r;
        const float hi = gt[i], lo = gt[kC + i];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int t = 16 * (ty + c) + 4 * g, end = 16 * (ty + c) + 15;
          if (ty + c < tx) {
            const float f = a.scale * exp_f32((hi - gt[end]) + (lo - gt[kC + end]));
            s[j][c] *= *reinterpret_cast<const f32x4*>(gt + 4 * kC + t) * f;
          } else {
            const f32x4 e = (hi - *reinterpret_cast<const f32x4*>(gt + t)) + (lo - *reinterpret_cast<const f32x4*>(gt + kC + t));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float v = s[j][c][x] * (a.scale * exp_f32(e[x]));
              s[j][c][x] = t + x <= i ? v : 0.f;
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      if (tiles.pairs()) {
        make_pair(0);
        make_pair(1);
      }
      __builtin_amdgcn_sched_barrier(0);
      load_y(next_chunk);
      if (w == 0 && it + 1 < count) put_gates(next_gate, (int)((it + 1) & 1));
      // (X S)^T, columns x tokens; operands are read a step ahead
      constexpr int kKB = DK / M::kDepth;
      typename M::Frag xi[2][4];
#pragma unroll
      for (int m = 0; m < 4; ++m) xi[0][m] = kt.rows(sm + Sm::kX, m, 0);
      auto f = M::template split<kPS>(&S[0]);
#pragma unroll
      for (int kb = 0; kb < kKB; ++kb) {
        __builtin_amdgcn_sched_barrier(0);
        auto next = f;
        if (kb + 1 < kKB) {
#pragma unroll
          for (int m = 0; m < 4; ++m) xi[(kb + 1) & 1][m] = kt.rows(sm + Sm::kX, m, kb + 1);
          next = M::template split<kPS>(&S[(kb + 1) * M::kTiles]);
        }
#pragma unroll
        for (int x = 0; x < kPS; ++x)
#pragma unroll
          for (int m = 0; m < 4; ++m) o[m] = M::mma(f.p[x], xi[kb & 1][m], o[m]);
        f = next;
      }
      __builtin_amdgcn_sched_barrier(0);
      load_x(next_chunk);
#pragma unroll
      for (int m = 0; m < 4; ++m) o[m] *= gt[2 * kC + 16 * m + r];
      __syncthreads();  // X has been read
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j < tiles.pairs())
#pragma unroll
          for (int c = 0; c < 2; c += M::kTiles) {
            const int kb = (tiles.y(j) + c) / M::kTiles, t = 16 * tiles.x(j);
            if (t < kb * M::kDepth) continue;  // (fp32: a tile past the diagonal)
            const auto f = M::template split<kPP>(&s[j][c]);
#pragma unroll
            for (int x = 0; x < kPP; ++x)
              *reinterpret_cast<typename M::Frag*>(smem + Sm::kX + x * TT::kBytes + TT::word_at(kb, t + r, g)) = f.p[x];
          }
    }
    // S' = last S + Y^T diag(fy) Z, two accumulators at a time, operands a step ahead.  The chunk's part is summed by
    // itself: added token by token to a state that hardly decays, its rounding would grow with the sequence.
    {
      const int l = opaque(lane), g = l >> 4;
      const KT kt(l);
      const VT vt(l, 16 * w);
      const float last = gt[5 * kC];
      auto entering = [&](int kb) {
        f32x4 e[M::kTiles];
#pragma unroll
        for (int x = 0; x < M::kTiles; ++x)
          e[x] = vt.tile(sz, kb * M::kTiles + x) *
                 *reinterpret_cast<const f32x4*>(gt + 3 * kC + 16 * (kb * M::kTiles + x) + 4 * g);
        return M::template split<kPE>(e);
      };
      constexpr int kPairs = DK / 32, kB = TT::kBlocks;
      typename M::Frag yc[2][2];
#pragma unroll
      for (int c = 0; c < 2; ++c) yc[0][c] = kt.cols(sy, c, 0);
      typename M::template Parts<kPE> es[kB];
      es[0] = entering(0);
#pragma unroll
      for (int m = 0; m < kPairs; ++m) {
        f32x4 own[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kb = 0; kb < kB; ++kb) {
          const int step = m * kB + kb, now = step & 1;
          __builtin_amdgcn_sched_barrier(0);
          if (step + 1 < kB * kPairs)
#pragma unroll
            for (int c = 0; c < 2; ++c) yc[now ^ 1][c] = kt.cols(sy, 2 * ((step + 1) / kB) + c, (step + 1) % kB);
          if (m == 0 && kb + 1 < kB) es[kb + 1] = entering(kb + 1);
#pragma unroll
          for (int x = 0; x < kPE; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c) own[c] = M::mma(yc[now][c], es[kb].p[x], own[c]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 0; x < 4; ++x) S[2 * m + c][x] = fmaf(S[2 * m + c][x], last, own[c][x]);
      }
    }
    if (!kO && w == 0 && it + 1 < count) put_gates(next_gate, (int)((it + 1) & 1));
    if constexpr (kO) {
      __syncthreads();  // Y has been read and the triangular matrix is whole
      const int l = opaque(lane), g = l >> 4, r = l & 15;
      const TT tt(l);
      const VT vt(l, 16 * w);
      const lds_ptr pm = sm + Sm::kX;
#pragma unroll
      for (int kb = 0; kb < TT::kBlocks; ++kb) {
        const auto z = vt.operand(sz, kb);
#pragma unroll
        for (int x = 0; x < kPP; ++x)
#pragma unroll
          for (int m = kb * M::kTiles; m < 4; ++m)
            o[m] = M::mma(z, tt.rows(pm + x * TT::kBytes, m, kb), o[m]);
      }
      cy.put(smem + Sm::kY, w, lane, next_y);
      __syncthreads();  // the triangular matrix and Z have been read
      // the output in Z's place, from where whole rows are stored behind the next barrier
#pragma unroll
      for (int m = 0; m < 4; ++m) put_out<E>(smem + Sm::kZ + st * Sm::kZBytes, 16 * m + r, 16 * w + 4 * g, o[m]);
      cx.put(smem + Sm::kX, w, lane, next_x);
    }
  }
  if (kO && count > 0) {
    __syncthreads();
    store_out(chunk_at(count - 1), (int)((count - 1) & 1));
  }
  if (kSum && col0 == 0 && w == 0 && lane == 0) p.seg_decay[seg_slot * a.hv + vh] = exp_f32((float)all);
  float* to = kSum ? a.seg_state + g_at
                   : a.last && (kRev ? first == 0 : end == nchunks) ? a.last + s_at : nullptr;
  if (to) {
    const auto buf = state_resource(to);
    const int l = opaque(lane);
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float v = S[m][x];
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), buf, (int)state_at(l, m, x), 0, 0);
      }
  }
}

template <typename E, int DK, int kWhat>
int launch_pass_t(PassArgs p, hipStream_t s) {
  const int cols = (p.f.dv + kCols - 1) / kCols;
  // Workgroups that read the same keys share an XCD's L2, up to 8 of them: with all 80 heads of a key head in one place
  // the slots that no sequence of a packed batch uses left XCDs without work (64 sequences of 300 tokens: 427 us).
  p.group = 8;
  while (p.f.rep * cols % p.group) --p.group;
  const uint32_t blocks = (uint32_t)(p.f.seg_slots * p.f.hv * cols);
  hipLaunchKernelGGL((linear_pass_kernel<E, DK, kWhat>), wide_grid(blocks, 256), dim3(256), 0, s, p, cols, blocks);
  return launch_status();
}
template <typename E, int kWhat>
int launch_pass(const PassArgs& p, hipStream_t s) {
  return p.f.dk <= 64 ? launch_pass_t<E, 64, kWhat>(p, s) : launch_pass_t<E, 128, kWhat>(p, s);
}

// What a chunk of an output pass takes in us where 1, 2 or `per_cu` workgroups share a CU (measured: 2048 tokens whole, 12 to
// 256, 320 and 384, and 640 workgroups).  fp32: LDS has room for one workgroup, or two of up to 64 values of dk.
struct ChunkTime {
  double us[3];
  int64_t per_cu;
};
inline ChunkTime chunk_time(const mamba_delta_dims* d) {
  if (d->io_dtype == MAMBA_BF16) return d->dk <= 64 ? ChunkTime{{2.8, 3.6, 4.8}, 3} : ChunkTime{{3.4, 4.6, 6.6}, 3};
  return d->dk <= 64 ? ChunkTime{{5.8, 9.3}, 2} : ChunkTime{{9.2}, 1};
}

// Chunks per segment (even), 0 for whole sequences.  Segments cost a second pass that leaves only states, a quarter of the
// time, half a chunk to begin one, the states' way through memory (twice, 5 TB/s) and 15 us of launches in place of 5.
//   Equal sequences: the time of the pass in its rounds of workgroups, with and without.
//   Packed ones, whose lengths are not known here: segments where one sequence of all tokens would take twice as long as
//   all work, which costs the launches where no sequence is long, as those whose chain takes no longer than about the
//   work (`limit` chunks) are not cut; the length for which a chain behind half the work and the states take least.
// Measured whole and cut, forward, dk and dv of 128 and 64 where nothing else is said: 65536 tokens, 12 heads of 128 x 128,
// bf16, 5.9 ms and 326 us; sequences of 2048, by 12, 96, 192, 256 and 384 workgroups, bf16 108 and 30, 109 and 61, 110 and
// 98, 110 and 122, 152 and 168 us; fp32 292 and 47, 295 and 189, 298 and 336, 299 and 443, 589 and 582; dk = 64, fp32, 182
// and 33, 186 and 101, 187 and 179, 190 and 258, 300 and 303.  Sequences of 512, 192 workgroups, dk = 64: bf16 27 and 33,
// fp32 52 and 63.  Packed, 80 heads: 8279 tokens in 8 sequences of up to 4099, bf16 228 and 202, fp32 595 and 588; 15 of 500
// and one of 12000, 617 and 360, 1705 and 1286; but 16 of 2048, 405 and 428, 1483 and 1867; 64 of 300, 252 and 297, 1072
// and 1246, which lengths on the host would tell apart.
struct SegPlan {
  int64_t chunks, limit;
};
inline SegPlan plan_segments(const mamba_delta_dims* d, bool packed) {
  const ChunkTime t = chunk_time(d);
  const double nseq = (double)(packed ? std::min(d->batch, d->seqlen) : d->batch);
  const double length = std::ceil((double)d->seqlen / kC);  // (packed: of a sequence of all tokens)
  const double heads = (double)d->v_heads * (double)((d->dv + kCols - 1) / kCols);
  const double full = t.us[t.per_cu - 1], work = full / (256.0 * (double)t.per_cu) * heads * (length + nseq);
  auto pass = [&](double c, double segments) {  // segments of c chunks
    if (packed) return full * c + 0.5 * work;
    const int64_t k = (int64_t)std::ceil(segments * heads / 256.0), rest = k % t.per_cu;
    return c * (full * (double)(k / t.per_cu) + (rest ? t.us[rest - 1] : 0.0));
  };
  double best = packed ? (t.us[0] * length > 2.0 * work ? 1e30 : 0.0) : 0.95 * (pass(length, nseq) + 5.0);
  SegPlan plan = {0, packed ? (int64_t)(work / full) : 0};
  for (int64_t c = 2; (double)c * 2.0 <= length; c += c < 32 ? 2 : c / 16 * 2) {
    const double segments = packed ? length / (double)c + nseq : std::ceil(length / (double)c) * nseq;
    const double states = segments * (double)d->v_heads * (double)(d->dk * d->dv) * 8.0 / 5e6;
    const double time = 1.25 * pass((double)c + 0.5, segments) + states + 15.0;
    if (time < best) best = time, plan.chunks = c;
  }
  return plan;
}

struct SegLayout {  // workspace regions in bytes
  int64_t chunks, limit, slots;
  size_t decay, total;
};
inline SegLayout seg_layout(const mamba_delta_dims* d, bool packed) {
  const SegPlan plan = plan_segments(d, packed);
  SegLayout l = {plan.chunks, plan.limit, d->batch, 0, 0};
  if (l.chunks) {
    l.slots = slots_of(d, packed, l.chunks * kC);
    const size_t heads = (size_t)l.slots * (size_t)d->v_heads;
    l.decay = (heads * (size_t)(d->dk * d->dv) * sizeof(float) + 255) / 256 * 256;
    l.total = l.decay + (heads * sizeof(float) + 255) / 256 * 256;
  }
  return l;
}
// The pass's arguments for these segments in a workspace that begins at ws.
inline void set_segments(PassArgs& p, const SegLayout& l, char* ws) {
  p.f.seg_chunks = l.chunks;
  p.seg_limit = l.limit;
  p.f.seg_slots = l.slots;
  p.f.seg_state = reinterpret_cast<float*>(ws);
  p.seg_decay = reinterpret_cast<float*>(ws + l.decay);
}
// Each segment's state from zero, then the states that the segments begin with, in their place.
__attribute__((visibility("hidden"))) int launch_segments(const PassArgs& p, bool bf, bool reverse, hipStream_t s);

inline int check_linear_inputs(const mamba_delta_dims* d, const void* q, const void* k, const void* v, const float* g,
                               const float* s0, const int64_t* offsets) {
  if (!q || !k || !v || !g) return MAMBA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || (s0 && !aligned(s0, 16)) ||
      (offsets && !aligned(offsets, 8)))
    return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

}  // namespace linear
}  // namespace mamba
