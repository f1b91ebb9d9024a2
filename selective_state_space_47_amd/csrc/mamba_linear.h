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
// one's operand, so that only the triangular matrix, a quarter of it made by each wave, goes through LDS.
#pragma once
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
  char* img;           // states before (backwards: after) every kUnit tokens, as tiles of dv x dk
  int64_t img_item;    // bytes of one unit and value head
};

template <typename E>
constexpr int kImgParts = Mma<E>::parts(2);
// bytes of one part of a state's image
template <typename E>
inline int64_t image_part(const mamba_delta_dims* d) {
  return (d->dv + 31) / 32 * 32 * (d->dk <= 64 ? 64 : 128) * (int64_t)sizeof(E);
}

// What a pass does: writes the output; keeps images of the states; goes backwards.
enum : int { kOutput = 1, kImages = 2, kReverse = 4, kSegmentOnly = 8 };

template <typename E, int DK, int kWhat>
struct Smem {
  static constexpr bool kO = kWhat & kOutput;
  static constexpr int kY = 0;
  static constexpr int kX = KeyTile<E, DK>::kBytes;
  // the triangular matrix takes the place of X once that has been read
  static constexpr int kTri = Mma<E>::parts(2) * TriTile<E>::kBytes;
  static constexpr int kXBytes = KeyTile<E, DK>::kBytes > kTri ? KeyTile<E, DK>::kBytes : kTri;
  static constexpr int kZ = kX + (kO ? kXBytes : 0);
  static constexpr int kStage = kZ + ValueTile<E, kCols>::kBytes;
  // gates of two chunks: G as two floats, fx, fy (64 each), last
  static constexpr int kGateFloats = 4 * kC + 4;
  static constexpr int bytes(int stages) { return stages * kStage + 2 * kGateFloats * 4; }
};

// RowCopy whose tile row x holds row 63 - x of memory where kRev
template <typename E, typename Tile, bool kRev>
struct TokenCopy {
  static constexpr int kI = kC * Tile::kRow / 1024 / kWaves4;
  uint32_t off[kI];
  __device__ __forceinline__ TokenCopy(int w, int lane, int64_t stride, int cols) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int at = (w + i * kWaves4) * 64 + lane, t = at / Tile::kWords;
      const int c = ((at % Tile::kWords) ^ Tile::key(t)) * (16 / (int)sizeof(E));
      off[i] = c < cols ? (uint32_t)((kRev ? kC - 1 - t : t) * stride + c) * (uint32_t)sizeof(E) : kOutside;
    }
  }
  __device__ __forceinline__ void operator()(i32x4 buf, uint32_t lds, int w) const {
#pragma unroll
    for (int i = 0; i < kI; ++i) copy_lds(buf, off[i], lds + (w + i * kWaves4) * 1024);
  }
};

// sum of v over lanes 0 .. lane
__device__ __forceinline__ double prefix_sum(double v, int lane) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const double t = __shfl_up(v, m);
    if (lane >= m) v += t;
  }
  return v;
}

// Below -200 exp is 0 in fp32; the clamp keeps -inf (a reset) out of differences and lets NaN through.
__device__ __forceinline__ float clamp_gate(float g) { return g < -200.f ? -200.f : g; }

// Rounding, bf16 storage: z times its factor enters the state as kPE bf16 parts (3: to 24 bits; 2, where the state
// is only kept as an image of two parts: to 16); the state and the triangular matrix enter the output as two parts
// each, so that its own rounding is the only one that shows.
template <typename E, int DK, int kWhat, int kStages>
__global__ __launch_bounds__(256, sizeof(E) == 2 && kStages == 1 ? 3 : 1) void linear_pass_kernel(
    PassArgs p, int32_t col_blocks, uint32_t blocks) {
  using M = Mma<E>;
  using Sm = Smem<E, DK, kWhat>;
  using KT = KeyTile<E, DK>;
  using TT = TriTile<E>;
  using VT = ValueTile<E, kCols>;
  constexpr bool kO = kWhat & kOutput, kI = kWhat & kImages, kRev = kWhat & kReverse, kSum = kWhat & kSegmentOnly;
  constexpr int kPS = M::parts(2), kPP = M::parts(2), kPE = M::parts(kI ? 2 : 3);
  __shared__ __align__(1024) char smem[Sm::bytes(kStages)];
  const Args& a = p.f;
  const uint32_t id = wide_index();
  if (id >= blocks) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wg = spread_index(id, blocks, a.rep * col_blocks);
  const int64_t sh = wg / col_blocks;
  const int64_t seg_slot = sh / a.hv;
  const int vh = (int)(sh - seg_slot * a.hv), kh = vh / a.rep;
  const int64_t unit = a.seg_chunks * kC;
  const int64_t seq = a.seg_chunks ? slot_seq(a, seg_slot, unit) : seq_by_length(a, seg_slot);
  const Span sp = seq_span(a, seq);
  const int64_t seg = a.seg_chunks ? seg_slot - slot_base(a, seq, sp.first, unit) : 0;
  const int64_t nchunks = (sp.len + kC - 1) / kC;
  const int64_t first = seg * a.seg_chunks;
  const int64_t end = a.seg_chunks ? min(first + a.seg_chunks, nchunks) : nchunks;
  if (seg < 0 || (first >= end && seg > 0)) return;  // an unused slot of a packed batch
  if (kSum && (kRev ? first == 0 : end == nchunks)) return;  // no segment follows
  const int col0 = (int)(wg - sh * col_blocks) * kCols;  // this workgroup's first column
  const int col = col0 + 16 * w;                         // this wave's
  const bool has_col = col + r < a.dv;
  const E* yp = static_cast<const E*>(a.k) + sp.first * a.k_stride + (int64_t)kh * a.dk;
  const E* xp = static_cast<const E*>(a.q) + sp.first * a.q_stride + (int64_t)kh * a.dk;
  const E* zp = static_cast<const E*>(a.v) + sp.first * a.v_stride + (int64_t)vh * a.dv + col0;
  const float* gp = p.gate + sp.first * a.hv + vh;
  const int64_t o_stride = (int64_t)a.hv * a.dv;
  E* op = static_cast<E*>(a.out) + sp.first * o_stride + (int64_t)vh * a.dv + col;
  const int64_t s_at = (seq * a.hv + vh) * (int64_t)a.dk * a.dv + col + r;
  const int64_t g_at = (seg_slot * a.hv + vh) * (int64_t)a.dk * a.dv + col + r;
  const float* from = kSum ? nullptr : a.seg_chunks ? a.seg_state + g_at : a.s0 ? a.s0 + s_at : nullptr;

  f32x4 S[DK / 16];
#pragma unroll
  for (int m = 0; m < DK / 16; ++m)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = KT::value(m, g, x);
      S[m][x] = from && has_col && row < a.dk ? from[(int64_t)row * a.dv] : 0.f;
    }

  const uint32_t lds0 = lds_address(smem);
  const int vcols = min(a.dv - col0, kCols);
  const TokenCopy<E, KT, kRev> cy(w, lane, a.k_stride, a.dk), cx(w, lane, a.q_stride, a.dk);
  const TokenCopy<E, VT, kRev> cz(w, lane, a.v_stride, vcols);
  // copies chunk ch into stage st; tokens past the sequence are past the buffers and read as zero
  auto copy = [&](int64_t ch, int st) {
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    const uint32_t to = lds0 + st * Sm::kStage;
    cy(rows_buffer(yp + t * a.k_stride, n, a.k_stride, a.dk), to + Sm::kY, w);
    if (kO) cx(rows_buffer(xp + t * a.q_stride, n, a.q_stride, a.dk), to + Sm::kX, w);
    cz(rows_buffer(zp + t * a.v_stride, n, a.v_stride, vcols), to + Sm::kZ, w);
  };
  float* const gates = reinterpret_cast<float*>(smem + kStages * Sm::kStage);
  // Wave 0: prefix sums of a chunk's log decays in fp64, kept as two floats, so that a difference of two of them is as
  // exact as its own size whatever came before in the chunk; lane = token.
  auto load_gate = [&](int64_t ch) {
    const int64_t t = ch * kC + lane;
    return t < sp.len ? clamp_gate(gp[t * a.hv]) : 0.f;
  };
  double all = 0.0;  // of the segment
  auto put_gates = [&](float v, int slot) {
    float* to = gates + slot * Sm::kGateFloats;
    const double G = prefix_sum((double)v, lane), total = __shfl(G, 63);
    const float hi = (float)G, lo = (float)(G - (double)hi);
    const float eg = a.scale * exp_f32(hi), c = exp_f32((float)(total - G));
    const int x = kRev ? kC - 1 - lane : lane;
    to[x] = kRev ? -hi : hi;
    to[kC + x] = kRev ? -lo : lo;
    to[2 * kC + x] = kRev ? c : eg;
    to[3 * kC + x] = kRev ? eg : c;
    if (lane == 0) to[4 * kC] = exp_f32((float)total);
    all += total;
  };

  const KT kt(lane);
  const TT tt(lane);
  const VT vt(lane, 16 * w);
  const int64_t count = end - first;
  auto chunk_at = [&](int64_t it) { return kRev ? end - 1 - it : first + it; };
  if (count > 0) {
    copy(chunk_at(0), 0);
    if (w == 0) put_gates(load_gate(chunk_at(0)), 0);
  }
  for (int64_t it = 0; it < count; ++it) {
    const int64_t ch = chunk_at(it);
    const int st = kStages == 2 ? (int)(it & 1) : 0;
    float next_gate = 0.f;
    copies_done();
    const lds_ptr sm = (lds_ptr)(smem + st * Sm::kStage);
    const float* gt = gates + (it & 1) * Sm::kGateFloats;
    if (w == 0 && it + 1 < count) next_gate = load_gate(chunk_at(it + 1));
    if (kStages == 2 && it + 1 < count) copy(chunk_at(it + 1), st ^ 1);
    const int n = (int)min((int64_t)kC, sp.len - ch * kC);

    if constexpr (kI) {
      // the state before the unit: 16 bytes of one column per operand
      constexpr int kPer = kUnit<E> / kC;
      if (kRev ? ch % kPer == kPer - 1 || ch == nchunks - 1 : ch % kPer == 0) {
        const int64_t part = (a.dv + 31) / 32 * 32 * (int64_t)KT::kRow;
        char* img = p.img + ((slot_base(a, seq, sp.first, kUnit<E>) + ch / kPer) * a.hv + vh) * p.img_item +
                    (int64_t)(col + r) * KT::kRow;
        if (col + r < (a.dv + 31) / 32 * 32) {
#pragma unroll
          for (int kb = 0; kb < DK / M::kDepth; ++kb) {
            const auto s = M::template split<kImgParts<E>>(&S[kb * M::kTiles]);
#pragma unroll
            for (int x = 0; x < kImgParts<E>; ++x)
              *reinterpret_cast<typename M::Frag*>(img + x * part + (((4 * kb + g) ^ KT::key(col + r)) << 4)) = s.p[x];
          }
        }
      }
    }
    f32x4 o[4], s[4];
    if constexpr (kO) {
      // columns x = 16 w + r of (Y X^T), rows y up to the diagonal: a lane holds 4 consecutive y of one x
#pragma unroll
      for (int m = 0; m < 4; ++m) s[m] = o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) {
        const auto xi = kt.rows(sm + Sm::kX, w, kb);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (m <= w) s[m] = M::mma(kt.rows(sm + Sm::kY, m, kb), xi, s[m]);
      }
      const int i = 16 * w + r;
      const float hi = gt[i], lo = gt[kC + i];
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (m <= w) {
          const f32x4 yh = *reinterpret_cast<const f32x4*>(gt + 16 * m + 4 * g),
                      yl = *reinterpret_cast<const f32x4*>(gt + kC + 16 * m + 4 * g);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            s[m][x] = 16 * m + 4 * g + x <= i ? s[m][x] * (a.scale * exp_f32((hi - yh[x]) + (lo - yl[x]))) : 0.f;
        }
      // (X S)^T, columns x tokens
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) {
        const auto f = M::template split<kPS>(&S[kb * M::kTiles]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const auto xi = kt.rows(sm + Sm::kX, m, kb);
#pragma unroll
          for (int x = 0; x < kPS; ++x) o[m] = M::mma(f.p[x], xi, o[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) o[m] *= gt[2 * kC + 16 * m + r];
    }
    // S' = last S + Y^T diag(fy) Z
    const float last = gt[4 * kC];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) S[m] *= last;
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      f32x4 e[M::kTiles];
#pragma unroll
      for (int x = 0; x < M::kTiles; ++x)
        e[x] = vt.tile(sm + Sm::kZ, kb * M::kTiles + x) *
               *reinterpret_cast<const f32x4*>(gt + 3 * kC + 16 * (kb * M::kTiles + x) + 4 * g);
      const auto es = M::template split<kPE>(e);
#pragma unroll
      for (int m = 0; m < DK / 16; ++m) {
        const auto yc = kt.cols(sm + Sm::kY, m, kb);
#pragma unroll
        for (int x = 0; x < kPE; ++x) S[m] = M::mma(yc, es.p[x], S[m]);
      }
    }
    if (w == 0 && it + 1 < count) put_gates(next_gate, (int)((it + 1) & 1));
    if constexpr (kO) {
      __syncthreads();  // X has been read
      char* const psm = smem + st * Sm::kStage + Sm::kX;
#pragma unroll
      for (int kb = 0; kb < TT::kBlocks; ++kb)
        if (16 * w >= kb * M::kDepth) {
          const auto f = M::template split<kPP>(&s[kb * M::kTiles]);
#pragma unroll
          for (int x = 0; x < kPP; ++x)
            *reinterpret_cast<typename M::Frag*>(psm + x * TT::kBytes + TT::word_at(kb, 16 * w + r, g)) = f.p[x];
        }
      __syncthreads();  // the triangular matrix is whole
      const lds_ptr pm = (lds_ptr)psm;
#pragma unroll
      for (int kb = 0; kb < TT::kBlocks; ++kb) {
        const auto z = vt.operand(sm + Sm::kZ, kb);
#pragma unroll
        for (int x = 0; x < kPP; ++x)
#pragma unroll
          for (int m = kb * M::kTiles; m < 4; ++m)
            o[m] = M::mma(z, tt.rows(pm + x * TT::kBytes, m, kb), o[m]);
      }
      const auto buf = __builtin_amdgcn_make_buffer_rsrc(
          op + ch * kC * o_stride, 0, (int)(((n - 1) * o_stride + max(a.dv - col, 0)) * (int64_t)sizeof(E)),
          0x00020000);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int t = kRev ? kC - 1 - (16 * m + r) : 16 * m + r;
        store_four<E>(buf, col + 4 * g < a.dv ? (uint32_t)(t * o_stride + 4 * g) * (uint32_t)sizeof(E) : kOutside,
                      o[m]);
      }
    }
    if (kStages == 1 && it + 1 < count) {
      __syncthreads();  // every wave has read the stage
      copy(chunk_at(it + 1), 0);
    }
  }
  if (kSum && col0 == 0 && w == 0 && lane == 0) p.seg_decay[seg_slot * a.hv + vh] = exp_f32((float)all);
  float* to = kSum ? a.seg_state + g_at
                   : a.last && (kRev ? first == 0 : end == nchunks) ? a.last + s_at : nullptr;
  if (to && has_col) {
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = KT::value(m, g, x);
        if (row < a.dk) to[(int64_t)row * a.dv] = S[m][x];
      }
  }
}

template <typename E, int DK, int kWhat>
int launch_pass_t(const PassArgs& p, hipStream_t s) {
  const int cols = (p.f.dv + kCols - 1) / kCols;
  const uint32_t blocks = (uint32_t)(p.f.seg_slots * p.f.hv * cols);
  hipLaunchKernelGGL((linear_pass_kernel<E, DK, kWhat, 1>), wide_grid(blocks, 256), dim3(256), 0, s, p, cols, blocks);
  return launch_status();
}
template <typename E, int kWhat>
int launch_pass(const PassArgs& p, hipStream_t s) {
  return p.f.dk <= 64 ? launch_pass_t<E, 64, kWhat>(p, s) : launch_pass_t<E, 128, kWhat>(p, s);
}

// Chunks per segment (even), 0 for whole sequences: segments where the sequences' workgroups alone leave CUs idle.
inline int64_t plan_segments(const mamba_delta_dims* d, bool packed) {
  const int64_t cols = (d->dv + kCols - 1) / kCols;
  const int64_t nseq = packed ? std::min(d->batch, d->seqlen) : d->batch;
  const double runs = (double)nseq * (double)d->v_heads * (double)cols;
  double chunks = (double)((d->seqlen + kC - 1) / kC);
  if (packed && nseq > 1) chunks = std::min(chunks, 2.0 * chunks / (double)nseq);
  const double want = 768.0 / runs;  // segments per sequence that fill the GPU
  if (want < 2.0 || chunks < 16.0) return 0;
  const int64_t c = std::max<int64_t>(4, (int64_t)(chunks / want));
  return (c + 1) / 2 * 2;
}

struct SegLayout {  // workspace regions in bytes
  int64_t chunks, slots;
  size_t decay, total;
};
inline SegLayout seg_layout(const mamba_delta_dims* d, bool packed) {
  SegLayout l = {plan_segments(d, packed), d->batch, 0, 0};
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
