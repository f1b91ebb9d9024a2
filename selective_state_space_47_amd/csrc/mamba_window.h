// mamba_window.h -- what the kernels of attention with a sliding window and sinks share (mamba_window.hip, _bwd.hip,
// _step.hip): launch arguments, where sequences and tiles lie, which keys a query sees, and host-side validation.
#pragma once
#include "mamba_delta.h"
#include "mamba_grid.h"

namespace mamba {
namespace window {

using namespace delta;  // matrix-core operands, LDS tiles and copies

constexpr int kKeys = 64;          // keys (or queries) of a tile in LDS
constexpr float kMinusInf = -__builtin_huge_valf();

struct WinArgs {
  const void* q;
  const void* k;
  const void* v;
  const int64_t* q_offsets;   // (nseq + 1) or NULL
  const int64_t* kv_offsets;
  void* out;
  float* lse;                 // (tokens, hq) or NULL
  const void* dout;           // gradients only
  void* dq;
  void* dk;
  void* dv;
  float* stat;                // (2 or 3, hq, tokens): log-sums times log2(e), sums of dout out, and inverse sums of weights
  float* far;                 // (far slots, hq, tiles of 16 sinks, 2, 16, dim): sums over queries past the sinks' windows
  int64_t seqlen, kv_len, nseq;
  int64_t q_stride, k_stride, v_stride;
  int64_t window, sinks;
  float* part;                // (2, groups, kv tokens, hk, dim): dv and dk where a key head's heads are split
  int64_t far_slots;
  int32_t hq, hk, rep, dim, sink_tiles;
  int32_t far_len;            // queries of a stretch
  int32_t groups;             // workgroups that share a key head's heads
  float scale;
};

// Tokens of sequence `seq`.  Offsets are clamped to the tokens there are, so that a wrong offset reads other tokens,
// never past them.
struct Seq {
  int64_t first;
  int len;
};
__device__ __forceinline__ Seq seq_of(const int64_t* offsets, int64_t total, int64_t seq) {
  if (!offsets) return {seq * total, (int)total};
  const int64_t b = min(max(offsets[seq], (int64_t)0), total), e = min(max(offsets[seq + 1], (int64_t)0), total);
  return {b, (int)max(e - b, (int64_t)0)};
}
// Slots of `unit` tokens: sequence s owns those from tile_base(s) on; first / unit + s leaves room for a partial
// last one in each.
__device__ __forceinline__ int64_t tile_base(const int64_t* offsets, int64_t total, int64_t seq, int64_t first, int unit) {
  return offsets ? first / unit + seq : seq * ((total + unit - 1) / unit);
}
// slot -> sequence (the last one whose base is not past the slot)
__device__ __forceinline__ int64_t tile_seq(const int64_t* offsets, int64_t total, int64_t nseq, int64_t slot, int unit) {
  if (!offsets) return slot / ((total + unit - 1) / unit);
  int64_t lo = 0, hi = nseq - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    const int64_t first = min(max(offsets[mid], (int64_t)0), total);
    if (first / unit + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// The sequence and the tile of a workgroup's slot; a tile below zero or past the sequence is an unused slot of a packed
// batch.  Equally long sequences go tile by tile, all of them beside each other, from the end where kLast: the tiles
// with the most work start first, and a sequence's (of one head) share an XCD where their number allows.
struct Tile {
  int64_t seq, tile;
};
template <bool kLast>
__device__ __forceinline__ Tile tile_of(const int64_t* offsets, int64_t total, int64_t nseq, int64_t slot, int unit) {
  if (!offsets) {
    const int64_t n = (total + unit - 1) / unit, t = slot / nseq;
    return {slot - t * nseq, kLast ? n - 1 - t : t};
  }
  const int64_t seq = tile_seq(offsets, total, nseq, slot, unit);
  return {seq, slot - tile_base(offsets, total, seq, min(max(offsets[seq], (int64_t)0), total), unit)};
}
inline int64_t tile_slots(int64_t total, int64_t nseq, bool packed, int unit) {
  return packed ? total / unit + nseq : nseq * ((total + unit - 1) / unit);
}

// Key j, query at position p.
struct Mask {
  int64_t window;
  int sinks;
  __device__ __forceinline__ bool sees(int p, int j) const { return j <= p && (p - j < window || j < sinks); }
  // all of queries [p0, p1] see all of keys [j0, j1]; none sees any
  __device__ __forceinline__ bool all(int p0, int p1, int j0, int j1) const {
    return j1 <= p0 && (p1 - j0 < window || j1 < sinks);
  }
  __device__ __forceinline__ bool none(int p0, int p1, int j0, int j1) const {
    return j0 > p1 || (p0 - j1 >= window && j0 >= sinks);
  }
};
__device__ __forceinline__ Mask mask_of(const WinArgs& a) {
  return {a.window, (int)min(a.sinks, (int64_t)0x7fffffff)};
}

template <typename V>
__device__ __forceinline__ V across_groups(V v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// values that an operand's accumulators hold, rounded, to 16-byte aligned memory
template <typename E>
__device__ __forceinline__ void store_operand(E* p, const f32x4* c) {
  *reinterpret_cast<typename Mma<E>::Frag*>(p) = Mma<E>::pack(c);
}

// rows of a (rows, DK) matrix as operands in registers, straight from memory: row `row` of `rows`, natural order
template <typename E, int DK>
__device__ __forceinline__ void load_rows(const E* p, int64_t stride, int row, int rows, int dim, int g,
                                          typename Mma<E>::Frag (&f)[DK / Mma<E>::kDepth]) {
  constexpr int kV = 16 / sizeof(E);
#pragma unroll
  for (int kb = 0; kb < DK / Mma<E>::kDepth; ++kb) {
    const int c = kb * Mma<E>::kDepth + g * kV;
    const bool in = row < rows && c < dim;
    f[kb] = in ? *reinterpret_cast<const typename Mma<E>::Frag*>(p + (int64_t)row * stride + c) : typename Mma<E>::Frag{};
  }
}

// Operands are read from LDS a step before the products that take them, as one or two waves per SIMD leave nobody
// else to hide the reads behind; nothing is moved past the end of a step.
__device__ __forceinline__ void end_step() { __builtin_amdgcn_sched_barrier(0); }

// fp32 storage: what a tile adds is summed by itself first.  Thousands of tokens one by one onto an accumulator leave an
// error of many times its rounding (2 x 2048 queries of 5 heads: dk and dv were off by 1.3e-6, a matrix product in blocks
// by 5e-7).
template <typename E>
constexpr bool kTileSums = sizeof(E) == 4;
template <int kC2, int kD>
__device__ __forceinline__ void clear(f32x4 (&t)[kC2][kD]) {
#pragma unroll
  for (int c = 0; c < kC2; ++c)
#pragma unroll
    for (int d = 0; d < kD; ++d) t[c][d] = f32x4{0.f, 0.f, 0.f, 0.f};
}
template <int kC2, int kD>
__device__ __forceinline__ void add_to(f32x4 (&to)[kC2][kD], const f32x4 (&t)[kC2][kD]) {
#pragma unroll
  for (int c = 0; c < kC2; ++c)
#pragma unroll
    for (int d = 0; d < kD; ++d) to[c][d] += t[c][d];
}

// Every load of this wave has landed, said so that the compiler counts it too.  Operands loaded before a loop would
// otherwise be waited for again at their first use in every turn, and with them the copies of the next tile.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

constexpr int64_t kMaxTokens = 0x7fffffff - 1024;
constexpr int64_t kMaxWindow = (int64_t)1 << 40;

inline int check_window(const mamba_window_dims* d, bool packed) {
  if (!d) return MAMBA_ERR_NULL;
  if (d->io_dtype != MAMBA_F32 && d->io_dtype != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (d->batch < 1 || d->seqlen < 1 || d->kv_len < 1 || d->q_heads < 1 || d->kv_heads < 1 || d->dim < 1 ||
      d->window < 1 || d->sinks < 0)
    return MAMBA_ERR_SHAPE;
  if (d->dim % 8 || d->dim > kMaxDk) return MAMBA_ERR_UNSUPPORTED;
  if (d->batch > ((int64_t)1 << 20) || d->seqlen > kMaxTokens || d->kv_len > kMaxTokens || d->window > kMaxWindow ||
      d->sinks > kMaxWindow || d->q_heads > 65535 || d->kv_heads > d->q_heads || d->q_heads % d->kv_heads)
    return MAMBA_ERR_SHAPE;
  const double seqs = packed ? 1.0 : (double)d->batch, lim = 1099511627776.0;
  if (seqs * (double)d->seqlen * (double)d->q_heads * (double)d->dim > lim ||
      seqs * (double)d->kv_len * (double)d->kv_heads * (double)d->dim > lim)
    return MAMBA_ERR_SHAPE;
  // the grids: one workgroup per 64 queries or 32 keys and head
  if ((seqs * (double)d->seqlen / kKeys + (double)d->batch) * (double)d->q_heads > 2147483647.0 ||
      (seqs * (double)d->kv_len / 32 + (double)d->batch) * (double)d->kv_heads > 2147483647.0)
    return MAMBA_ERR_SHAPE;
  // tokens are read as 16-byte words
  const int64_t vec = d->io_dtype == MAMBA_BF16 ? 8 : 4;
  const int64_t s[3] = {d->q_stride, d->k_stride, d->v_stride};
  const int64_t w[3] = {d->q_heads * d->dim, d->kv_heads * d->dim, d->kv_heads * d->dim};
  for (int i = 0; i < 3; ++i) {
    if (w[i] > kMaxStride || s[i] > kMaxStride || (s[i] && s[i] < w[i])) return MAMBA_ERR_SHAPE;
    if (s[i] % vec) return MAMBA_ERR_ALIGN;
  }
  return MAMBA_OK;
}

inline WinArgs window_args(const mamba_window_dims* d, float scale, const void* q, const void* k, const void* v,
                           const int64_t* q_offsets, const int64_t* kv_offsets) {
  WinArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_offsets = q_offsets;
  a.kv_offsets = kv_offsets;
  a.seqlen = d->seqlen;
  a.kv_len = d->kv_len;
  a.nseq = d->batch;
  a.hq = (int32_t)d->q_heads;
  a.hk = (int32_t)d->kv_heads;
  a.rep = (int32_t)(d->q_heads / d->kv_heads);
  a.dim = (int32_t)d->dim;
  a.q_stride = d->q_stride ? d->q_stride : d->q_heads * d->dim;
  a.k_stride = d->k_stride ? d->k_stride : d->kv_heads * d->dim;
  a.v_stride = d->v_stride ? d->v_stride : d->kv_heads * d->dim;
  a.window = d->window;
  a.sinks = d->sinks;
  a.scale = scale;
  return a;
}

inline int check_window_inputs(const void* q, const void* k, const void* v, const int64_t* q_offsets,
                               const int64_t* kv_offsets) {
  if (!q || !k || !v || !q_offsets != !kv_offsets) return MAMBA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || (q_offsets && !aligned(q_offsets, 8)) ||
      (kv_offsets && !aligned(kv_offsets, 8)))
    return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

}  // namespace window
}  // namespace mamba
