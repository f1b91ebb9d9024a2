// mamba_delta.h -- what the gated delta rule's kernels share (mamba_delta.hip, mamba_delta_bwd.hip):
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
#include "mamba_common.h"

namespace mamba {
namespace delta {

constexpr int kC = 64;          // tokens per chunk
constexpr int kMaxDk = 128;
constexpr int64_t kMaxDv = 1024;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Operands of the 16 x 16 matrix instructions.  Lane l (g = l / 16, r = l % 16) holds for operand A
// the row r, for operand B the column r, and of the accumulator C the column r and rows 4g .. 4g+3.
// A lane's k values may be any permutation of the depth, the same in A and B.  `chain` and `chain_t`
// read an operand in the order in which accumulators hold their rows, so that the accumulators of
// one product are (converted in place) the operand of the next: no exchange between lanes.
//   row     natural order, from a row with k contiguous
//   chain   accumulator order, from a row with k contiguous
//   chain_t accumulator order, from rows of k: element (k, r) at tile[k ld + r]
//   ctile   rows 4g .. 4g+3 of column r of a 16-row tile, as an accumulator
//   pack    accumulators -> operand (kDepth / 16 of them)
//   split   the same as a sum of kParts operands that together hold (about) the fp32 value
template <typename E>
struct Mma;

template <>
struct Mma<uint16_t> {
  static constexpr int kDepth = 32;
  static constexpr int kParts = 2;  // bf16 high part and remainder: 16 bits of the mantissa
  static constexpr int kPad = 8;
  using Frag = bf16x8;
  struct Parts { Frag p[kParts]; };
  __device__ static __forceinline__ Frag row(const uint16_t* p, int g) {
    return *reinterpret_cast<const bf16x8*>(p + 8 * g);
  }
  __device__ static __forceinline__ Frag join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ static __forceinline__ Frag chain(const uint16_t* p, int g) {
    return join(*reinterpret_cast<const bf16x4*>(p + 4 * g),
                *reinterpret_cast<const bf16x4*>(p + 16 + 4 * g));
  }
  // transposing LDS read: 16 lanes address 4 rows of 16 values (lane r: row r / 4, values
  // 4 (r % 4) ..) and lane r receives column r of the 4 rows
  __device__ static __forceinline__ bf16x4 tr(const uint16_t* tile, int ld, int g, int r) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const uint16_t* p = tile + (4 * g + (r >> 2)) * ld + 4 * (r & 3);
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
  }
  __device__ static __forceinline__ Frag chain_t(const uint16_t* tile, int ld, int g, int r) {
    return join(tr(tile, ld, g, r), tr(tile + 16 * ld, ld, g, r));
  }
  __device__ static __forceinline__ f32x4 ctile(const uint16_t* tile, int ld, int g, int r) {
    return __builtin_convertvector(tr(tile, ld, g, r), f32x4);
  }
  __device__ static __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ Frag pack(const f32x4* c) {
    return join(__builtin_convertvector(c[0], bf16x4), __builtin_convertvector(c[1], bf16x4));
  }
  __device__ static __forceinline__ Parts split(const f32x4* c) {
    const bf16x4 h0 = __builtin_convertvector(c[0], bf16x4);
    const bf16x4 h1 = __builtin_convertvector(c[1], bf16x4);
    const f32x4 l0 = c[0] - __builtin_convertvector(h0, f32x4);
    const f32x4 l1 = c[1] - __builtin_convertvector(h1, f32x4);
    return {{join(h0, h1), join(__builtin_convertvector(l0, bf16x4),
                                __builtin_convertvector(l1, bf16x4))}};
  }
};

template <>
struct Mma<float> {
  static constexpr int kDepth = 16;
  static constexpr int kParts = 1;
  static constexpr int kPad = 4;
  using Frag = f32x4;
  struct Parts { Frag p[kParts]; };
  __device__ static __forceinline__ Frag row(const float* p, int g) {
    return *reinterpret_cast<const f32x4*>(p + 4 * g);
  }
  __device__ static __forceinline__ Frag chain(const float* p, int g) { return row(p, g); }
  __device__ static __forceinline__ Frag chain_t(const float* tile, int ld, int g, int r) {
    const float* p = tile + 4 * g * ld + r;
    return Frag{p[0], p[ld], p[2 * ld], p[3 * ld]};
  }
  __device__ static __forceinline__ f32x4 ctile(const float* tile, int ld, int g, int r) {
    return chain_t(tile, ld, g, r);
  }
  // four 4-deep fp32 instructions: step j takes element j of both operands (k = 4g + j)
  __device__ static __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ Frag pack(const f32x4* c) { return c[0]; }
  __device__ static __forceinline__ Parts split(const f32x4* c) { return {{c[0]}}; }
};

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
  char* ws;                // per (chunk slot, value head): T, P, gates
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  int64_t seqlen;          // tokens per sequence (packed: of all sequences)
  int64_t nseq;
  int64_t slots;           // chunk slots
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

// Chunk slots: sequence s owns the slots from slot_base(s) on.  For packed sequences
// offset / 64 + s leaves room for a last, partial chunk in each, without a scan over the lengths.
__device__ __forceinline__ int64_t slot_base(const Args& a, int64_t seq, int64_t first) {
  return a.offsets ? first / kC + seq : seq * ((a.seqlen + kC - 1) / kC);
}

// slot -> sequence (the last one whose base is not past the slot)
__device__ __forceinline__ int64_t slot_seq(const Args& a, int64_t slot) {
  if (!a.offsets) return slot / ((a.seqlen + kC - 1) / kC);
  int64_t lo = 0, hi = a.nseq - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    const int64_t first = min(max(a.offsets[mid], (int64_t)0), a.seqlen);
    if (first / kC + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Workspace of one chunk and value head: T (64 x 64; bf16: high parts, then remainders), P
// (64 x 64), then exp(G_i) (64 floats), c_j (64 floats), exp(G_64).
template <typename E>
struct ChunkWs {
  static constexpr int kT = kC * kC * 4;  // bytes: 64 x 64 fp32, or two bf16 parts
  static constexpr int kP = kC * kC * (int)sizeof(E);
  static constexpr int kGate = 192 * 4;
  static constexpr int kBytes = kT + kP + kGate;
};

inline int64_t chunk_slots(const mamba_delta_dims* d, bool packed) {
  return packed ? d->seqlen / kC + d->batch : d->batch * ((d->seqlen + kC - 1) / kC);
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
  // the grids: one workgroup per chunk slot and head, and per sequence, value head and 16 columns
  if ((tokens / kC + (double)d->batch) * (double)d->v_heads > 2147483647.0 ||
      (double)d->batch * (double)d->v_heads * 64.0 > 2147483647.0)
    return MAMBA_ERR_SHAPE;
  // tokens are read as 16-byte words
  const int64_t vec = d->io_dtype == MAMBA_BF16 ? 8 : 4;
  const int64_t s[3] = {d->q_stride, d->k_stride, d->v_stride};
  const int64_t w[3] = {d->qk_heads * d->dk, d->qk_heads * d->dk, d->v_heads * d->dv};
  for (int i = 0; i < 3; ++i) {
    if (s[i] && (s[i] < w[i] || s[i] > lim)) return MAMBA_ERR_SHAPE;
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
  a.hk = (int32_t)d->qk_heads;
  a.hv = (int32_t)d->v_heads;
  a.rep = (int32_t)(d->v_heads / d->qk_heads);
  a.dk = (int32_t)d->dk;
  a.dv = (int32_t)d->dv;
  a.scale = scale;
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

// Launches the chunk products (T, P and gates of every chunk and value head) into a.ws.
__attribute__((visibility("hidden"))) int launch_chunks(const Args& a, bool bf, hipStream_t s);

}  // namespace delta
}  // namespace mamba
