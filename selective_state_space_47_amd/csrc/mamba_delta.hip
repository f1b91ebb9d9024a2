// mamba_delta.hip -- the gated delta rule on gfx950: whole sequences in chunks of 64 tokens on the
// matrix cores, and one generation step.  The formulas are in mamba_delta.h.
//
//   chunk_kernel  one workgroup per chunk and key head: T, P and the gate factors, for every value
//                 head that shares the key head (K K^T and Q K^T are made once).
//   scan_kernel   one workgroup per sequence, value head and 16 NW columns of the state: the state
//                 goes through the chunks.  A wave owns 16 columns; its state stays in accumulators
//                 from the first chunk to the last, and every product's accumulators are the next
//                 product's operand, so that waves share nothing but the tiles they read.
//   step_kernel   one token: the state is read and written once.
//
// Rounding (bf16 storage): products take bf16 operands into fp32 accumulators.  Whatever reaches the
// state (S in K S, Y, T, E in K^T E) goes in as three bf16 parts, the fp32 value to 24 bits, so that
// the state is fp32 in earnest; the output O takes S and E as two parts and P as one, whose rounding
// is that of the output again.  fp32 storage uses fp32 matrix instructions throughout.
#include "mamba_delta.h"

namespace mamba {
namespace delta {
namespace {

// 16-byte word `i` (of W E-values) of row `row` of a (64 x cols) tile, zero outside
template <typename E>
__device__ __forceinline__ uint4 tile_word(const E* base, int64_t stride, int row, int col, int rows,
                                           int cols) {
  return row < rows && col < cols
             ? *reinterpret_cast<const uint4*>(base + (int64_t)row * stride + col)
             : make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ chunk products

template <typename E, int DK>
struct ChunkSmem {
  static constexpr int kLd = DK + 16 / (int)sizeof(E);
  static constexpr int kLf = kC + 4;
  union {
    struct { E k[kC * kLd], q[kC * kLd]; } in;
    struct { float a[kC * kLf], t[kC * kLf]; } m;
  };
  float d[4][16 * 20];      // inverted diagonal blocks
  float ghi[kC], glo[kC], beta[kC];
};

// 16 bytes of storage: bf16 takes the 4 values of each of two tiles, fp32 those of one
template <typename E>
__device__ __forceinline__ uint4 pack_word(const float (&a)[4], const float (&b)[4]) {
  if constexpr (sizeof(E) == 2)
    return make_uint4(pack_bf16(make_float2(a[0], a[1])), pack_bf16(make_float2(a[2], a[3])),
                      pack_bf16(make_float2(b[0], b[1])), pack_bf16(make_float2(b[2], b[3])));
  else
    return __builtin_bit_cast(uint4, make_float4(a[0], a[1], a[2], a[3]));
}

// sum of v over lanes 0 .. lane
__device__ __forceinline__ double wave_prefix(double v, int lane) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const double t = __shfl_up(v, m);
    if (lane >= m) v += t;
  }
  return v;
}

template <typename E, int DK>
__global__ __launch_bounds__(256) void chunk_kernel(Args a) {
  using M = Mma<E>;
  using Sm = ChunkSmem<E, DK>;
  __shared__ __align__(16) Sm sm;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r = lane & 15;
  const int64_t slot = blockIdx.x / a.hk;
  const int kh = (int)(blockIdx.x - slot * a.hk);
  const int64_t seq = slot_seq(a, slot);
  const Span sp = seq_span(a, seq);
  const int64_t c0 = (slot - slot_base(a, seq, sp.first)) * kC;
  if (c0 < 0 || c0 >= sp.len) return;  // an unused slot of a packed batch
  const int n = (int)min((int64_t)kC, sp.len - c0);
  const int64_t t0 = sp.first + c0;

  constexpr int kV = 16 / sizeof(E);
  constexpr int kRowWords = DK / kV;
  const E* kp = static_cast<const E*>(a.k) + t0 * a.k_stride + (int64_t)kh * a.dk;
  const E* qp = static_cast<const E*>(a.q) + t0 * a.q_stride + (int64_t)kh * a.dk;
#pragma unroll
  for (int i = tid; i < kC * kRowWords; i += 256) {
    const int row = i / kRowWords, col = i % kRowWords * kV;
    *reinterpret_cast<uint4*>(&sm.in.k[row * Sm::kLd + col]) =
        tile_word(kp, a.k_stride, row, col, n, a.dk);
    *reinterpret_cast<uint4*>(&sm.in.q[row * Sm::kLd + col]) =
        tile_word(qp, a.q_stride, row, col, n, a.dk);
  }
  __syncthreads();

  // Wave w: columns i = 16w .. of (K K^T)^T and (Q K^T)^T, rows j up to the diagonal, so that a lane
  // holds 4 consecutive j of one token i.
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) kk[jt] = qk[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kb = 0; kb < DK / M::kDepth; ++kb) {
    const int at = r * Sm::kLd + kb * M::kDepth + g * kV;
    const auto ki = *reinterpret_cast<const typename M::Frag*>(&sm.in.k[16 * w * Sm::kLd + at]);
    const auto qi = *reinterpret_cast<const typename M::Frag*>(&sm.in.q[16 * w * Sm::kLd + at]);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
      if (jt <= w) {
        const auto kj = *reinterpret_cast<const typename M::Frag*>(&sm.in.k[16 * jt * Sm::kLd + at]);
        kk[jt] = M::mma(kj, ki, kk[jt]);
        qk[jt] = M::mma(kj, qi, qk[jt]);
      }
  }

  const int i = 16 * w + r;  // this lane's token
  for (int h = 0; h < a.rep; ++h) {
    const int vh = kh * a.rep + h;
    char* ws = a.ws + (slot * a.hv + vh) * (int64_t)ChunkWs<E>::kBytes;
    __syncthreads();  // the tiles of the previous head (or K and Q) have been read
    if (w == 0) {
      // Prefix sums of the log decays in fp64, kept as two floats: a difference of two of them is
      // then as exact as its own size, whatever came before in the chunk.  Below -200 exp is 0 in
      // fp32; the clamp keeps -inf (a reset) out of the differences and lets NaN through.
      float gl = 0.f, bt = 0.f;
      if (lane < n) {
        const int64_t at = (t0 + lane) * a.hv + vh;
        gl = ld_f32(static_cast<const E*>(a.g), at);
        bt = ld_f32(static_cast<const E*>(a.beta), at);
        gl = gl < -200.f ? -200.f : gl;
      }
      const double G = wave_prefix((double)gl, lane);
      const double total = __shfl(G, 63);
      const float hi = (float)G;
      sm.ghi[lane] = hi;
      sm.glo[lane] = (float)(G - (double)hi);
      sm.beta[lane] = bt;
      float* gate = reinterpret_cast<float*>(ws + ChunkWs<E>::kT + ChunkWs<E>::kP);
      gate[lane] = exp_f32(hi);
      gate[kC + lane] = exp_f32((float)(total - G)) * bt;
      if (lane == 0) gate[2 * kC] = exp_f32((float)total);
    }
    __syncthreads();
    const float gi = sm.ghi[i], gil = sm.glo[i];
    float p[4][4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int j = 16 * jt + 4 * g;
      float A[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float d = jt <= w && j + x <= i
                            ? exp_f32((gi - sm.ghi[j + x]) + (gil - sm.glo[j + x])) * sm.beta[j + x]
                            : 0.f;
        A[x] = j + x < i ? d * kk[jt][x] : 0.f;
        p[jt][x] = d * qk[jt][x] * a.scale;
      }
      *reinterpret_cast<float4*>(&sm.m.a[i * Sm::kLf + j]) = make_float4(A[0], A[1], A[2], A[3]);
    }
    // a lane's accumulators of one block of P are one word of its image
#pragma unroll
    for (int kb = 0; kb < TriTile<E>::kBlocks; ++kb)
      if (16 * w >= kb * M::kDepth)
        *reinterpret_cast<uint4*>(ws + ChunkWs<E>::kT + TriTile<E>::word_at(kb, i, g)) =
            pack_word<E>(p[kb * M::kTiles], p[(kb + 1) * M::kTiles - 1]);
    __syncthreads();
    // T = (I + A)^-1 by blocks of 16.  Wave w inverts diagonal block w by substitution, lane r its
    // column r: x_m = [m = r] - sum_{j < m} A_mj x_j.
    {
      const float* Ab = &sm.m.a[16 * w * Sm::kLf + 16 * w];
      float x[16];
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        float t = m == r ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < m; ++j) t = fmaf(-Ab[m * Sm::kLf + j], x[j], t);
        x[m] = t;
      }
#pragma unroll
      for (int m = 0; m < 4; ++m)  // the four lane groups hold the same columns: 4 rows each
        sm.d[w][(4 * g + m) * 20 + r] = g == 0 ? x[m] : g == 1 ? x[4 + m] : g == 2 ? x[8 + m] : x[12 + m];
    }
    __syncthreads();
    // Wave w makes block column w below the diagonal: T_iw = -T_ii (sum_{k=w}^{i-1} A_ik T_kw), its
    // own blocks staying in accumulators.
    {
      using F = Mma<float>;
      f32x4 T[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) T[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b == w)
#pragma unroll
          for (int x = 0; x < 4; ++x) T[b][x] = sm.d[w][(4 * g + x) * 20 + r];
        if (b > w) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < b; ++k)
            if (k >= w) acc = F::mma(*reinterpret_cast<const f32x4*>(&sm.m.a[(16 * b + r) * Sm::kLf + 16 * k + 4 * g]), T[k], acc);
          f32x4 z = {0.f, 0.f, 0.f, 0.f};
          T[b] = F::mma(*reinterpret_cast<const f32x4*>(&sm.d[b][r * 20 + 4 * g]), -acc, z);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) sm.m.t[(16 * b + 4 * g + x) * Sm::kLf + 16 * w + r] = T[b][x];
      }
    }
    __syncthreads();
    // the image of T: one word per turn
    for (int x = tid; x < TriTile<E>::kRows * 4; x += 256) {
      int kb = 0, t = x >> 2;
      while (t >= kC - kb * M::kDepth) t -= kC - M::kDepth * kb++;
      t += kb * M::kDepth;
      const float* src = &sm.m.t[t * Sm::kLf + kb * M::kDepth + 4 * (x & 3)];
      float lo[4], hi[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        lo[y] = src[y];
        hi[y] = sizeof(E) == 2 ? src[16 + y] : src[y];
      }
#pragma unroll
      for (int part = 0; part < M::kParts; ++part) {
        const uint4 word = pack_word<E>(lo, hi);
        *reinterpret_cast<uint4*>(ws + part * TriTile<E>::kBytes +
                                  TriTile<E>::word_at(kb, t, x & 3)) = word;
        if (sizeof(E) == 2) {
          const float2 a0 = unpack(word.x), a1 = unpack(word.y), b0 = unpack(word.z),
                       b1 = unpack(word.w);
          lo[0] -= a0.x; lo[1] -= a0.y; lo[2] -= a1.x; lo[3] -= a1.y;
          hi[0] -= b0.x; hi[1] -= b0.y; hi[2] -= b1.x; hi[3] -= b1.y;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the state through the chunks

// One stage of a workgroup's LDS: the chunk's K and Q, the chunk's workspace image (T, P, gates) and V.
template <typename E, int DK, int NW, int NC>
struct Stage {
  static constexpr int kK = 0;
  static constexpr int kQ = KeyTile<E, DK>::kBytes;
  static constexpr int kWs = 2 * KeyTile<E, DK>::kBytes;
  static constexpr int kGate = kWs + ChunkWs<E>::kT + ChunkWs<E>::kP;
  static constexpr int kVv = kWs + ChunkWs<E>::kBytes;
  static constexpr int kVRow = 16 * NC * NW * (int)sizeof(E);
  static constexpr int kBytes = kVv + kC * kVRow;
  static constexpr int kCount = 2 * kBytes <= 160 * 1024 ? 2 : 1;
};

template <typename E, int DK, int NW, int NC>
__global__ __launch_bounds__(64 * NW) void scan_kernel(Args a, int32_t col_blocks) {
  using M = Mma<E>;
  using St = Stage<E, DK, NW, NC>;
  using KT = KeyTile<E, DK>;
  using TT = TriTile<E>;
  constexpr int kV = 16 / sizeof(E);  // values per word
  __shared__ __align__(1024) char smem[St::kCount * St::kBytes];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wg = placed_index(blockIdx.x, gridDim.x);
  const int64_t sh = wg / col_blocks;
  const int64_t seq = sh / a.hv;
  const int vh = (int)(sh - seq * a.hv), kh = vh / a.rep;
  const int col0 = (int)(wg - sh * col_blocks) * 16 * NC * NW;  // this workgroup's first column
  const int col = col0 + 16 * NC * w;                        // this wave's
  const Span sp = seq_span(a, seq);
  const int64_t slot0 = slot_base(a, seq, sp.first);
  const E* kp = static_cast<const E*>(a.k) + sp.first * a.k_stride + (int64_t)kh * a.dk;
  const E* qp = static_cast<const E*>(a.q) + sp.first * a.q_stride + (int64_t)kh * a.dk;
  const E* vp = static_cast<const E*>(a.v) + sp.first * a.v_stride + (int64_t)vh * a.dv + col0;
  E* op = static_cast<E*>(a.out) + (sp.first * a.hv + vh) * (int64_t)a.dv + col;
  const int64_t s_at = (seq * a.hv + vh) * (int64_t)a.dk * a.dv + col + r;

  f32x4 S[NC][DK / 16];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = KT::value(m, g, x);
        S[c][m][x] = a.s0 && col + 16 * c + r < a.dv && row < a.dk
                         ? a.s0[s_at + (int64_t)row * a.dv + 16 * c] : 0.f;
      }

  // Byte offsets of the words this lane copies: instruction j of a tile fills its j-th KB, wave w the
  // instructions w, w + NW, ...
  constexpr int kKI = KT::kBytes / 1024 / NW;
  constexpr int kVI = kC * St::kVRow / 1024 / NW;
  static_assert(kKI * NW * 1024 == KT::kBytes && kVI * NW * 1024 == kC * St::kVRow, "whole KBs");
  uint32_t ok[kKI], oq[kKI], ov[kVI];
#pragma unroll
  for (int i = 0; i < kKI; ++i) {
    const int at = (w + i * NW) * 64 + lane, t = at / KT::kWords;
    const int c = ((at % KT::kWords) ^ KT::key(t)) * kV;
    ok[i] = c < a.dk ? (uint32_t)(t * a.k_stride + c) * sizeof(E) : kOutside;
    oq[i] = c < a.dk ? (uint32_t)(t * a.q_stride + c) * sizeof(E) : kOutside;
  }
#pragma unroll
  for (int i = 0; i < kVI; ++i) {
    const int at = (w + i * NW) * 64 + lane, t = at / (St::kVRow / 16);
    const int c = at % (St::kVRow / 16) * kV;
    ov[i] = c < a.dv - col0 ? (uint32_t)(t * a.v_stride + c) * sizeof(E) : kOutside;
  }
  const uint32_t lds0 = lds_address(smem);
  const int64_t nchunks = (sp.len + kC - 1) / kC;
  const int vcols = min(a.dv - col0, 16 * NC * NW);
  // copies chunk ch into stage st; tokens past the sequence are past the buffers and read as zero
  auto copy = [&](int64_t ch, int st) {
    const int64_t n = min((int64_t)kC, sp.len - ch * kC);
    const i32x4 bk = buffer_of(kp + ch * kC * a.k_stride,
                               (uint32_t)(((n - 1) * a.k_stride + a.dk) * sizeof(E)));
    const i32x4 bq = buffer_of(qp + ch * kC * a.q_stride,
                               (uint32_t)(((n - 1) * a.q_stride + a.dk) * sizeof(E)));
    const i32x4 bv = buffer_of(vp + ch * kC * a.v_stride,
                               (uint32_t)(((n - 1) * a.v_stride + vcols) * sizeof(E)));
    const i32x4 bw = buffer_of(a.ws + ((slot0 + ch) * a.hv + vh) * (int64_t)ChunkWs<E>::kBytes,
                               ChunkWs<E>::kBytes);
    const uint32_t to = lds0 + st * St::kBytes + w * 1024;
#pragma unroll
    for (int i = 0; i < kKI; ++i) copy_lds(bk, ok[i], to + St::kK + i * NW * 1024);
#pragma unroll
    for (int i = 0; i < kVI; ++i) copy_lds(bv, ov[i], to + St::kVv + i * NW * 1024);
#pragma unroll
    for (int i = 0; i < kKI; ++i) copy_lds(bq, oq[i], to + St::kQ + i * NW * 1024);
#pragma unroll
    for (int i = 0; i < (ChunkWs<E>::kBytes / 1024 + NW - 1) / NW; ++i)
      if ((i + 1) * NW <= ChunkWs<E>::kBytes / 1024 || w + i * NW < ChunkWs<E>::kBytes / 1024)
        copy_lds(bw, (w + i * NW) * 1024 + lane * 16, to + St::kWs + i * NW * 1024);
  };

  const KT kt(lane);
  const TT tt(lane);
  const int vrow = sizeof(E) == 2 ? (4 * g + (r >> 2)) * St::kVRow + 32 * NC * w + 8 * (r & 3)
                                  : 4 * g * St::kVRow + (16 * NC * w + r) * 4;
  if (nchunks > 0) copy(0, 0);
  for (int64_t ch = 0; ch < nchunks; ++ch) {
    const int st = St::kCount == 2 ? (int)(ch & 1) : 0;
    copies_done();
    // with two stages the next chunk is copied while this one is worked on
    if (St::kCount == 2 && ch + 1 < nchunks) copy(ch + 1, st ^ 1);
    const lds_ptr sm = (lds_ptr)(smem + st * St::kBytes);
    const int n = (int)min((int64_t)kC, sp.len - ch * kC);

    // K S (tokens x columns) and (Q S)^T (columns x tokens)
    f32x4 y[NC][4], o[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) y[c][m] = o[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < DK / M::kDepth; ++kb) {
      typename M::Parts s[NC];
      typename M::Frag kf[4], qf[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        kf[m] = kt.rows(sm + St::kK, m, kb);
        qf[m] = kt.rows(sm + St::kQ, m, kb);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) s[c] = M::split(&S[c][kb * M::kTiles]);
#pragma unroll
      for (int p = 0; p < M::kParts; ++p)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int m = 0; m < 4; ++m) y[c][m] = M::mma(kf[m], s[c].p[p], y[c][m]);
#pragma unroll
      for (int p = 0; p < (M::kParts + 1) / 2; ++p)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int m = 0; m < 4; ++m) o[c][m] = M::mma(s[c].p[p], qf[m], o[c][m]);
    }
    // Y = V - diag(exp G) K S;  O scaled by its token's factor
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 eg = lds_read<f32x4>(sm + St::kGate + (16 * m + 4 * g) * 4);
      const float so = a.scale * lds_read<float>(sm + St::kGate + (16 * m + r) * 4);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        f32x4 v;
        const lds_ptr vt = sm + St::kVv + 16 * m * St::kVRow + 16 * c * (int)sizeof(E) + vrow;
        if constexpr (sizeof(E) == 2) {
          v = __builtin_convertvector(lds_tr(vt), f32x4);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = lds_read<float>(vt + x * St::kVRow);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          y[c][m][x] = fmaf(-eg[x], y[c][m][x], v[x]);
          o[c][m][x] *= so;
        }
      }
    }
    // E = T Y, T lower triangular; of the parts' products those above 2^-24
    f32x4 e[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) e[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      typename M::Parts ys[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) ys[c] = M::split(&y[c][kb * M::kTiles]);
#pragma unroll
      for (int p = 0; p < M::kParts; ++p) {
        typename M::Frag tf[4];
#pragma unroll
        for (int m = kb * M::kTiles; m < 4; ++m) tf[m] = tt.rows(sm + St::kWs + p * TT::kBytes, m, kb);
#pragma unroll
        for (int x = 0; x + p < M::kParts; ++x)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int m = kb * M::kTiles; m < 4; ++m) e[c][m] = M::mma(tf[m], ys[c].p[x], e[c][m]);
      }
    }
    // O += P E, transposed: a lane ends with 4 consecutive columns of one token
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      typename M::Parts es[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) es[c] = M::split(&e[c][kb * M::kTiles]);
      typename M::Frag pf[4];
#pragma unroll
      for (int m = kb * M::kTiles; m < 4; ++m) pf[m] = tt.rows(sm + St::kWs + ChunkWs<E>::kT, m, kb);
#pragma unroll
      for (int p = 0; p < (M::kParts + 1) / 2; ++p)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int m = kb * M::kTiles; m < 4; ++m) o[c][m] = M::mma(es[c].p[p], pf[m], o[c][m]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int t = 16 * m + r;
        if (t < n && col + 16 * c + 4 * g < a.dv) {
          E* dst = op + (ch * kC + t) * (int64_t)a.hv * a.dv + 16 * c + 4 * g;
          if constexpr (sizeof(E) == 2)
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16(make_float2(o[c][m][0], o[c][m][1])),
                           pack_bf16(make_float2(o[c][m][2], o[c][m][3])));
          else
            *reinterpret_cast<f32x4*>(dst) = o[c][m];
        }
      }
    // S = exp(G_64) S + K^T diag(c) E
    const float last = lds_read<float>(sm + St::kGate + 2 * kC * 4);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 cj = lds_read<f32x4>(sm + St::kGate + (kC + 16 * m + 4 * g) * 4);
#pragma unroll
      for (int c = 0; c < NC; ++c) e[c][m] *= cj;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < DK / 16; ++m) S[c][m] *= last;
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      typename M::Parts es[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) es[c] = M::split(&e[c][kb * M::kTiles]);
#pragma unroll
      for (int m0 = 0; m0 < DK / 16; m0 += 4) {
        typename M::Frag kf[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) kf[m] = kt.cols(sm + St::kK, m0 + m, kb);
#pragma unroll
        for (int p = 0; p < M::kParts; ++p)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int m = 0; m < 4; ++m) S[c][m0 + m] = M::mma(kf[m], es[c].p[p], S[c][m0 + m]);
      }
    }
    if (St::kCount == 1 && ch + 1 < nchunks) {
      __syncthreads();  // every wave has read the stage
      copy(ch + 1, 0);
    }
  }
  if (a.last) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < DK / 16; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = KT::value(m, g, x);
          if (row < a.dk && col + 16 * c + r < a.dv)
            a.last[s_at + (int64_t)row * a.dv + 16 * c] = S[c][m][x];
        }
  }
}

// ------------------------------------------------------------------ one token

constexpr int kStepThreads = 256;

struct StepArgs {
  float* state;
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  const void* beta;
  void* out;
  int64_t q_stride, k_stride, v_stride;
  int32_t hv, rep, dk, dv;
  float scale;
};

// One token of one value head and 4 TC columns: TC lanes hold a row's float4s, kStepThreads / TC
// rows are held at a time, kRows per thread.  Bound by the state's traffic (read and written once,
// fp32): with a = exp(g), both dots go through the old state in one pass,
//     x = a S^T k,  e = v - x,  o = scale (a S^T q + beta (k . q) e),  S <- a S + beta k e^T,
// so that one reduction across the rows' lanes serves both.
template <typename E, int TC, int kRows>
__global__ __launch_bounds__(kStepThreads) void step_kernel(StepArgs a, int32_t col_blocks) {
  constexpr int kStride = kStepThreads / TC;  // rows held at a time
  __shared__ float sk[kMaxDk], sq[kMaxDk];
  __shared__ float red[kStepThreads / 64][2][4 * TC];
  __shared__ float skq[2];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t sh = blockIdx.x / col_blocks;
  const int64_t seq = sh / a.hv;
  const int vh = (int)(sh - seq * a.hv), kh = vh / a.rep;
  const int c = (int)(blockIdx.x - sh * col_blocks) * 4 * TC + tid % TC * 4;
  const int row0 = tid / TC;
  float* sp = a.state + sh * (int64_t)a.dk * a.dv + c;
  const bool live = c < a.dv;
  f32x4 s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStride;
    s[i] = live && row < a.dk ? *reinterpret_cast<const f32x4*>(sp + (int64_t)row * a.dv)
                              : f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float kv = 0.f, qv = 0.f;
  if (tid < a.dk) {
    kv = ld_f32(static_cast<const E*>(a.k), seq * a.k_stride + (int64_t)kh * a.dk + tid);
    qv = ld_f32(static_cast<const E*>(a.q), seq * a.q_stride + (int64_t)kh * a.dk + tid);
  }
  const float ga = exp_f32(ld_f32(static_cast<const E*>(a.g), seq * a.hv + vh));
  const float bt = ld_f32(static_cast<const E*>(a.beta), seq * a.hv + vh);
  float v[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    v[x] = live ? ld_f32(static_cast<const E*>(a.v), seq * a.v_stride + (int64_t)vh * a.dv + c + x)
                : 0.f;
  if (tid < kMaxDk) {
    sk[tid] = kv;
    sq[tid] = qv;
    float t = kv * qv;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) t += __shfl_xor(t, m);
    if (lane == 0) skq[w] = t;
  }
  __syncthreads();
  f32x4 xk = {0.f, 0.f, 0.f, 0.f}, xq = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStride;
    if (row < kMaxDk) {
      s[i] *= ga;
      xk += s[i] * sk[row];
      xq += s[i] * sq[row];
    }
  }
  // rows of a wave, then of the workgroup
#pragma unroll
  for (int m = TC; m < 64; m *= 2)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      xk[x] += __shfl_xor(xk[x], m);
      xq[x] += __shfl_xor(xq[x], m);
    }
  if (lane < TC) {
    *reinterpret_cast<f32x4*>(&red[w][0][4 * lane]) = xk;
    *reinterpret_cast<f32x4*>(&red[w][1][4 * lane]) = xq;
  }
  __syncthreads();
  xk = xq = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kStepThreads / 64; ++i) {
    xk += *reinterpret_cast<const f32x4*>(&red[i][0][tid % TC * 4]);
    xq += *reinterpret_cast<const f32x4*>(&red[i][1][tid % TC * 4]);
  }
  const float kq = skq[0] + skq[1];
  if (!live) return;
  f32x4 u;
  float o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    u[x] = bt * (v[x] - xk[x]);
    o[x] = a.scale * fmaf(kq, u[x], xq[x]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStride;
    if (row < a.dk) *reinterpret_cast<f32x4*>(sp + (int64_t)row * a.dv) = s[i] + u * sk[row];
  }
  if (row0 == 0)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      st_out(static_cast<E*>(a.out), sh * (int64_t)a.dv + c + x, o[x]);
}

template <typename E>
int launch_step(const StepArgs& a, int64_t heads, hipStream_t s) {
  // 128 columns per workgroup make full 512-byte rows; where that leaves CUs idle, 32 columns give
  // four times the workgroups
  const int64_t wide = (a.dv + 127) / 128, narrow = (a.dv + 31) / 32;
  if (heads * wide >= 512)
    hipLaunchKernelGGL((step_kernel<E, 32, kMaxDk / 8>), dim3((unsigned)(heads * wide)),
                       dim3(kStepThreads), 0, s, a, (int32_t)wide);
  else
    hipLaunchKernelGGL((step_kernel<E, 8, kMaxDk / 32>), dim3((unsigned)(heads * narrow)),
                       dim3(kStepThreads), 0, s, a, (int32_t)narrow);
  return launch_status();
}

template <typename E, int DK>
int launch_chunks_t(const Args& a, hipStream_t s) {
  hipLaunchKernelGGL((chunk_kernel<E, DK>), dim3((unsigned)(a.slots * a.hk)), dim3(256), 0, s, a);
  return launch_status();
}

template <typename E, int DK, int NW, int NC>
int launch_scan_t(const Args& a, hipStream_t s) {
  const int cols = (a.dv + 16 * NC * NW - 1) / (16 * NC * NW);
  hipLaunchKernelGGL((scan_kernel<E, DK, NW, NC>), dim3((unsigned)(a.nseq * a.hv * cols)),
                     dim3(64 * NW), 0, s, a, cols);
  return launch_status();
}

template <typename E, int DK>
int launch_scan_d(const Args& a, hipStream_t s) {
  return a.dv <= 64 ? launch_scan_t<E, DK, 4, 1>(a, s) : launch_scan_t<E, DK, 8, 1>(a, s);
}

}  // namespace

int launch_chunks(const Args& a, bool bf, hipStream_t s) {
  if (bf) return a.dk <= 64 ? launch_chunks_t<uint16_t, 64>(a, s) : launch_chunks_t<uint16_t, 128>(a, s);
  return a.dk <= 64 ? launch_chunks_t<float, 64>(a, s) : launch_chunks_t<float, 128>(a, s);
}

}  // namespace delta
}  // namespace mamba

using namespace mamba;
using namespace mamba::delta;

extern "C" {

size_t mamba_delta_workspace_bytes(const mamba_delta_dims* dims, int packed) {
  if (check_delta(dims, packed != 0) != MAMBA_OK) return 0;
  return (size_t)chunk_slots(dims, packed != 0) * (size_t)dims->v_heads * chunk_ws_bytes(dims);
}

int mamba_delta_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                    const float* initial_state, const int64_t* seq_offsets, float scale, void* out,
                    float* last_state, const mamba_delta_dims* dims, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = check_delta(dims, seq_offsets != nullptr);
  if (st != MAMBA_OK) return st;
  if (!out) return MAMBA_ERR_NULL;
  if ((st = check_delta_inputs(dims, q, k, v, g, beta, initial_state, seq_offsets)) != MAMBA_OK)
    return st;
  if (!aligned(out, 16) || (last_state && !aligned(last_state, 16))) return MAMBA_ERR_ALIGN;
  if (!workspace || workspace_bytes < mamba_delta_workspace_bytes(dims, seq_offsets != nullptr))
    return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  Args a = make_args(dims, scale, q, k, v, g, beta, initial_state, seq_offsets);
  a.out = out;
  a.last = last_state;
  a.ws = static_cast<char*>(workspace);
  const bool bf = dims->io_dtype == MAMBA_BF16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = launch_chunks(a, bf, s)) != MAMBA_OK) return st;
  if (bf) return a.dk <= 64 ? launch_scan_d<uint16_t, 64>(a, s) : launch_scan_d<uint16_t, 128>(a, s);
  return a.dk <= 64 ? launch_scan_d<float, 64>(a, s) : launch_scan_d<float, 128>(a, s);
}

int mamba_delta_update(float* state, const void* q, const void* k, const void* v, const void* g,
                       const void* beta, float scale, void* out, const mamba_delta_dims* dims,
                       void* stream) {
  int st = check_delta(dims, false);
  if (st != MAMBA_OK) return st;
  if (dims->seqlen != 1) return MAMBA_ERR_SHAPE;
  if (!state || !out) return MAMBA_ERR_NULL;
  if ((st = check_delta_inputs(dims, q, k, v, g, beta, state, nullptr)) != MAMBA_OK) return st;
  if (!aligned(out, dims->io_dtype == MAMBA_BF16 ? 2 : 4)) return MAMBA_ERR_ALIGN;
  const Args d = make_args(dims, scale, q, k, v, g, beta, nullptr, nullptr);
  StepArgs a = {state, q, k, v, g, beta, out, d.q_stride, d.k_stride, d.v_stride,
                d.hv, d.rep, d.dk, d.dv, scale};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dims->io_dtype == MAMBA_BF16 ? launch_step<uint16_t>(a, dims->batch * dims->v_heads, s)
                                      : launch_step<float>(a, dims->batch * dims->v_heads, s);
}

}  // extern "C"
