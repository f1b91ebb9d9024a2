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
// state (S in K S, Y, T, E in K^T E) goes in as a bf16 pair (high part and remainder, 16 bits), so
// that the fp32 state is right to about 1e-6; S and E enter the output O as one bf16 value, whose
// error is that of rounding the output.  fp32 storage uses fp32 matrix instructions throughout.
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
  static constexpr int kLd = DK + Mma<E>::kPad;
  static constexpr int kLf = kC + 4;
  union {
    struct { E k[kC * kLd], q[kC * kLd]; } in;
    struct { float a[kC * kLf], t[kC * kLf]; } m;
  };
  float d[4][16 * 20];      // inverted diagonal blocks
  float ghi[kC], glo[kC], beta[kC];
};

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
    const auto ki = M::row(&sm.in.k[(16 * w + r) * Sm::kLd + kb * M::kDepth], g);
    const auto qi = M::row(&sm.in.q[(16 * w + r) * Sm::kLd + kb * M::kDepth], g);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
      if (jt <= w) {
        const auto kj = M::row(&sm.in.k[(16 * jt + r) * Sm::kLd + kb * M::kDepth], g);
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
    E* P = reinterpret_cast<E*>(ws + ChunkWs<E>::kT);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int j = 16 * jt + 4 * g;
      float A[4], p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float d = jt <= w && j + x <= i
                            ? exp_f32((gi - sm.ghi[j + x]) + (gil - sm.glo[j + x])) * sm.beta[j + x]
                            : 0.f;
        A[x] = j + x < i ? d * kk[jt][x] : 0.f;
        p[x] = d * qk[jt][x] * a.scale;
      }
      *reinterpret_cast<float4*>(&sm.m.a[i * Sm::kLf + j]) = make_float4(A[0], A[1], A[2], A[3]);
      if constexpr (sizeof(E) == 2)
        *reinterpret_cast<uint2*>(P + i * kC + j) =
            make_uint2(pack_bf16(make_float2(p[0], p[1])), pack_bf16(make_float2(p[2], p[3])));
      else
        *reinterpret_cast<float4*>(P + i * kC + j) = make_float4(p[0], p[1], p[2], p[3]);
    }
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
        if (b == w) T[b] = F::ctile(&sm.d[w][0], 20, g, r);
        if (b > w) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < b; ++k)
            if (k >= w) acc = F::mma(F::row(&sm.m.a[(16 * b + r) * Sm::kLf + 16 * k], g), T[k], acc);
          f32x4 z = {0.f, 0.f, 0.f, 0.f};
          T[b] = F::mma(F::row(&sm.d[b][r * 20], g), -acc, z);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) sm.m.t[(16 * b + 4 * g + x) * Sm::kLf + 16 * w + r] = T[b][x];
      }
    }
    __syncthreads();
    {
      const int row = tid >> 2, c = (tid & 3) * 16;
      const float* t = &sm.m.t[row * Sm::kLf + c];
      if constexpr (sizeof(E) == 4) {
        float* T = reinterpret_cast<float*>(ws) + row * kC + c;
#pragma unroll
        for (int x = 0; x < 16; x += 4)
          *reinterpret_cast<float4*>(T + x) = *reinterpret_cast<const float4*>(t + x);
      } else {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float2 f = make_float2(t[2 * x], t[2 * x + 1]);
          hi[x] = pack_bf16(f);
          const float2 h = unpack(hi[x]);
          lo[x] = pack_bf16(make_float2(f.x - h.x, f.y - h.y));
        }
        uint4* T = reinterpret_cast<uint4*>(ws) + (row * kC + c) / 8;
        T[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        T[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        T[kC * kC / 8] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        T[kC * kC / 8 + 1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      }
    }
  }
}

// ------------------------------------------------------------------ the state through the chunks

template <typename E, int DK, int NW>
struct ScanSmem {
  static constexpr int kLd = DK + Mma<E>::kPad;
  static constexpr int kLt = kC + Mma<E>::kPad;
  static constexpr int kLv = 16 * NW + Mma<E>::kPad;
  static constexpr int kParts = Mma<E>::kParts;
  E k[kC * kLd], q[kC * kLd], t[kParts][kC * kLt], p[kC * kLt], v[kC * kLv];
  float eg[kC], c[kC];
};

template <typename E, int DK, int NW>
__global__ __launch_bounds__(64 * NW) void scan_kernel(Args a, int32_t col_blocks) {
  using M = Mma<E>;
  using Sm = ScanSmem<E, DK, NW>;
  constexpr int kThreads = 64 * NW;
  constexpr int kV = 16 / sizeof(E);       // values per 16-byte word
  constexpr int kTPF = M::kDepth / 16;     // accumulator tiles per operand
  constexpr int kWk = kC * DK / kV / kThreads, kWt = kC * kC / kV / kThreads;
  constexpr int kWv = kC * 16 * NW / kV / kThreads;
  __shared__ __align__(16) Sm sm;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r = lane & 15;
  const int64_t wg = placed_index(blockIdx.x, gridDim.x);
  const int64_t sh = wg / col_blocks;
  const int64_t seq = sh / a.hv;
  const int vh = (int)(sh - seq * a.hv), kh = vh / a.rep;
  const int col0 = (int)(wg - sh * col_blocks) * 16 * NW;  // this workgroup's first column
  const int col = col0 + 16 * w;                           // this wave's
  const Span sp = seq_span(a, seq);
  const int64_t slot0 = slot_base(a, seq, sp.first);
  const E* kp = static_cast<const E*>(a.k) + sp.first * a.k_stride + (int64_t)kh * a.dk;
  const E* qp = static_cast<const E*>(a.q) + sp.first * a.q_stride + (int64_t)kh * a.dk;
  const E* vp = static_cast<const E*>(a.v) + sp.first * a.v_stride + (int64_t)vh * a.dv + col0;
  E* op = static_cast<E*>(a.out) + (sp.first * a.hv + vh) * (int64_t)a.dv + col;
  const int64_t s_at = (seq * a.hv + vh) * (int64_t)a.dk * a.dv + col + r;
  const bool has_col = col + r < a.dv;

  f32x4 S[DK / 16];
#pragma unroll
  for (int m = 0; m < DK / 16; ++m)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = 16 * m + 4 * g + x;
      S[m][x] = a.s0 && has_col && row < a.dk ? a.s0[s_at + (int64_t)row * a.dv] : 0.f;
    }

  const int64_t nchunks = (sp.len + kC - 1) / kC;
  uint4 rk[kWk], rq[kWk], rt[M::kParts][kWt], rp[kWt], rv[kWv];
  float rg;
  float eg_last = 0.f, eg_next;
  auto load = [&](int64_t ch) {
    const int n = (int)min((int64_t)kC, sp.len - ch * kC);
    const E* k0 = kp + ch * kC * a.k_stride;
    const E* q0 = qp + ch * kC * a.q_stride;
    const E* v0 = vp + ch * kC * a.v_stride;
    const char* ws = a.ws + ((slot0 + ch) * a.hv + vh) * (int64_t)ChunkWs<E>::kBytes;
#pragma unroll
    for (int i = 0; i < kWk; ++i) {
      const int x = tid + i * kThreads, row = x / (DK / kV), c = x % (DK / kV) * kV;
      rk[i] = tile_word(k0, a.k_stride, row, c, n, a.dk);
      rq[i] = tile_word(q0, a.q_stride, row, c, n, a.dk);
    }
#pragma unroll
    for (int i = 0; i < kWt; ++i) {
#pragma unroll
      for (int p = 0; p < M::kParts; ++p)
        rt[p][i] = reinterpret_cast<const uint4*>(ws)[p * (kC * kC / kV) + tid + i * kThreads];
      rp[i] = reinterpret_cast<const uint4*>(ws + ChunkWs<E>::kT)[tid + i * kThreads];
    }
#pragma unroll
    for (int i = 0; i < kWv; ++i) {
      const int x = tid + i * kThreads, row = x / (16 * NW / kV), c = x % (16 * NW / kV) * kV;
      rv[i] = tile_word(v0, a.v_stride, row, c, n, a.dv - col0);
    }
    const float* gate = reinterpret_cast<const float*>(ws + ChunkWs<E>::kT + ChunkWs<E>::kP);
    if (tid < 2 * kC) rg = gate[tid];
    eg_next = gate[2 * kC];
  };

  if (nchunks > 0) load(0);
  for (int64_t ch = 0; ch < nchunks; ++ch) {
    __syncthreads();  // the previous chunk's tiles have been read
#pragma unroll
    for (int i = 0; i < kWk; ++i) {
      const int x = tid + i * kThreads, at = x / (DK / kV) * Sm::kLd + x % (DK / kV) * kV;
      *reinterpret_cast<uint4*>(&sm.k[at]) = rk[i];
      *reinterpret_cast<uint4*>(&sm.q[at]) = rq[i];
    }
#pragma unroll
    for (int i = 0; i < kWt; ++i) {
      const int x = tid + i * kThreads, at = x / (kC / kV) * Sm::kLt + x % (kC / kV) * kV;
#pragma unroll
      for (int p = 0; p < M::kParts; ++p) *reinterpret_cast<uint4*>(&sm.t[p][at]) = rt[p][i];
      *reinterpret_cast<uint4*>(&sm.p[at]) = rp[i];
    }
#pragma unroll
    for (int i = 0; i < kWv; ++i) {
      const int x = tid + i * kThreads, at = x / (16 * NW / kV) * Sm::kLv + x % (16 * NW / kV) * kV;
      *reinterpret_cast<uint4*>(&sm.v[at]) = rv[i];
    }
    if (tid < kC) sm.eg[tid] = rg;
    else if (tid < 2 * kC) sm.c[tid - kC] = rg;
    eg_last = eg_next;
    __syncthreads();
    if (ch + 1 < nchunks) load(ch + 1);
    const int n = (int)min((int64_t)kC, sp.len - ch * kC);

    // K S (tokens x columns) and (Q S)^T (columns x tokens)
    f32x4 y[4], o[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < DK / M::kDepth; ++kb) {
      const auto s = M::split(&S[kb * kTPF]);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const auto kf = M::chain(&sm.k[(16 * m + r) * Sm::kLd + kb * M::kDepth], g);
        const auto qf = M::chain(&sm.q[(16 * m + r) * Sm::kLd + kb * M::kDepth], g);
#pragma unroll
        for (int p = 0; p < M::kParts; ++p) y[m] = M::mma(kf, s.p[p], y[m]);
        o[m] = M::mma(s.p[0], qf, o[m]);
      }
    }
    // Y = V - diag(exp G) K S;  O scaled by its token's factor
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 v = M::ctile(&sm.v[16 * m * Sm::kLv + 16 * w], Sm::kLv, g, r);
      const f32x4 eg = *reinterpret_cast<const f32x4*>(&sm.eg[16 * m + 4 * g]);
      const float so = a.scale * sm.eg[16 * m + r];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        y[m][x] = fmaf(-eg[x], y[m][x], v[x]);
        o[m][x] *= so;
      }
    }
    // E = T Y, T lower triangular
    f32x4 e[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) e[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < kC / M::kDepth; ++kb) {
      const auto ys = M::split(&y[kb * kTPF]);
#pragma unroll
      for (int m = kb * kTPF; m < 4; ++m) {
        const auto th = M::chain(&sm.t[0][(16 * m + r) * Sm::kLt + kb * M::kDepth], g);
        e[m] = M::mma(th, ys.p[0], e[m]);
        if constexpr (M::kParts == 2) {
          const auto tl = M::chain(&sm.t[1][(16 * m + r) * Sm::kLt + kb * M::kDepth], g);
          e[m] = M::mma(th, ys.p[1], e[m]);
          e[m] = M::mma(tl, ys.p[0], e[m]);
        }
      }
    }
    // O += P E, transposed: a lane ends with 4 consecutive columns of one token
#pragma unroll
    for (int kb = 0; kb < kC / M::kDepth; ++kb) {
      const auto ef = M::pack(&e[kb * kTPF]);
#pragma unroll
      for (int m = kb * kTPF; m < 4; ++m)
        o[m] = M::mma(ef, M::chain(&sm.p[(16 * m + r) * Sm::kLt + kb * M::kDepth], g), o[m]);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t = 16 * m + r;
      if (t < n && col + 4 * g < a.dv) {
        E* dst = op + (ch * kC + t) * (int64_t)a.hv * a.dv + 4 * g;
        if constexpr (sizeof(E) == 2)
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(make_float2(o[m][0], o[m][1])),
                                                      pack_bf16(make_float2(o[m][2], o[m][3])));
        else
          *reinterpret_cast<f32x4*>(dst) = o[m];
      }
    }
    // S = exp(G_64) S + K^T diag(c) E
#pragma unroll
    for (int m = 0; m < 4; ++m) e[m] *= *reinterpret_cast<const f32x4*>(&sm.c[16 * m + 4 * g]);
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) S[m] *= eg_last;
#pragma unroll
    for (int kb = 0; kb < kC / M::kDepth; ++kb) {
      const auto es = M::split(&e[kb * kTPF]);
#pragma unroll
      for (int m = 0; m < DK / 16; ++m) {
        const auto kt = M::chain_t(&sm.k[kb * M::kDepth * Sm::kLd + 16 * m], Sm::kLd, g, r);
#pragma unroll
        for (int p = 0; p < M::kParts; ++p) S[m] = M::mma(kt, es.p[p], S[m]);
      }
    }
  }
  if (a.last && has_col) {
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 16 * m + 4 * g + x;
        if (row < a.dk) a.last[s_at + (int64_t)row * a.dv] = S[m][x];
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

template <typename E, int DK, int NW>
int launch_scan_t(const Args& a, hipStream_t s) {
  const int cols = (a.dv + 16 * NW - 1) / (16 * NW);
  hipLaunchKernelGGL((scan_kernel<E, DK, NW>), dim3((unsigned)(a.nseq * a.hv * cols)),
                     dim3(64 * NW), 0, s, a, cols);
  return launch_status();
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
  if (bf) return a.dk <= 64 ? launch_scan_t<uint16_t, 64, 4>(a, s) : launch_scan_t<uint16_t, 128, 4>(a, s);
  return a.dk <= 64 ? launch_scan_t<float, 64, 4>(a, s) : launch_scan_t<float, 128, 4>(a, s);
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
