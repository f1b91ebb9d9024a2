// mamba_delta.hip -- the gated delta rule on gfx950: whole sequences in chunks of 64 tokens on the
// matrix cores.  The formulas are in mamba_delta.h.
//
//   chunk_kernel     one workgroup per chunk and key head: T, P and the gate factors, for every value
//                    head that shares the key head (K K^T and Q K^T are made once).
//   scan_kernel      the state goes through the chunks (mamba_delta_scan.h).
//   segments_kernel  a long sequence of few heads goes through scan_kernel in segments, side by side: first
//                    each segment's effect on the state, then the states before them one after another,
//                    then every segment from its own.
//
// Rounding (bf16 storage): products take bf16 operands into fp32 accumulators.  What makes E and enters the
// state by K^T E goes in as three bf16 parts (Y and c E: the fp32 value to 24 bits) or two (S, and T, which
// is one on its diagonal and small off it): the state is within about 3e-7 of fp64.  The output takes S, P
// and E as two parts each (2^-17 of every product), so that its own rounding to bf16 is the only one that
// shows; with S and P in one part its error was 1.4 to 1.8 times as large.  fp32 storage uses fp32 matrix
// instructions throughout.
#include "mamba_delta_scan.h"
#include "mamba_grid.h"

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
  float ghi[4][kC], glo[4][kC], beta[4][kC];  // of four value heads
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

// what a bf16 word leaves of its values
__device__ __forceinline__ void subtract_word(float (&a)[4], float (&b)[4], uint4 word) {
  const float2 a0 = unpack(word.x), a1 = unpack(word.y), b0 = unpack(word.z), b1 = unpack(word.w);
  a[0] -= a0.x; a[1] -= a0.y; a[2] -= a1.x; a[3] -= a1.y;
  b[0] -= b0.x; b[1] -= b0.y; b[2] -= b1.x; b[3] -= b1.y;
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

// T, P and the gates of one chunk, for the value heads of a key head.  Four waves share the 64 tokens, a wave's
// block of 16 x 16 products being what one matrix instruction makes; T comes from the inverses of its four
// diagonal blocks, which 16 substitution steps make in registers, and fp32 matrix products below them, so that
// no chain of steps is as long as the chunk.  10240 chunks x heads of dk = 128, bf16: 128 us, 0.45 GB read and
// written (3.5 TB/s); bound by the substitution's dependent steps and the barriers between the parts, which
// four workgroups per CU overlap.
template <typename E, int DK>
__global__ __launch_bounds__(256, sizeof(E) * DK <= 256 ? 4 : 2) void chunk_kernel(Args a) {
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
  // value heads blockIdx.y, blockIdx.y + gridDim.y, ... of the key head
  const int step = gridDim.y;
  for (int h = blockIdx.y, turn = 0; h < a.rep; h += step, ++turn) {
    const int vh = kh * a.rep + h;
    char* ws = a.ws + (slot * a.hv + vh) * a.ws_item;
    __syncthreads();  // the tiles of the previous head (or K and Q) have been read
    const int hs = turn & 3;
    if (hs == 0 && h + w * step < a.rep) {
      // Wave w: prefix sums of the w-th next head's log decays in fp64, kept as two floats: a difference of two
      // of them is then as exact as its own size, whatever came before in the chunk.  Below -200 exp is
      // 0 in fp32; the clamp keeps -inf (a reset) out of the differences and lets NaN through.
      float gl = 0.f, bt = 0.f;
      if (lane < n) {
        const int64_t at = (t0 + lane) * a.hv + vh + w * step;
        gl = ld_f32(static_cast<const E*>(a.g), at);
        bt = ld_f32(static_cast<const E*>(a.beta), at);
        gl = gl < -200.f ? -200.f : gl;
      }
      const double G = wave_prefix((double)gl, lane);
      const double total = __shfl(G, 63);
      const float hi = (float)G, lo = (float)(G - (double)hi);
      sm.ghi[w][lane] = hi;
      sm.glo[w][lane] = lo;
      sm.beta[w][lane] = bt;
      float* gate = reinterpret_cast<float*>(ws + w * step * a.ws_item + ChunkWs<E>::kGate);
      gate[lane] = exp_f32(hi);
      gate[kC + lane] = exp_f32((float)(total - G)) * bt;
      if (lane == 0) gate[2 * kC] = exp_f32((float)total);
      float* decay = reinterpret_cast<float*>(ws + w * step * a.ws_item + ChunkWs<E>::kDecay);
      decay[lane] = hi;
      decay[kC + lane] = lo;
      decay[2 * kC + lane] = bt;
    }
    __syncthreads();
    const float gi = sm.ghi[hs][i], gil = sm.glo[hs][i];
    float p[4][4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int j = 16 * jt + 4 * g;
      float A[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float d = jt <= w && j + x <= i ? exp_f32((gi - sm.ghi[hs][j + x]) +
                                                        (gil - sm.glo[hs][j + x])) *
                                                    sm.beta[hs][j + x]
                                              : 0.f;
        A[x] = j + x < i ? d * kk[jt][x] : 0.f;
        p[jt][x] = d * qk[jt][x] * a.scale;
      }
      *reinterpret_cast<float4*>(&sm.m.a[i * Sm::kLf + j]) = make_float4(A[0], A[1], A[2], A[3]);
    }
    // a lane's accumulators of one block of P are one word of its image
#pragma unroll
    for (int kb = 0; kb < TriTile<E>::kBlocks; ++kb)
      if (16 * w >= kb * M::kDepth) {
        float (&lo)[4] = p[kb * M::kTiles], (&hi)[4] = p[(kb + 1) * M::kTiles - 1];
        const int at = TriTile<E>::word_at(kb, i, g);
        const uint4 word = pack_word<E>(lo, hi);
        *reinterpret_cast<uint4*>(ws + ChunkWs<E>::kP + at) = word;
        if (M::parts(2) > 1) {
          subtract_word(lo, hi, word);
          *reinterpret_cast<uint4*>(ws + ChunkWs<E>::kP + ChunkWs<E>::kPart + at) = pack_word<E>(lo, hi);
        }
      }
    __syncthreads();
    // T = (I + A)^-1 by blocks of 16.  Wave w inverts diagonal block w by substitution, lane r its
    // column r: x_m = [m = r] - sum_{j < m} A_mj x_j, in four partial sums.
    {
      const float* Ab = &sm.m.a[16 * w * Sm::kLf + 16 * w];
      float x[16];
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        f32x4 t = {m == r ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < m; j += 4) {
          const f32x4 row = *reinterpret_cast<const f32x4*>(Ab + m * Sm::kLf + j);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (j + y < m) t[y] = fmaf(-row[y], x[j + y], t[y]);
        }
        x[m] = (t[0] + t[1]) + (t[2] + t[3]);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m)  // the four lane groups hold the same columns: 4 rows each
        sm.m.t[(16 * w + 4 * g + m) * Sm::kLf + 16 * w + r] =
            g == 0 ? x[m] : g == 1 ? x[4 + m] : g == 2 ? x[8 + m] : x[12 + m];
    }
    __syncthreads();
    // Wave w makes block column w below the diagonal: T_iw = -T_ii (sum_{k=w}^{i-1} A_ik T_kw), its
    // own blocks staying in accumulators.  (Blocks above the diagonal inside a block of the image are
    // zero.)
    {
      using F = Mma<float>;
      f32x4 T[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        T[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (b == w)
#pragma unroll
          for (int x = 0; x < 4; ++x) T[b][x] = sm.m.t[(16 * b + 4 * g + x) * Sm::kLf + 16 * w + r];
        if (b > w) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < b; ++k)
            if (k >= w)
              acc = F::mma(*reinterpret_cast<const f32x4*>(
                               &sm.m.a[(16 * b + r) * Sm::kLf + 16 * k + 4 * g]), T[k], acc);
          T[b] = F::mma(*reinterpret_cast<const f32x4*>(
                            &sm.m.t[(16 * b + r) * Sm::kLf + 16 * b + 4 * g]), -acc,
                        f32x4{0.f, 0.f, 0.f, 0.f});
        }
        if (b != w)
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
      for (int part = 0; part < M::parts(kTParts); ++part) {
        const uint4 word = pack_word<E>(lo, hi);
        *reinterpret_cast<uint4*>(ws + ChunkWs<E>::kT + part * ChunkWs<E>::kPart +
                                  TriTile<E>::word_at(kb, t, x & 3)) = word;
        if (sizeof(E) == 2) subtract_word(lo, hi, word);
      }
    }
  }
}

// ------------------------------------------------------------------ the state through the chunks

template <typename E, int DK, int NW, Pass kPass>
__global__ __launch_bounds__(kPassThreads) void scan_kernel(Args a, int32_t col_blocks, uint32_t blocks) {
  __shared__ __align__(1024) char smem[Stage<E, DK, NW, kPass>::kLds];
  const uint32_t id = wide_index();
  if (id < blocks) scan_pass<E, DK, NW, kPass>(a, col_blocks, smem, id, blocks);
}

// The states before the segments, one after another: S <- map S + (the segment's own).  A workgroup has 16
// columns, its waves 16 rows each; fp32 matrix instructions, S handed round through LDS.  Bound by that chain:
// 65 us for 65536 tokens x 12 heads of 128, bf16.  seg_state holds each segment's own result on
// entry and the state before it on return, the first segment's (of sequences without tokens, too) being a copy
// of the initial state: the output pass reads only these, as it may write the last state over the initial one.
template <int DK>
__global__ __launch_bounds__(DK * 4) void segments_kernel(Args a, int32_t col_blocks) {
  using M = Mma<float>;
  constexpr int kLd = DK + 4;
  __shared__ __align__(16) float sm[2][16 * kLd];  // S transposed: column r, then row
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, w = threadIdx.x >> 6;
  const int64_t sh = blockIdx.x / col_blocks;
  const int64_t seq = sh / a.hv;
  const int vh = (int)(sh - seq * a.hv);
  const int col = (int)(blockIdx.x - sh * col_blocks) * 16 + r;
  const int64_t unit = a.seg_chunks * kC;
  const Span sp = seq_span(a, seq);
  const int64_t base = slot_base(a, seq, sp.first, unit);
  const int64_t nseg = (sp.len + unit - 1) / unit;
  const bool has_col = col < a.dv;
  const int row0 = 16 * w + 4 * g;  // this lane's rows of S
  auto state = [&](int64_t slot) {
    return a.seg_state + (slot * a.hv + vh) * (int64_t)a.dk * a.dv + (int64_t)row0 * a.dv + col;
  };
  auto load_own = [&](int64_t s) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (has_col && row0 < a.dk)
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = state(base + s)[(int64_t)x * a.dv];
    return v;
  };
  // operands: row 16 w + r of the segment's map; the next segment's are on their way meanwhile
  f32x4 map[2][DK / 16];
  auto load_map = [&](int64_t s, f32x4 (&map)[DK / 16]) {
    const float* p = a.seg_map + ((base + s) * a.hv + vh) * (int64_t)a.dk * a.dk +
                     (int64_t)(16 * w + r) * a.dk + 4 * g;
#pragma unroll
    for (int kb = 0; kb < DK / 16; ++kb)
      map[kb] = 16 * w + r < a.dk && 16 * kb + 4 * g < a.dk
                    ? *reinterpret_cast<const f32x4*>(p + 16 * kb) : f32x4{0.f, 0.f, 0.f, 0.f};
  };
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (a.s0 && has_col && row0 < a.dk)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      S[x] = a.s0[((seq * a.hv + vh) * (int64_t)a.dk + row0 + x) * a.dv + col];
  f32x4 own[2] = {S, S};
  auto store = [&](int64_t s) {
    if (has_col && row0 < a.dk)
#pragma unroll
      for (int x = 0; x < 4; ++x) state(base + s)[(int64_t)x * a.dv] = S[x];
  };
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (i + 1 < nseg) {
      load_map(i, map[i]);
      own[i] = load_own(i);
    }
  store(0);
  for (int64_t s0 = 0; s0 + 1 < nseg; s0 += 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t s = s0 + i;
      if (s + 1 >= nseg) break;
      *reinterpret_cast<f32x4*>(&sm[i][r * kLd + row0]) = S;
      __syncthreads();
      f32x4 acc[2] = {own[i], f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int kb = 0; kb < DK / 16; ++kb)
        acc[kb & 1] = M::mma(map[i][kb],
                             *reinterpret_cast<const f32x4*>(&sm[i][r * kLd + 16 * kb + 4 * g]),
                             acc[kb & 1]);
      S = acc[0] + acc[1];
      if (s + 3 < nseg) {
        load_map(s + 2, map[i]);
        own[i] = load_own(s + 2);
      }
      store(s + 1);
    }
  }
}

template <typename E, int DK>
int launch_chunks_t(const Args& a, hipStream_t s) {
  // value heads of a key head one after another share K K^T and Q K^T; where that leaves CUs idle, each
  // has a workgroup of its own (whole forward, each and together, two value heads per key head, the only ratio
  // measured: 40 chunks x heads 17 and 22 us, 400 47 and 51 us, 800 76 and 80 us, 10240 480 and 446 us)
  const unsigned split = a.slots * a.hk * a.rep <= 512 ? (unsigned)a.rep : 1;
  hipLaunchKernelGGL((chunk_kernel<E, DK>), dim3((unsigned)(a.slots * a.hk), split), dim3(256), 0, s, a);
  return launch_status();
}

template <typename E, int DK, int NW, Pass kPass>
int launch_scan_t(const Args& a, hipStream_t s) {
  const int cols = (a.dv + 16 * NW - 1) / (16 * NW) +
                   (kPass == kSummary ? (a.dk + 16 * NW - 1) / (16 * NW) : 0);
  const uint32_t blocks = (uint32_t)(a.seg_slots * a.hv * cols);
  hipLaunchKernelGGL((scan_kernel<E, DK, NW, kPass>), wide_grid(blocks, 64 * NW), dim3(64 * NW), 0, s, a, cols,
                     blocks);
  return launch_status();
}

template <typename E, Pass kPass>
int launch_scan(const Args& a, hipStream_t s) {
  const bool even = !a.offsets || a.nseq == 1;
  const bool narrow = narrow_pass(a.hv, a.seg_slots, even, a.dv);
  if (a.dk <= 64)
    return narrow ? launch_scan_t<E, 64, 4, kPass>(a, s) : launch_scan_t<E, 64, 8, kPass>(a, s);
  return narrow ? launch_scan_t<E, 128, 4, kPass>(a, s) : launch_scan_t<E, 128, 8, kPass>(a, s);
}

template <typename E>
int launch_forward(const Args& a, hipStream_t s) {
  if (a.seg_chunks) {
    int st = launch_scan<E, kSummary>(a, s);
    if (st != MAMBA_OK) return st;
    const int cols = (a.dv + 15) / 16;
    if (a.dk <= 64)
      hipLaunchKernelGGL(segments_kernel<64>, dim3((unsigned)(a.nseq * a.hv * cols)), dim3(256), 0, s,
                         a, cols);
    else
      hipLaunchKernelGGL(segments_kernel<128>, dim3((unsigned)(a.nseq * a.hv * cols)), dim3(512), 0, s,
                         a, cols);
    if ((st = launch_status()) != MAMBA_OK) return st;
  }
  return launch_scan<E, kOut>(a, s);
}

// Chunks per segment, 0 for whole sequences.  A pass costs one unit per chunk and round of 256
// workgroups (one per CU, counted as 128 columns each, also where narrow_pass then takes 64); segments add a
// summary pass over their own and the map's columns, about 0.65 of a unit per chunk (65536 tokens x 12 heads: 378 us
// in two rounds, the output pass 281 us in one), and a quarter of a unit per segment to join them.  Packed sequences
// are taken to be up to twice as long as their mean.  Segments are used where that model gains a quarter.
// Measured, heads of 128, bf16, whole and in segments: 65536 tokens x 12 heads 3025 and 778 us, 16384 x 12
// 713 and 259 us.
int64_t plan_segments(const mamba_delta_dims* d, bool packed) {
  constexpr double kCUs = 256.0;
  const int64_t per = d->dv <= 64 ? 64 : 128;
  const double vb = (double)((d->dv + per - 1) / per), kb = (double)((d->dk + per - 1) / per);
  const int64_t nseq = packed ? std::min(d->batch, d->seqlen) : d->batch;
  const double heads = (double)nseq * (double)d->v_heads;
  double chunks = (double)((d->seqlen + kC - 1) / kC);
  if (packed && nseq > 1) chunks = std::min(chunks, 2.0 * chunks / (double)nseq);
  const double whole = std::ceil(heads * vb / kCUs) * chunks;
  double best = 0.75 * whole;
  int64_t pick = 0;
  for (int64_t c = 8; c <= 256; ++c) {
    const double n = std::ceil(chunks / (double)c);
    if (n < 2) break;
    if ((n + 1) * heads * (vb + kb) > 2147483647.0) continue;  // one grid
    const double t = std::ceil((n - 1) * heads * (vb + kb) / kCUs) * (double)c * 0.65 +
                     std::ceil(n * heads * vb / kCUs) * (double)c + 0.25 * n + 4.0;
    if (t < best) {
      best = t;
      pick = c;
    }
  }
  return pick;
}

struct FwdLayout {  // workspace regions in bytes
  int64_t seg_chunks, seg_slots;
  size_t state, map, total;
};
FwdLayout fwd_layout(const mamba_delta_dims* d, bool packed) {
  FwdLayout l = {plan_segments(d, packed), d->batch, 0, 0, 0};
  l.state = (size_t)chunk_slots(d, packed) * (size_t)d->v_heads * chunk_ws_bytes(d);
  l.map = l.total = l.state;
  if (l.seg_chunks) {
    l.seg_slots = slots_of(d, packed, l.seg_chunks * kC);
    const size_t rows = (size_t)l.seg_slots * (size_t)d->v_heads * (size_t)d->dk * sizeof(float);
    l.map = l.state + rows * (size_t)d->dv;
    l.total = l.map + rows * (size_t)d->dk;
  }
  return l;
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
  return fwd_layout(dims, packed != 0).total;
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
  const FwdLayout l = fwd_layout(dims, seq_offsets != nullptr);
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  Args a = make_args(dims, scale, q, k, v, g, beta, initial_state, seq_offsets);
  a.out = out;
  a.last = last_state;
  a.ws = static_cast<char*>(workspace);
  a.seg_chunks = l.seg_chunks;
  a.seg_slots = l.seg_slots;
  a.seg_state = reinterpret_cast<float*>(a.ws + l.state);
  a.seg_map = reinterpret_cast<float*>(a.ws + l.map);
  const bool bf = dims->io_dtype == MAMBA_BF16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = launch_chunks(a, bf, s)) != MAMBA_OK) return st;
  return bf ? launch_forward<uint16_t>(a, s) : launch_forward<float>(a, s);
}

}  // extern "C"
