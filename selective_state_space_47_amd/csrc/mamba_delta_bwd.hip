// mamba_delta_bwd.hip -- gradients of the gated delta rule on gfx950.
//
// In chunks (mamba_delta.h), with dS' the adjoint of the state after the chunk and dO that of O:
//     dE = P^T dO + diag(c) K dS',   dV = dY = T^T dE
//     dS = exp(G_64) dS' + Q^T diag(scale exp G) dO - K^T diag(exp G) dY
//     M_ij = dO_i . e_j (j <= i),  N_ij = dY_i . e_j (j < i)
//     B1_ij = scale D_ij beta_j M_ij,  B2_ij = -D_ij beta_j N_ij
//     dQ_i = sum_j B1_ij k_j + scale exp(G_i) S dO_i
//     dK_i = sum_j B2_ij k_j - exp(G_i) S dY_i + sum_t (B2_ti k_t + B1_ti q_t) + c_i dS' e_i
//     dbeta_j = sum_i D_ij (scale (q_i . k_j) M_ij - (k_i . k_j) N_ij) + exp(G_64 - G_j) k_j . dS' e_j
//     dg_t = exp(G_64) <dS', S> + sum_{j < t} Z_j + sum_{i >= t} R_i + sum_{i >= t > j} X_ij,
//         Z_j = c_j k_j . dS' e_j,  X_ij = B1_ij (q_i . k_j) + B2_ij (k_i . k_j)
//         R_i = exp(G_i) (scale q_i . S dO_i - k_i . S dY_i)
// The last sum is that of the rows i >= t of X less that of its columns j >= t, whose common pairs cancel: they are
// added in fp64, so that nothing of them is left where a strong decay makes the pairs that cross t small.
//
// Three launches: the chunk products of mamba_delta.hip, then
//   passes_kernel   the state forwards through the chunks (mamba_delta_scan.h; it leaves E and the state before
//                   every chunk) and, beside it, the adjoint of the state backwards: dV, and dS' of every
//                   chunk; laid out like the state's pass (16 columns per wave, in accumulators)
//   grad_kernel     one workgroup per chunk and key head: everything else.  The value heads that share
//                   the key head add their dQ and dK in accumulators, in a fixed order: no atomics.
// Every gradient is rounded once.  Rounding inside, bf16 storage: two bf16 parts of every factor; S to 17 bits
// (a byte beside its bf16).  One part of S and dY, which dQ, dK and the sums of dg take, cost up to 1.6 times the
// error of rounding once where queries lie near their keys.
#include "mamba_delta_scan.h"

namespace mamba {
namespace delta {
namespace {

struct BwdArgs {
  Args f;
  const void* dout;    // (tokens, hv, dv)
  const float* dlast;  // (nseq, hv, dk, dv) or NULL: zero
  void* dq;            // (tokens, hk, dk)
  void* dk;
  void* dv;            // (tokens, hv, dv)
  void* dg;            // (tokens, hv)
  void* dbeta;
  float* ds0;          // (nseq, hv, dk, dv) or NULL
  void* dy_low;        // bf16 storage: what bf16 leaves of dY, like dv
};

// 8 (bf16) or 4 (fp32) consecutive values from one operand's accumulators
template <typename E>
__device__ __forceinline__ void store_values(E* p, const f32x4* c) {
  *reinterpret_cast<typename Mma<E>::Frag*>(p) = Mma<E>::pack(c);
}

// what bf16 leaves of four values
__device__ __forceinline__ f32x4 after_bf16(f32x4 v) {
  const float2 a = unpack(pack_bf16(make_float2(v[0], v[1]))), b = unpack(pack_bf16(make_float2(v[2], v[3])));
  return f32x4{v[0] - a.x, v[1] - a.y, v[2] - b.x, v[3] - b.y};
}

// sum over the four groups
template <typename V>
__device__ __forceinline__ V across_groups(V v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// ------------------------------------------------------------------ the adjoint of the state

template <typename E, int DK, int NW>
struct AdjStage {
  using VT = ValueTile<E, 16 * NW>;
  static constexpr int kK = 0;
  static constexpr int kQ = KeyTile<E, DK>::kBytes;
  static constexpr int kWs = 2 * KeyTile<E, DK>::kBytes;  // P, T, gates
  static constexpr int kP = kWs + ChunkWs<E>::kP;
  static constexpr int kT = kWs + ChunkWs<E>::kT;
  static constexpr int kGate = kWs + ChunkWs<E>::kGate;
  static constexpr int kDO = kWs + ChunkWs<E>::kDecay;
  static constexpr int kBytes = kDO + VT::kBytes;
  static constexpr int kCount = 2 * kBytes <= 160 * 1024 ? 2 : 1;
  static constexpr int kLds = kCount * kBytes;
};

template <typename E, int DK, int NW>
__device__ __forceinline__ void adjoint_pass(const BwdArgs& b, int32_t col_blocks, char* smem, uint32_t id,
                                             uint32_t grid) {
  using M = Mma<E>;
  using St = AdjStage<E, DK, NW>;
  using KT = KeyTile<E, DK>;
  using TT = TriTile<E>;
  using VT = typename St::VT;
  using CW = ChunkWs<E>;
  constexpr int kP2 = M::parts(2);
  const Args& a = b.f;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wg = spread_index(id, grid, a.rep * col_blocks);
  const int64_t sh = wg / col_blocks;
  const int64_t rank = sh / a.hv, seq = seq_by_length(a, rank);
  const int vh = (int)(sh - rank * a.hv), kh = vh / a.rep;
  const int col0 = (int)(wg - sh * col_blocks) * 16 * NW;
  const int col = col0 + 16 * w;
  const Span sp = seq_span(a, seq);
  const int64_t slot0 = slot_base(a, seq, sp.first);
  const E* kp = static_cast<const E*>(a.k) + sp.first * a.k_stride + (int64_t)kh * a.dk;
  const E* qp = static_cast<const E*>(a.q) + sp.first * a.q_stride + (int64_t)kh * a.dk;
  const int64_t o_stride = (int64_t)a.hv * a.dv;
  const int64_t o_at = (sp.first * a.hv + vh) * (int64_t)a.dv;
  const E* dop = static_cast<const E*>(b.dout) + o_at + col0;
  E* dvp = static_cast<E*>(b.dv) + o_at + col;
  E* low = static_cast<E*>(b.dy_low) + o_at + col;
  const int64_t s_at = (seq * a.hv + vh) * (int64_t)a.dk * a.dv + col + r;
  const bool has_col = col + r < a.dv;

  f32x4 S[DK / 16];  // the adjoint, rows (keys' values) permuted as in KeyTile
#pragma unroll
  for (int m = 0; m < DK / 16; ++m)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = KT::value(m, g, x);
      S[m][x] = b.dlast && has_col && row < a.dk ? b.dlast[s_at + (int64_t)row * a.dv] : 0.f;
    }

  const uint32_t lds0 = lds_address(smem);
  const int64_t nchunks = (sp.len + kC - 1) / kC;
  const int vcols = min(a.dv - col0, 16 * NW);
  const RowCopy<E, KT, kC, NW> ck(w, lane, a.k_stride, a.dk), cq(w, lane, a.q_stride, a.dk);
  const RowCopy<E, VT, kC, NW> co(w, lane, o_stride, vcols);
  auto copy = [&](int64_t ch, int st) {
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    const uint32_t to = lds0 + st * St::kBytes;
    const char* ws = a.ws + ((slot0 + ch) * a.hv + vh) * a.ws_item;
    ck(rows_buffer(kp + t * a.k_stride, n, a.k_stride, a.dk), to + St::kK, w);
    co(rows_buffer(dop + t * o_stride, n, o_stride, vcols), to + St::kDO, w);
    copy_linear<CW::kDecay, NW>(ws, to + St::kWs, w, lane);
    cq(rows_buffer(qp + t * a.q_stride, n, a.q_stride, a.dk), to + St::kQ, w);
  };

  const int dv_pad = (a.dv + BwdBlock<E>::kDB - 1) / BwdBlock<E>::kDB * BwdBlock<E>::kDB;
  const int64_t img_bytes = (int64_t)dv_pad * KT::kRow;
  const KT kt(lane);
  const TT tt(lane);
  const VT ot(lane, 16 * w);
  uint32_t s_off[DK / M::kDepth];  // this lane's words of the images
#pragma unroll
  for (int kb = 0; kb < DK / M::kDepth; ++kb)
    s_off[kb] = (col + r) * KT::kRow + (((4 * kb + g) ^ KT::key(col + r)) << 4);
  if (nchunks > 0) copy(nchunks - 1, 0);
  for (int64_t ch = nchunks - 1; ch >= 0; --ch) {
    const int st = St::kCount == 2 ? (int)((nchunks - 1 - ch) & 1) : 0;
    copies_done();
    const lds_ptr sm = (lds_ptr)(smem + st * St::kBytes);
    const int n = (int)min((int64_t)kC, sp.len - ch * kC);
    // (operands are read a step before their products, as in the state's pass)
    auto step = [] { __builtin_amdgcn_sched_barrier(0); };
    typename M::Frag kf[2][4];
    auto read_k = [&](int kb) {
#pragma unroll
      for (int m = 0; m < 4; ++m) kf[kb & 1][m] = kt.rows(sm + St::kK, m, kb);
    };
    read_k(0);
    if (St::kCount == 2 && ch > 0) copy(ch - 1, st ^ 1);
    // dS' goes to its image, and K dS'
    const int64_t at = ((slot0 + ch) * a.hv + vh) * img_bytes;
    f32x4 e[4], cf[4];
    typename M::Frag pf[2][kP2][4], df[2];
    auto read_p = [&](int ib) {
      df[ib & 1] = ot.operand(sm + St::kDO, ib);
#pragma unroll
      for (int m = 0; m < (ib + 1) * M::kTiles; ++m) {
#pragma unroll
        for (int p = 0; p < kP2; ++p) pf[ib & 1][p][m] = tt.cols(sm + St::kP + p * TT::kBytes, m, ib);
      }
    };
#pragma unroll
    for (int m = 0; m < 4; ++m) e[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < DK / M::kDepth; ++kb) {
      step();
      if (kb + 1 < DK / M::kDepth) {
        read_k(kb + 1);
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) cf[m] = lds_read<f32x4>(sm + St::kGate + (kC + 16 * m + 4 * g) * 4);
        read_p(0);
      }
      const auto ds = M::template split<kP2>(&S[kb * M::kTiles]);
      if (col < dv_pad) {
        *reinterpret_cast<typename M::Frag*>(a.ds_img + at + s_off[kb]) = ds.p[0];
        if constexpr (kP2 == 2) *reinterpret_cast<typename M::Frag*>(a.ds_low + at + s_off[kb]) = ds.p[1];
      }
#pragma unroll
      for (int p = 0; p < kP2; ++p)
#pragma unroll
        for (int m = 0; m < 4; ++m) e[m] = M::mma(kf[kb & 1][m], ds.p[p], e[m]);
    }
    // dE = diag(c) K dS' + P^T dO
    typename M::Frag tf[2][kP2][4];
    auto read_t = [&](int ib) {
#pragma unroll
      for (int p = 0; p < kP2; ++p)
#pragma unroll
        for (int m = 0; m < (ib + 1) * M::kTiles; ++m)
          tf[ib & 1][p][m] = tt.cols(sm + St::kT + p * TT::kBytes, m, ib);
    };
#pragma unroll
    for (int ib = 0; ib < TT::kBlocks; ++ib) {
      step();
      if (ib + 1 < TT::kBlocks) read_p(ib + 1); else read_t(0);
      if (ib == 0)
#pragma unroll
        for (int m = 0; m < 4; ++m) e[m] *= cf[m];
#pragma unroll
      for (int p = 0; p < kP2; ++p)
#pragma unroll
        for (int m = 0; m < (ib + 1) * M::kTiles; ++m) e[m] = M::mma(pf[ib & 1][p][m], df[ib & 1], e[m]);
    }
    // dY = T^T dE, and transposed for the store; then what dS takes
    f32x4 eg[4], o[4];
    float last = 0.f;
    typename M::Frag qc[2][4], kc[2][4];
    auto read_cols = [&](int i) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        qc[i & 1][m] = kt.cols(sm + St::kQ, i % (DK / 64) * 4 + m, i / (DK / 64));
        kc[i & 1][m] = kt.cols(sm + St::kK, i % (DK / 64) * 4 + m, i / (DK / 64));
      }
    };
    f32x4 y[4], yt[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = yt[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ib = 0; ib < TT::kBlocks; ++ib) {
      step();
      if (ib + 1 < TT::kBlocks) {
        read_t(ib + 1);
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          eg[m] = lds_read<f32x4>(sm + St::kGate + (16 * m + 4 * g) * 4);
          o[m] = ot.tile(sm + St::kDO, m);
        }
        last = lds_read<float>(sm + St::kGate + 2 * kC * 4);
        read_cols(0);
      }
      const auto es = M::template split<kP2>(&e[ib * M::kTiles]);
#pragma unroll
      for (int m = 0; m < (ib + 1) * M::kTiles; ++m)
#pragma unroll
        for (int p = 0; p < kP2; ++p) {
#pragma unroll
          for (int x = 0; x + p < kP2; ++x) {
            y[m] = M::mma(tf[ib & 1][p][m], es.p[x], y[m]);
            yt[m] = M::mma(es.p[x], tf[ib & 1][p][m], yt[m]);
          }
        }
    }
    step();
    // token 16 m + r, columns col + 4 g .. +3
    const int bytes = (int)(((n - 1) * o_stride + max(a.dv - col, 0)) * (int64_t)sizeof(E));
    const auto buf = __builtin_amdgcn_make_buffer_rsrc(dvp + ch * kC * o_stride, 0, bytes, 0x00020000);
    const auto buf_low = __builtin_amdgcn_make_buffer_rsrc(low + ch * kC * o_stride, 0, bytes, 0x00020000);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t to = col + 4 * g < a.dv ? (uint32_t)((16 * m + r) * o_stride + 4 * g) * (uint32_t)sizeof(E)
                                             : kOutside;
      store_four<E>(buf, to, yt[m]);
      if constexpr (kP2 == 2) store_four<E>(buf_low, to, after_bf16(yt[m]));
    }
    // dS = exp(G_64) dS' + Q^T diag(scale exp G) dO - K^T diag(exp G) dY
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      o[m] *= a.scale * eg[m];
      y[m] *= -eg[m];
    }
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) S[m] *= last;
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      const auto of = M::template split<kP2>(&o[kb * M::kTiles]);
      const auto yf = M::template split<kP2>(&y[kb * M::kTiles]);
#pragma unroll
      for (int j = 0; j < DK / 64; ++j) {
        const int i = kb * (DK / 64) + j;
        if (i + 1 < TT::kBlocks * (DK / 64)) read_cols(i + 1);
#pragma unroll
        for (int p = 0; p < kP2; ++p)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            S[4 * j + m] = M::mma(qc[i & 1][m], of.p[p], S[4 * j + m]);
            S[4 * j + m] = M::mma(kc[i & 1][m], yf.p[p], S[4 * j + m]);
          }
        step();
      }
    }
    if (St::kCount == 1 && ch > 0) {
      __syncthreads();  // every wave has read the stage
      copy(ch - 1, 0);
    }
  }
  if (b.ds0 && has_col) {
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = KT::value(m, g, x);
        if (row < a.dk) b.ds0[s_at + (int64_t)row * a.dv] = S[m][x];
      }
  }
}

// The state forwards and its adjoint backwards need nothing of each other: their workgroups share a launch,
// the adjoint's first (they take longer).  8 x 2048 tokens x 40 heads of 128, bf16: 714 us (before dY had a second
// part 670, and in launches of their own, two rounds of the CUs each, 371 and 608), 2.8 GB read and written, 3.9 TB/s:
// the memory's rate but for the last round's idle CUs.  S and dS' of every chunk are 1.2 GB of it; making them again
// from the chunks' inputs would take the passes' products a second time.  (fp32 tiles of 128 keys do not fit 256
// registers.)
template <typename E, int DK, int NW>
__global__ __launch_bounds__((sizeof(E) * DK <= 256 ? kPassThreads : 64 * NW)) void passes_kernel(
    BwdArgs b, int32_t col_blocks, uint32_t each) {
  constexpr int kA = AdjStage<E, DK, NW>::kLds, kS = Stage<E, DK, NW, kBackward>::kLds;
  __shared__ __align__(1024) char smem[kA > kS ? kA : kS];
  if (blockIdx.x < each)
    adjoint_pass<E, DK, NW>(b, col_blocks, smem, blockIdx.x, each);
  else
    scan_pass<E, DK, NW, kBackward>(b.f, col_blocks, smem, blockIdx.x - each, each);
}

// ------------------------------------------------------------------ dQ, dK, dg, dbeta

// every wave's LDS accesses are done (its copies may still be on their way)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// sum over the 16 lanes of a group, in every lane of it
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_row<0x128>(v);
  v += dpp_row<0x124>(v);
  v += dpp_row<0x122>(v);
  v += dpp_row<0x121>(v);
  return v;
}
// the same in fp64
template <int kCtrl>
__device__ __forceinline__ double dpp_row64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __float_as_uint(dpp_row<kCtrl>(__uint_as_float((uint32_t)b)));
  const uint32_t hi = __float_as_uint(dpp_row<kCtrl>(__uint_as_float((uint32_t)(b >> 32))));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double group_sum(double v) {
  v += dpp_row64<0x128>(v);
  v += dpp_row64<0x124>(v);
  v += dpp_row64<0x122>(v);
  v += dpp_row64<0x121>(v);
  return v;
}
// sum over lanes lane .. 63
template <typename V>
__device__ __forceinline__ V wave_suffix(V v, int lane) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const V t = __shfl_down(v, m);
    if (lane + m < 64) v += t;
  }
  return v;
}

template <typename E, int DK>
struct GradSmem {
  using B = BwdBlock<E>;
  // one block of columns of the state: dO, dY, E, S, dS', and what bf16 leaves of dY, S and dS'
  static constexpr int kDO = 0;
  static constexpr int kDY = kDO + B::kE;
  static constexpr int kE = kDY + B::kE;
  static constexpr int kS = kE + B::kEParts * B::kE;
  static constexpr int kDS = kS + B::kDB * KeyTile<E, DK>::kRow;
  static constexpr int kBlock = B::kDB * KeyTile<E, DK>::kRow;
  static constexpr bool kLow = sizeof(E) == 2;
  static constexpr int kDSLow = kDS + kBlock;
  static constexpr int kSLow = kDSLow + (kLow ? kBlock : 0);  // (of S: bytes)
  static constexpr int kDYLow = kSLow + (kLow ? kBlock / 2 : 0);
  static constexpr int kStage = kDYLow + (kLow ? B::kE : 0);
  static constexpr int kBParts = Mma<E>::parts(2);
  static constexpr int kK = 0;
  static constexpr int kQ = KeyTile<E, DK>::kBytes;
  static constexpr int kSLowTile = 2 * KeyTile<E, DK>::kBytes;  // what bf16 leaves of the block's S, as bf16
  // B1 and B2, after a head's last block: in its stage where there are two
  static constexpr int kB = 2 * kBParts * TriTile<E>::kBytes;
  static constexpr bool kBInStage = kLow;
  static constexpr int kOwnB = kSLowTile + (kLow ? kBlock : 0);
  static constexpr int kGate = kOwnB + (kBInStage ? 0 : kB);  // gates and decays of two heads
  static constexpr int kSumX = kGate + 2 * 2048;  // per wave and column: sum of X (fp64)
  static constexpr int kSumB = kSumX + 8 * kC * 8;  // and for dbeta
  static constexpr int kRowX = kSumB + 8 * kC * 4;  // per half and token: row sum of X (fp64),
  static constexpr int kTok = kRowX + 2 * kC * 8;   // R, then k . dS' e
  static constexpr int kDot = kTok + 4 * kC * 4;    // per wave: <dS', S>
  static constexpr int kStages = (kDot + 32 + 1023) / 1024 * 1024;
  static constexpr int kCount = kStages + 2 * kStage <= 160 * 1024 ? 2 : 1;
  static constexpr int kBytes = kStages + kCount * kStage;
  static_assert(!kBInStage || (kCount == 2 && kB <= kStage), "a stage is free while the next block comes");
};

// Eight waves: wave (tile, half) has the tokens 16 tile .. 16 tile + 15.  Half 0 makes M and B1, half 1 N
// and B2; of dQ and dK each half has half of the keys' values.  The state's columns come in blocks of kDB,
// head after head: the next block is copied while one is worked on.
// 10240 chunks x heads of 128 x 128, bf16: 731 us, 2.4 GB, 3.3 TB/s; 619 us of it without the products and what is
// made of them: bound first by the copies of the images, 48 KB of them on their way to a CU at a time (the LDS that
// is left), then by what follows a head's last block, which nothing else on the CU overlaps.
template <typename E, int DK>
__global__ __launch_bounds__(512) void grad_kernel(BwdArgs b) {
  using M = Mma<E>;
  using Sm = GradSmem<E, DK>;
  using KT = KeyTile<E, DK>;
  using TT = TriTile<E>;
  using BB = BwdBlock<E>;
  using ET = KeyTile<E, BB::kDB>;
  using CW = ChunkWs<E>;
  constexpr int kTiles = DK / 32, kBP = Sm::kBParts;  // accumulator tiles of a wave's values
  __shared__ __align__(1024) char smem[Sm::kBytes];
  const Args& a = b.f;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = w & 3, half = w >> 2, m0 = half * kTiles;
  const int64_t wg = placed_index(blockIdx.x, gridDim.x);
  const int64_t slot = wg / a.hk;
  const int kh = (int)(wg - slot * a.hk);
  const int64_t seq = slot_seq(a, slot);
  const Span sp = seq_span(a, seq);
  const int64_t c0 = (slot - slot_base(a, seq, sp.first)) * kC;
  if (c0 < 0 || c0 >= sp.len) return;
  const int n = (int)min((int64_t)kC, sp.len - c0);
  const int64_t t0 = sp.first + c0;
  const uint32_t lds0 = lds_address(smem);
  const lds_ptr sm = (lds_ptr)smem;
  const int64_t o_stride = (int64_t)a.hv * a.dv;
  const int blocks = (a.dv + BB::kDB - 1) / BB::kDB;
  const int64_t img_bytes = (int64_t)blocks * BB::kDB * KT::kRow;
  const int64_t e_bytes = (int64_t)blocks * BB::kEParts * BB::kE;
  const KT kt(lane);
  const TT tt(lane);
  const ET et(lane);
  const int i = 16 * tile + r;  // this lane's token

  // block db of head h into a stage, the head's gates with its first block
  auto copy = [&](int h, int db, int st) {
    const int64_t vh = kh * a.rep + h, item = slot * a.hv + vh;
    const uint32_t to = lds0 + Sm::kStages + st * Sm::kStage;
    const int cols = min(a.dv - db * BB::kDB, BB::kDB);
    const int64_t at = (t0 * a.hv + vh) * (int64_t)a.dv + db * BB::kDB;
    // dO and dY: a tile of 4 (bf16) or 8 KB each, the first (and what bf16 leaves of dY) by waves 0-3, dY by 4-7
    const RowCopy<E, ET, kC, 4> co(tile, lane, o_stride, cols);
    co(rows_buffer(static_cast<const E*>(half ? b.dv : b.dout) + at, n, o_stride, cols),
       to + (half ? Sm::kDY : Sm::kDO), tile);
    if constexpr (Sm::kLow)
      if (!half) co(rows_buffer(static_cast<const E*>(b.dy_low) + at, n, o_stride, cols), to + Sm::kDYLow, tile);
    constexpr int kBlock = Sm::kBlock;
    copy_linear<BB::kEParts * BB::kE, 8>(
        a.e_img + item * e_bytes + (int64_t)db * BB::kEParts * BB::kE, to + Sm::kE, w, lane);
    copy_linear<kBlock, 8>(a.s_img + item * img_bytes + (int64_t)db * kBlock, to + Sm::kS, w, lane);
    copy_linear<kBlock, 8>(a.ds_img + item * img_bytes + (int64_t)db * kBlock, to + Sm::kDS, w, lane);
    if constexpr (Sm::kLow) {
      copy_linear<kBlock, 8>(a.ds_low + item * img_bytes + (int64_t)db * kBlock, to + Sm::kDSLow, w, lane);
      copy_linear<kBlock / 2, 8>(a.s_low + (item * img_bytes + (int64_t)db * kBlock) / 2, to + Sm::kSLow, w, lane);
    }
    if (db == 0)
      copy_linear<2048, 8>(a.ws + item * a.ws_item + CW::kGate, lds0 + Sm::kGate + (h & 1) * 2048, w, lane);
  };

  {
    const RowCopy<E, KT, kC, 8> ck(w, lane, a.k_stride, a.dk), cq(w, lane, a.q_stride, a.dk);
    ck(rows_buffer(static_cast<const E*>(a.k) + t0 * a.k_stride + (int64_t)kh * a.dk, n, a.k_stride,
                   a.dk), lds0 + Sm::kK, w);
    cq(rows_buffer(static_cast<const E*>(a.q) + t0 * a.q_stride + (int64_t)kh * a.dk, n, a.q_stride,
                   a.dk), lds0 + Sm::kQ, w);
    copy(0, 0, 0);
    copies_done();
  }
  // rows j (tiles up to this one), column i: k_j . q_i, or k_j . k_i
  f32x4 kx[4], dQ[kTiles], dK[kTiles];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) kx[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int m = 0; m < kTiles; ++m) dQ[m] = dK[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kb = 0; kb < DK / M::kDepth; ++kb) {
    const auto xi = kt.rows(sm + (half ? Sm::kK : Sm::kQ), tile, kb);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
      if (jt <= tile) kx[jt] = M::mma(kt.rows(sm + Sm::kK, jt, kb), xi, kx[jt]);
  }

  int st = 0;
  for (int h = 0; h < a.rep; ++h) {
    const int64_t vh = kh * a.rep + h, item = slot * a.hv + vh;
    float dot = 0.f;  // this thread's part of <dS', S>
    f32x4 mn[4], sdo[kTiles], sdy[kTiles], dse[kTiles];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) mn[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < kTiles; ++m) sdo[m] = sdy[m] = dse[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int db = 0; db < blocks; ++db) {
      const bool more = db + 1 < blocks || h + 1 < a.rep;
      const int nh = db + 1 < blocks ? h : h + 1, nb = db + 1 < blocks ? db + 1 : 0;
      if (h + db > 0) copies_done();
      if (Sm::kCount == 2 && more) copy(nh, nb, st ^ 1);
      const lds_ptr bl = sm + Sm::kStages + st * Sm::kStage;
      // <dS', S>, and what bf16 leaves of S from its bytes to operands
      for (int x = threadIdx.x; x < Sm::kBlock / 16; x += 512) {
        const auto s = lds_read<typename M::Frag>(bl + Sm::kS + 16 * x);
        const auto d = lds_read<typename M::Frag>(bl + Sm::kDS + 16 * x);
        if constexpr (Sm::kLow) {
          typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
          typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
          const u32x4 sw = __builtin_bit_cast(u32x4, s);
          const u32x2 lw = lds_read<u32x2>(bl + Sm::kSLow + 8 * x);
          const auto dl = lds_read<typename M::Frag>(bl + Sm::kDSLow + 16 * x);
          float sl[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint32_t high = y & 1 ? sw[y >> 1] & 0xffff0000u : sw[y >> 1] << 16;
            const float whole = with_low(high, lw[y >> 2], y & 3);
            dot = fmaf(whole, (float)d[y] + (float)dl[y], dot);
            sl[y] = whole - __uint_as_float(high);  // (7 bits and a sign: exact as bf16)
          }
          *reinterpret_cast<uint4*>(smem + Sm::kSLowTile + 16 * x) =
              make_uint4(pack_bf16(make_float2(sl[0], sl[1])), pack_bf16(make_float2(sl[2], sl[3])),
                         pack_bf16(make_float2(sl[4], sl[5])), pack_bf16(make_float2(sl[6], sl[7])));
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) dot = fmaf((float)s[y], (float)d[y], dot);
        }
      }
      if constexpr (Sm::kLow) lds_barrier();
#pragma unroll
      for (int kb = 0; kb < BB::kDB / M::kDepth; ++kb) {
        const auto of = et.rows(bl + Sm::kDO, tile, kb), yf = et.rows(bl + Sm::kDY, tile, kb);
        const auto xf = half ? yf : of;
        typename M::Frag ef[BB::kEParts];
#pragma unroll
        for (int p = 0; p < BB::kEParts; ++p) ef[p] = et.rows(bl + Sm::kE + p * BB::kE, tile, kb);
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
          if (jt <= tile)
#pragma unroll
            for (int p = 0; p < BB::kEParts; ++p)
              mn[jt] = M::mma(et.rows(bl + Sm::kE + p * BB::kE, jt, kb), xf, mn[jt]);
        typename M::Frag yl{};
        if constexpr (Sm::kLow) {
          yl = et.rows(bl + Sm::kDYLow, tile, kb);
          if (half)
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
              if (jt <= tile) mn[jt] = M::mma(et.rows(bl + Sm::kE, jt, kb), yl, mn[jt]);
        }
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const auto sf = kt.template cols<true>(bl + Sm::kS, m0 + m, kb);
          const auto df = kt.template cols<true>(bl + Sm::kDS, m0 + m, kb);
          sdo[m] = M::mma(sf, of, sdo[m]);
          sdy[m] = M::mma(sf, yf, sdy[m]);
#pragma unroll
          for (int p = 0; p < BB::kEParts; ++p) dse[m] = M::mma(df, ef[p], dse[m]);
          if constexpr (Sm::kLow) {
            dse[m] = M::mma(kt.template cols<true>(bl + Sm::kDSLow, m0 + m, kb), ef[0], dse[m]);
            const auto sl = kt.template cols<true>(sm + Sm::kSLowTile, m0 + m, kb);
            sdo[m] = M::mma(sl, of, sdo[m]);
            sdy[m] = M::mma(sl, yf, sdy[m]);
            sdy[m] = M::mma(sf, yl, sdy[m]);
          }
        }
      }
      if (Sm::kCount == 2) {
        st ^= 1;
      } else if (more) {
        __syncthreads();  // every wave has read the stage
        copy(nh, nb, 0);
      }
    }
    const lds_ptr gate = sm + Sm::kGate + (h & 1) * 2048, decay = gate + 1024;
    // B1 or B2, and the sums that reach dbeta and dg
    const int b1 = Sm::kBInStage ? Sm::kStages + (st ^ 1) * Sm::kStage : Sm::kOwnB;
    const int b2 = b1 + kBP * TT::kBytes;
    if (Sm::kBInStage) lds_barrier();  // every wave has read the last block
    {
      double row_x = 0.0;
      const float gi = lds_read<float>(decay + 4 * i), gil = lds_read<float>(decay + 4 * (kC + i));
      const float sign = half ? -1.f : a.scale;
      const int last = half ? i - 1 : i;  // j up to here
      double* sum_x = reinterpret_cast<double*>(smem + Sm::kSumX) + w * kC + 4 * g;
      float* sum_b = reinterpret_cast<float*>(smem + Sm::kSumB) + w * kC + 4 * g;
      f32x4 bx[4];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        const int j = 16 * jt + 4 * g;
        const f32x4 gj = lds_read<f32x4>(decay + 4 * j), gjl = lds_read<f32x4>(decay + 4 * (kC + j));
        const f32x4 bj = lds_read<f32x4>(decay + 4 * (2 * kC + j));
        f32x4 cx, cb;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool in = jt <= tile && j + x <= last;
          const float m = in ? sign * exp_f32((gi - gj[x]) + (gil - gjl[x])) * mn[jt][x] : 0.f;
          bx[jt][x] = m * bj[x];
          cb[x] = m * kx[jt][x];
          cx[x] = cb[x] * bj[x];
          row_x += (double)cx[x];
        }
        if (jt <= tile) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const double sx = group_sum((double)cx[x]);
            const float sb = group_sum(cb[x]);
            if (r == 0) {
              sum_x[16 * jt + x] = sx;
              sum_b[16 * jt + x] = sb;
            }
          }
        }
      }
      row_x = across_groups(row_x);
      if (g == 0) reinterpret_cast<double*>(smem + Sm::kRowX)[half * kC + i] = row_x;
#pragma unroll
      for (int kb = 0; kb < TT::kBlocks; ++kb)
        if (16 * tile >= kb * M::kDepth) {
          const auto f = M::template split<kBP>(&bx[kb * M::kTiles]);
#pragma unroll
          for (int p = 0; p < kBP; ++p)
            *reinterpret_cast<typename M::Frag*>(smem + (half ? b2 : b1) + p * TT::kBytes +
                                                 TT::word_at(kb, i, g)) = f.p[p];
        }
    }
    // the state's terms, and their dots with q_i and k_i (half of the values each half)
    {
      const float eg = lds_read<float>(gate + 4 * i), ci = lds_read<float>(gate + 4 * (kC + i));
      float rdot = 0.f, kd = 0.f;
#pragma unroll
      for (int kb = 0; kb < kTiles / M::kTiles; ++kb) {
        const auto ki = kt.rows(sm + Sm::kK, tile, m0 / M::kTiles + kb);
        const auto qi = kt.rows(sm + Sm::kQ, tile, m0 / M::kTiles + kb);
#pragma unroll
        for (int y = 0; y < M::kTiles; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int m = kb * M::kTiles + y;
            const float so = a.scale * eg * sdo[m][x], sy = -eg * sdy[m][x];
            rdot = fmaf((float)qi[4 * y + x], so, fmaf((float)ki[4 * y + x], sy, rdot));
            kd = fmaf((float)ki[4 * y + x], dse[m][x], kd);
            dQ[m][x] += so;
            dK[m][x] += fmaf(ci, dse[m][x], sy);
          }
      }
      rdot = across_groups(rdot);
      kd = across_groups(kd);
      float* tok = reinterpret_cast<float*>(smem + Sm::kTok);
      if (g == 0) {
        tok[half * kC + i] = rdot;
        tok[(2 + half) * kC + i] = kd;
      }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) dot += __shfl_xor(dot, m);
      if (lane == 0) reinterpret_cast<float*>(smem + Sm::kDot)[w] = dot;
    }
    lds_barrier();  // B1 and B2 are whole
    // sums over j (rows i of B1, B2), then over i (their columns)
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      if (16 * tile >= kb * M::kDepth) {
        typename M::Frag f1[kBP], f2[kBP];
#pragma unroll
        for (int p = 0; p < kBP; ++p) {
          f1[p] = tt.rows(sm + b1 + p * TT::kBytes, tile, kb);
          f2[p] = tt.rows(sm + b2 + p * TT::kBytes, tile, kb);
        }
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const auto kf = kt.cols(sm + Sm::kK, m0 + m, kb);
#pragma unroll
          for (int p = 0; p < kBP; ++p) {
            dQ[m] = M::mma(kf, f1[p], dQ[m]);
            dK[m] = M::mma(kf, f2[p], dK[m]);
          }
        }
      }
      if (16 * tile < (kb + 1) * M::kDepth) {
        typename M::Frag f1[kBP], f2[kBP];
#pragma unroll
        for (int p = 0; p < kBP; ++p) {
          f1[p] = tt.cols(sm + b1 + p * TT::kBytes, tile, kb);
          f2[p] = tt.cols(sm + b2 + p * TT::kBytes, tile, kb);
        }
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const auto qf = kt.cols(sm + Sm::kQ, m0 + m, kb), kf = kt.cols(sm + Sm::kK, m0 + m, kb);
#pragma unroll
          for (int p = 0; p < kBP; ++p) {
            dK[m] = M::mma(qf, f1[p], dK[m]);
            dK[m] = M::mma(kf, f2[p], dK[m]);
          }
        }
      }
    }
    if (w == 0) {
      const double* sum_x = reinterpret_cast<const double*>(smem + Sm::kSumX);
      const float* sum_b = reinterpret_cast<const float*>(smem + Sm::kSumB);
      const double* rows = reinterpret_cast<const double*>(smem + Sm::kRowX);
      const float* tok = reinterpret_cast<const float*>(smem + Sm::kTok);
      const float* gt = reinterpret_cast<const float*>(smem + Sm::kGate + (h & 1) * 2048);
      const float* dec = gt + 256;
      const float* dots = reinterpret_cast<const float*>(smem + Sm::kDot);
      const float kdt = tok[2 * kC + lane] + tok[3 * kC + lane];
      float all = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) all += dots[x];
      double cx = 0.0;
      float cb = 0.f;
      for (int x = lane >> 4; x < 8; x = x == 3 ? 4 + (lane >> 4) : x + 1) {
        cx += sum_x[x * kC + lane];
        cb += sum_b[x * kC + lane];
      }
      const float e = exp_f32((dec[kC - 1] - dec[lane]) + (dec[2 * kC - 1] - dec[kC + lane]));
      const float z = gt[kC + lane] * kdt;
      const float after = wave_suffix(tok[lane] + tok[kC + lane], lane) +
                          (float)wave_suffix((rows[lane] + rows[kC + lane]) - cx, lane);
      float before = z;  // sum of z over the tokens before
#pragma unroll
      for (int m = 1; m < 64; m *= 2) {
        const float t = __shfl_up(before, m);
        if (lane >= m) before += t;
      }
      before = __shfl_up(before, 1);
      const float whole = gt[2 * kC] * all;
      if (lane < n) {
        const int64_t at = (t0 + lane) * a.hv + vh;
        st_out(static_cast<E*>(b.dg), at, whole + (lane ? before : 0.f) + after);
        st_out(static_cast<E*>(b.dbeta), at, fmaf(e, kdt, cb));
      }
    }
  }
  if (i < n) {
    E* dqp = static_cast<E*>(b.dq) + ((t0 + i) * a.hk + kh) * (int64_t)a.dk;
    E* dkp = static_cast<E*>(b.dk) + ((t0 + i) * a.hk + kh) * (int64_t)a.dk;
#pragma unroll
    for (int m = 0; m < kTiles; m += M::kTiles) {
      const int v = KT::value(m0 + m, g, 0);
      if (v < a.dk) {
        store_values(dqp + v, &dQ[m]);
        store_values(dkp + v, &dK[m]);
      }
    }
  }
}

template <typename E, int DK, int NW>
int launch_passes_t(const BwdArgs& b, hipStream_t s) {
  const int cols = (b.f.dv + 16 * NW - 1) / (16 * NW);
  const uint32_t each = (uint32_t)(b.f.nseq * b.f.hv * cols);
  hipLaunchKernelGGL((passes_kernel<E, DK, NW>), dim3(2 * each), dim3(64 * NW), 0, s, b, cols, each);
  return launch_status();
}
template <typename E, int DK>
int launch_bwd(const BwdArgs& b, hipStream_t s) {
  // 64 or 128 columns per workgroup as in the forward (8 waves of fp32 operands would not fit the
  // registers)
  const bool narrow = sizeof(E) == 4 ||
                      narrow_pass(b.f.hv, 2 * b.f.nseq, !b.f.offsets || b.f.nseq == 1, b.f.dv);
  const int st = narrow ? launch_passes_t<E, DK, 4>(b, s)
                        : launch_passes_t<E, DK, sizeof(E) == 2 ? 8 : 4>(b, s);
  if (st != MAMBA_OK) return st;
  hipLaunchKernelGGL((grad_kernel<E, DK>), dim3((unsigned)(b.f.slots * b.f.hk)), dim3(512), 0, s, b);
  return launch_status();
}

struct BwdLayout {  // workspace regions in bytes
  size_t item, e, s, ds, s_low, ds_low, dy_low, total;
};
template <typename E>
BwdLayout layout_t(const mamba_delta_dims* d, bool packed) {
  const size_t items = (size_t)chunk_slots(d, packed) * (size_t)d->v_heads;
  const size_t blocks = (size_t)BwdBlock<E>::blocks(d->dv);
  const size_t row = (d->dk <= 64 ? 64 : 128) * sizeof(E);
  BwdLayout l;
  l.item = ChunkWs<E>::kBytes;
  l.e = items * l.item;
  l.s = l.e + items * blocks * BwdBlock<E>::kEParts * BwdBlock<E>::kE;
  l.ds = l.s + items * blocks * BwdBlock<E>::kDB * row;
  const size_t img = items * blocks * BwdBlock<E>::kDB * row, low = sizeof(E) == 2 ? img : 0;
  l.s_low = l.ds + img;
  l.ds_low = l.s_low + low / 2;
  l.dy_low = l.ds_low + low;
  l.total = l.dy_low;
  if (sizeof(E) == 2)
    l.total += (size_t)(packed ? d->seqlen : d->batch * d->seqlen) * (size_t)(d->v_heads * d->dv) * sizeof(E);
  return l;
}
BwdLayout layout(const mamba_delta_dims* d, bool packed) {
  return d->io_dtype == MAMBA_BF16 ? layout_t<uint16_t>(d, packed) : layout_t<float>(d, packed);
}

}  // namespace
}  // namespace delta
}  // namespace mamba

using namespace mamba;
using namespace mamba::delta;

extern "C" {

size_t mamba_delta_bwd_workspace_bytes(const mamba_delta_dims* dims, int packed) {
  if (check_delta(dims, packed != 0) != MAMBA_OK) return 0;
  return layout(dims, packed != 0).total;
}

int mamba_delta_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                    const float* initial_state, const int64_t* seq_offsets, float scale,
                    const void* dout, const float* dlast, void* dq, void* dk, void* dv, void* dg,
                    void* dbeta, float* dinitial_state, const mamba_delta_dims* dims,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const bool packed = seq_offsets != nullptr;
  int st = check_delta(dims, packed);
  if (st != MAMBA_OK) return st;
  if (!dout || !dq || !dk || !dv || !dg || !dbeta) return MAMBA_ERR_NULL;
  if ((st = check_delta_inputs(dims, q, k, v, g, beta, initial_state, seq_offsets)) != MAMBA_OK)
    return st;
  const size_t es = dims->io_dtype == MAMBA_BF16 ? 2 : 4;
  if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(dg, es) || !aligned(dbeta, es) || (dlast && !aligned(dlast, 16)) ||
      (dinitial_state && !aligned(dinitial_state, 16)))
    return MAMBA_ERR_ALIGN;
  const BwdLayout l = layout(dims, packed);
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  BwdArgs b = {};
  b.f = make_args(dims, scale, q, k, v, g, beta, initial_state, seq_offsets);
  b.f.ws = static_cast<char*>(workspace);
  b.f.e_img = b.f.ws + l.e;
  b.f.s_img = b.f.ws + l.s;
  b.f.ds_img = b.f.ws + l.ds;
  b.f.s_low = b.f.ws + l.s_low;
  b.f.ds_low = b.f.ws + l.ds_low;
  b.dy_low = b.f.ws + l.dy_low;
  b.dout = dout;
  b.dlast = dlast;
  b.dq = dq;
  b.dk = dk;
  b.dv = dv;
  b.dg = dg;
  b.dbeta = dbeta;
  b.ds0 = dinitial_state;
  const bool bf = dims->io_dtype == MAMBA_BF16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = launch_chunks(b.f, bf, s)) != MAMBA_OK) return st;
  if (bf) return b.f.dk <= 64 ? launch_bwd<uint16_t, 64>(b, s) : launch_bwd<uint16_t, 128>(b, s);
  return b.f.dk <= 64 ? launch_bwd<float, 64>(b, s) : launch_bwd<float, 128>(b, s);
}

}  // extern "C"
