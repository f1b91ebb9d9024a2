// mamba_linear_bwd.hip -- gradients of linear attention with a decay per head on gfx950.
//
// Over a unit of 128 tokens (fp32 storage: 64), with S the state before it, dS' the adjoint of the state after it,
// G_i the sum of its log decays up to token i, D_ij = exp(G_i - G_j) and c_j = exp(G_end - G_j):
//     B_ij = scale D_ij (dO_i . v_j)  (j <= i)
//     dQ_i = sum_j B_ij k_j + scale exp(G_i) S dO_i
//     dK_j = sum_i B_ij q_i + c_j dS' v_j
//     dg_t = sum_{i >= t > j} B_ij (q_i . k_j) + sum_{i >= t} R_i + sum_{j < t} Z_j + exp(G_end) <S, dS'>
//         R_i = scale exp(G_i) q_i . S dO_i,   Z_j = c_j k_j . dS' v_j
// Every term of dg_t is of pairs of tokens on both sides of t, so that nothing cancels: the gradient of a strong
// decay is as small as its pairs make it, and that of a reset is zero.
//
// Launches: linear_pass_kernel (mamba_linear.h) backwards leaves dV and the adjoints, forwards the states and <S, dS'>;
// linear_grad_kernel first dK and the part of dg that comes from keys, then dQ and dg, a workgroup per unit and key
// head, value heads added in accumulators in a fixed order.  Where units and key heads alone would leave CUs idle the
// value heads of a key head are split among workgroups, whose fp32 sums linear_fold_kernel adds in order.  No atomics.
//
// Measured (8 x 2048 tokens, 20 and 40 heads of 128, bf16): dK 259 us at 4.7 TB/s, dQ and dg 326 at 4.5, bound by memory:
// the states' images, 4 bytes a value, are a quarter of the bytes, V or dO comes in twice, as tiles and as a wave's own
// operands.  Both sides in one kernel, with 154 KB of LDS and so one workgroup per CU, took 739.  Images of units of
// 256 tokens would be half as large, for twice the pairs of tokens and tiles that do not fit two workgroups' LDS.
#include "mamba_linear.h"

namespace mamba {
namespace linear {
namespace {

struct GradArgs {
  Args f;            // q, k, v, offsets and sizes
  const float* gate;
  const void* dout;  // (tokens, hv, dv)
  const float* s_img;
  const float* ds_img;
  int64_t img_item;
  const float* dots; // (units, hv, dot_parts): parts of <S, dS'>
  int32_t dot_parts;
  float* dgz;        // (tokens, hv): what keys and <S, dS'> give dg
  void* dq;          // (tokens, hk, dk)
  void* dk;
  float* dg;         // (tokens, hv)
  float* part;       // (2, groups, tokens, hk, dk) where value heads are split
  int64_t tokens;
  int32_t groups;    // workgroups that share a key head's value heads
};

// Parts that stand for a state's value: with bf16 storage three, all of its 24 bits, for the sake of dg, which is
// fp32 and made of the same products as dQ and dK.
template <typename E>
constexpr int kImgParts = Mma<E>::parts(3);

// One of the two sides of a unit: dQ, of queries, dO and S, or dK, of keys, V and dS'.  LDS of a workgroup: the other
// side's keys or queries of the unit throughout; two stages of 32 columns of the other side's V or dO; 32 of the
// state's rows.  Two workgroups fit a CU, so that one's products hide the other's reads.
template <typename E, int DK>
struct GradSmem {
  static constexpr int kT = kUnit<E>;
  static constexpr int kNT = kT / 16;   // tiles of 16 tokens
  static constexpr int kNW = kT / 32;   // a wave has 32 tokens
  using KT = KeyTile<E, DK>;
  using BT = KeyTile<E, 32>;
  static constexpr int kX = 0;
  static constexpr int kA = kT * KT::kRow;
  static constexpr int kABytes = kT * BT::kRow;
  static constexpr int kState = 32 * KT::kRow;               // a part of 32 rows
  static constexpr int kS = kA + 2 * kABytes;
  static constexpr int kGate = kS + kImgParts<E> * kState;   // G as two floats, the tokens' factors (kT each), exp(G_end)
  static constexpr int kRed = kGate + (3 * kT + 4) * 4;      // pairs' sums of a tile's tokens: (kNT, kT)
  static constexpr int kTok = kRed + kNT * kT * 4;           // R or Z (kT)
  static constexpr int kBytes = kTok + kT * 4;
  static_assert(2 * kBytes <= 160 * 1024, "two workgroups per CU");
};

// A thread's share of 32 columns of a state's image: words of 16 bytes of an operand, on their way in registers.
template <typename E, int DK, int kThreads>
struct StateRows {
  static constexpr int kV = 16 / sizeof(E), kF = kV / 4, kItems = 32 * DK / kV;
  static constexpr int kN = (kItems + kThreads - 1) / kThreads;
  f32x4 v[kN][kF];
  __device__ __forceinline__ void load(const float* p) {
    const int thread = opaque(threadIdx.x);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = thread + i * kThreads;  // word at / 64 of the image's kF KBs each
#pragma unroll
      for (int x = 0; x < kF; ++x)
        v[i][x] = at < kItems ? *reinterpret_cast<const f32x4*>(p + (at / 64 * kF + x) * 256 + at % 64 * 4)
                              : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  // as parts to LDS, laid out like a tile of keys
  __device__ __forceinline__ void put(char* lds) const {
    using KT = KeyTile<E, DK>;
    constexpr int kPer = DK / 4 / kV;  // words of 64 lanes for 16 columns
    const int thread = opaque(threadIdx.x);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = thread + i * kThreads, lane = at % 64;
      const int row = at / 64 / kPer * 16 + (lane & 15), word = at / 64 % kPer * 4 + (lane >> 4);
      if (kItems % kThreads && at >= kItems) continue;
      const auto f = Mma<E>::template split<kImgParts<E>>(v[i]);
#pragma unroll
      for (int x = 0; x < kImgParts<E>; ++x)
        *reinterpret_cast<typename Mma<E>::Frag*>(lds + x * 32 * KT::kRow + row * KT::kRow + ((word ^ KT::key(row)) << 4)) =
            f.p[x];
    }
  }
};

// 16 bytes of a buffer, zeros past its end
template <typename F>
__device__ __forceinline__ F load_16(__amdgpu_buffer_rsrc_t buf, uint32_t offset) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(F, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(buf, (int)offset, 0, 0));
}
template <typename V>
__device__ __forceinline__ V across_groups(V v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// One side.  Per value head first the pairs of tokens (tiles of dO V^T, columns = a wave's own 32 tokens, which both sides make in
// their own orientation: no wave needs another's), then the state's terms.
template <typename E, int DK, bool kKeys>
__global__ __launch_bounds__((GradSmem<E, DK>::kNW * 64), sizeof(E) == 2 || DK == 64 ? 2 : 1) void linear_grad_kernel(GradArgs b, uint32_t blocks) {
  using M = Mma<E>;
  using Sm = GradSmem<E, DK>;
  using KT = typename Sm::KT;
  using BT = typename Sm::BT;
  constexpr int kT = Sm::kT, kNT = Sm::kNT, kNW = Sm::kNW, kTiles = DK / 16, kP = kImgParts<E>, kV = 16 / sizeof(E);
  constexpr int kDB = 32 / M::kDepth;  // depths of a block of columns
  __shared__ __align__(1024) char smem[Sm::kBytes];
  const Args& a = b.f;
  const uint32_t wg = wide_index();
  if (wg >= blocks) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // This wave's tiles of 16 tokens: one of each half, so that the waves have equally many pairs.  The first meets only
  // the other side's tiles of one half, from kFirst on, the second all.
  constexpr int kFirst = kKeys ? kNT / 2 : 0;
  const int tile_of[2] = {kKeys ? kNT - 1 - w : w, kKeys ? w : kNT - 1 - w};
  const uint32_t grp = wg % (uint32_t)b.groups, rest = wg / (uint32_t)b.groups;
  const int64_t slot = rest / (uint32_t)a.hk;
  const int kh = (int)(rest - slot * a.hk);
  const int64_t seq = slot_seq(a, slot, kT);
  const Span sp = seq_span(a, seq);
  const int64_t c0 = (slot - slot_base(a, seq, sp.first, kT)) * kT;
  if (c0 < 0 || c0 >= sp.len) return;  // an unused slot of a packed batch
  const int n = (int)min((int64_t)kT, sp.len - c0);
  const int64_t t0 = sp.first + c0;
  const int per = (a.rep + b.groups - 1) / b.groups;
  const int h0 = (int)grp * per, h1 = min(a.rep, h0 + per);

  const uint32_t lds0 = lds_address(smem);
  const lds_ptr sm = (lds_ptr)smem;
  const int64_t o_stride = (int64_t)a.hv * a.dv;
  // own: q and dO, or k and v; other: k and v, or q and dO
  const E* const q = static_cast<const E*>(a.q) + t0 * a.q_stride + (int64_t)kh * a.dk;
  const E* const k = static_cast<const E*>(a.k) + t0 * a.k_stride + (int64_t)kh * a.dk;
  const E* const v = static_cast<const E*>(a.v) + t0 * a.v_stride;
  const E* const o = static_cast<const E*>(b.dout) + t0 * o_stride;
  const E *const own_x = kKeys ? k : q, *const other_x = kKeys ? q : k, *const own_y = kKeys ? v : o,
          *const other_y = kKeys ? o : v;
  const int64_t own_xs = kKeys ? a.k_stride : a.q_stride, other_xs = kKeys ? a.q_stride : a.k_stride;
  const int64_t own_ys = kKeys ? a.v_stride : o_stride, other_ys = kKeys ? o_stride : a.v_stride;
  const RowCopy<E, KT, kT, kNW> cx(w, lane, other_xs, a.dk);
  cx(rows_buffer(other_x, n, other_xs, a.dk), lds0 + Sm::kX, w);
  const int dblocks = (a.dv + 31) / 32;
  // columns [32 db, ...) of the other side's V or dO of value head vh into a stage
  auto copy = [&](int vh, int db, int st) {
    const int cols = min(a.dv - 32 * db, 32);
    const RowCopy<E, BT, kT, kNW> cy(w, opaque(lane), other_ys, cols);
    cy(rows_buffer(other_y + (int64_t)vh * a.dv + 32 * db, n, other_ys, cols), lds0 + Sm::kA + st * Sm::kABytes, w);
  };
  // this wave's own tokens of dO or V as operands
  typename M::Frag own[2][kDB];
  auto fetch_own = [&](int vh, int db) {
    const auto buf = rows_resource(own_y + (int64_t)vh * a.dv, n, own_ys, a.dv);
    const int l = opaque(lane), g = l >> 4, r = l & 15;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int kb = 0; kb < kDB; ++kb) {
        const int col = 32 * db + kb * M::kDepth + g * kV;
        const uint32_t at = (uint32_t)((16 * tile_of[c] + r) * own_ys + col) * (uint32_t)sizeof(E);
        own[c][kb] = load_16<typename M::Frag>(buf, col < a.dv ? at : kOutside);
      }
  };
  // and of q or k
  typename M::Frag xs[2][DK / M::kDepth];
  auto fetch_x = [&]() {
    const auto buf = rows_resource(own_x, n, own_xs, a.dk);
    const int l = opaque(lane), g = l >> 4, r = l & 15;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) {
        const int col = kb * M::kDepth + g * kV;
        const uint32_t at = (uint32_t)((16 * tile_of[c] + r) * own_xs + col) * (uint32_t)sizeof(E);
        xs[c][kb] = load_16<typename M::Frag>(buf, col < a.dk ? at : kOutside);
      }
  };
  StateRows<E, DK, kNW * 64> rows;
  auto fetch_state = [&](int vh, int db) {
    rows.load((kKeys ? b.ds_img : b.s_img) + (slot * a.hv + vh) * b.img_item + (int64_t)db * 32 * DK);
  };
  float* const gate = reinterpret_cast<float*>(smem + Sm::kGate);
  float* const red = reinterpret_cast<float*>(smem + Sm::kRed);
  float* const tok = reinterpret_cast<float*>(smem + Sm::kTok);

  f32x4 X[2][kTiles];  // dQ or dK, transposed: rows = values, column = token
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int m = 0; m < kTiles; ++m) X[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  copy(kh * a.rep + h0, 0, 0);
  int st = 0;
  for (int h = h0; h < h1; ++h) {
    const int vh = kh * a.rep + h;
    fetch_own(vh, 0);
    if (!kKeys) fetch_x();
    // gates: wave 0, prefix sums in fp64, kept as two floats
    if (w == 0) {
      const int l = opaque(lane);
      double before = 0.0, G[kT / 64];
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        const int t = 64 * x + l;
        const float v = t < n ? clamp_gate(b.gate[(t0 + t) * a.hv + vh]) : 0.f;
        G[x] = before + prefix_sum((double)v);
        before = last_lane(G[x]);
      }
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        const int t = 64 * x + l;
        const float hi = (float)G[x];
        gate[t] = hi;
        gate[kT + t] = (float)(G[x] - (double)hi);
        gate[2 * kT + t] = kKeys ? exp_f32((float)(before - G[x])) : a.scale * exp_f32(hi);
      }
      if (lane == 0) gate[3 * kT] = exp_f32((float)before);
    }
    {
      // dO V^T: rows of tile t of the other side, columns = own tokens (tiles past the diagonal too: they cost less
      // than branches)
      f32x4 B0[kNT / 2], B1[kNT];
#pragma unroll
      for (int t = 0; t < kNT; ++t) B0[t / 2] = B1[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const BT bt(opaque(lane));
      for (int db = 0; db < dblocks; ++db) {
        copies_done();
        const lds_ptr sa = sm + Sm::kA + st * Sm::kABytes;
        typename M::Frag x[2][kDB];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int kb = 0; kb < kDB; ++kb) x[c][kb] = own[c][kb];
        fetch_own(vh, db + 1 < dblocks ? db + 1 : 0);  // (the last turn: for the state's terms)
        if (db + 1 < dblocks) copy(vh, db + 1, st ^ 1);
        else if (h + 1 < h1) copy(vh + 1, 0, st ^ 1);
#pragma unroll
        for (int kb = 0; kb < kDB; ++kb)
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            const auto f = bt.rows(sa, t, kb);
            if (t >= kFirst && t < kFirst + kNT / 2) B0[t - kFirst] = M::mma(f, x[0][kb], B0[t - kFirst]);
            B1[t] = M::mma(f, x[1][kb], B1[t]);
          }
        st ^= 1;
      }
      const KT kt(opaque(lane));
      // times scale D; on the queries' side the sums of q_i . k_t B for dg.  (The barriers keep the compiler from drawing
      // the tiles into each other: it spilled 168 registers.)
      auto weigh = [&](int tile, f32x4& Bt, int t, float hi, float lo) {
        if (kKeys ? t < tile : t > tile) {
          Bt = f32x4{0.f, 0.f, 0.f, 0.f};
          return;
        }
        const f32x4 rh = *reinterpret_cast<const f32x4*>(gate + 16 * t + 4 * g),
                    rl = *reinterpret_cast<const f32x4*>(gate + kT + 16 * t + 4 * g);
        const f32x4 e = (hi - rh) + (lo - rl);
#pragma unroll
        for (int x = 0; x < 4; ++x) Bt[x] *= a.scale * exp_f32(kKeys ? -e[x] : e[x]);
        if (t == tile)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (kKeys ? 4 * g + x < r : 4 * g + x > r) Bt[x] = 0.f;
      };
      // pairs of own token i and tokens of tile t: of a tile before i's the sums over i, at red[i's tile][t's tokens], and
      // `rows`, the sums over t; of i's own tile the sums over i >= t' > t for every t'
      auto sum_pairs = [&](int tile, f32x4 s, int t, float& rows) {
        f32x4 v = s;
        const float sum = (s[0] + s[1]) + (s[2] + s[3]);
        if (t < tile) {
          rows += sum;
        } else {
          const float up1 = __shfl_up(sum, 16), up2 = __shfl_up(sum, 32), up3 = __shfl_up(sum, 48);
          float before = (g > 0 ? up1 : 0.f) + (g > 1 ? up2 : 0.f) + (g > 2 ? up3 : 0.f);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            v[x] = 4 * g + x <= r ? before : 0.f;
            before += s[x];
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v[x] += dpp_row<0x128>(v[x]);
          v[x] += dpp_row<0x124>(v[x]);
          v[x] += dpp_row<0x122>(v[x]);
          v[x] += dpp_row<0x121>(v[x]);
        }
        if (r == 0) *reinterpret_cast<f32x4*>(red + tile * kT + 16 * t + 4 * g) = v;
      };
      float rows_sum[2] = {0.f, 0.f};
      {
        const int l = opaque(lane), i0 = 16 * tile_of[0] + (l & 15), i1 = 16 * tile_of[1] + (l & 15);
        const float hi0 = gate[i0], lo0 = gate[kT + i0], hi1 = gate[i1], lo1 = gate[kT + i1];
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          __builtin_amdgcn_sched_barrier(0);
          const bool two = t >= kFirst && t < kFirst + kNT / 2;
          f32x4 qk0 = {0.f, 0.f, 0.f, 0.f}, qk1 = qk0;
          if constexpr (!kKeys) {
            if (t <= tile_of[1]) {
#pragma unroll
              for (int kb = 0; kb < DK / M::kDepth; ++kb) {
                const auto f = kt.rows(sm + Sm::kX, t, kb);
                if (two) qk0 = M::mma(f, xs[0][kb], qk0);
                qk1 = M::mma(f, xs[1][kb], qk1);
              }
            }
          }
          if (two) weigh(tile_of[0], B0[t - kFirst], t, hi0, lo0);
          weigh(tile_of[1], B1[t], t, hi1, lo1);
          if constexpr (!kKeys) {
            if (two && t <= tile_of[0]) sum_pairs(tile_of[0], qk0 * B0[t - kFirst], t, rows_sum[0]);
            if (t <= tile_of[1]) sum_pairs(tile_of[1], qk1 * B1[t], t, rows_sum[1]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      fetch_state(vh, 0);
      // dQ += K^T B, or dK += Q^T B
#pragma unroll
      for (int kb = 0; kb < kT / M::kDepth; ++kb) {
        const int t = kb * M::kTiles;
        const bool two = t >= kFirst && t < kFirst + kNT / 2;
        if (kKeys ? t + M::kTiles <= tile_of[1] : t > tile_of[1]) continue;
        const auto f1 = M::template split<M::parts(2)>(&B1[t]);
        const auto f0 = M::template split<M::parts(2)>(&B0[two ? t - kFirst : 0]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const auto xc = kt.cols(sm + Sm::kX, m, kb);
#pragma unroll
          for (int x = 0; x < M::parts(2); ++x) {
            if (two) X[0][m] = M::mma(xc, f0.p[x], X[0][m]);
            X[1][m] = M::mma(xc, f1.p[x], X[1][m]);
          }
        }
      }
      if constexpr (!kKeys) {
        // of each own tile: the pairs with tokens before t as sums over the tokens before it; the own tile's with the
        // tokens of the tiles before
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int tile = tile_of[c];
          float* const to = red + tile * kT;
          float v = across_groups(rows_sum[c]);  // of token r
          v += dpp_or_zero<0x101, 0xf>(v);       // and those behind it
          v += dpp_or_zero<0x102, 0xf>(v);
          v += dpp_or_zero<0x104, 0xf>(v);
          v += dpp_or_zero<0x108, 0xf>(v);
          float before = 0.f;
#pragma unroll
          for (int x = 0; x < kT / 64; ++x) {
            const int t = 64 * x + lane;
            const float s = t < 16 * tile ? to[t] : 0.f;
            const float p = prefix_sum(s), q = __shfl_up(p, 1);
            if (t < 16 * tile) to[t] = before + (lane ? q : 0.f);
            before += __shfl(p, 63);
          }
          if (lane < 16) to[16 * tile + lane] += v;
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // the state's terms: S dO_i, or dS' v_j
    f32x4 s[2][kTiles];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int m = 0; m < kTiles; ++m) s[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const KT kt(opaque(lane));
    for (int db = 0; db < dblocks; ++db) {
      rows.put(smem + Sm::kS);
      typename M::Frag x[2][kDB];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int kb = 0; kb < kDB; ++kb) x[c][kb] = own[c][kb];
      __syncthreads();
      if (db + 1 < dblocks) {
        fetch_state(vh, db + 1);
        fetch_own(vh, db + 1);
      } else if (!kKeys) {
        fetch_x();
      }
#pragma unroll
      for (int kb = 0; kb < kDB; ++kb)
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            const auto f = kt.template cols<true>(sm + Sm::kS + p * Sm::kState, m, kb);
            s[0][m] = M::mma(f, x[0][kb], s[0][m]);
            s[1][m] = M::mma(f, x[1][kb], s[1][m]);
          }
      __syncthreads();  // the state's rows have been read
    }
    if (kKeys) fetch_x();  // (registers for it sooner would be spilled ones: 274 -> 300 us)
    // with their token's factor, and their dots with q_i or k_j
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      __builtin_amdgcn_sched_barrier(0);
      const int l = opaque(lane), i = 16 * tile_of[c] + (l & 15);
      const float f = gate[2 * kT + i];
      float sum = 0.f;
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb)
#pragma unroll
        for (int y = 0; y < M::kTiles; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float v = f * s[c][kb * M::kTiles + y][x];
            sum = fmaf((float)xs[c][kb][4 * y + x], v, sum);
            X[c][kb * M::kTiles + y][x] += v;
          }
      sum = across_groups(sum);
      if (l < 16) tok[i] = sum;
    }
    __syncthreads();
    if (w == 0) {
      const int l = opaque(lane);
      float sums[kT / 64], whole = 0.f;
      if constexpr (kKeys) {
        // <S, dS'> and the sums of Z before each token: 64 x + lane
        const float* d = b.dots + (slot * a.hv + vh) * b.dot_parts;
        float all = 0.f;
        for (int x = 0; x < b.dot_parts; ++x) all += d[x];
        whole = all * gate[3 * kT];
#pragma unroll
        for (int x = 0; x < kT / 64; ++x) {
          float sum = tok[64 * x + l];
#pragma unroll
          for (int m = 1; m < 64; m *= 2) {
            const float t = __shfl_up(sum, m);
            if (lane >= m) sum += t;
          }
          const float one = __shfl_up(sum, 1);
          sums[x] = whole + (lane ? one : 0.f);
          whole += __shfl(sum, 63);
        }
      } else {
        // the sums of R from each token on
#pragma unroll
        for (int x = kT / 64 - 1; x >= 0; --x) {
          float sum = tok[64 * x + l];
#pragma unroll
          for (int m = 1; m < 64; m *= 2) {
            const float t = __shfl_down(sum, m);
            if (lane + m < 64) sum += t;
          }
          sums[x] = whole + sum;
          whole += __shfl(sum, 0);
        }
      }
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        const int t = 64 * x + l;
        const int64_t at = (t0 + t) * a.hv + vh;
        if (t >= n) continue;
        if constexpr (kKeys) {
          b.dgz[at] = sums[x];
        } else {
          float pairs = 0.f;
          for (int y = t / 16; y < kNT; ++y) pairs += red[y * kT + t];
          b.dg[at] = (b.dgz[at] + sums[x]) + pairs;
        }
      }
    }
    __syncthreads();  // gates and sums have been read
  }
  E* const out = static_cast<E*>(kKeys ? b.dk : b.dq);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int i = 16 * tile_of[c] + r;
    if (i >= n) continue;
    const int64_t at = ((t0 + i) * a.hk + kh) * (int64_t)a.dk;
    if (b.groups > 1) {
      float* to = b.part + ((kKeys ? b.groups : 0) + (int64_t)grp) * (b.tokens * a.hk * (int64_t)a.dk) + at;
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
        if (KT::value(m, g, 0) < a.dk) *reinterpret_cast<f32x4*>(to + KT::value(m, g, 0)) = X[c][m];
      continue;
    }
#pragma unroll
    for (int m = 0; m < kTiles; m += M::kTiles) {
      const int v = KT::value(m, g, 0);
      if (v < a.dk) *reinterpret_cast<typename M::Frag*>(out + at + v) = M::pack(&X[c][m]);
    }
  }
}

// dq (y = 0) and dk (y = 1) of 64 tokens of a sequence, in pieces (z): the groups' sums in order
template <typename E>
__global__ __launch_bounds__(256) void linear_fold_kernel(GradArgs b) {
  const Args& a = b.f;
  const int64_t seq = slot_seq(a, blockIdx.x);
  const Span sp = seq_span(a, seq);
  const int64_t c0 = ((int64_t)blockIdx.x - slot_base(a, seq, sp.first)) * kC;
  if (c0 < 0 || c0 >= sp.len) return;
  const int64_t row = (int64_t)a.hk * a.dk, size = b.tokens * row;
  const int64_t first = (sp.first + c0) * row, count = min((int64_t)kC, sp.len - c0) * row;
  const float* part = b.part + (blockIdx.y ? (int64_t)b.groups * size : 0) + first;
  E* out = static_cast<E*>(blockIdx.y ? b.dk : b.dq) + first;
  for (int64_t x = (blockIdx.z * 256 + threadIdx.x) * 4; x < count; x += gridDim.z * 1024) {
    f32x4 s = *reinterpret_cast<const f32x4*>(part + x);
#pragma unroll 4
    for (int y = 1; y < b.groups; ++y) s += *reinterpret_cast<const f32x4*>(part + y * size + x);
    if constexpr (sizeof(E) == 2)
      *reinterpret_cast<uint2*>(out + x) = make_uint2(pack_bf16(make_float2(s[0], s[1])), pack_bf16(make_float2(s[2], s[3])));
    else
      *reinterpret_cast<f32x4*>(out + x) = s;
  }
}

struct BwdLayout {  // workspace regions in bytes
  SegLayout seg;
  size_t s, ds, dots, dgz, part, total;
  int64_t item, units;
  int32_t groups;
};
template <typename E>
BwdLayout layout_t(const mamba_delta_dims* d, bool packed) {
  BwdLayout l = {};
  l.seg = seg_layout(d, packed);
  l.units = slots_of(d, packed, kUnit<E>);
  l.item = image_size(d);
  const size_t img = (size_t)l.units * (size_t)d->v_heads * (size_t)l.item * sizeof(float);
  l.s = (l.seg.total + 1023) / 1024 * 1024;
  l.ds = l.s + img;
  l.dots = l.ds + img;
  const size_t tokens = (size_t)(packed ? d->seqlen : d->batch * d->seqlen);
  l.dgz = l.dots + ((size_t)l.units * (size_t)d->v_heads * (size_t)((d->dv + kCols - 1) / kCols) * kWaves4 * sizeof(float) +
                    255) / 256 * 256;
  l.part = l.dgz + (tokens * (size_t)d->v_heads * sizeof(float) + 255) / 256 * 256;
  // enough workgroups for one round of two per CU
  const int64_t rep = d->v_heads / d->qk_heads, wgs = l.units * d->qk_heads;
  l.groups = (int32_t)std::max<int64_t>(1, std::min<int64_t>(rep, 512 / std::max<int64_t>(wgs, 1)));
  const int64_t per = (rep + l.groups - 1) / l.groups;
  l.groups = (int32_t)((rep + per - 1) / per);  // (none without heads)
  l.total = l.part;
  if (l.groups > 1)
    l.total += 2 * (size_t)l.groups * tokens * (size_t)(d->qk_heads * d->dk) * sizeof(float);
  return l;
}
BwdLayout layout(const mamba_delta_dims* d, bool packed) {
  return d->io_dtype == MAMBA_BF16 ? layout_t<uint16_t>(d, packed) : layout_t<float>(d, packed);
}

template <typename E, int DK>
int launch_grad(const GradArgs& b, int64_t units, hipStream_t s) {
  using Sm = GradSmem<E, DK>;
  const uint32_t blocks = (uint32_t)(units * b.f.hk * b.groups);
  const dim3 grid = wide_grid(blocks, Sm::kNW * 64), threads(Sm::kNW * 64);
  hipLaunchKernelGGL((linear_grad_kernel<E, DK, true>), grid, threads, 0, s, b, blocks);
  const int st = launch_status();
  if (st != MAMBA_OK) return st;
  hipLaunchKernelGGL((linear_grad_kernel<E, DK, false>), grid, threads, 0, s, b, blocks);
  return launch_status();
}

template <typename E>
int launch_bwd(const PassArgs& fwd, const PassArgs& rev, const GradArgs& b, int64_t units, hipStream_t s) {
  constexpr bool bf = sizeof(E) == 2;
  int st = MAMBA_OK;
  if (rev.f.seg_chunks && (st = launch_segments(rev, bf, true, s)) != MAMBA_OK) return st;
  if ((st = launch_pass<E, kOutput | kImages | kReverse>(rev, s)) != MAMBA_OK) return st;
  if (fwd.f.seg_chunks && (st = launch_segments(fwd, bf, false, s)) != MAMBA_OK) return st;
  if ((st = launch_pass<E, kImages | kDots>(fwd, s)) != MAMBA_OK) return st;
  st = b.f.dk <= 64 ? launch_grad<E, 64>(b, units, s) : launch_grad<E, 128>(b, units, s);
  if (st != MAMBA_OK || b.groups == 1) return st;
  const int64_t pieces = std::min<int64_t>((kC * (int64_t)b.f.hk * b.f.dk + 4095) / 4096, 256);
  hipLaunchKernelGGL((linear_fold_kernel<E>), dim3((unsigned)b.f.slots, 2, (unsigned)pieces), dim3(256), 0, s, b);
  return launch_status();
}

}  // namespace
}  // namespace linear
}  // namespace mamba

using namespace mamba;
using namespace mamba::linear;

extern "C" {

size_t mamba_linear_attn_bwd_workspace_bytes(const mamba_delta_dims* dims, int packed) {
  if (check_delta(dims, packed != 0) != MAMBA_OK) return 0;
  return mamba::linear::layout(dims, packed != 0).total;
}

int mamba_linear_attn_bwd(const void* q, const void* k, const void* v, const float* g, const float* initial_state,
                          const int64_t* seq_offsets, float scale, const void* dout, const float* dlast, void* dq,
                          void* dk, void* dv, float* dg, float* dinitial_state, const mamba_delta_dims* dims,
                          void* workspace, size_t workspace_bytes, void* stream) {
  const bool packed = seq_offsets != nullptr;
  int st = check_delta(dims, packed);
  if (st != MAMBA_OK) return st;
  if (!dout || !dq || !dk || !dv || !dg) return MAMBA_ERR_NULL;
  if ((st = check_linear_inputs(dims, q, k, v, g, initial_state, seq_offsets)) != MAMBA_OK) return st;
  if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dg, 4) ||
      (dlast && !aligned(dlast, 16)) || (dinitial_state && !aligned(dinitial_state, 16)))
    return MAMBA_ERR_ALIGN;
  const BwdLayout l = mamba::linear::layout(dims, packed);
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  PassArgs fwd = {}, rev = {};
  fwd.f = make_args(dims, scale, q, k, v, g, nullptr, initial_state, seq_offsets);
  fwd.gate = g;
  fwd.img = reinterpret_cast<float*>(ws + l.s);
  fwd.img_item = l.item;
  set_segments(fwd, l.seg, ws);
  rev = fwd;
  rev.f.q = k;
  rev.f.k = q;
  rev.f.q_stride = fwd.f.k_stride;
  rev.f.k_stride = fwd.f.q_stride;
  rev.f.v = dout;
  rev.f.v_stride = dims->v_heads * dims->dv;
  rev.f.out = dv;
  rev.f.s0 = dlast;
  rev.f.last = dinitial_state;
  rev.img = reinterpret_cast<float*>(ws + l.ds);
  fwd.other = rev.img;
  fwd.dots = reinterpret_cast<float*>(ws + l.dots);
  GradArgs b = {};
  b.f = fwd.f;
  b.gate = g;
  b.dout = dout;
  b.s_img = fwd.img;
  b.ds_img = rev.img;
  b.img_item = l.item;
  b.dots = fwd.dots;
  b.dot_parts = (int32_t)((dims->dv + kCols - 1) / kCols) * kWaves4;
  b.dgz = reinterpret_cast<float*>(ws + l.dgz);
  b.dq = dq;
  b.dk = dk;
  b.dg = dg;
  b.part = reinterpret_cast<float*>(ws + l.part);
  b.tokens = packed ? dims->seqlen : dims->batch * dims->seqlen;
  b.groups = l.groups;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dims->io_dtype == MAMBA_BF16 ? launch_bwd<uint16_t>(fwd, rev, b, l.units, s)
                                      : launch_bwd<float>(fwd, rev, b, l.units, s);
}

}  // extern "C"
