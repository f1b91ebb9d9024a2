// mamba_window_bwd.hip -- gradients of attention with a sliding window and sinks on gfx950.
//
//     P_ij = exp(s_ij - lse_i),  D_i = sum_j P_ij (dO_i . v_j) = dO_i . out_i,  dS_ij = P_ij (dO_i . v_j - D_i)
//     dV_j = sum_i P_ij dO_i,   dK_j = scale sum_i dS_ij q_i,   dQ_i = scale sum_j dS_ij k_j
//
//   window_stat_kernel  fp32 storage: lse log2(e) and D = dO . out of every query and head, head by head
//   window_dq_kernel    as the forward, 128 queries (fp32 storage: 64) through their keys; with bf16 storage twice, first
//                       for D, which it leaves for the next kernel with lse log2(e)
//   window_dkv_kernel   64 keys (32) of one head, through the queries that see them, heads that share it one after
//                       another: sums in accumulators in a fixed order, no atomics
// The sinks are seen by every later query: the queries past the windows of a sinks' tile are cut into stretches,
// which window_dkv_kernel takes first, as workgroups of their own that leave fp32 sums; the tile's own workgroup, of
// a launch after that, adds them in order.  Without this one workgroup would go through a whole long sequence; where the
// sinks are many they are many workgroups, which do.
//
// The scores are made again in each kernel (with bf16 storage six products in the queries' pass and seven in the keys', ten
// in all without the second parts of P and dS, with fp32 storage eight, in place of five): dQ summed over the keys'
// workgroups would need atomics, whose order changes results, or a sum in memory per tile of keys.  And D from the rounded
// out would carry 2^-8 of dO . out into dS, which is the small difference of two numbers of that size where a few keys have
// all the weight (4 keys, scores of deviation 3.4: dq was off by 5.4e-3).
//
// lse is a number of fp32 and so is its product with log2(e): each is off by 2^-24 of itself, and the weights made from
// them by as many powers of e, up to 6e-5 of themselves at a score of 500.  The queries' pass therefore sums the weights
// and takes D as sum P (dO . v) / sum P: dO . v - D, which is small where a key has nearly all the weight, does not see
// their common factor.  With bf16 storage log2(sum P) goes into lse log2(e) (which leaves 2^-24 of that, far below the
// gradients' rounding); with fp32 storage dQ is divided by the sum, and the keys' pass, which sums the scores' products in
// the same order and so makes the same weights, reads its inverse as a third number.
// (Scores of 300 to 650, every query with one key, bf16: dq was off by 2.2e-6 of its terms, more at larger ones; fp32:
// dv by 7e-5 of its norm.)
//
// Rounding, bf16 storage: P and dS enter their products as two bf16 parts (2^-17 of each), so that the gradients' own
// rounding is the only one that shows, 1.66e-3 of the norm (one part of P: dV off by 2.3e-3; one of dS, whose rows sum to
// zero: dK and dQ by up to 1.48 times their rounding.  8 x 2048 tokens, 20 and 4 heads of 128: the second part of P costs
// 23 of 785 us, that of dS 103).  The rest is fp32.
#include <cstdint>

#include "mamba_window.h"

namespace mamba {
namespace window {
namespace {

template <typename E>
constexpr int kTilesW = sizeof(E) == 2 ? 2 : 1;  // 16-row tiles of a wave
template <typename E>
constexpr int kRows = 4 * 16 * kTilesW<E>;       // of a workgroup
constexpr int kPairs = 2;                        // pairs of waves that share the keys of a workgroup of the keys' pass
template <typename E>
constexpr int kKeyRows = kPairs * 16 * kTilesW<E>;
template <typename E>
constexpr int kStats = sizeof(E) == 2 ? 2 : 3;   // numbers of a query and head that the keys' pass reads
constexpr int kFar = 512;                        // queries of a stretch past the sinks' windows where there are few sinks
constexpr double kSinkWG = 96.0;                 // workgroups of sinks from which on there are no stretches
constexpr int64_t kFarBytes = (int64_t)256 << 20;  // sums of stretches: up to so much, or four times dk and dv in fp32

// 8 lanes per row; a row without a key has weights of zero: its log-sum counts as +infinity
template <typename E>
__global__ __launch_bounds__(256) void window_stat_kernel(WinArgs a, int64_t tokens) {
  const int64_t row = ((int64_t)wide_index() * 256 + threadIdx.x) / 8;  // head by head, token by token
  if (row >= tokens * a.hq) return;
  const int64_t h = row / tokens, t = row - h * tokens;
  const int64_t at = t * a.hq + h;
  const E* x = static_cast<const E*>(a.out) + at * a.dim;
  const E* y = static_cast<const E*>(a.dout) + at * a.dim;
  constexpr int kV = 16 / sizeof(E);
  typedef typename Mma<E>::Frag Frag;
  float s = 0.f;
  for (int c = (threadIdx.x & 7) * kV; c < a.dim; c += 8 * kV) {
    const Frag u = *reinterpret_cast<const Frag*>(x + c), v = *reinterpret_cast<const Frag*>(y + c);
#pragma unroll
    for (int i = 0; i < kV; ++i) s = fmaf((float)u[i], (float)v[i], s);
  }
  s += __shfl_xor(s, 1);
  s += __shfl_xor(s, 2);
  s += __shfl_xor(s, 4);
  if ((threadIdx.x & 7) == 0) {
    const float lse = a.lse[at];
    a.stat[row] = lse == kMinusInf ? -kMinusInf : lse * kLog2e;
    a.stat[tokens * a.hq + row] = s;
  }
}

// What a wave of the keys' pass makes: dV (from P), or dK (from P and dO V^T).  Two waves share 32 keys (fp32 storage:
// 16): with both sums in one wave there is room for one wave on a SIMD, which has nobody to hide its waits behind.
// (8 x 2048 tokens, 20 and 4 heads of 128, window 1024, dS in one part: 395 us; both sums in one wave and 128 keys per
// workgroup 491, by roles with 128 keys 503, as the longest workgroups then ran alone at the end; these on a GPU whose clocks
// had not risen.  Warm, with P and dS in two parts: 418, matrix unit 54% busy.)
enum Role { kMakeDv, kMakeDk };

// The queries' tiles of a workgroup of the keys' pass
struct KeyWork {
  int q_lo, q_hi;    // queries
  int t_lo, tiles;   // their tiles
  int count;         // tiles times heads, the heads one after another
  int shift;         // position of query 0
};

// A wave's share: 16 kC2 keys from jw0 on against the tiles of queries that come into the stages.
template <typename E, int DK, bool kFarPart, int kC2, Role kRole, typename Copy, typename Load, typename Put>
__device__ __forceinline__ void key_sums(const WinArgs& a, const KeyWork& k, const Mask& mask, char* smem,
                                         const float (&stats)[2][kStats<E>][kKeys], int jw0, float sc,
                                         const typename Mma<E>::Frag (&kf)[kC2][DK / Mma<E>::kDepth],
                                         const typename Mma<E>::Frag (&vf)[kC2][DK / Mma<E>::kDepth],
                                         f32x4 (&acc)[kC2][DK / 16], Copy copy, Load load_stat, Put put_stat) {
  using M = Mma<E>;
  using KT = KeyTile<E, DK>;
  constexpr int kStage = 2 * KT::kBytes;
  constexpr int kPer = kRole == kMakeDv ? 2 : 1;  // depths of a step of the scores
  constexpr bool kSplit = kRole == kMakeDv && sizeof(E) == 2;
  constexpr int kStepsK = DK / M::kDepth / kPer, kGroups = DK / 64, kStepsV = 32 / M::kDepth * kGroups;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const KT kt(lane);
  const int jw1 = jw0 + 16 * kC2 - 1;
  for (int i = 0; i < k.count; ++i) {
    const int st = i & 1, h = i / k.tiles, q0 = (k.t_lo + i - h * k.tiles) * kKeys;
    float3 next = make_float3(0.f, 0.f, 0.f);
    copies_done();
    if (i + 1 < k.count) {
      next = load_stat(i + 1);
      copy(i + 1, st ^ 1);
    }
    const lds_ptr sq = (lds_ptr)(smem + st * kStage), so = sq + KT::kBytes;
    const lds_ptr sums = kRole == kMakeDv ? so : sq;  // whose transpose the sums take
    const int p0 = q0 + k.shift;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int ph = p0 + 32 * half;
      if (mask.none(ph, ph + 31, jw0, jw1)) continue;
      const bool whole = !kFarPart && mask.all(ph, ph + 31, jw0, jw1) && q0 + 32 * half + 32 <= k.q_hi;
      // 32 queries: scores and dO V^T, rows = queries, column = key; then P or dS, as operands
      f32x4 s[kC2][2], e[kC2][2];
#pragma unroll
      for (int c = 0; c < kC2; ++c)
#pragma unroll
        for (int m = 0; m < 2; ++m) s[c][m] = e[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
      typename M::Frag f[2][4];
      auto read_k = [&](int i) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          f[i & 1][m] = kt.rows(sq, 2 * half + m, kPer * i);
          f[i & 1][2 + m] = kRole == kMakeDv ? kt.rows(sq, 2 * half + m, kPer * i + 1) : kt.rows(so, 2 * half + m, i);
        }
      };
      auto read_v = [&](int i) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          f[(i + kStepsK) & 1][x] = kt.cols(sums, i % kGroups * 4 + x, half * (32 / M::kDepth) + i / kGroups);
      };
      read_k(0);
#pragma unroll
      for (int kb = 0; kb < kStepsK; ++kb) {
        end_step();
        if (kb + 1 < kStepsK) read_k(kb + 1); else read_v(0);
        end_step();
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < kC2; ++c) {
            s[c][m] = M::mma(f[kb & 1][m], kf[c][kPer * kb], s[c][m]);
            if constexpr (kRole == kMakeDk) {
              e[c][m] = M::mma(f[kb & 1][2 + m], vf[c][kb], e[c][m]);
            } else {  // the other half of the scores (fp32 storage: in the order of the queries' pass)
              f32x4& to = kSplit ? e[c][m] : s[c][m];
              to = M::mma(f[kb & 1][2 + m], kf[c][kPer * kb + 1], to);
            }
          }
      }
      end_step();
      if (kStepsV > 1) read_v(1);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const f32x4 ls = *reinterpret_cast<const f32x4*>(&stats[st][0][32 * half + 16 * m + 4 * g]);
#pragma unroll
        for (int c = 0; c < kC2; ++c) {
          if (kSplit) s[c][m] += e[c][m];
#pragma unroll
          for (int x = 0; x < 4; ++x) s[c][m][x] = fast_exp2(fmaf(s[c][m][x], sc, -ls[x]));
          if constexpr (kStats<E> == 3)
            s[c][m] *= *reinterpret_cast<const f32x4*>(&stats[st][2][32 * half + 16 * m + 4 * g]);
        }
      }
      if (!whole)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < kC2; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int qi = q0 + 32 * half + 16 * m + 4 * g + x, j = jw0 + 16 * c + r;
              if (!(mask.sees(qi + k.shift, j) && qi < k.q_hi && (!kFarPart || qi >= k.q_lo))) s[c][m][x] = 0.f;
            }
      if constexpr (kRole == kMakeDk)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const f32x4 ds = *reinterpret_cast<const f32x4*>(&stats[st][1][32 * half + 16 * m + 4 * g]);
#pragma unroll
          for (int c = 0; c < kC2; ++c) s[c][m] = s[c][m] * (e[c][m] - ds);
        }
      constexpr int kP = M::parts(2);
      typename M::template Parts<kP> pf[kC2];
      f32x4 part[kTileSums<E> ? kC2 : 1][DK / 16];
      if constexpr (kTileSums<E>) clear(part);
#pragma unroll
      for (int i = 0; i < kStepsV; ++i) {
        if (i % kGroups == 0)
#pragma unroll
          for (int c = 0; c < kC2; ++c) pf[c] = M::template split<kP>(&s[c][i / kGroups * M::kTiles]);
        end_step();
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int c = 0; c < kC2; ++c) {
              f32x4& to = (kTileSums<E> ? part : acc)[c][i % kGroups * 4 + x];
              to = M::mma(f[(i + kStepsK) & 1][x], pf[c].p[p], to);
            }
        end_step();
        if (i + 2 < kStepsV) read_v(i + 2);
      }
      if constexpr (kTileSums<E>) add_to(acc, part);
      end_step();
    }
    if (i + 1 < k.count) put_stat(next, st ^ 1);
  }
}

// floats of dk or dv
__device__ __forceinline__ int64_t part_floats(const WinArgs& a) {
  return (a.kv_offsets ? 1 : a.nseq) * a.kv_len * (int64_t)a.hk * a.dim;
}

// kFarPart: 16 sinks and one query head over a stretch of queries past the sinks' windows; otherwise a tile of keys, the
// heads that share it one after another.  (Far part of 4 sinks and 8 x 2048 tokens: 27 us; with the sinks' tile as one
// workgroup's work it was 564.)
template <typename E, int DK, bool kFarPart>
__global__ __launch_bounds__(kFarPart ? 128 : 128 * kPairs, kFarPart ? 1 : sizeof(E) == 2 ? 2 : 1) void window_dkv_kernel(WinArgs a, uint32_t blocks, int64_t tokens) {
  using M = Mma<E>;
  using KT = KeyTile<E, DK>;
  constexpr int kP = kFarPart ? 1 : kPairs, kNW = 2 * kP, kC2 = kFarPart ? 1 : kTilesW<E>;
  constexpr int kN = kFarPart ? 16 : kKeyRows<E>, kStage = 2 * KT::kBytes;
  __shared__ __align__(1024) char smem[2 * kStage];
  __shared__ __align__(16) float stats[2][kStats<E>][kKeys];
  const uint32_t id = wide_index();
  if (id >= blocks) return;
  int64_t seq, tile, far_slot = 0, stretch = 0;
  int kh, h0, heads;
  if (kFarPart) {
    const uint32_t per = (uint32_t)(a.hq * a.sink_tiles);
    far_slot = id / per;
    const int rest = (int)(id - far_slot * per), h = rest / a.sink_tiles;
    tile = rest - h * a.sink_tiles;
    kh = h / a.rep;
    h0 = h - kh * a.rep;
    heads = 1;
    seq = tile_seq(a.q_offsets, a.seqlen, a.nseq, far_slot, a.far_len);
  } else {
    const uint32_t rest = id / (uint32_t)a.groups, per = (uint32_t)((a.rep + a.groups - 1) / a.groups);
    const int64_t slot = rest / (uint32_t)a.hk;
    kh = (int)(rest - slot * a.hk);
    h0 = (int)((id - rest * (uint32_t)a.groups) * per);
    heads = min((int)per, a.rep - h0);
    const Tile t = tile_of<false>(a.kv_offsets, a.kv_len, a.nseq, slot, kN);
    seq = t.seq;
    tile = t.tile;
  }
  const Seq qs = seq_of(a.q_offsets, a.seqlen, seq), ks = seq_of(a.kv_offsets, a.kv_len, seq);
  if (kFarPart) stretch = far_slot - tile_base(a.q_offsets, a.seqlen, seq, qs.first, a.far_len);
  if (tile < 0 || tile * kN >= ks.len || stretch < 0) return;
  const int j0 = (int)tile * kN, nk = min(ks.len - j0, kN);
  const Mask mask = mask_of(a);
  KeyWork k;
  k.shift = ks.len - qs.len;
  // Queries: those whose position is not before the tile's first key, up to the last that has a key of the tile in its
  // window; the queries behind those, which see only sinks, go by stretches.  (Both kinds of tile begin them with
  // the same query: that past the window of the last of the kKeyRows keys that the sinks lie in.)
  auto near = [&](int64_t t) {  // first query past the windows of the t-th kKeyRows keys
    const int64_t last = min((t + 1) * kKeyRows<E>, (int64_t)ks.len) - 1;
    return max(min(last + a.window - k.shift, (int64_t)qs.len), max(t * kKeyRows<E> - k.shift, (int64_t)0));
  };
  if (kFarPart) {
    const int64_t b = near(j0 / kKeyRows<E>) + stretch * a.far_len;
    k.q_lo = (int)min(b, (int64_t)qs.len);
    k.q_hi = (int)min(b + a.far_len, (int64_t)qs.len);
    if (k.q_lo >= k.q_hi) return;
  } else {
    k.q_lo = max(j0 - k.shift, 0);
    k.q_hi = a.sink_tiles || j0 >= mask.sinks ? (int)min(near(tile), (int64_t)qs.len) : qs.len;  // (no far part: all)
  }
  k.t_lo = k.q_lo / kKeys;
  k.tiles = k.q_hi > k.q_lo ? (k.q_hi - 1) / kKeys - k.t_lo + 1 : 0;
  k.count = k.tiles * heads;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w0 = 16 * kC2 * (w % kP);
  const bool makes_dk = w >= kP;

  const int64_t o_stride = (int64_t)a.hq * a.dim;
  const int hq0 = kh * a.rep + h0;
  const E* qp = static_cast<const E*>(a.q) + qs.first * a.q_stride + (int64_t)hq0 * a.dim;
  const E* op = static_cast<const E*>(a.dout) + qs.first * o_stride + (int64_t)hq0 * a.dim;
  const uint32_t lds0 = lds_address(smem);
  const RowCopy<E, KT, kKeys, kNW> cq(w, lane, a.q_stride, a.dim), co(w, lane, o_stride, a.dim);
  auto copy = [&](int i, int st) {
    const int h = i / k.tiles, t = (k.t_lo + i - h * k.tiles) * kKeys;
    const int64_t n = min(kKeys, qs.len - t);
    cq(rows_buffer(qp + t * a.q_stride + (int64_t)h * a.dim, n, a.q_stride, a.dim), lds0 + st * kStage, w);
    co(rows_buffer(op + t * o_stride + (int64_t)h * a.dim, n, o_stride, a.dim), lds0 + st * kStage + KT::kBytes, w);
  };
  // wave 0: the log-sums, the dots and the inverse sums; past the sequence +infinity and 0
  auto load_stat = [&](int i) {
    const int h = i / k.tiles, t = (k.t_lo + i - h * k.tiles) * kKeys + lane;
    const float* p = a.stat + (int64_t)(hq0 + h) * tokens + qs.first + t;
    return w == 0 && t < qs.len ? make_float3(p[0], p[tokens * a.hq], kStats<E> == 3 ? p[2 * tokens * a.hq] : 0.f)
                                : make_float3(-kMinusInf, 0.f, 0.f);
  };
  auto put_stat = [&](float3 v, int st) {
    if (w == 0) {
      stats[st][0][lane] = v.x;
      stats[st][1][lane] = v.y;
      if constexpr (kStats<E> == 3) stats[st][2][lane] = v.z;
    }
  };
  if (k.count) {
    copy(0, 0);
    put_stat(load_stat(0), 0);
  }
  typename M::Frag kf[kC2][DK / M::kDepth], vf[kC2][DK / M::kDepth];
  const E* kp = static_cast<const E*>(a.k) + (ks.first + j0) * a.k_stride + (int64_t)kh * a.dim;
  const E* vp = static_cast<const E*>(a.v) + (ks.first + j0) * a.v_stride + (int64_t)kh * a.dim;
  f32x4 acc[kC2][DK / 16];
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    load_rows<E, DK>(kp, a.k_stride, w0 + 16 * c + r, nk, a.dim, g, kf[c]);
    if (makes_dk) load_rows<E, DK>(vp, a.v_stride, w0 + 16 * c + r, nk, a.dim, g, vf[c]);
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) acc[c][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float sc = a.scale * kLog2e;
  loads_done();
  if (makes_dk)
    key_sums<E, DK, kFarPart, kC2, kMakeDk>(a, k, mask, smem, stats, j0 + w0, sc, kf, vf, acc, copy, load_stat, put_stat);
  else
    key_sums<E, DK, kFarPart, kC2, kMakeDv>(a, k, mask, smem, stats, j0 + w0, sc, kf, vf, acc, copy, load_stat, put_stat);
  // sums of a stretch: (far slot, query head, tile of 16 sinks, dk and dv, 16, dim)
  auto far_at = [&](int64_t slot, int h, int64_t t) {
    return a.far + (((slot * a.hq + h) * a.sink_tiles + t) * 32 + (makes_dk ? 0 : 16) + r) * (int64_t)a.dim;
  };
  if (kFarPart) {
    if (r < nk) {
      float* to = far_at(far_slot, hq0, tile);
#pragma unroll
      for (int d = 0; d < DK / 16; ++d) {
        const int v = KT::value(d, g, 0);
        if (v < a.dim) *reinterpret_cast<f32x4*>(to + v) = acc[0][d];
      }
    }
    return;
  }
  const int64_t first = near(tile), stretches = first < qs.len ? (qs.len - first + a.far_len - 1) / a.far_len : 0;
  const int64_t far_base = tile_base(a.q_offsets, a.seqlen, seq, qs.first, a.far_len);
  E* const out = static_cast<E*>(makes_dk ? a.dk : a.dv);
  const float scale = makes_dk ? a.scale : 1.f;
  const int64_t part_size = part_floats(a);
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    const int j = w0 + 16 * c + r;
    const int64_t t16 = (j0 + w0) / 16 + c;  // these 16 keys among the sinks' tiles
    if (t16 < a.sink_tiles && j < nk)
      for (int64_t x = 0; x < stretches; ++x)
        for (int h = 0; h < heads; ++h) {
          const float* from = far_at(far_base + x, hq0 + h, t16);
#pragma unroll
          for (int d = 0; d < DK / 16; ++d) {
            const int v = KT::value(d, g, 0);
            if (v < a.dim) acc[c][d] += *reinterpret_cast<const f32x4*>(from + v);
          }
        }
    if (j >= nk) continue;
    const int64_t at = ((ks.first + j0 + j) * a.hk + kh) * (int64_t)a.dim;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) acc[c][d] *= scale;
    if (a.groups > 1) {
      float* to = a.part + ((makes_dk ? a.groups : 0) + h0 / ((a.rep + a.groups - 1) / a.groups)) * part_size + at;
#pragma unroll
      for (int d = 0; d < DK / 16; ++d)
        if (KT::value(d, g, 0) < a.dim) *reinterpret_cast<f32x4*>(to + KT::value(d, g, 0)) = acc[c][d];
      continue;
    }
#pragma unroll
    for (int d = 0; d < DK / 16; d += M::kTiles) {
      const int v = KT::value(d, g, 0);
      if (v < a.dim) store_operand(out + at + v, &acc[c][d]);
    }
  }
}

// dv (y = 0) and dk (y = 1) where a key head's heads are split: the groups' sums in order, four values a thread.  Tokens
// that no sequence holds are left as they were.
template <typename E>
__global__ __launch_bounds__(256) void window_fold_kernel(WinArgs a) {
  const int64_t seq = tile_seq(a.kv_offsets, a.kv_len, a.nseq, blockIdx.x, kKeys);
  const Seq ks = seq_of(a.kv_offsets, a.kv_len, seq);
  const int64_t tile = blockIdx.x - tile_base(a.kv_offsets, a.kv_len, seq, ks.first, kKeys);
  if (tile < 0 || tile * kKeys >= ks.len) return;
  const int64_t row = (int64_t)a.hk * a.dim, size = part_floats(a);
  const int64_t first = (ks.first + tile * kKeys) * row, count = min((int64_t)kKeys, ks.len - tile * kKeys) * row;
  const float* from = a.part + blockIdx.y * a.groups * size + first;
  E* out = static_cast<E*>(blockIdx.y ? a.dk : a.dv) + first;
  for (int64_t x = (blockIdx.z * 256 + threadIdx.x) * 4; x < count; x += gridDim.z * 1024) {
    f32x4 s = *reinterpret_cast<const f32x4*>(from + x);
    for (int y = 1; y < a.groups; ++y) s += *reinterpret_cast<const f32x4*>(from + y * size + x);
    if constexpr (sizeof(E) == 2)
      *reinterpret_cast<uint2*>(out + x) = uint2{pack_bf16(make_float2(s[0], s[1])), pack_bf16(make_float2(s[2], s[3]))};
    else
      *reinterpret_cast<f32x4*>(out + x) = s;
  }
}

// 8 x 2048 tokens, 20 and 4 heads of 128, window 1024, bf16: 365 us for six products per pair of tiles (S and dO V^T
// twice, dS K in two parts; the exponentials are made twice too), matrix unit 51% busy.
template <typename E, int DK>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void window_dq_kernel(WinArgs a, uint32_t blocks,
                                                                                int64_t tokens) {
  using M = Mma<E>;
  using KT = KeyTile<E, DK>;
  constexpr int kC2 = kTilesW<E>, kQ = kRows<E>, kStage = 2 * KT::kBytes;
  __shared__ __align__(1024) char smem[2 * kStage];
  const uint32_t id = wide_index();
  if (id >= blocks) return;
  const int64_t wg = spread_index(id, blocks, a.rep);
  const int64_t slot = wg / a.hq;
  const int h = (int)(wg - slot * a.hq), kh = h / a.rep;
  const auto [seq, tile] = tile_of<true>(a.q_offsets, a.seqlen, a.nseq, slot, kQ);
  const Seq qs = seq_of(a.q_offsets, a.seqlen, seq), ks = seq_of(a.kv_offsets, a.kv_len, seq);
  if (tile < 0 || tile * kQ >= qs.len) return;
  const int q0 = (int)tile * kQ, nq = min(qs.len - q0, kQ);
  const int shift = ks.len - qs.len;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w0 = 16 * kC2 * w;
  const Mask mask = mask_of(a);
  const int p0 = q0 + shift, p1 = p0 + nq - 1;
  const int lo = (int)(max((int64_t)p0 - a.window + 1, (int64_t)0) / kKeys);
  const int sink_tiles = min((mask.sinks + (kKeys - 1ll)) / kKeys, (int64_t)lo);
  const int count = p1 < 0 ? 0 : sink_tiles + p1 / kKeys - lo + 1;
  auto tile_at = [&](int i) { return i < sink_tiles ? i : lo + i - sink_tiles; };
  const E* kp = static_cast<const E*>(a.k) + ks.first * a.k_stride + (int64_t)kh * a.dim;
  const E* vp = static_cast<const E*>(a.v) + ks.first * a.v_stride + (int64_t)kh * a.dim;
  const uint32_t lds0 = lds_address(smem);
  const RowCopy<E, KT, kKeys, 4> ck(w, lane, a.k_stride, a.dim), cv(w, lane, a.v_stride, a.dim);
  auto copy = [&](int t, int st) {
    const int64_t j = (int64_t)t * kKeys, n = min((int64_t)kKeys, ks.len - j);
    ck(rows_buffer(kp + j * a.k_stride, n, a.k_stride, a.dim), lds0 + st * kStage, w);
    cv(rows_buffer(vp + j * a.v_stride, n, a.v_stride, a.dim), lds0 + st * kStage + KT::kBytes, w);
  };
  if (count) copy(tile_at(0), 0);
  typename M::Frag qf[kC2][DK / M::kDepth], of[kC2][DK / M::kDepth];
  const int64_t o_stride = (int64_t)a.hq * a.dim;
  const E* qp = static_cast<const E*>(a.q) + (qs.first + q0) * a.q_stride + (int64_t)h * a.dim;
  const E* op = static_cast<const E*>(a.dout) + (qs.first + q0) * o_stride + (int64_t)h * a.dim;
  constexpr bool kTwice = sizeof(E) == 2;
  float ls[kC2], ds[kC2], sums[kC2];  // sums of P: see the head of this file
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    const int i = w0 + 16 * c + r;
    sums[c] = 0.f;
    load_rows<E, DK>(qp, a.q_stride, i, nq, a.dim, g, qf[c]);
    load_rows<E, DK>(op, o_stride, i, nq, a.dim, g, of[c]);
    const int64_t at = (int64_t)h * tokens + qs.first + q0 + i;
    ls[c] = -kMinusInf;
    ds[c] = 0.f;
    if (i < nq && !kTwice) {
      ls[c] = a.stat[at];
      ds[c] = a.stat[tokens * a.hq + at];
    }
    if (i < nq && kTwice) {
      const float lse = a.lse[(qs.first + q0 + i) * a.hq + h];
      ls[c] = lse == kMinusInf ? -kMinusInf : lse * kLog2e;
    }
  }
  const float sc = a.scale * kLog2e;
  f32x4 dq[kC2][DK / 16];
#pragma unroll
  for (int c = 0; c < kC2; ++c)
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) dq[c][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  const KT kt(lane);
  const int pw0 = p0 + w0, pw1 = pw0 + 16 * kC2 - 1;
  constexpr int kStepsK = DK / M::kDepth, kGroups = DK / 64, kStepsV = 32 / M::kDepth * kGroups;
  typename M::Frag f[2][4];
  auto read_cols = [&](lds_ptr sk, int half, int i) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      f[i & 1][x] = kt.cols(sk, i % kGroups * 4 + x, half * (32 / M::kDepth) + i / kGroups);
  };
  // 32 keys of the stage at sk: P and dO V^T, rows = keys, column = query; `then` reads what the products after them
  // take first
  auto scores = [&](lds_ptr sk, int j0, int half, f32x4 (&s)[kC2][2], f32x4 (&e)[kC2][2], auto then,
                    auto behind) {
    const lds_ptr sv = sk + KT::kBytes;
    const int jh = j0 + 32 * half;
#pragma unroll
    for (int c = 0; c < kC2; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m) s[c][m] = e[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto read = [&](int kb) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f[kb & 1][m] = kt.rows(sk, 2 * half + m, kb);
        f[kb & 1][2 + m] = kt.rows(sv, 2 * half + m, kb);
      }
    };
    read(0);
#pragma unroll
    for (int kb = 0; kb < kStepsK; ++kb) {
      end_step();
      if (kb + 1 < kStepsK) read(kb + 1); else then();
      end_step();
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < kC2; ++c) {
          s[c][m] = M::mma(f[kb & 1][m], qf[c][kb], s[c][m]);
          e[c][m] = M::mma(f[kb & 1][2 + m], of[c][kb], e[c][m]);
        }
    }
    end_step();
    behind();
#pragma unroll
    for (int c = 0; c < kC2; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[c][m][x] = fast_exp2(fmaf(s[c][m][x], sc, -ls[c]));
    if (!mask.all(pw0, pw1, jh, jh + 31))
#pragma unroll
      for (int c = 0; c < kC2; ++c)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (!mask.sees(pw0 + 16 * c + r, jh + 16 * m + 4 * g + x)) s[c][m][x] = 0.f;
  };
  auto add_sums = [&](const f32x4 (&s)[kC2][2]) {
#pragma unroll
    for (int c = 0; c < kC2; ++c) {
      const f32x4 t = s[c][0] + s[c][1];
      sums[c] += (t[0] + t[1]) + (t[2] + t[3]);
    }
  };
  int turn = 0;  // stages
  loads_done();
  if constexpr (kTwice) {
    for (int i = 0; i < count; ++i, ++turn) {
      const int st = turn & 1, j0 = tile_at(i) * kKeys;
      copies_done();
      copy(tile_at(i + 1 < count ? i + 1 : 0), st ^ 1);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (mask.none(pw0, pw1, j0 + 32 * half, j0 + 32 * half + 31)) continue;
        f32x4 s[kC2][2], e[kC2][2];
        scores((lds_ptr)(smem + st * kStage), j0, half, s, e, [] {}, [] {});
        add_sums(s);
#pragma unroll
        for (int c = 0; c < kC2; ++c)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int x = 0; x < 4; ++x) ds[c] = fmaf(s[c][m][x], e[c][m][x], ds[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < kC2; ++c) {
      const float sum = across_groups(sums[c]);
      ds[c] = across_groups(ds[c]);
      if (sum != 0.f) {
        ds[c] /= sum;
        ls[c] += __builtin_amdgcn_logf(sum);
      }
      const int i = w0 + 16 * c + r;
      const int64_t at = (int64_t)h * tokens + qs.first + q0 + i;
      if (g == 0 && i < nq) {
        a.stat[at] = ls[c];
        a.stat[tokens * a.hq + at] = ds[c];
      }
    }
  }
  for (int i = 0; i < count; ++i, ++turn) {
    const int st = turn & 1, j0 = tile_at(i) * kKeys;
    copies_done();
    if (i + 1 < count) copy(tile_at(i + 1), st ^ 1);
    const lds_ptr sk = (lds_ptr)(smem + st * kStage);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (mask.none(pw0, pw1, j0 + 32 * half, j0 + 32 * half + 31)) continue;
      f32x4 s[kC2][2], e[kC2][2];
      scores(sk, j0, half, s, e, [&] { read_cols(sk, half, 0); }, [&] { if (kStepsV > 1) read_cols(sk, half, 1); });
      if constexpr (!kTwice) add_sums(s);
#pragma unroll
      for (int c = 0; c < kC2; ++c)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          e[c][m] = s[c][m] * (e[c][m] - ds[c]);
      constexpr int kP = M::parts(2);
      typename M::template Parts<kP> ef[kC2];
      f32x4 part[kTileSums<E> ? kC2 : 1][DK / 16];
      if constexpr (kTileSums<E>) clear(part);
#pragma unroll
      for (int i = 0; i < kStepsV; ++i) {
        if (i % kGroups == 0)
#pragma unroll
          for (int c = 0; c < kC2; ++c) ef[c] = M::template split<kP>(&e[c][i / kGroups * M::kTiles]);
        end_step();
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int c = 0; c < kC2; ++c) {
              f32x4& to = (kTileSums<E> ? part : dq)[c][i % kGroups * 4 + x];
              to = M::mma(f[i & 1][x], ef[c].p[p], to);
            }
        end_step();
        if (i + 2 < kStepsV) read_cols(sk, half, i + 2);
      }
      if constexpr (kTileSums<E>) add_to(dq, part);
      end_step();
    }
  }
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    const int i = w0 + 16 * c + r;
    float f = a.scale;
    if constexpr (!kTwice) {
      const float sum = across_groups(sums[c]), inv = sum == 0.f ? 0.f : 1.f / sum;
      f *= inv;
      if (g == 0 && i < nq) a.stat[2 * tokens * a.hq + (int64_t)h * tokens + qs.first + q0 + i] = inv;
    }
    if (i >= nq) continue;
    E* to = static_cast<E*>(a.dq) + ((qs.first + q0 + i) * a.hq + h) * (int64_t)a.dim;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) dq[c][d] *= f;
#pragma unroll
    for (int d = 0; d < DK / 16; d += M::kTiles)
      if (KT::value(d, g, 0) < a.dim) store_operand(to + KT::value(d, g, 0), &dq[c][d]);
  }
}

struct BwdLayout {  // workspace regions in bytes
  size_t far, part, total;
  int64_t far_slots, tokens;
  int32_t sink_tiles, far_len, groups;
};
BwdLayout layout(const mamba_window_dims* d, bool packed) {
  BwdLayout l = {};
  l.far_len = kFar;
  l.groups = 1;
  l.tokens = packed ? d->seqlen : d->batch * d->seqlen;
  const size_t stats = d->io_dtype == MAMBA_BF16 ? kStats<uint16_t> : kStats<float>;
  l.far = ((size_t)l.tokens * (size_t)d->q_heads * stats * sizeof(float) + 255) / 256 * 256;
  l.total = l.far;
  // (queries times sinks for which inputs alone are past any memory are said to take a workspace that is)
  if (d->window < d->kv_len && (double)l.tokens * (double)(d->q_heads * d->dim) * (double)std::min(d->sinks, d->kv_len) > 6.4e19) {
    l.total = SIZE_MAX;
    return l;
  }
  // Many sinks are many workgroups by themselves, which go through all their queries (1 x 16384 tokens, 20 and 4 heads of
  // 128, window 1024, bf16, by stretches and so: 1024 sinks, 64 workgroups, 2.80 and 3.51 ms; 2048, 128 of them, 4.28 and
  // 3.87; 4096 6.98 and 4.53; 12 and 12 heads, 512 sinks, 96, 1.26 and 1.06).  Packed: those of one sequence count.
  const int64_t rows = d->io_dtype == MAMBA_BF16 ? kKeyRows<uint16_t> : kKeyRows<float>;
  const double sink_wgs = (packed ? 1.0 : (double)d->batch) * (double)d->kv_heads * (double)((d->sinks + rows - 1) / rows);
  // (as many sinks, or a window of as many tokens, as there are keys: every earlier key is seen, no query is far)
  if (d->sinks && d->window < d->kv_len && d->sinks < d->kv_len && sink_wgs < kSinkWG) {
    l.sink_tiles = (int32_t)((d->sinks + 15) / 16);
    // shorter stretches where they would leave CUs idle (2 x 333 tokens, 12 heads of 64, fp32: 22 -> 13 us)
    auto slots = [&] { return tile_slots(d->seqlen, d->batch, packed, l.far_len); };
    while (l.far_len > kKeys && (double)slots() * (double)d->q_heads * (double)l.sink_tiles < 256.0) l.far_len /= 2;
    // longer ones where the sums would grow with queries times sinks, none where one for each sequence is too much
    auto bytes = [&] { return (double)slots() * (double)d->q_heads * (double)l.sink_tiles * 128.0 * (double)d->dim; };
    const double most = std::max((double)kFarBytes, 32.0 * (packed ? 1.0 : (double)d->batch) * (double)d->kv_len *
                                                        (double)(d->kv_heads * d->dim));
    while (bytes() > most && l.far_len < d->seqlen && l.far_len < 1 << 30) l.far_len *= 2;
    if (bytes() > most) {
      l.sink_tiles = 0;
    } else {
      l.far_slots = slots();
      l.total += (size_t)l.far_slots * (size_t)d->q_heads * (size_t)l.sink_tiles * 32 * (size_t)d->dim * sizeof(float);
    }
  }
  // A key head's heads go to several workgroups where tiles of keys alone leave CUs idle and that shortens the longest
  // chain by four tiles, which the sum of the parts costs (the same case: 42 -> 24 us and 5 for the sum).
  const int64_t rep = d->q_heads / d->kv_heads, keys = d->io_dtype == MAMBA_BF16 ? kKeyRows<uint16_t> : kKeyRows<float>;
  const int64_t wgs = tile_slots(d->kv_len, d->batch, packed, (int)keys) * d->kv_heads;
  const int64_t groups = std::min<int64_t>(rep, 512 / std::max<int64_t>(wgs, 1));
  const int64_t chain = (std::min(d->window + keys, d->seqlen) + kKeys - 1) / kKeys;
  if (groups > 1) {
    const int64_t per = (rep + groups - 1) / groups;
    if ((rep - per) * chain >= 4) l.groups = (int32_t)((rep + per - 1) / per);
  }
  l.part = (l.total + 255) / 256 * 256;
  if (l.groups > 1)
    l.total = l.part + 2 * (size_t)l.groups * (size_t)(packed ? 1 : d->batch) * (size_t)d->kv_len *
                           (size_t)(d->kv_heads * d->dim) * sizeof(float);
  return l;
}

template <typename E, int DK>
int launch_bwd(const WinArgs& a, int64_t tokens, hipStream_t s) {
  const bool packed = a.q_offsets != nullptr;
  int st = MAMBA_OK;
  if constexpr (sizeof(E) == 4) {
    const int64_t rows = tokens * a.hq;
    hipLaunchKernelGGL((window_stat_kernel<E>), wide_grid((uint64_t)((rows + 31) / 32), 256), dim3(256), 0, s, a, tokens);
    if ((st = launch_status()) != MAMBA_OK) return st;
  }
  const uint32_t queries = (uint32_t)(tile_slots(a.seqlen, a.nseq, packed, kRows<E>) * a.hq);
  hipLaunchKernelGGL((window_dq_kernel<E, DK>), wide_grid(queries, 256), dim3(256), 0, s, a, queries, tokens);
  if ((st = launch_status()) != MAMBA_OK) return st;
  if (a.sink_tiles) {
    const uint32_t blocks = (uint32_t)(a.far_slots * a.hq * a.sink_tiles);
    hipLaunchKernelGGL((window_dkv_kernel<E, DK, true>), wide_grid(blocks, 128), dim3(128), 0, s, a, blocks, tokens);
    if ((st = launch_status()) != MAMBA_OK) return st;
  }
  const uint32_t keys = (uint32_t)(tile_slots(a.kv_len, a.nseq, packed, kKeyRows<E>) * a.hk * a.groups);
  hipLaunchKernelGGL((window_dkv_kernel<E, DK, false>), wide_grid(keys, 128 * kPairs), dim3(128 * kPairs), 0, s, a, keys, tokens);
  if ((st = launch_status()) != MAMBA_OK || a.groups == 1) return st;
  const int64_t pieces = std::min<int64_t>((kKeys * (int64_t)a.hk * a.dim + 4095) / 4096, 256);
  hipLaunchKernelGGL((window_fold_kernel<E>), dim3((unsigned)tile_slots(a.kv_len, a.nseq, packed, kKeys), 2, (unsigned)pieces),
                     dim3(256), 0, s, a);
  return launch_status();
}

}  // namespace
}  // namespace window
}  // namespace mamba

using namespace mamba;
using namespace mamba::window;

extern "C" {

size_t mamba_window_attn_bwd_workspace_bytes(const mamba_window_dims* dims, int packed) {
  if (check_window(dims, packed != 0) != MAMBA_OK) return 0;
  return layout(dims, packed != 0).total;
}

int mamba_window_attn_bwd(const void* q, const void* k, const void* v, const int64_t* q_offsets,
                          const int64_t* kv_offsets, float scale, const void* out, const float* lse, const void* dout,
                          void* dq, void* dk, void* dv, const mamba_window_dims* dims, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const bool packed = q_offsets != nullptr;
  int st = check_window(dims, packed);
  if (st != MAMBA_OK) return st;
  if (!out || !lse || !dout || !dq || !dk || !dv) return MAMBA_ERR_NULL;
  if ((st = check_window_inputs(q, k, v, q_offsets, kv_offsets)) != MAMBA_OK) return st;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dv, 16))
    return MAMBA_ERR_ALIGN;
  const BwdLayout l = layout(dims, packed);
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGN;
  WinArgs a = window_args(dims, scale, q, k, v, q_offsets, kv_offsets);
  a.out = const_cast<void*>(out);
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.stat = static_cast<float*>(workspace);
  a.far = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.far);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.part);
  a.far_slots = l.far_slots;
  a.far_len = l.far_len;
  a.groups = l.groups;
  a.sink_tiles = l.sink_tiles;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dims->io_dtype == MAMBA_BF16)
    return a.dim <= 64 ? launch_bwd<uint16_t, 64>(a, l.tokens, s) : launch_bwd<uint16_t, 128>(a, l.tokens, s);
  return a.dim <= 64 ? launch_bwd<float, 64>(a, l.tokens, s) : launch_bwd<float, 128>(a, l.tokens, s);
}

}  // extern "C"
