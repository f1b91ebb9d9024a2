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
// Launches: linear_pass_kernel (mamba_linear.h) forwards leaves the states, backwards dV and the adjoints;
// linear_grad_kernel the rest, a workgroup per unit and key head, value heads added in accumulators in a fixed
// order.  Where units and key heads alone would leave CUs idle the value heads of a key head are split among
// workgroups, whose fp32 sums linear_fold_kernel adds in order.  No atomics.
#include "mamba_linear.h"

namespace mamba {
namespace linear {
namespace {

struct GradArgs {
  Args f;            // q, k, v, offsets and sizes
  const float* gate;
  const void* dout;  // (tokens, hv, dv)
  const char* s_img;
  const char* ds_img;
  int64_t img_item;
  void* dq;          // (tokens, hk, dk)
  void* dk;
  float* dg;         // (tokens, hv)
  float* part;       // (2, groups, tokens, hk, dk) where value heads are split
  int64_t tokens;
  int32_t groups;    // workgroups that share a key head's value heads
};

// LDS of a workgroup: Q and K of the unit throughout; two stages of 32 columns of V and dO with the state's rows of
// them; one of the adjoint's.
template <typename E, int DK>
struct GradSmem {
  static constexpr int kT = kUnit<E>;
  static constexpr int kNW = kT / 16;  // a wave has 16 tokens
  using KT = KeyTile<E, DK>;
  using BT = KeyTile<E, 32>;
  static constexpr int kQ = 0;
  static constexpr int kK = kT * KT::kRow;
  static constexpr int kA = 2 * kT * KT::kRow;
  static constexpr int kV = 0, kO = kT * BT::kRow, kS = 2 * kT * BT::kRow;  // inside a stage
  static constexpr int kState = 32 * KT::kRow;                             // a part of 32 rows
  static constexpr int kABytes = kS + kImgParts<E> * kState;
  static constexpr int kDS = kA + 2 * kABytes;
  static constexpr int kGate = kDS + kImgParts<E> * kState;  // G as two floats, eg, c (kT each), exp(G_end)
  static constexpr int kRed = kGate + (4 * kT + 4) * 4;      // pairs' sums of a wave's tokens: (kNW, kT)
  static constexpr int kTok = kRed + kNW * kT * 4;           // R, Z (kT each)
  static constexpr int kDot = kTok + 2 * kT * 4;             // a wave's part of <S, dS'>
  static constexpr int kBytes = kDot + 2 * kNW * 4;
  static_assert(kBytes <= 160 * 1024, "LDS");
};

template <typename V>
__device__ __forceinline__ V across_groups(V v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <typename E, int DK>
__global__ __launch_bounds__((GradSmem<E, DK>::kNW * 64)) void linear_grad_kernel(GradArgs b, uint32_t blocks) {
  using M = Mma<E>;
  using Sm = GradSmem<E, DK>;
  using KT = typename Sm::KT;
  using BT = typename Sm::BT;
  constexpr int kT = Sm::kT, kNW = Sm::kNW, kTiles = DK / 16, kP = kImgParts<E>;
  __shared__ __align__(1024) char smem[Sm::kBytes];
  const Args& a = b.f;
  const uint32_t wg = wide_index();
  if (wg >= blocks) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  {
    const RowCopy<E, KT, kT, kNW> cq(w, lane, a.q_stride, a.dk), ck(w, lane, a.k_stride, a.dk);
    cq(rows_buffer(static_cast<const E*>(a.q) + t0 * a.q_stride + (int64_t)kh * a.dk, n, a.q_stride, a.dk),
       lds0 + Sm::kQ, w);
    ck(rows_buffer(static_cast<const E*>(a.k) + t0 * a.k_stride + (int64_t)kh * a.dk, n, a.k_stride, a.dk),
       lds0 + Sm::kK, w);
  }
  const int dblocks = (a.dv + 31) / 32;
  const int64_t part = (int64_t)dblocks * Sm::kState;
  // columns [32 db, ...) of V and dO and the state's rows of them, of value head vh
  auto copy_a = [&](int vh, int db, int st) {
    const int cols = min(a.dv - 32 * db, 32);
    const uint32_t to = lds0 + Sm::kA + st * Sm::kABytes;
    const RowCopy<E, BT, kT, kNW> cv(w, lane, a.v_stride, cols), co(w, lane, o_stride, cols);
    cv(rows_buffer(static_cast<const E*>(a.v) + t0 * a.v_stride + (int64_t)vh * a.dv + 32 * db, n, a.v_stride, cols),
       to + Sm::kV, w);
    co(rows_buffer(static_cast<const E*>(b.dout) + t0 * o_stride + (int64_t)vh * a.dv + 32 * db, n, o_stride, cols),
       to + Sm::kO, w);
    const char* img = b.s_img + (slot * a.hv + vh) * b.img_item + (int64_t)db * Sm::kState;
#pragma unroll
    for (int x = 0; x < kP; ++x) copy_linear<Sm::kState, kNW>(img + x * part, to + Sm::kS + x * Sm::kState, w, lane);
  };
  auto copy_ds = [&](int vh, int db) {
    const char* img = b.ds_img + (slot * a.hv + vh) * b.img_item + (int64_t)db * Sm::kState;
#pragma unroll
    for (int x = 0; x < kP; ++x) copy_linear<Sm::kState, kNW>(img + x * part, lds0 + Sm::kDS + x * Sm::kState, w, lane);
  };
  const KT kt(lane);
  const BT bt(lane);
  float* const gate = reinterpret_cast<float*>(smem + Sm::kGate);
  float* const red = reinterpret_cast<float*>(smem + Sm::kRed);
  float* const tok = reinterpret_cast<float*>(smem + Sm::kTok);
  float* const dots = reinterpret_cast<float*>(smem + Sm::kDot);
  const int i = 16 * w + r;  // this lane's token

  // Slot t <= w: rows j of tile t, column i; t > w, and slot kNW for tile w: rows i' of tile t, column j' = i.  With both
  // orientations no wave needs another's tiles, and every wave has kNW + 1.
  f32x4 B[kNW + 1], dQ[kTiles], dK[kTiles];
#pragma unroll
  for (int t = 0; t <= kNW; ++t) B[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int m = 0; m < kTiles; ++m) dQ[m] = dK[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  copy_a(kh * a.rep + h0, 0, 0);
  int st = 0;
  for (int h = h0; h < h1; ++h) {
    const int vh = kh * a.rep + h;
    // gates: wave 0, prefix sums in fp64, kept as two floats
    if (w == 0) {
      double before = 0.0, G[kT / 64];
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        const int t = 64 * x + lane;
        const float v = t < n ? clamp_gate(b.gate[(t0 + t) * a.hv + vh]) : 0.f;
        G[x] = before + prefix_sum((double)v, lane);
        before = __shfl(G[x], 63);
      }
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        const int t = 64 * x + lane;
        const float hi = (float)G[x];
        gate[t] = hi;
        gate[kT + t] = (float)(G[x] - (double)hi);
        gate[2 * kT + t] = a.scale * exp_f32(hi);
        gate[3 * kT + t] = exp_f32((float)(before - G[x]));
      }
      if (lane == 0) gate[4 * kT] = exp_f32((float)before);
    }
    f32x4 bb[kNW + 1], sq[kTiles], sk[kTiles];
#pragma unroll
    for (int t = 0; t <= kNW; ++t) bb[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < kTiles; ++m) sq[m] = sk[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    float dot = 0.f;
    for (int db = 0; db < dblocks; ++db) {
      copies_done();
      const lds_ptr sa = sm + Sm::kA + st * Sm::kABytes;
      copy_ds(vh, db);
      if (db + 1 < dblocks) copy_a(vh, db + 1, st ^ 1);
      else if (h + 1 < h1) copy_a(vh + 1, 0, st ^ 1);
#pragma unroll
      for (int kb = 0; kb < 32 / M::kDepth; ++kb) {
        const auto vw = bt.rows(sa + Sm::kV, w, kb), ow = bt.rows(sa + Sm::kO, w, kb);
#pragma unroll
        for (int t = 0; t < kNW; ++t) {
          if (t <= w) bb[t] = M::mma(bt.rows(sa + Sm::kV, t, kb), ow, bb[t]);
          else bb[t] = M::mma(bt.rows(sa + Sm::kO, t, kb), vw, bb[t]);
        }
        bb[kNW] = M::mma(ow, vw, bb[kNW]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int x = 0; x < kP; ++x)
            sq[m] = M::mma(kt.template cols<true>(sa + Sm::kS + x * Sm::kState, m, kb), ow, sq[m]);
      }
      copies_done();
#pragma unroll
      for (int kb = 0; kb < 32 / M::kDepth; ++kb) {
        const auto vw = bt.rows(sa + Sm::kV, w, kb);
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int x = 0; x < kP; ++x)
            sk[m] = M::mma(kt.template cols<true>(sm + Sm::kDS + x * Sm::kState, m, kb), vw, sk[m]);
      }
      // <S, dS'> of these columns (the images are alike, so their order does not matter)
      for (int x = threadIdx.x; x < Sm::kState / 16; x += kNW * 64) {
        float s[16 / sizeof(E)], d[16 / sizeof(E)];
#pragma unroll
        for (int y = 0; y < kP; ++y) {
          const auto fs = lds_read<typename M::Frag>(sa + Sm::kS + y * Sm::kState + 16 * x);
          const auto fd = lds_read<typename M::Frag>(sm + Sm::kDS + y * Sm::kState + 16 * x);
#pragma unroll
          for (int z = 0; z < (int)(16 / sizeof(E)); ++z) {
            s[z] = (y ? s[z] : 0.f) + (float)fs[z];
            d[z] = (y ? d[z] : 0.f) + (float)fd[z];
          }
        }
#pragma unroll
        for (int z = 0; z < (int)(16 / sizeof(E)); ++z) dot = fmaf(s[z], d[z], dot);
      }
      st ^= 1;
    }
    // pairs of tokens
    const float hi = gate[i], lo = gate[kT + i];
    float base = 0.f;  // sum over the rows of the tiles before
#pragma unroll
    for (int t = 0; t <= kNW; ++t) {
      const bool lower = t <= w && t < kNW;
      const int tile = t < kNW ? t : w;
      const f32x4 rh = *reinterpret_cast<const f32x4*>(gate + 16 * tile + 4 * g),
                  rl = *reinterpret_cast<const f32x4*>(gate + kT + 16 * tile + 4 * g);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 16 * tile + 4 * g + x;
        const float e = (hi - rh[x]) + (lo - rl[x]);
        const bool live = lower ? row <= i : row >= i;
        bb[t][x] = live ? bb[t][x] * (a.scale * exp_f32(lower ? e : -e)) : 0.f;
      }
      B[t] += bb[t];
      if (lower) {
        // B_ij (q_i . k_j), then for every row t of the tile the sum over the rows before it, over columns i >= t
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < DK / M::kDepth; ++kb)
          s = M::mma(kt.rows(sm + Sm::kK, t, kb), kt.rows(sm + Sm::kQ, w, kb), s);
        s *= bb[t];
        float own = (s[0] + s[1]) + (s[2] + s[3]);
        const float up1 = __shfl_up(own, 16), up2 = __shfl_up(own, 32), up3 = __shfl_up(own, 48);
        float before = base + (g > 0 ? up1 : 0.f) + (g > 1 ? up2 : 0.f) + (g > 2 ? up3 : 0.f);
        base += across_groups(own);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 16 * t + 4 * g + x;
          float v = row <= i ? before : 0.f;
          before += s[x];
          v += dpp_row<0x128>(v);
          v += dpp_row<0x124>(v);
          v += dpp_row<0x122>(v);
          v += dpp_row<0x121>(v);
          if (r == 0) red[w * kT + row] = v;
        }
      }
    }
    // the state's terms, and their dots with q_i and k_i
    {
      const float eg = gate[2 * kT + i], ci = gate[3 * kT + i];
      float rq = 0.f, rk = 0.f;
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) {
        const auto qi = kt.rows(sm + Sm::kQ, w, kb), ki = kt.rows(sm + Sm::kK, w, kb);
#pragma unroll
        for (int y = 0; y < M::kTiles; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int m = kb * M::kTiles + y;
            const float fq = eg * sq[m][x], fk = ci * sk[m][x];
            rq = fmaf((float)qi[4 * y + x], fq, rq);
            rk = fmaf((float)ki[4 * y + x], fk, rk);
            dQ[m][x] += fq;
            dK[m][x] += fk;
          }
      }
      rq = across_groups(rq);
      rk = across_groups(rk);
      if (g == 0) {
        tok[i] = rq;
        tok[kT + i] = rk;
      }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) dot += __shfl_xor(dot, m);
      if (lane == 0) dots[w] = dot;
    }
    __syncthreads();
    if (w == 0) {
      float all = 0.f;
#pragma unroll
      for (int x = 0; x < kNW; ++x) all += dots[x];
      all *= gate[4 * kT];
      // tokens lane, 64 + lane: sums of Z before and of R from there on, fp32: all have one sign or are independent
      float z0 = 0.f, later[kT / 64], earlier[kT / 64];
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        float z = tok[kT + 64 * x + lane], s = z;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const float t = __shfl_up(s, m);
          if (lane >= m) s += t;
        }
        const float one = __shfl_up(s, 1);
        earlier[x] = z0 + (lane ? one : 0.f);
        z0 += __shfl(s, 63);
      }
      float r0 = 0.f;
#pragma unroll
      for (int x = kT / 64 - 1; x >= 0; --x) {
        float s = tok[64 * x + lane];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const float t = __shfl_down(s, m);
          if (lane + m < 64) s += t;
        }
        later[x] = r0 + s;
        r0 += __shfl(s, 0);
      }
#pragma unroll
      for (int x = 0; x < kT / 64; ++x) {
        const int t = 64 * x + lane;
        float pairs = 0.f;
        for (int y = t / 16; y < kNW; ++y) pairs += red[y * kT + t];
        if (t < n) b.dg[(t0 + t) * a.hv + vh] = ((all + earlier[x]) + later[x]) + pairs;
      }
    }
    __syncthreads();  // gates and sums have been read
  }
  // dQ += K^T B^T, dK += Q^T B
#pragma unroll
  for (int kb = 0; kb < kT / M::kDepth; ++kb) {
    f32x4 lo[M::kTiles], up[M::kTiles];
#pragma unroll
    for (int y = 0; y < M::kTiles; ++y) {
      const int t = kb * M::kTiles + y;
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      lo[y] = t <= w ? B[t] : zero;
      up[y] = t == w ? B[kNW] : t > w ? B[t] : zero;
    }
    if (kb * M::kTiles <= w) {
      const auto f = M::template split<M::parts(2)>(lo);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        const auto kc = kt.cols(sm + Sm::kK, m, kb);
#pragma unroll
        for (int x = 0; x < M::parts(2); ++x) dQ[m] = M::mma(kc, f.p[x], dQ[m]);
      }
    }
    if (kb * M::kTiles + M::kTiles > w) {
      const auto f = M::template split<M::parts(2)>(up);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        const auto qc = kt.cols(sm + Sm::kQ, m, kb);
#pragma unroll
        for (int x = 0; x < M::parts(2); ++x) dK[m] = M::mma(qc, f.p[x], dK[m]);
      }
    }
  }
  if (i >= n) return;
  const int64_t at = ((t0 + i) * a.hk + kh) * (int64_t)a.dk;
  if (b.groups > 1) {
    const int64_t size = b.tokens * a.hk * (int64_t)a.dk;
    float* pq = b.part + (int64_t)grp * size + at;
    float* pk = pq + (int64_t)b.groups * size;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const int v = KT::value(m, g, 0);
      if (v < a.dk) {
        *reinterpret_cast<f32x4*>(pq + v) = dQ[m];
        *reinterpret_cast<f32x4*>(pk + v) = dK[m];
      }
    }
    return;
  }
#pragma unroll
  for (int m = 0; m < kTiles; m += M::kTiles) {
    const int v = KT::value(m, g, 0);
    if (v < a.dk) {
      *reinterpret_cast<typename M::Frag*>(static_cast<E*>(b.dq) + at + v) = M::pack(&dQ[m]);
      *reinterpret_cast<typename M::Frag*>(static_cast<E*>(b.dk) + at + v) = M::pack(&dK[m]);
    }
  }
}

// dq (y = 0) and dk (y = 1) of 64 tokens of a sequence: the groups' sums in order
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
  for (int64_t x = threadIdx.x * 4; x < count; x += 1024) {
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
  size_t s, ds, part, total;
  int64_t item, units;
  int32_t groups;
};
template <typename E>
BwdLayout layout_t(const mamba_delta_dims* d, bool packed) {
  BwdLayout l = {};
  l.seg = seg_layout(d, packed);
  l.units = slots_of(d, packed, kUnit<E>);
  l.item = kImgParts<E> * image_part<E>(d);
  const size_t img = (size_t)l.units * (size_t)d->v_heads * (size_t)l.item;
  l.s = (l.seg.total + 1023) / 1024 * 1024;
  l.ds = l.s + img;
  l.part = l.ds + img;
  // enough workgroups for two rounds of the CUs
  const int64_t rep = d->v_heads / d->qk_heads, wgs = l.units * d->qk_heads;
  l.groups = (int32_t)std::max<int64_t>(1, std::min<int64_t>(rep, 512 / std::max<int64_t>(wgs, 1)));
  const int64_t per = (rep + l.groups - 1) / l.groups;
  l.groups = (int32_t)((rep + per - 1) / per);  // (none without heads)
  l.total = l.part;
  if (l.groups > 1)
    l.total += 2 * (size_t)l.groups * (size_t)(packed ? d->seqlen : d->batch * d->seqlen) *
               (size_t)(d->qk_heads * d->dk) * sizeof(float);
  return l;
}
BwdLayout layout(const mamba_delta_dims* d, bool packed) {
  return d->io_dtype == MAMBA_BF16 ? layout_t<uint16_t>(d, packed) : layout_t<float>(d, packed);
}

template <typename E, int DK>
int launch_grad(const GradArgs& b, int64_t units, hipStream_t s) {
  using Sm = GradSmem<E, DK>;
  const uint32_t blocks = (uint32_t)(units * b.f.hk * b.groups);
  hipLaunchKernelGGL((linear_grad_kernel<E, DK>), wide_grid(blocks, Sm::kNW * 64), dim3(Sm::kNW * 64), 0, s, b,
                     blocks);
  return launch_status();
}

template <typename E>
int launch_bwd(const PassArgs& fwd, const PassArgs& rev, const GradArgs& b, int64_t units, hipStream_t s) {
  constexpr bool bf = sizeof(E) == 2;
  int st = MAMBA_OK;
  if (fwd.f.seg_chunks && (st = launch_segments(fwd, bf, false, s)) != MAMBA_OK) return st;
  if ((st = launch_pass<E, kImages>(fwd, s)) != MAMBA_OK) return st;
  if (rev.f.seg_chunks && (st = launch_segments(rev, bf, true, s)) != MAMBA_OK) return st;
  if ((st = launch_pass<E, kOutput | kImages | kReverse>(rev, s)) != MAMBA_OK) return st;
  st = b.f.dk <= 64 ? launch_grad<E, 64>(b, units, s) : launch_grad<E, 128>(b, units, s);
  if (st != MAMBA_OK || b.groups == 1) return st;
  hipLaunchKernelGGL((linear_fold_kernel<E>), dim3((unsigned)b.f.slots, 2), dim3(256), 0, s, b);
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
  fwd.img = ws + l.s;
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
  rev.img = ws + l.ds;
  GradArgs b = {};
  b.f = fwd.f;
  b.gate = g;
  b.dout = dout;
  b.s_img = fwd.img;
  b.ds_img = rev.img;
  b.img_item = l.item;
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
