// mamba_window.hip -- causal attention with a sliding window and sinks on gfx950, forward.
//
// For a query at position p, over the keys j <= p with p - j < window or j < sinks:
//     s_j = scale q . k_j,  out = sum_j exp(s_j - lse) v_j,  lse = log sum_j exp(s_j)
// in one pass over the keys with the running maximum m and sum l:
//     m' = max(m, max s),  P = exp(s - m'),  l' = exp(m - m') l + sum P,  O' = exp(m - m') O + P V
//
// A workgroup has 4 waves of 32 queries (fp32 storage: 16) of one head and goes through the keys in tiles of 64: the
// sinks' tiles first, then those that its queries' windows reach.  Products are made transposed, keys x queries and
// values x queries: a lane holds one query's scores, so that the softmax needs two exchanges per tile, and the
// accumulators of P are, rounded, the operand of the next product.
//
// Rounding, bf16 storage: P enters the product with V as two bf16 parts (2^-17 of each weight), so that out's own rounding
// is the only one that shows, as in the step and as fp32 arithmetic promises (one part: 2^-8 of a weight at most, out off
// by 2.0e-3 to 2.4e-3 of its norm where rounding it is 1.66e-3; 169 us of the layer below in place of 211, 108 of the
// packed prompts in place of 132); scores, m, l and O are fp32.  The reference of the weights follows the maximum only
// past a factor of 2^8, so that in a tile with a new maximum the sums are seldom rescaled (7% of the time).
//
// Measured (8 x 2048 tokens, 20 and 4 heads of 128, window 1024, bf16): 211 us, 615 TFLOP/s of the pairs that are seen, 1.5
// times as many of products made.  The matrix unit is busy for 45% of that, the vector unit for 55%, in turn: softmax,
// conversions and products of the two waves of a SIMD add up.  Two workgroups share a CU, 8 waves of 32 queries: with 16 each a tile's operands would
// be read twice as often.
#include "mamba_window.h"

namespace mamba {
namespace window {
namespace {

template <typename E>
constexpr int kTilesQ = sizeof(E) == 2 ? 2 : 1;  // 16-query tiles of a wave
template <typename E>
constexpr int kQueries = 4 * 16 * kTilesQ<E>;    // of a workgroup

template <typename E, int DK>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void window_fwd_kernel(WinArgs a, uint32_t blocks) {
  using M = Mma<E>;
  using KT = KeyTile<E, DK>;
  constexpr int kC2 = kTilesQ<E>, kQ = kQueries<E>, kStage = 2 * KT::kBytes;
  __shared__ __align__(1024) char smem[2 * kStage];
  const uint32_t id = wide_index();
  if (id >= blocks) return;
  const int64_t wg = spread_index(id, blocks, a.rep);
  const int64_t slot = wg / a.hq;
  const int h = (int)(wg - slot * a.hq), kh = h / a.rep;
  const auto [seq, tile] = tile_of<true>(a.q_offsets, a.seqlen, a.nseq, slot, kQ);
  const Seq qs = seq_of(a.q_offsets, a.seqlen, seq), ks = seq_of(a.kv_offsets, a.kv_len, seq);
  if (tile < 0 || tile * kQ >= qs.len) return;  // an unused slot of a packed batch
  const int q0 = (int)tile * kQ, nq = min(qs.len - q0, kQ);
  const int shift = ks.len - qs.len;  // position of query 0
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w0 = 16 * kC2 * w;  // this wave's first query in the tile
  const Mask mask = mask_of(a);

  // tiles of keys: the sinks' that lie before the windows, then the windows'
  const int p0 = q0 + shift, p1 = p0 + nq - 1;  // positions
  const int lo = (int)(max((int64_t)p0 - a.window + 1, (int64_t)0) / kKeys);
  const int sink_tiles = min((mask.sinks + (kKeys - 1ll)) / kKeys, (int64_t)lo);
  const int count = p1 < 0 ? 0 : sink_tiles + p1 / kKeys - lo + 1;
  auto tile_at = [&](int i) { return i < sink_tiles ? i : lo + i - sink_tiles; };

  const E* kp = static_cast<const E*>(a.k) + ks.first * a.k_stride + (int64_t)kh * a.dim;
  const E* vp = static_cast<const E*>(a.v) + ks.first * a.v_stride + (int64_t)kh * a.dim;
  const uint32_t lds0 = lds_address(smem);
  const RowCopy<E, KT, kKeys, 4> ck(w, lane, a.k_stride, a.dim), cv(w, lane, a.v_stride, a.dim);
  auto copy = [&](int t, int st) {  // keys past the sequence are past the buffers and read as zero
    const int64_t j = (int64_t)t * kKeys, n = min((int64_t)kKeys, ks.len - j);
    ck(rows_buffer(kp + j * a.k_stride, n, a.k_stride, a.dim), lds0 + st * kStage, w);
    cv(rows_buffer(vp + j * a.v_stride, n, a.v_stride, a.dim), lds0 + st * kStage + KT::kBytes, w);
  };
  if (count) copy(tile_at(0), 0);

  // operands: column = query; a negative scale goes into the sign of q, so that a maximum of q . k is one of s
  typename M::Frag qf[kC2][DK / M::kDepth];
  const E* qp = static_cast<const E*>(a.q) + (qs.first + q0) * a.q_stride + (int64_t)h * a.dim;
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    load_rows<E, DK>(qp, a.q_stride, w0 + 16 * c + r, nq, a.dim, g, qf[c]);
    if (a.scale < 0.f)
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) qf[c][kb] = -qf[c][kb];
    if (a.scale == 0.f)  // (in q as well: of a masked score it would make NaN)
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) qf[c][kb] *= typename M::Frag{};
  }
  const float sc = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  f32x4 o[kC2][DK / 16];
  float mx[kC2], l[kC2];
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    mx[c] = kMinusInf;
    l[c] = 0.f;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) o[c][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const KT kt(lane);
  const int pw0 = p0 + w0, pw1 = pw0 + 16 * kC2 - 1;
  loads_done();
  for (int i = 0; i < count; ++i) {
    const int st = i & 1, j0 = tile_at(i) * kKeys;
    copies_done();
    if (i + 1 < count) copy(tile_at(i + 1), st ^ 1);
    if (mask.none(pw0, pw1, j0, j0 + kKeys - 1)) continue;
    const lds_ptr sk = (lds_ptr)(smem + st * kStage), sv = sk + KT::kBytes;
    f32x4 s[kC2][4];
#pragma unroll
    for (int c = 0; c < kC2; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) s[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kStepsK = DK / M::kDepth, kGroups = DK / 64, kStepsV = kKeys / M::kDepth * kGroups;
    typename M::Frag f[2][4];
    auto read_k = [&](int i) {
#pragma unroll
      for (int m = 0; m < 4; ++m) f[i & 1][m] = kt.rows(sk, m, i);
    };
    auto read_v = [&](int i) {  // (kStepsK is even)
#pragma unroll
      for (int x = 0; x < 4; ++x) f[i & 1][x] = kt.cols(sv, i % kGroups * 4 + x, i / kGroups);
    };
    read_k(0);
#pragma unroll
    for (int kb = 0; kb < kStepsK; ++kb) {
      end_step();
      if (kb + 1 < kStepsK) read_k(kb + 1); else read_v(0);
      end_step();
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int c = 0; c < kC2; ++c) s[c][m] = M::mma(f[kb & 1][m], qf[c][kb], s[c][m]);
    }
    end_step();
    if (kStepsV > 1) read_v(1);  // (two steps ahead: transposing reads take longer than a step's products)
    const bool whole = mask.all(pw0, pw1, j0, j0 + kKeys - 1);
#pragma unroll
    for (int c = 0; c < kC2; ++c) {
      const int p = pw0 + 16 * c + r;
      if (!whole) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (!mask.sees(p, j0 + 16 * m + 4 * g + x)) s[c][m][x] = kMinusInf;
      }
      float top = mx[c];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, s[c][m][x]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      // the maximum is followed only where weights would grow past 2^8: any reference gives the same softmax, and a
      // wave's queries together would have nearly every tile rescale all sums
      if (__any(top * sc > fmaf(mx[c], sc, 8.f))) {
        const float f = mx[c] == kMinusInf ? 0.f : fast_exp2((mx[c] - top) * sc);
        l[c] *= f;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) o[c][d] *= f;
        mx[c] = top;
      }
      const float use = mx[c] == kMinusInf ? 0.f : mx[c] * sc;  // (nothing seen yet)
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[c][m][x] = fast_exp2(fmaf(s[c][m][x], sc, -use));
#pragma unroll
      for (int m = 0; m < 4; ++m) sum += (s[c][m][0] + s[c][m][1]) + (s[c][m][2] + s[c][m][3]);
      l[c] += sum;
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
            f32x4& to = (kTileSums<E> ? part : o)[c][i % kGroups * 4 + x];
            to = M::mma(f[i & 1][x], pf[c].p[p], to);
          }
      end_step();
      if (i + 2 < kStepsV) read_v(i + 2);
    }
    if constexpr (kTileSums<E>) add_to(o, part);
    end_step();
  }
#pragma unroll
  for (int c = 0; c < kC2; ++c) {
    const int i = w0 + 16 * c + r;
    const float sum = across_groups(l[c]);
    if (i >= nq) continue;
    const int64_t row = (qs.first + q0 + i) * a.hq + h;
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    if (a.lse && g == 0)
      a.lse[row] = sum == 0.f ? kMinusInf : fmaf(mx[c], sc, __builtin_amdgcn_logf(sum)) * kLn2;
    E* to = static_cast<E*>(a.out) + row * a.dim;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) o[c][d] *= inv;
#pragma unroll
    for (int d = 0; d < DK / 16; d += M::kTiles)
      if (KT::value(d, g, 0) < a.dim) store_operand(to + KT::value(d, g, 0), &o[c][d]);
  }
}

template <typename E, int DK>
int launch_fwd(const WinArgs& a, hipStream_t s) {
  const uint32_t blocks =
      (uint32_t)(tile_slots(a.seqlen, a.nseq, a.q_offsets != nullptr, kQueries<E>) * a.hq);
  hipLaunchKernelGGL((window_fwd_kernel<E, DK>), wide_grid(blocks, 256), dim3(256), 0, s, a, blocks);
  return launch_status();
}

}  // namespace
}  // namespace window
}  // namespace mamba

using namespace mamba;
using namespace mamba::window;

extern "C" {

int mamba_window_attn_fwd(const void* q, const void* k, const void* v, const int64_t* q_offsets,
                          const int64_t* kv_offsets, float scale, void* out, float* lse, const mamba_window_dims* dims,
                          void* stream) {
  int st = check_window(dims, q_offsets != nullptr);
  if (st != MAMBA_OK) return st;
  if (!out) return MAMBA_ERR_NULL;
  if ((st = check_window_inputs(q, k, v, q_offsets, kv_offsets)) != MAMBA_OK) return st;
  if (!aligned(out, 16) || (lse && !aligned(lse, 4))) return MAMBA_ERR_ALIGN;
  WinArgs a = window_args(dims, scale, q, k, v, q_offsets, kv_offsets);
  a.out = out;
  a.lse = lse;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dims->io_dtype == MAMBA_BF16)
    return a.dim <= 64 ? launch_fwd<uint16_t, 64>(a, s) : launch_fwd<uint16_t, 128>(a, s);
  return a.dim <= 64 ? launch_fwd<float, 64>(a, s) : launch_fwd<float, 128>(a, s);
}

}  // extern "C"
