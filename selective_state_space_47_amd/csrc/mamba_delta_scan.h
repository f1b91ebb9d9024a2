// mamba_delta_scan.h -- the state of the gated delta rule through the chunks (formulas in mamba_delta.h): the
// forward's pass, its summary of a segment, and the backward's state pass, which runs beside the adjoint's.
//
// One workgroup per sequence (or segment), value head and 16 NW columns of the state.  A wave owns 16
// columns; its state stays in accumulators from the first chunk to the last, and every product's accumulators
// are the next product's operand, so that waves share nothing but the tiles they read.  Those come by copies
// straight into LDS, a chunk ahead.
//
// Bound by the chain of a chunk's products (K S, T Y, K^T E: a wave waits for the matrix unit, for LDS and for
// its own conversions in turn), 4.5 us a chunk of the output pass with 8 waves on a CU and 3.6 us with 4.  8 x 2048
// tokens x 40 heads of 128, bf16: 316 us; 320 workgroups are two rounds of 256 CUs.
#pragma once
#include "mamba_delta.h"

namespace mamba {
namespace delta {

// Threads that a pass is compiled for: 512 (256 registers each), though a workgroup of 4 waves could have 512
// registers.  With no more than 256 the compiler keeps accumulators where vector instructions reach them;
// otherwise a fifth of its vector instructions move values to and from the accumulation registers.
constexpr int kPassThreads = 512;

// What a pass leaves: the output and the last state; the backward's E and the state before each chunk; or,
// for a segment of a long sequence, the state that it makes from zero (columns of the state) and from the
// identity without values (dk more columns: the segment's map of the state before it).
enum Pass { kOut, kBackward, kSummary };

// One stage of a workgroup's LDS: the chunk's K and Q, what the pass reads of the chunk's workspace (P for an
// output; T and gates) and V.
template <typename E, int DK, int NW, Pass kPass>
struct Stage {
  using CW = ChunkWs<E>;
  static constexpr int kK = 0;
  static constexpr int kQ = KeyTile<E, DK>::kBytes;
  static constexpr int kWs = 2 * KeyTile<E, DK>::kBytes;
  static constexpr int kFrom = kPass == kOut ? CW::kP : CW::kT;
  static constexpr int kWsBytes = CW::kDecay - kFrom;
  static constexpr int kP = kWs + CW::kP - kFrom;
  static constexpr int kT = kWs + CW::kT - kFrom;
  static constexpr int kGate = kWs + CW::kGate - kFrom;
  static constexpr int kVv = kWs + kWsBytes;
  static constexpr int kBytes = kVv + ValueTile<E, 16 * NW>::kBytes;
  static constexpr int kCount = 2 * kBytes <= 160 * 1024 ? 2 : 1;
  static constexpr int kLds = kCount * kBytes;
};

// The results of the backward's pass only enter gradients that are rounded to the storage type: with bf16
// storage two parts of each factor keep them clear of those roundings, also where a sum of them cancels (dg).
template <typename E, int DK, int NW, Pass kPass>
__device__ __forceinline__ void scan_pass(const Args& a, int32_t col_blocks, char* smem, uint32_t id,
                                          uint32_t grid) {
  using M = Mma<E>;
  using St = Stage<E, DK, NW, kPass>;
  using KT = KeyTile<E, DK>;
  using TT = TriTile<E>;
  using VT = ValueTile<E, 16 * NW>;
  constexpr bool kStates = kPass == kBackward, kO = kPass == kOut;
  constexpr int kPS = M::parts(2), kPT = M::parts(kTParts);
  constexpr int kPY = M::parts(kStates ? 2 : 3), kPE = M::parts(kStates ? 2 : 3);
  constexpr int kPO = M::parts(2);  // of S, of P and of E in the output
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wg = spread_index(id, grid, a.rep * col_blocks);
  const int64_t sh = wg / col_blocks;
  const int64_t seg_slot = sh / a.hv;
  const int vh = (int)(sh - seg_slot * a.hv), kh = vh / a.rep;
  const int64_t unit = a.seg_chunks * kC;
  const int64_t seq = a.seg_chunks ? slot_seq(a, seg_slot, unit) : seq_by_length(a, seg_slot);
  const Span sp = seq_span(a, seq);
  const int64_t seg = a.seg_chunks ? seg_slot - slot_base(a, seq, sp.first, unit) : 0;
  const int64_t nchunks = (sp.len + kC - 1) / kC;
  const int64_t first = seg * a.seg_chunks;  // this segment's chunks
  const int64_t end = a.seg_chunks ? min(first + a.seg_chunks, nchunks) : nchunks;
  if (seg < 0 || (first >= end && seg > 0)) return;  // an unused slot of a packed batch
  if (kPass == kSummary && end == nchunks) return;   // nothing follows the last segment
  const int vblocks = (a.dv + 16 * NW - 1) / (16 * NW);
  const int cb = (int)(wg - sh * col_blocks);
  const bool map = kPass == kSummary && cb >= vblocks;  // columns of the identity
  const int width = map ? a.dk : a.dv;
  const int col0 = (map ? cb - vblocks : cb) * 16 * NW;  // this workgroup's first column
  const int col = col0 + 16 * w;                         // this wave's
  const int64_t slot0 = slot_base(a, seq, sp.first);
  const E* kp = static_cast<const E*>(a.k) + sp.first * a.k_stride + (int64_t)kh * a.dk;
  const E* qp = static_cast<const E*>(a.q) + sp.first * a.q_stride + (int64_t)kh * a.dk;
  const E* vp = static_cast<const E*>(a.v) + sp.first * a.v_stride + (int64_t)vh * a.dv + col0;
  const int64_t o_stride = (int64_t)a.hv * a.dv;
  E* op = static_cast<E*>(a.out) + sp.first * o_stride + (int64_t)vh * a.dv + col;
  const bool has_col = col + r < width;
  // (dk, width) matrices of this head: the sequence's states, and this segment's
  const int64_t s_at = (seq * a.hv + vh) * (int64_t)a.dk * a.dv + col + r;
  const int64_t g_at = (seg_slot * a.hv + vh) * (int64_t)a.dk * width + col + r;
  const float* from = kPass == kSummary ? nullptr : a.seg_chunks ? a.seg_state + g_at : a.s0 ? a.s0 + s_at : nullptr;

  f32x4 S[DK / 16];
#pragma unroll
  for (int m = 0; m < DK / 16; ++m)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = KT::value(m, g, x);
      S[m][x] = map ? (row == col + r ? 1.f : 0.f)
                    : from && has_col && row < a.dk ? from[(int64_t)row * a.dv] : 0.f;
    }

  const uint32_t lds0 = lds_address(smem);
  const int vcols = map ? 0 : min(a.dv - col0, 16 * NW);  // (without values: words outside, zeros)
  const RowCopy<E, KT, kC, NW> ck(w, lane, a.k_stride, a.dk), cq(w, lane, a.q_stride, a.dk);
  const RowCopy<E, VT, kC, NW> cv(w, lane, a.v_stride, vcols);
  // copies chunk ch into stage st; tokens past the sequence are past the buffers and read as zero
  auto copy = [&](int64_t ch, int st) {
    const int64_t t = ch * kC, n = min((int64_t)kC, sp.len - t);
    const uint32_t to = lds0 + st * St::kBytes;
    ck(rows_buffer(kp + t * a.k_stride, n, a.k_stride, a.dk), to + St::kK, w);
    cv(rows_buffer(vp + t * a.v_stride, n, a.v_stride, vcols), to + St::kVv, w);
    if (kO) cq(rows_buffer(qp + t * a.q_stride, n, a.q_stride, a.dk), to + St::kQ, w);
    copy_linear<St::kWsBytes, NW>(a.ws + ((slot0 + ch) * a.hv + vh) * a.ws_item + St::kFrom,
                                  to + St::kWs, w, lane);
  };

  // bytes of the backward's images of one chunk and value head
  const int dv_pad = (a.dv + BwdBlock<E>::kDB - 1) / BwdBlock<E>::kDB * BwdBlock<E>::kDB;
  const int64_t img_bytes = (int64_t)dv_pad * KT::kRow;
  const int64_t e_bytes = (int64_t)dv_pad * kC * sizeof(E) * BwdBlock<E>::kEParts;
  const KT kt(lane);
  const TT tt(lane);
  const VT vt(lane, 16 * w);
  if (first < end) copy(first, 0);
  for (int64_t ch = first; ch < end; ++ch) {
    const int st = St::kCount == 2 ? (int)((ch - first) & 1) : 0;
    copies_done();
    const lds_ptr sm = (lds_ptr)(smem + st * St::kBytes);
    const int n = (int)min((int64_t)kC, sp.len - ch * kC);
    // Operands are read a step before the products that take them: one or two waves per SIMD leave nobody
    // else to hide the reads behind (an eighth more time with reads where they are used).  Nothing is moved past
    // the end of a step.
    typename M::Frag kf[2][4], qf[2][4];
    auto read_kq = [&](int kb) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        kf[kb & 1][m] = kt.rows(sm + St::kK, m, kb);
        if (kO) qf[kb & 1][m] = kt.rows(sm + St::kQ, m, kb);
      }
    };
    auto step = [] { __builtin_amdgcn_sched_barrier(0); };
    read_kq(0);
    // with two stages the next chunk is copied while this one is worked on
    if (St::kCount == 2 && ch + 1 < end) copy(ch + 1, st ^ 1);

    if constexpr (kStates) {
      // the state before the chunk: 16 bytes of one column per operand
      const int64_t item = (slot0 + ch) * a.hv + vh;
      char* img = a.s_img + item * img_bytes;
      if (col < dv_pad) {
#pragma unroll
        for (int kb = 0; kb < DK / M::kDepth; ++kb) {
          const auto f = M::pack(&S[kb * M::kTiles]);
          *reinterpret_cast<typename M::Frag*>(img + (int64_t)(col + r) * KT::kRow +
                                               (((4 * kb + g) ^ KT::key(col + r)) << 4)) = f;
          if constexpr (sizeof(E) == 2) {  // a byte per value beside it, in the same order
            const uint4 h = __builtin_bit_cast(uint4, f);
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
            uint32_t low[2] = {0, 0};
#pragma unroll
            for (int x = 0; x < 8; ++x)
              low[x >> 2] |= low_byte(S[2 * kb + (x >> 2)][x & 3],
                                      x & 1 ? hw[x >> 1] & 0xffff0000u : hw[x >> 1] << 16)
                             << (8 * (x & 3));
            *reinterpret_cast<uint2*>(a.s_low + item * (img_bytes / 2) + (int64_t)(col + r) * (KT::kRow / 2) +
                                      (((4 * kb + g) ^ KT::key(col + r)) << 3)) = make_uint2(low[0], low[1]);
          }
        }
      }
    }
    // K S (tokens x columns) and (Q S)^T (columns x tokens)
    f32x4 y[4], o[4], vv[4], eg[4];
    float so[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < DK / M::kDepth; ++kb) {
      step();
      if (kb + 1 < DK / M::kDepth) {
        read_kq(kb + 1);
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          vv[m] = vt.tile(sm + St::kVv, m);
          eg[m] = lds_read<f32x4>(sm + St::kGate + (16 * m + 4 * g) * 4);
          so[m] = lds_read<float>(sm + St::kGate + (16 * m + r) * 4);
        }
      }
      const auto s = M::template split<kPS>(&S[kb * M::kTiles]);
#pragma unroll
      for (int p = 0; p < kPS; ++p)
#pragma unroll
        for (int m = 0; m < 4; ++m) y[m] = M::mma(kf[kb & 1][m], s.p[p], y[m]);
      if constexpr (kO) {
#pragma unroll
        for (int p = 0; p < kPO; ++p)
#pragma unroll
          for (int m = 0; m < 4; ++m) o[m] = M::mma(s.p[p], qf[kb & 1][m], o[m]);
      }
    }
    // Y = V - diag(exp G) K S;  O scaled by its token's factor
    step();
    typename M::Frag tf[2][kPT][4], pf[2][kPO][4];
    auto read_t = [&](int kb) {
#pragma unroll
      for (int p = 0; p < kPT; ++p)
#pragma unroll
        for (int m = kb * M::kTiles; m < 4; ++m)
          tf[kb & 1][p][m] = tt.rows(sm + St::kT + p * TT::kBytes, m, kb);
    };
    auto read_p = [&](int kb) {
#pragma unroll
      for (int p = 0; p < kPO; ++p)
#pragma unroll
        for (int m = kb * M::kTiles; m < 4; ++m)
          pf[kb & 1][p][m] = tt.rows(sm + St::kP + p * TT::kBytes, m, kb);
    };
    read_t(0);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        y[m][x] = fmaf(-eg[m][x], y[m][x], vv[m][x]);
        if (kO) o[m][x] *= a.scale * so[m];
      }
    // what the state takes: factors c, then operands of K in fours
    constexpr int kFours = TT::kBlocks * (DK / 64);
    f32x4 cf[4];
    float last = 0.f;
    auto read_c = [&] {
#pragma unroll
      for (int m = 0; m < 4; ++m) cf[m] = lds_read<f32x4>(sm + St::kGate + (kC + 16 * m + 4 * g) * 4);
      last = lds_read<float>(sm + St::kGate + 2 * kC * 4);
    };
    typename M::Frag cols[2][4];
    auto read_cols = [&](int i) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
        cols[i & 1][m] = kt.cols(sm + St::kK, i % (DK / 64) * 4 + m, i / (DK / 64));
    };
    // E = T Y, T lower triangular; the parts' products down to the last part's size.  The state pass
    // also makes it transposed, to store it row by row.
    f32x4 e[4], et[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) e[m] = et[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      step();
      if (kb + 1 < TT::kBlocks) {
        read_t(kb + 1);
      } else {
        if (kO) read_p(0); else read_cols(0);
        read_c();
      }
      const auto ys = M::template split<kPY>(&y[kb * M::kTiles]);
#pragma unroll
      for (int p = 0; p < kPT; ++p)
#pragma unroll
        for (int x = 0; x + p < kPY; ++x)
#pragma unroll
          for (int m = kb * M::kTiles; m < 4; ++m) {
            e[m] = M::mma(tf[kb & 1][p][m], ys.p[x], e[m]);
            if (kStates) et[m] = M::mma(ys.p[x], tf[kb & 1][p][m], et[m]);
          }
    }
    step();
    if constexpr (kStates) {
      // token 16 m + r, columns col + 4 g .. +3 of the image of E
      if (col + 4 * g < dv_pad) {
        using ET = KeyTile<E, BwdBlock<E>::kDB>;
        constexpr int kDB = BwdBlock<E>::kDB;
        const int cw = (col + 4 * g) % kDB * (int)sizeof(E);  // byte in the block's rows
        char* img = a.e_img + ((slot0 + ch) * a.hv + vh) * e_bytes +
                    (int64_t)((col + 4 * g) / kDB) * BwdBlock<E>::kEParts * BwdBlock<E>::kE;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int t = 16 * m + r;
          char* to = img + t * ET::kRow + (((cw >> 4) ^ ET::key(t)) << 4) + (cw & 15);
          if constexpr (sizeof(E) == 2) {
            const uint32_t h0 = pack_bf16(make_float2(et[m][0], et[m][1]));
            const uint32_t h1 = pack_bf16(make_float2(et[m][2], et[m][3]));
            const float2 f0 = unpack(h0), f1 = unpack(h1);
            *reinterpret_cast<uint2*>(to) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(to + BwdBlock<E>::kE) =
                make_uint2(pack_bf16(make_float2(et[m][0] - f0.x, et[m][1] - f0.y)),
                           pack_bf16(make_float2(et[m][2] - f1.x, et[m][3] - f1.y)));
          } else {
            *reinterpret_cast<f32x4*>(to) = et[m];
          }
        }
      }
    } else if constexpr (kO) {
      // O += P E, transposed: a lane ends with 4 consecutive columns of one token
#pragma unroll
      for (int kb = 0; kb < TT::kBlocks; ++kb) {
        if (kb + 1 < TT::kBlocks) read_p(kb + 1); else read_cols(0);
        const auto es = M::template split<kPO>(&e[kb * M::kTiles]);
#pragma unroll
        for (int p = 0; p < kPO; ++p)
#pragma unroll
          for (int x = 0; x + p < kPO; ++x)
#pragma unroll
            for (int m = kb * M::kTiles; m < 4; ++m) o[m] = M::mma(es.p[x], pf[kb & 1][p][m], o[m]);
        step();
      }
      const auto buf = __builtin_amdgcn_make_buffer_rsrc(
          op + ch * kC * o_stride, 0, (int)(((n - 1) * o_stride + max(a.dv - col, 0)) * (int64_t)sizeof(E)),
          0x00020000);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        store_four<E>(buf, col + 4 * g < a.dv ? (uint32_t)((16 * m + r) * o_stride + 4 * g) * (uint32_t)sizeof(E)
                                              : kOutside, o[m]);
    }
    // S = exp(G_64) S + K^T diag(c) E
#pragma unroll
    for (int m = 0; m < 4; ++m) e[m] *= cf[m];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) S[m] *= last;
#pragma unroll
    for (int kb = 0; kb < TT::kBlocks; ++kb) {
      const auto es = M::template split<kPE>(&e[kb * M::kTiles]);
#pragma unroll
      for (int j = 0; j < DK / 64; ++j) {
        const int i = kb * (DK / 64) + j;
        if (i + 1 < kFours) read_cols(i + 1);
#pragma unroll
        for (int p = 0; p < kPE; ++p)
#pragma unroll
          for (int m = 0; m < 4; ++m) S[4 * j + m] = M::mma(cols[i & 1][m], es.p[p], S[4 * j + m]);
        step();
      }
    }
    if (St::kCount == 1 && ch + 1 < end) {
      __syncthreads();  // every wave has read the stage
      copy(ch + 1, 0);
    }
  }
  float* to = kPass == kSummary ? (map ? a.seg_map : a.seg_state) + g_at
              : kO && a.last && end == nchunks ? a.last + s_at : nullptr;
  if (to && has_col) {
#pragma unroll
    for (int m = 0; m < DK / 16; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = KT::value(m, g, x);
        if (row < a.dk) to[(int64_t)row * width] = S[m][x];
      }
  }
}

}  // namespace delta
}  // namespace mamba
