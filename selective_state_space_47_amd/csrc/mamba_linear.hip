// mamba_linear.hip -- linear attention with a decay per head on gfx950: whole sequences in chunks of 64 tokens on the
// matrix cores (the pass is in mamba_linear.h), and one generation step.
//
//   linear_pass_kernel   the state through the chunks of a sequence, or of a segment of one
//   linear_join_kernel   where sequences go through in segments side by side: the states before the segments
//   linear_step_kernel   one token for each sequence
#include "mamba_linear.h"

namespace mamba {
namespace linear {
namespace {

// The states that the segments begin with, one after another: S <- decay S + (the segment's own); seg_state holds each
// segment's own on entry.  Bound by memory (packed prompts, 80 heads of 128 x 64: 28 us, 5.5 TB/s).  The first one's is a
// copy of the initial state: the output pass reads only these, as it may write the last state over the initial one.
template <bool kRev>
__global__ __launch_bounds__(256) void linear_join_kernel(PassArgs p, int32_t blocks) {
  const Args& a = p.f;
  const uint32_t id = wide_index();
  const int64_t sh = id / (uint32_t)blocks;
  const int64_t seq = sh / a.hv;
  if (seq >= a.nseq) return;
  const int vh = (int)(sh - seq * a.hv);
  const int64_t size = (int64_t)a.dk * a.dv, at = ((int64_t)(id - sh * blocks) * 256 + threadIdx.x) * 4;
  if (at >= size) return;
  const int64_t unit = a.seg_chunks * kC;
  const Span sp = seq_span(a, seq);
  const int64_t base = slot_base(a, seq, sp.first, unit), nseg = (sp.len + unit - 1) / unit;
  if ((sp.len + kC - 1) / kC <= p.seg_limit) return;  // goes through whole, from the initial state itself
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (a.s0) S = *reinterpret_cast<const f32x4*>(a.s0 + (seq * a.hv + vh) * size + at);
  constexpr int kAhead = 4;  // segments on their way
  for (int64_t s0 = 0; s0 < nseg; s0 += kAhead) {
    f32x4 own[kAhead];
    float decay[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s0 + i + 1 < nseg) {  // (nothing follows the last one)
        const int64_t slot = (base + (kRev ? nseg - 1 - s0 - i : s0 + i)) * a.hv + vh;
        own[i] = *reinterpret_cast<const f32x4*>(a.seg_state + slot * size + at);
        decay[i] = p.seg_decay[slot];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s0 + i < nseg) {
        const int64_t slot = (base + (kRev ? nseg - 1 - s0 - i : s0 + i)) * a.hv + vh;
        *reinterpret_cast<f32x4*>(a.seg_state + slot * size + at) = S;
        if (s0 + i + 1 < nseg) S = S * decay[i] + own[i];
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
  const float* g;
  void* out;
  int64_t q_stride, k_stride, v_stride;
  int64_t heads;  // sequences x hv
  int32_t hv, rep, dk, dv;
  float scale;
};

// One token of one value head and 32 columns: 8 lanes hold a row's float4s, 32 rows are held at a time, 4 per thread,
// all of them loaded before the first is used.  Bound by the state's traffic, read and written once in fp32 (256
// sequences, 80 heads of 128 x 64: 268 us, 5.0 TB/s, a copy's rate).
template <typename E>
__global__ __launch_bounds__(kStepThreads) void linear_step_kernel(StepArgs a, int32_t col_blocks) {
  constexpr int TC = 8, kStride = kStepThreads / TC, kRows = kMaxDk / kStride;
  __shared__ float sk[kMaxDk], sq[kMaxDk];
  __shared__ float red[kStepThreads / 64][4 * TC];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const uint32_t wg = wide_index();
  const int64_t sh = wg / (uint32_t)col_blocks;
  if (sh >= a.heads) return;
  const int64_t seq = sh / a.hv;
  const int vh = (int)(sh - seq * a.hv), kh = vh / a.rep;
  const int c = (int)(wg - sh * col_blocks) * 4 * TC + tid % TC * 4;
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
  if (tid < kMaxDk) {
    const bool in = tid < a.dk;
    sk[tid] = in ? ld_f32(static_cast<const E*>(a.k), seq * a.k_stride + (int64_t)kh * a.dk + tid) : 0.f;
    sq[tid] = in ? ld_f32(static_cast<const E*>(a.q), seq * a.q_stride + (int64_t)kh * a.dk + tid) : 0.f;
  }
  const float ga = exp_f32(clamp_gate(a.g[seq * a.hv + vh]));
  f32x4 v = {0.f, 0.f, 0.f, 0.f}, o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (live) v[x] = ld_f32(static_cast<const E*>(a.v), seq * a.v_stride + (int64_t)vh * a.dv + c + x);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStride;
    s[i] = s[i] * ga + v * sk[row];
    o += s[i] * sq[row];
    if (live && row < a.dk) *reinterpret_cast<f32x4*>(sp + (int64_t)row * a.dv) = s[i];
  }
  // rows of a wave, then of the workgroup
#pragma unroll
  for (int m = TC; m < 64; m *= 2)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] += __shfl_xor(o[x], m);
  if (lane < TC) *reinterpret_cast<f32x4*>(&red[w][4 * lane]) = o;
  __syncthreads();
  if (tid < 4 * TC && (int)(wg - sh * col_blocks) * 4 * TC + tid < a.dv) {
    float t = red[0][tid];
#pragma unroll
    for (int i = 1; i < kStepThreads / 64; ++i) t += red[i][tid];
    st_out(static_cast<E*>(a.out), sh * (int64_t)a.dv + (int64_t)(wg - sh * col_blocks) * 4 * TC + tid, a.scale * t);
  }
}

template <typename E>
int launch_step(const StepArgs& a, hipStream_t s) {
  const int64_t blocks = (a.dv + 31) / 32;
  hipLaunchKernelGGL((linear_step_kernel<E>), wide_grid(a.heads * blocks, kStepThreads), dim3(kStepThreads), 0, s, a,
                     (int32_t)blocks);
  return launch_status();
}

template <typename E>
int launch_forward(const PassArgs& p, hipStream_t s) {
  if (p.f.seg_chunks) {
    const int st = launch_segments(p, sizeof(E) == 2, false, s);
    if (st != MAMBA_OK) return st;
  }
  return launch_pass<E, kOutput>(p, s);
}

template <typename E, bool kRev>
int launch_segments_t(const PassArgs& p, hipStream_t s) {
  const int st = launch_pass<E, kSegmentOnly | (kRev ? kReverse : 0)>(p, s);
  if (st != MAMBA_OK) return st;
  const int blocks = (p.f.dk * p.f.dv + 1023) / 1024;
  hipLaunchKernelGGL((linear_join_kernel<kRev>), wide_grid((uint64_t)p.f.nseq * p.f.hv * blocks, 256), dim3(256), 0, s, p,
                     blocks);
  return launch_status();
}

}  // namespace

int launch_segments(const PassArgs& p, bool bf, bool reverse, hipStream_t s) {
  if (bf) return reverse ? launch_segments_t<uint16_t, true>(p, s) : launch_segments_t<uint16_t, false>(p, s);
  return reverse ? launch_segments_t<float, true>(p, s) : launch_segments_t<float, false>(p, s);
}

}  // namespace linear
}  // namespace mamba

using namespace mamba;
using namespace mamba::linear;

extern "C" {

size_t mamba_linear_attn_workspace_bytes(const mamba_delta_dims* dims, int packed) {
  if (check_delta(dims, packed != 0) != MAMBA_OK) return 0;
  return seg_layout(dims, packed != 0).total;
}

int mamba_linear_attn_fwd(const void* q, const void* k, const void* v, const float* g, const float* initial_state,
                          const int64_t* seq_offsets, float scale, void* out, float* last_state,
                          const mamba_delta_dims* dims, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_delta(dims, seq_offsets != nullptr);
  if (st != MAMBA_OK) return st;
  if (!out) return MAMBA_ERR_NULL;
  if ((st = check_linear_inputs(dims, q, k, v, g, initial_state, seq_offsets)) != MAMBA_OK) return st;
  if (!aligned(out, 16) || (last_state && !aligned(last_state, 16))) return MAMBA_ERR_ALIGN;
  const SegLayout l = seg_layout(dims, seq_offsets != nullptr);
  if (l.total && (!workspace || workspace_bytes < l.total)) return MAMBA_ERR_WORKSPACE;
  if (l.total && !aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  PassArgs p = {};
  p.f = make_args(dims, scale, q, k, v, g, nullptr, initial_state, seq_offsets);
  p.f.out = out;
  p.f.last = last_state;
  p.gate = g;
  set_segments(p, l, static_cast<char*>(workspace));
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dims->io_dtype == MAMBA_BF16 ? launch_forward<uint16_t>(p, s) : launch_forward<float>(p, s);
}

int mamba_linear_attn_update(float* state, const void* q, const void* k, const void* v, const float* g, float scale,
                             void* out, const mamba_delta_dims* dims, void* stream) {
  int st = check_delta(dims, false);
  if (st != MAMBA_OK) return st;
  if (dims->seqlen != 1) return MAMBA_ERR_SHAPE;
  if (!state || !out) return MAMBA_ERR_NULL;
  if ((st = check_linear_inputs(dims, q, k, v, g, state, nullptr)) != MAMBA_OK) return st;
  if (!aligned(out, dims->io_dtype == MAMBA_BF16 ? 2 : 4)) return MAMBA_ERR_ALIGN;
  const Args d = make_args(dims, scale, q, k, v, g, nullptr, nullptr, nullptr);
  const StepArgs a = {state, q, k, v, g, out, d.q_stride, d.k_stride, d.v_stride, dims->batch * dims->v_heads,
                      d.hv, d.rep, d.dk, d.dv, scale};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dims->io_dtype == MAMBA_BF16 ? launch_step<uint16_t>(a, s) : launch_step<float>(a, s);
}

}  // extern "C"
