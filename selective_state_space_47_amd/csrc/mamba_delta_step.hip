// mamba_delta_step.hip -- one generation step of the gated delta rule on gfx950 (formulas in mamba_delta.h).
#include "mamba_delta.h"
#include "mamba_grid.h"

namespace mamba {
namespace delta {
namespace {

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
  int64_t heads;  // sequences x hv
  int32_t hv, rep, dk, dv;
  float scale;
};

// One token of one value head and 32 columns: 8 lanes hold a row's float4s, 32 rows are held at a time, 4 per
// thread, all of them loaded before the first is used.  Bound by the state's traffic (read and written once,
// fp32): with a = exp(g), both dots go through the old state in one pass,
//     x = a S^T k,  e = v - x,  o = scale (a S^T q + beta (k . q) e),  S <- a S + beta k e^T,
// so that one reduction across the rows' lanes serves both.  256 tokens x 40 heads of 128 x 128: 270 us,
// 5.0 TB/s, what a copy of that size reaches; 12 heads: 4 us, latency.  (128 columns
// per workgroup are no faster at either end, and leave lanes idle below 128.)
template <typename E>
__global__ __launch_bounds__(kStepThreads) void step_kernel(StepArgs a, int32_t col_blocks) {
  constexpr int TC = 8, kStride = kStepThreads / TC, kRows = kMaxDk / kStride;
  __shared__ float sk[kMaxDk], sq[kMaxDk];
  __shared__ float red[kStepThreads / 64][2][4 * TC];
  __shared__ float skq[2];
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
int launch_step(const StepArgs& a, hipStream_t s) {
  const int64_t blocks = (a.dv + 31) / 32;
  hipLaunchKernelGGL((step_kernel<E>), wide_grid(a.heads * blocks, kStepThreads), dim3(kStepThreads), 0, s, a,
                     (int32_t)blocks);
  return launch_status();
}

}  // namespace
}  // namespace delta
}  // namespace mamba

using namespace mamba;
using namespace mamba::delta;

extern "C" {

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
                dims->batch * dims->v_heads, d.hv, d.rep, d.dk, d.dv, scale};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dims->io_dtype == MAMBA_BF16 ? launch_step<uint16_t>(a, s) : launch_step<float>(a, s);
}

}  // extern "C"
