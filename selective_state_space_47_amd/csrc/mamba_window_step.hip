// mamba_window_step.hip -- attention with a sliding window and sinks on gfx950: one generation step against the ring
// caches, and the caches filled from a prompt's keys and values.
//
// Position p lies in slot p below `sinks` and in slot sinks + (p - sinks) mod window from there on, so that the slots
// of a sequence hold, without an order that matters, exactly what its newest query sees.
#include "mamba_window.h"

namespace mamba {
namespace window {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepHeads = 8;        // query heads that share a pass over a key head's slots
constexpr int64_t kStepWG = 1024;    // workgroups that fill the GPU
constexpr int64_t kStepSlots = 128;  // slots of a part, at least

struct StepArgs {
  void* k_cache;
  void* v_cache;
  const void* q;
  const void* k;
  const void* v;
  const int64_t* positions;
  void* out;
  float* part;  // (parts, batch * hq, 2 + 128): maximum, sum, unnormalised output
  int64_t q_stride, k_stride, v_stride;
  int64_t batch, slots, window, sinks;
  int32_t hq, hk, rep, dim, parts;
  float scale;
};

template <typename E>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack(u[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// sum over the T lanes of a slot, in each of them
template <int T>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (T == 16) {
    v += dpp_row<0x128>(v);
    v += dpp_row<0x124>(v);
    v += dpp_row<0x122>(v);
    v += dpp_row<0x121>(v);
  } else {
    v += dpp_row<0xb1>(v);   // lane ^ 1
    v += dpp_row<0x4e>(v);   // lane ^ 2
    v += dpp_row<0x141>(v);  // half row mirrored
  }
  return v;
}

// One sequence, key head and part of the slots; R query heads of it at a time.  T lanes hold a slot's key and value,
// 8 values each, so that a wave reads 64 / T slots at once, kAhead of those on their way; each group of lanes
// goes through its own slots with its own maximum and sum, which are joined at the end.  Bound by the caches'
// traffic (read once; fp32 arithmetic).  The new key and value are taken from the inputs and written to their slot
// by the lanes that come to it: nobody reads that slot.
template <typename E, int T, int R>
__global__ __launch_bounds__(kStepThreads) void window_step_kernel(StepArgs a, uint32_t blocks) {
  constexpr int kGroups = kStepThreads / T, kAhead = 4, kWaves = kStepThreads / 64;
  __shared__ float sm[kWaves][R][2], so[kWaves][R][8 * T];
  const uint32_t wg = wide_index();
  if (wg >= blocks) return;
  const uint32_t part = wg % (uint32_t)a.parts, rest = wg / (uint32_t)a.parts;
  const int64_t seq = rest / (uint32_t)a.hk;
  const int kh = (int)(rest - seq * a.hk);
  const int tid = threadIdx.x, l = tid % T, grp = tid / T, lane = tid & 63, w = tid >> 6;
  const int c = 8 * l;
  const bool has = c < a.dim;
  const int64_t p = a.positions[seq];
  const int64_t live = p < 0 ? 0 : min(p + 1, a.slots);  // slots that hold a position
  const int64_t mine = p < a.sinks ? p : a.sinks + (p - a.sinks) % a.window;
  const int64_t per = (live + a.parts - 1) / a.parts;
  const int64_t s0 = (int64_t)part * per, s1 = min(s0 + per, live);
  const int64_t row = (int64_t)a.hk * a.dim;
  E* kc = static_cast<E*>(a.k_cache) + (seq * a.slots * a.hk + kh) * (int64_t)a.dim + c;
  E* vc = static_cast<E*>(a.v_cache) + (seq * a.slots * a.hk + kh) * (int64_t)a.dim + c;
  const E* kn = static_cast<const E*>(a.k) + seq * a.k_stride + (int64_t)kh * a.dim + c;
  const E* vn = static_cast<const E*>(a.v) + seq * a.v_stride + (int64_t)kh * a.dim + c;
  for (int h0 = 0; h0 < a.rep; h0 += R) {
    float q[R][8], o[R][8], m[R], sum[R];
#pragma unroll
    for (int x = 0; x < R; ++x) {
      m[x] = kMinusInf;
      sum[x] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q[x][i] = o[x][i] = 0.f;
      if (has && h0 + x < a.rep) {
        Vec8<E> v;
        v.load(static_cast<const E*>(a.q) + seq * a.q_stride + (int64_t)(kh * a.rep + h0 + x) * a.dim + c);
        v.get(q[x]);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[x][i] *= a.scale * kLog2e;
      }
    }
    for (int64_t s = s0 + grp; s < s1; s += kAhead * kGroups) {
      Vec8<E> kv[kAhead], vv[kAhead];
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        const int64_t at = s + y * kGroups;
        kv[y].zero();
        vv[y].zero();
        if (has && at < s1) {
          const bool now = at == mine;
          kv[y].load(now ? kn : kc + at * row);
          vv[y].load(now ? vn : vc + at * row);
        }
      }
      float e[R][kAhead];
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        float kf[8];
        kv[y].get(kf);
#pragma unroll
        for (int x = 0; x < R; ++x) {
          float d = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) d = fmaf(q[x][i], kf[i], d);
          d = lanes_sum<T>(d);
          e[x][y] = s + y * kGroups < s1 ? d : kMinusInf;
        }
      }
#pragma unroll
      for (int x = 0; x < R; ++x) {
        float top = m[x];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) top = fmaxf(top, e[x][y]);
        const float use = top == kMinusInf ? 0.f : top, f = fast_exp2(m[x] - use);
        m[x] = top;
        sum[x] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[x][i] *= f;
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          e[x][y] = fast_exp2(e[x][y] - use);
          sum[x] += e[x][y];
        }
      }
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        float vf[8];
        vv[y].get(vf);
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
          for (int i = 0; i < 8; ++i) o[x][i] = fmaf(e[x][y], vf[i], o[x][i]);
      }
      if (h0 == 0)
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
          if (has && s + y * kGroups == mine) {
            kv[y].store(kc + mine * row);
            vv[y].store(vc + mine * row);
          }
    }
    // groups of a wave, then waves
#pragma unroll
    for (int x = 0; x < R; ++x) {
#pragma unroll
      for (int d = T; d < 64; d *= 2) {
        const float mo = __shfl_xor(m[x], d), so_ = __shfl_xor(sum[x], d);
        const float top = fmaxf(m[x], mo), use = top == kMinusInf ? 0.f : top;
        const float fa = fast_exp2(m[x] - use), fb = fast_exp2(mo - use);
        sum[x] = sum[x] * fa + so_ * fb;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[x][i] = o[x][i] * fa + __shfl_xor(o[x][i], d) * fb;
        m[x] = top;
      }
      if (lane < T) {
#pragma unroll
        for (int i = 0; i < 8; ++i) so[w][x][c + i] = o[x][i];
        if (lane == 0) {
          sm[w][x][0] = m[x];
          sm[w][x][1] = sum[x];
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < R * 8 * T; i += kStepThreads) {
      const int x = i / (8 * T), d = i % (8 * T);
      if (h0 + x >= a.rep || d >= a.dim) continue;
      float top = kMinusInf;
#pragma unroll
      for (int y = 0; y < kWaves; ++y) top = fmaxf(top, sm[y][x][0]);
      const float use = top == kMinusInf ? 0.f : top;
      float t = 0.f, v = 0.f;
#pragma unroll
      for (int y = 0; y < kWaves; ++y) {
        const float f = fast_exp2(sm[y][x][0] - use);
        t = fmaf(f, sm[y][x][1], t);
        v = fmaf(f, so[y][x][d], v);
      }
      const int64_t head = seq * a.hq + kh * a.rep + h0 + x;
      if (a.parts == 1) {
        st_out(static_cast<E*>(a.out), head * a.dim + d, t == 0.f ? 0.f : v / t);
      } else {
        float* to = a.part + ((int64_t)part * a.batch * a.hq + head) * (2 + kMaxDk);
        to[2 + d] = v;
        if (d == 0) {
          to[0] = top;
          to[1] = t;
        }
      }
    }
    __syncthreads();  // before the next heads' sums
  }
}

// The parts of one sequence and head, in order: a lane has two values.
template <typename E>
__global__ __launch_bounds__(64) void window_join_kernel(StepArgs a) {
  const int64_t head = blockIdx.x, all = a.batch * a.hq;
  const float* from = a.part + head * (2 + kMaxDk);
  const int64_t step = all * (2 + kMaxDk);
  float top = kMinusInf;
  for (int y = 0; y < a.parts; ++y) top = fmaxf(top, from[y * step]);
  const float use = top == kMinusInf ? 0.f : top;
  float t = 0.f, v[2] = {0.f, 0.f};
  const int d = threadIdx.x;
  for (int y = 0; y < a.parts; ++y) {
    const float f = fast_exp2(from[y * step] - use);
    t = fmaf(f, from[y * step + 1], t);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (d + 64 * i < a.dim) v[i] = fmaf(f, from[y * step + 2 + d + 64 * i], v[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (d + 64 * i < a.dim) st_out(static_cast<E*>(a.out), head * a.dim + d + 64 * i, t == 0.f ? 0.f : v[i] / t);
}

// A thread per 16 bytes of a slot: the last position of the sequence that lies there.
__global__ __launch_bounds__(256) void window_store_kernel(WinArgs a, char* k_cache, char* v_cache, int32_t words,
                                                           int32_t esize, uint64_t total) {
  const uint64_t id = (uint64_t)wide_index() * 256 + threadIdx.x;
  if (id >= total) return;
  const int64_t slots = a.window + a.sinks;
  const int64_t slot_at = (int64_t)(id / (uint64_t)words);
  const int word = (int)(id - (uint64_t)slot_at * words);
  const int64_t seq = slot_at / slots, slot = slot_at - seq * slots;
  const Seq ks = seq_of(a.kv_offsets, a.kv_len, seq);
  int64_t p = slot;
  if (slot >= a.sinks) {
    const int64_t last = ks.len - 1 - a.sinks, i = slot - a.sinks;  // behind the sinks
    if (last < i) return;
    p = a.sinks + last - (last - i) % a.window;
  }
  if (p >= ks.len) return;
  const int64_t to = slot_at * words + word;
  reinterpret_cast<uint4*>(k_cache)[to] = *reinterpret_cast<const uint4*>(
      static_cast<const char*>(a.k) + (ks.first + p) * a.k_stride * esize + 16 * (int64_t)word);
  reinterpret_cast<uint4*>(v_cache)[to] = *reinterpret_cast<const uint4*>(
      static_cast<const char*>(a.v) + (ks.first + p) * a.v_stride * esize + 16 * (int64_t)word);
}

// Parts that a sequence's slots are split into: where sequences and key heads alone leave CUs idle.
int32_t step_parts(const mamba_window_dims* d) {
  const int64_t wgs = d->batch * d->kv_heads, slots = d->window + d->sinks;
  return (int32_t)std::max<int64_t>(
      1, std::min<int64_t>({(slots + kStepSlots - 1) / kStepSlots, kStepWG / std::max<int64_t>(wgs, 1), 256}));
}

template <typename E, int T, int R>
int launch_step_t(const StepArgs& a, hipStream_t s) {
  const uint32_t blocks = (uint32_t)(a.batch * a.hk * a.parts);
  hipLaunchKernelGGL((window_step_kernel<E, T, R>), wide_grid(blocks, kStepThreads), dim3(kStepThreads), 0, s, a,
                     blocks);
  int st = launch_status();
  if (st != MAMBA_OK || a.parts == 1) return st;
  hipLaunchKernelGGL((window_join_kernel<E>), dim3((unsigned)(a.batch * a.hq)), dim3(64), 0, s, a);
  return launch_status();
}
template <typename E, int T>
int launch_step(const StepArgs& a, hipStream_t s) {
  if (a.rep == 1) return launch_step_t<E, T, 1>(a, s);
  if (a.rep == 2) return launch_step_t<E, T, 2>(a, s);
  if (a.rep <= 4) return launch_step_t<E, T, 4>(a, s);
  return launch_step_t<E, T, kStepHeads>(a, s);
}

int check_cache(const mamba_window_dims* d) {
  // every slot of every sequence is addressed: the caches' size is bounded like a tensor's
  const double size = (double)d->batch * ((double)d->window + (double)d->sinks) * (double)(d->kv_heads * d->dim);
  return size > 1099511627776.0 ? MAMBA_ERR_SHAPE : MAMBA_OK;
}

}  // namespace
}  // namespace window
}  // namespace mamba

using namespace mamba;
using namespace mamba::window;

extern "C" {

int mamba_window_cache_store(const void* k, const void* v, const int64_t* kv_offsets, void* k_cache, void* v_cache,
                             const mamba_window_dims* dims, void* stream) {
  if (!dims) return MAMBA_ERR_NULL;
  mamba_window_dims d = *dims;  // (seqlen, q_heads and q's stride do not count)
  d.seqlen = 1;
  d.q_heads = d.kv_heads;
  d.q_stride = 0;
  int st = check_window(&d, kv_offsets != nullptr);
  if (st == MAMBA_OK) st = check_cache(&d);
  if (st != MAMBA_OK) return st;
  if (!k || !v || !k_cache || !v_cache) return MAMBA_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      (kv_offsets && !aligned(kv_offsets, 8)))
    return MAMBA_ERR_ALIGN;
  const WinArgs a = window_args(&d, 1.f, k, k, v, kv_offsets, kv_offsets);
  const int32_t es = d.io_dtype == MAMBA_BF16 ? 2 : 4, words = (int32_t)(d.kv_heads * d.dim * es / 16);
  const uint64_t total = (uint64_t)d.batch * (uint64_t)(d.window + d.sinks) * (uint64_t)words;
  hipLaunchKernelGGL(window_store_kernel, wide_grid((total + 255) / 256, 256), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a, static_cast<char*>(k_cache), static_cast<char*>(v_cache),
                     words, es, total);
  return launch_status();
}

size_t mamba_window_attn_update_workspace_bytes(const mamba_window_dims* dims) {
  if (check_window(dims, false) != MAMBA_OK || check_cache(dims) != MAMBA_OK || dims->seqlen != 1 || dims->kv_len != 1)
    return 0;
  const int32_t parts = step_parts(dims);
  return parts == 1 ? 0 : (size_t)parts * (size_t)(dims->batch * dims->q_heads) * (2 + kMaxDk) * sizeof(float);
}

int mamba_window_attn_update(void* k_cache, void* v_cache, const void* q, const void* k, const void* v,
                             const int64_t* positions, float scale, void* out, const mamba_window_dims* dims,
                             void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_window(dims, false);
  if (st == MAMBA_OK) st = check_cache(dims);
  if (st != MAMBA_OK) return st;
  if (dims->seqlen != 1 || dims->kv_len != 1) return MAMBA_ERR_SHAPE;
  if (!k_cache || !v_cache || !positions || !out) return MAMBA_ERR_NULL;
  if ((st = check_window_inputs(q, k, v, nullptr, nullptr)) != MAMBA_OK) return st;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(positions, 8) ||
      !aligned(out, dims->io_dtype == MAMBA_BF16 ? 2 : 4))
    return MAMBA_ERR_ALIGN;
  const size_t need = mamba_window_attn_update_workspace_bytes(dims);
  if (need && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return MAMBA_ERR_ALIGN;
  const WinArgs w = window_args(dims, scale, q, k, v, nullptr, nullptr);
  StepArgs a = {};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  a.q_stride = w.q_stride;
  a.k_stride = w.k_stride;
  a.v_stride = w.v_stride;
  a.batch = dims->batch;
  a.slots = dims->window + dims->sinks;
  a.window = dims->window;
  a.sinks = dims->sinks;
  a.hq = w.hq;
  a.hk = w.hk;
  a.rep = w.rep;
  a.dim = w.dim;
  a.parts = step_parts(dims);
  a.scale = scale;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dims->io_dtype == MAMBA_BF16)
    return a.dim <= 64 ? launch_step<uint16_t, 8>(a, s) : launch_step<uint16_t, 16>(a, s);
  return a.dim <= 64 ? launch_step<float, 8>(a, s) : launch_step<float, 16>(a, s);
}

}  // extern "C"
