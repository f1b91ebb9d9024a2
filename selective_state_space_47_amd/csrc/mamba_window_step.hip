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
constexpr int kStepHeads = 16;       // query heads that share a pass over a key head's slots: columns of a product
constexpr int64_t kStepWG = 512;     // workgroups that fill the GPU
constexpr int64_t kStepSlots = 256;  // slots of a part, at least

struct StepArgs {
  void* k_cache;
  void* v_cache;
  const void* q;
  const void* k;
  const void* v;
  const int64_t* positions;
  void* out;
  float* part;  // (parts, batch * hq, 2 + 128): maximum times log2(e), sum, unnormalised output
  int64_t q_stride, k_stride, v_stride;
  int64_t batch, slots, window, sinks;
  int32_t hq, hk, rep, dim, parts;
  float scale;
};

// One sequence, key head and part of the slots; up to 16 query heads of it are the columns of the products.  Each wave
// goes through its own tiles of slots with its own maximum and sum, without a barrier: keys come from memory as
// operands, values straight into the wave's LDS, both of a whole tile at once; the waves are joined at the end.
// Bound by the caches' traffic (read once).  The new key and value are taken from the inputs and written to their slot
// by the wave that comes to it: nobody reads that slot.  With bf16 storage the weights enter the product with V as two
// bf16 parts (2^-17 of each), so that the output's rounding is the only one that shows.  256 sequences, 20 and 4 heads of
// 128, 1024 + 4 slots, bf16: 100 us, 4.7 TB/s, a copy's rate (heads one after another on the vector unit: 221).
template <typename E, int DK>
__global__ __launch_bounds__(kStepThreads, 2) void window_step_kernel(StepArgs a, uint32_t blocks) {
  using M = Mma<E>;
  using KT = KeyTile<E, DK>;
  constexpr int kWaves = kStepThreads / 64, kSlots = sizeof(E) == 2 ? 64 : 32, kT = kSlots / 16, kV = 16 / sizeof(E);
  constexpr int kTile = kSlots * KT::kRow, kP = M::parts(2);
  static_assert(kTile >= kStepHeads * DK * 4, "a wave's output takes its tile's place");
  __shared__ __align__(1024) char smem[kWaves * kTile];
  __shared__ float sm[kWaves][kStepHeads][2];
  const uint32_t wg = wide_index();
  if (wg >= blocks) return;
  const uint32_t part = wg % (uint32_t)a.parts, rest = wg / (uint32_t)a.parts;
  const int64_t seq = rest / (uint32_t)a.hk;
  const int kh = (int)(rest - seq * a.hk);
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t p = a.positions[seq];
  const int64_t live = p < 0 ? 0 : min(p + 1, a.slots);  // slots that hold a position
  const int64_t mine = p < a.sinks ? p : a.sinks + (p - a.sinks) % a.window;
  const int64_t per = (live + a.parts - 1) / a.parts;
  const int64_t s0 = (int64_t)part * per, s1 = min(s0 + per, live);
  const int64_t row = (int64_t)a.hk * a.dim;
  E* kc = static_cast<E*>(a.k_cache) + (seq * a.slots * a.hk + kh) * (int64_t)a.dim;
  E* vc = static_cast<E*>(a.v_cache) + (seq * a.slots * a.hk + kh) * (int64_t)a.dim;
  const E* kn = static_cast<const E*>(a.k) + seq * a.k_stride + (int64_t)kh * a.dim;
  const E* vn = static_cast<const E*>(a.v) + seq * a.v_stride + (int64_t)kh * a.dim;
  char* const mem = smem + w * kTile;
  const lds_ptr sv = (lds_ptr)mem;
  const uint32_t lds = lds_address(smem) + w * kTile;
  const RowCopy<E, KT, kSlots, 1> cv(0, lane, row, a.dim);
  const KT kt(lane);
  const float sc = fabsf(a.scale) * kLog2e;
  for (int h0 = 0; h0 < a.rep; h0 += kStepHeads) {
    const int heads = min(a.rep - h0, kStepHeads);
    typename M::Frag q[DK / M::kDepth];  // column = head; a negative scale goes into the sign of q
    load_rows<E, DK>(static_cast<const E*>(a.q) + seq * a.q_stride + (int64_t)(kh * a.rep + h0) * a.dim, a.dim, r, heads,
                     a.dim, g, q);
    if (a.scale < 0.f)
#pragma unroll
      for (int kb = 0; kb < DK / M::kDepth; ++kb) q[kb] = -q[kb];
    f32x4 o[DK / 16];
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = kMinusInf, l = 0.f;
    for (int64_t s = s0 + w * kSlots; s < s1; s += kWaves * kSlots) {
      const int n = (int)min((int64_t)kSlots, s1 - s);
      cv(rows_buffer(vc + s * row, n, row, a.dim), lds, 0);  // (slots past the part read as zero)
      typename M::Frag kf[kT][DK / M::kDepth];
#pragma unroll
      for (int m = 0; m < kT; ++m) {
        const int i = 16 * m + r;
        const E* from = s + i == mine ? kn : kc + (s + i) * row;
#pragma unroll
        for (int kb = 0; kb < DK / M::kDepth; ++kb) {
          const int c = kb * M::kDepth + g * kV;
          kf[m][kb] = i < n && c < a.dim ? *reinterpret_cast<const typename M::Frag*>(from + c) : typename M::Frag{};
        }
      }
      f32x4 e[kT];
#pragma unroll
      for (int m = 0; m < kT; ++m) {
        e[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < DK / M::kDepth; ++kb) e[m] = M::mma(kf[m][kb], q[kb], e[m]);
      }
      float top = mx;
#pragma unroll
      for (int m = 0; m < kT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (16 * m + 4 * g + x >= n) e[m][x] = kMinusInf;
          top = fmaxf(top, e[m][x]);
        }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float use = top == kMinusInf ? 0.f : top * sc, f = mx == kMinusInf ? 0.f : fast_exp2(fmaf(mx, sc, -use));
      mx = top;
      l *= f;
#pragma unroll
      for (int d = 0; d < DK / 16; ++d) o[d] *= f;
#pragma unroll
      for (int m = 0; m < kT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          e[m][x] = 16 * m + 4 * g + x < n ? fast_exp2(fmaf(e[m][x], sc, -use)) : 0.f;
          l += e[m][x];
        }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's values have landed
      if (mine >= s && mine < s + n) {
        const int at = (int)(mine - s);
        if (lane * kV < a.dim) {
          const uint4 nv = *reinterpret_cast<const uint4*>(vn + lane * kV);
          *reinterpret_cast<uint4*>(mem + at * KT::kRow + ((lane ^ KT::key(at)) << 4)) = nv;
          if (h0 == 0) {
            *reinterpret_cast<uint4*>(vc + mine * row + lane * kV) = nv;
            *reinterpret_cast<uint4*>(kc + mine * row + lane * kV) = *reinterpret_cast<const uint4*>(kn + lane * kV);
          }
        }
        wave_lds_fence();
      }
#pragma unroll
      for (int kb = 0; kb < kSlots / M::kDepth; ++kb) {
        const auto f = M::template split<kP>(&e[kb * M::kTiles]);
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) {
          const auto vf = kt.cols(sv, d, kb);
#pragma unroll
          for (int x = 0; x < kP; ++x) o[d] = M::mma(vf, f.p[x], o[d]);
        }
      }
      wave_lds_fence();  // (the tile has been read)
    }
    l = across_groups(l);
    if (g == 0) {
      sm[w][r][0] = mx;
      sm[w][r][1] = l;
    }
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
      *reinterpret_cast<f32x4*>(mem + (r * DK + KT::value(d, g, 0)) * 4) = o[d];
    __syncthreads();
    for (int i = tid; i < heads * DK; i += kStepThreads) {
      const int x = i / DK, d = i % DK;
      if (d >= a.dim) continue;
      float top = kMinusInf;
#pragma unroll
      for (int y = 0; y < kWaves; ++y) top = fmaxf(top, sm[y][x][0]);
      const float use = top == kMinusInf ? 0.f : top * sc;
      float t = 0.f, v = 0.f;
#pragma unroll
      for (int y = 0; y < kWaves; ++y) {
        const float f = sm[y][x][0] == kMinusInf ? 0.f : fast_exp2(fmaf(sm[y][x][0], sc, -use));
        t = fmaf(f, sm[y][x][1], t);
        v = fmaf(f, reinterpret_cast<const float*>(smem + y * kTile)[i], v);
      }
      const int64_t head = seq * a.hq + kh * a.rep + h0 + x;
      if (a.parts == 1) {
        st_out(static_cast<E*>(a.out), head * a.dim + d, t == 0.f ? 0.f : v / t);
      } else {
        float* to = a.part + ((int64_t)part * a.batch * a.hq + head) * (2 + kMaxDk);
        to[2 + d] = v;
        if (d == 0) {
          to[0] = top == kMinusInf ? top : use;
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

template <typename E, int DK>
int launch_step(const StepArgs& a, hipStream_t s) {
  const uint32_t blocks = (uint32_t)(a.batch * a.hk * a.parts);
  hipLaunchKernelGGL((window_step_kernel<E, DK>), wide_grid(blocks, kStepThreads), dim3(kStepThreads), 0, s, a,
                     blocks);
  int st = launch_status();
  if (st != MAMBA_OK || a.parts == 1) return st;
  hipLaunchKernelGGL((window_join_kernel<E>), dim3((unsigned)(a.batch * a.hq)), dim3(64), 0, s, a);
  return launch_status();
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
    return a.dim <= 64 ? launch_step<uint16_t, 64>(a, s) : launch_step<uint16_t, 128>(a, s);
  return a.dim <= 64 ? launch_step<float, 64>(a, s) : launch_step<float, 128>(a, s);
}

}  // extern "C"
