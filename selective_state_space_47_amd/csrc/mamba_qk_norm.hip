// mamba_qk_norm.hip -- the RMS norm of queries and keys per head with the position rotation in the same pass on
// gfx950, forward and gradients.  Per row (token) and head of `dim` values x, weight w (one for queries, one for keys):
//     h = x rsqrt(mean(x^2) + eps) w
//     pairs (h_i, h_{i + R/2}), or (h_2i, h_{2i+1}), i < R/2, turned by the angle position * inv_freq_i
//     out = (h_i cos - h_j sin, h_j cos + h_i sin);  values from R on as they are
// and with dh the gradient turned back:
//     a = dh w,  n = x rs,  dx = rs (a - n mean(a n)),  dw = sum dh n        (rs the inverse root)
//
// Bound by memory: each value is read and written once.  A lane holds both values of its eight pairs, so that the
// rotation needs no exchange: a head of 128 is a team of 8 lanes, 16 values each.  The cosines and sines of a
// workgroup's rows are made once for all heads, in LDS: the angle in turns is a product in fp64 less its nearest
// integer (a position of a million at one radian each would leave fp32 two digits), its sine and cosine fp32.
// The weights' gradients are partial rows, one per workgroup, added by a second launch in a fixed order: no atomics.
// 16384 rows, 20 and 4 heads of 128, bf16: 33 us (6.0 TB/s, some of it from the caches), gradients 87 (3.4 TB/s: some of
// a copy's rate is lost to the conversions and sums, the vector unit is busy 67% of the time) and 5.
#include "mamba_common.h"
#include "mamba_grid.h"

namespace mamba {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 256;
constexpr int64_t kQkMaxHeads = 65535, kQkMaxRows = 0x7fffffff;
constexpr int kQkRows = 4;          // rows of a workgroup's table
constexpr int64_t kQkBwdWG = 1024;  // workgroups of a gradient launch
constexpr int kQkFoldCols = 32;     // columns of a workgroup that adds partial rows

struct QkArgs {
  const void* x[2];        // queries, keys
  const float* w[2];
  const void* dout[2];     // gradients only
  void* out[2];            // outputs, or the inputs' gradients
  const int64_t* pos;
  const double* freq;      // radians per position
  float* part;             // partial weight gradients: (workgroups, dim)
  int64_t rows, x_stride[2];
  uint32_t split;          // gradients: workgroups of the queries
  int32_t heads[2], dim, rotary;
  float eps;
};

// 8 values as they are stored, at a 16-byte aligned address (those on their way take no more registers)
template <typename E>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p, bool in) {
    w = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack(u[k]);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool in) {
    a = in ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    b = in ? *reinterpret_cast<const float4*>(p + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <typename E>
using Pair = Vec8<E>[2];
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(make_float2(v[0], v[1])), pack_bf16(make_float2(v[2], v[3])),
                 pack_bf16(make_float2(v[4], v[5])), pack_bf16(make_float2(v[6], v[7])));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// A lane's two vectors of a head: where they begin, whether they exist, whether their pairs turn.  Halves: vector
// a of the first half with the same of the second, then the unturned rest two by two.  Interleaved: two vectors
// one after the other, whose own neighbours are pairs.
template <int T, bool kInter>
struct Lane {
  int l, a, b;
  bool has_a, has_b, turns;
  __device__ __forceinline__ Lane(const QkArgs& q) : l(threadIdx.x % T) {
    const int pairs = q.rotary / 16;  // lanes that turn 8 pairs each
    turns = l < pairs;
    if (kInter) {
      a = 16 * l;
      b = a + 8;
    } else {
      a = turns ? 8 * l : q.rotary + 16 * (l - pairs);
      b = turns ? q.rotary / 2 + a : a + 8;
    }
    has_a = a < q.dim;
    has_b = b < q.dim;
  }
  template <typename E>
  __device__ __forceinline__ void load(const E* p, Pair<E>& v, bool in = true) const {
    v[0].load(p + a, in && has_a);
    v[1].load(p + b, in && has_b);
  }
  __device__ __forceinline__ void load(const float* p, float (&v)[2][8]) const {
    Pair<float> x;
    load(p, x);
    get<float>(x, v);
  }
  template <typename E>
  __device__ __forceinline__ void get(const Pair<E>& x, float (&v)[2][8]) const {
    x[0].get(v[0]);
    x[1].get(v[1]);
  }
  template <typename E>
  __device__ __forceinline__ void store(E* p, const float (&v)[2][8]) const {
    if (has_a) store8(p + a, v[0]);
    if (has_b) store8(p + b, v[1]);
  }
  // turn by the table's angle (sign 1) or back (-1)
  __device__ __forceinline__ void turn(const float2* row, float sign, float (&v)[2][8]) const {
    if (!turns) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 cs = row[8 * l + k];
      const float s = sign * cs.y;
      float& x = kInter ? v[k >> 2][2 * (k & 3)] : v[0][k];
      float& y = kInter ? v[k >> 2][2 * (k & 3) + 1] : v[1][k];
      const float t = x;
      x = fmaf(x, cs.x, -y * s);
      y = fmaf(y, cs.x, t * s);
    }
  }
};

// Sum over the T lanes of a team, in every one of them, by lane permutations inside a row of 16.
template <int T>
__device__ __forceinline__ float team_sum(float v) {
  if constexpr (T == 16) {
    v += dpp_row<0x128>(v);
    v += dpp_row<0x124>(v);
    v += dpp_row<0x122>(v);
    v += dpp_row<0x121>(v);
  } else {
    v += dpp_row<0xb1>(v);                         // lane ^ 1
    v += dpp_row<0x4e>(v);                         // lane ^ 2
    if constexpr (T == 8) v += dpp_row<0x141>(v);  // half row mirrored
  }
  return v;
}
template <int T>
__device__ __forceinline__ double team_sum(double v) {
  auto add = [&](auto other) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __float_as_uint(other(__uint_as_float((uint32_t)b)));
    const uint32_t hi = __float_as_uint(other(__uint_as_float((uint32_t)(b >> 32))));
    v += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  if constexpr (T == 16) {
    add([](float x) { return dpp_row<0x128>(x); });
    add([](float x) { return dpp_row<0x124>(x); });
    add([](float x) { return dpp_row<0x122>(x); });
    add([](float x) { return dpp_row<0x121>(x); });
  } else {
    add([](float x) { return dpp_row<0xb1>(x); });
    add([](float x) { return dpp_row<0x4e>(x); });
    if constexpr (T == 8) add([](float x) { return dpp_row<0x141>(x); });
  }
  return v;
}

// cosines and sines of rows row0 .. row0 + n - 1
__device__ __forceinline__ void angles(const QkArgs& a, int64_t row0, int n, float2 (*table)[kQkMaxDim / 2]) {
  const int half = a.rotary / 2;
  for (int i = threadIdx.x; i < n * half; i += kQkThreads) {
    const int r = i / half, p = i - r * half;
    const double turns = (double)a.pos[row0 + r] * (a.freq[p] * 0.15915494309189533577);
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    table[r][p] = make_float2(c, s);
  }
}

template <typename E, int T, bool kInter>
__global__ __launch_bounds__(kQkThreads) void qk_norm_kernel(QkArgs a, int32_t per) {
  __shared__ float2 table[kQkRows][kQkMaxDim / 2];
  const Lane<T, kInter> lane(a);
  const int64_t row0 = (int64_t)wide_index() * per;
  if (row0 >= a.rows) return;
  const int n = (int)min((int64_t)per, a.rows - row0);
  const int heads = a.heads[0] + a.heads[1], units = n * heads;
  // a unit's values are read a turn ahead, the first before the angles are made (lanes of one team run together)
  Pair<E> ahead;
  auto load = [&](int u) {
    const int r = u / heads, h = u - r * heads, key = h >= a.heads[0], hh = key ? h - a.heads[0] : h;
    lane.load(static_cast<const E*>(a.x[key]) + (row0 + r) * a.x_stride[key] + (int64_t)hh * a.dim, ahead, u < units);
  };
  load(threadIdx.x / T);
  angles(a, row0, n, table);
  __syncthreads();
  for (int u = threadIdx.x / T; u < units; u += kQkThreads / T) {
    const int r = u / heads, h = u - r * heads;
    const int key = h >= a.heads[0];
    const int hh = key ? h - a.heads[0] : h;
    const int64_t row = row0 + r;
    float v[2][8], w[2][8];
    lane.template get<E>(ahead, v);
    load(u + kQkThreads / T);
    lane.load(a.w[key], w);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(v[i >> 3][i & 7], v[i >> 3][i & 7], s);
    const float rs = rsqrtf(team_sum<T>(s) / a.dim + a.eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] *= rs * w[i >> 3][i & 7];
    lane.turn(table[r], 1.f, v);
    lane.store(static_cast<E*>(a.out[key]) + (row * a.heads[key] + hh) * (int64_t)a.dim, v);
  }
}

// A workgroup takes rows of the queries or of the keys, so that its weight sums are of one kind.
template <typename E, int T, bool kInter>
__global__ __launch_bounds__(kQkThreads, sizeof(E) == 2 ? 4 : 3) void qk_norm_bwd_kernel(QkArgs a) {
  __shared__ float2 table[kQkRows][kQkMaxDim / 2];
  __shared__ float sum[kQkThreads / 64][kQkMaxDim];
  const Lane<T, kInter> lane(a);
  const int key = blockIdx.x >= a.split;
  const uint32_t wg = key ? blockIdx.x - a.split : blockIdx.x, wgs = key ? gridDim.x - a.split : a.split;
  const int heads = a.heads[key];
  float w[2][8], acc[2][8];
  lane.load(a.w[key], w);
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i >> 3][i & 7] = 0.f;
  const double inv = 1.0 / a.dim;
  Pair<E> ax, ad;  // a unit's values a turn ahead
  auto load = [&](int64_t row0, int u, int units) {
    const int r = u / heads, h = u - r * heads;
    const int64_t row = row0 + r;
    lane.load(static_cast<const E*>(a.x[key]) + row * a.x_stride[key] + (int64_t)h * a.dim, ax, u < units);
    lane.load(static_cast<const E*>(a.dout[key]) + (row * heads + h) * (int64_t)a.dim, ad, u < units);
  };
  for (int64_t row0 = (int64_t)wg * kQkRows; row0 < a.rows; row0 += (int64_t)wgs * kQkRows) {
    const int n = (int)min((int64_t)kQkRows, a.rows - row0), units = n * heads;
    load(row0, threadIdx.x / T, units);
    __syncthreads();  // the table of the rows before has been read
    angles(a, row0, n, table);
    __syncthreads();
#pragma unroll 1
    for (int u = threadIdx.x / T; u < units; u += kQkThreads / T) {
      const int r = u / heads, h = u - r * heads;
      const int64_t row = row0 + r, at = (row * heads + h) * (int64_t)a.dim;
      float x[2][8], d[2][8];
      lane.template get<E>(ax, x);
      lane.template get<E>(ad, d);
      load(row0, u + kQkThreads / T, units);
      lane.turn(table[r], -1.f, d);
      // statistics in fp64: next to nothing is left of a where it is nearly parallel to n
      double sq = 0.0, dot = 0.0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double v = x[i >> 3][i & 7];
        sq = fma(v, v, sq);
        dot = fma((double)(d[i >> 3][i & 7] * w[i >> 3][i & 7]), v, dot);
      }
      sq = team_sum<T>(sq);
      dot = team_sum<T>(dot);
      const double ms = fma(sq, inv, (double)a.eps), r2 = 1.0 / ms;
      const float rs = ms > 1e-37 && ms < 1e37 ? rsqrtf((float)ms) : (float)(1.0 / sqrt(ms));
      const double m = dot * r2 * inv;
      // (opaque: the values are widened again rather than kept wide, which would take 64 registers more)
#pragma unroll
      for (int i = 0; i < 16; ++i) asm("" : "+v"(x[i >> 3][i & 7]), "+v"(d[i >> 3][i & 7]));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float& v = x[i >> 3][i & 7];
        const float e = d[i >> 3][i & 7];
        acc[i >> 3][i & 7] = fmaf(e, v * rs, acc[i >> 3][i & 7]);
        v = rs * (float)fma(-(double)v, m, (double)(e * w[i >> 3][i & 7]));
      }
      lane.store(static_cast<E*>(a.out[key]) + at, x);
    }
  }
  // teams of a wave, then its waves
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float& v = acc[i >> 3][i & 7];
#pragma unroll
    for (int m = T; m < 64; m *= 2) v += __shfl_xor(v, m);
  }
  if ((threadIdx.x & 63) < T) lane.store(sum[threadIdx.x >> 6], acc);
  __syncthreads();
  for (int c = threadIdx.x; c < a.dim; c += kQkThreads) {
    float t = sum[0][c];
#pragma unroll
    for (int i = 1; i < kQkThreads / 64; ++i) t += sum[i][c];
    a.part[(int64_t)blockIdx.x * a.dim + c] = t;
  }
}

// Column sums of the partial rows; y: queries' rows [0, split), keys' [split, wgs).
__global__ __launch_bounds__(1024) void qk_fold_kernel(const float* part, float* dwq, float* dwk, int split, int wgs,
                                                       int dim) {
  constexpr int kLanes = 1024 / kQkFoldCols;
  __shared__ double s[kLanes][kQkFoldCols + 1];
  const int c = threadIdx.x % kQkFoldCols, l = threadIdx.x / kQkFoldCols;
  const int col = blockIdx.x * kQkFoldCols + c;
  const int first = blockIdx.y ? split : 0, end = blockIdx.y ? wgs : split;
  double t = 0.0;
  if (col < dim) {
#pragma unroll 8
    for (int r = first + l; r < end; r += kLanes) t += (double)part[(int64_t)r * dim + col];
  }
  s[l][c] = t;
  __syncthreads();
  if (l == 0 && col < dim) {
    for (int i = 1; i < kLanes; ++i) t += s[i][c];
    (blockIdx.y ? dwk : dwq)[col] = (float)t;
  }
}

int check_qk(const mamba_qk_norm_rope_dims* d) {
  if (!d) return MAMBA_ERR_NULL;
  if (d->io_dtype != MAMBA_F32 && d->io_dtype != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (d->rows < 1 || d->q_heads < 1 || d->k_heads < 1 || d->dim < 1 || d->rotary_dim < 0)
    return MAMBA_ERR_SHAPE;
  if (d->dim % 8 || d->dim > kQkMaxDim || d->rotary_dim % 16 || d->rotary_dim > d->dim)
    return MAMBA_ERR_UNSUPPORTED;
  if (d->rows > kQkMaxRows || d->q_heads > kQkMaxHeads || d->k_heads > kQkMaxHeads) return MAMBA_ERR_SHAPE;
  const int64_t lim = (int64_t)1 << 32, vec = d->io_dtype == MAMBA_BF16 ? 8 : 4;
  const int64_t s[2] = {d->q_stride, d->k_stride}, w[2] = {d->q_heads * d->dim, d->k_heads * d->dim};
  for (int i = 0; i < 2; ++i) {
    if ((s[i] && s[i] < w[i]) || s[i] > lim) return MAMBA_ERR_SHAPE;
    if (s[i] % vec) return MAMBA_ERR_ALIGN;
  }
  return MAMBA_OK;
}

int check_qk_inputs(const mamba_qk_norm_rope_dims* d, const void* q, const void* k, const float* qw, const float* kw,
                    const int64_t* pos, const double* freq, float eps) {
  if (!q || !k || !qw || !kw || (d->rotary_dim && (!pos || !freq))) return MAMBA_ERR_NULL;
  if (!(eps >= 0.f && eps < 3e38f)) return MAMBA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(qw, 16) || !aligned(kw, 16) || (pos && !aligned(pos, 8)) ||
      (freq && !aligned(freq, 8)))
    return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

QkArgs qk_args(const mamba_qk_norm_rope_dims* d, const void* q, const void* k, const float* qw, const float* kw,
               const int64_t* pos, const double* freq, float eps) {
  QkArgs a = {};
  a.x[0] = q;
  a.x[1] = k;
  a.w[0] = qw;
  a.w[1] = kw;
  a.pos = pos;
  a.freq = freq;
  a.rows = d->rows;
  a.heads[0] = (int32_t)d->q_heads;
  a.heads[1] = (int32_t)d->k_heads;
  a.x_stride[0] = d->q_stride ? d->q_stride : d->q_heads * d->dim;
  a.x_stride[1] = d->k_stride ? d->k_stride : d->k_heads * d->dim;
  a.dim = (int32_t)d->dim;
  a.rotary = (int32_t)d->rotary_dim;
  a.eps = eps;
  return a;
}

// Gradient launch: workgroups of the queries and of all, in proportion to their work.
struct QkGrid {
  uint32_t split, all;
};
QkGrid qk_grid(const mamba_qk_norm_rope_dims* d) {
  const int64_t most = (d->rows + kQkRows - 1) / kQkRows;
  const double share = (double)d->q_heads / (double)(d->q_heads + d->k_heads);
  const int64_t q = std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)(share * kQkBwdWG)));
  const int64_t k = std::max<int64_t>(1, std::min<int64_t>(most, kQkBwdWG - (int64_t)(share * kQkBwdWG)));
  return {(uint32_t)q, (uint32_t)(q + k)};
}

template <typename E, int T, bool kInter>
int launch_qk_t(const QkArgs& a, bool bwd, QkGrid grid, hipStream_t s) {
  if (bwd) {
    hipLaunchKernelGGL((qk_norm_bwd_kernel<E, T, kInter>), dim3(grid.all), dim3(kQkThreads), 0, s, a);
  } else {
    // few rows: a workgroup each
    const int per = a.rows >= 1024 ? kQkRows : 1;
    hipLaunchKernelGGL((qk_norm_kernel<E, T, kInter>), wide_grid((uint64_t)((a.rows + per - 1) / per), kQkThreads),
                       dim3(kQkThreads), 0, s, a, per);
  }
  return launch_status();
}
template <typename E, bool kInter>
int launch_qk_d(const QkArgs& a, bool bwd, QkGrid grid, hipStream_t s) {
  if (a.dim <= 64) return launch_qk_t<E, 4, kInter>(a, bwd, grid, s);
  if (a.dim <= 128) return launch_qk_t<E, 8, kInter>(a, bwd, grid, s);
  return launch_qk_t<E, 16, kInter>(a, bwd, grid, s);
}
int launch_qk(const QkArgs& a, const mamba_qk_norm_rope_dims* d, bool bwd, QkGrid grid, hipStream_t s) {
  if (d->io_dtype == MAMBA_BF16)
    return d->interleaved ? launch_qk_d<uint16_t, true>(a, bwd, grid, s) : launch_qk_d<uint16_t, false>(a, bwd, grid, s);
  return d->interleaved ? launch_qk_d<float, true>(a, bwd, grid, s) : launch_qk_d<float, false>(a, bwd, grid, s);
}

}  // namespace
}  // namespace mamba

using namespace mamba;

extern "C" {

int mamba_qk_norm_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                           const int64_t* positions, const double* inv_freq, float eps, void* q_out, void* k_out,
                           const mamba_qk_norm_rope_dims* dims, void* stream) {
  int st = check_qk(dims);
  if (st != MAMBA_OK) return st;
  if (!q_out || !k_out) return MAMBA_ERR_NULL;
  if ((st = check_qk_inputs(dims, q, k, q_weight, k_weight, positions, inv_freq, eps)) != MAMBA_OK) return st;
  if (!aligned(q_out, 16) || !aligned(k_out, 16)) return MAMBA_ERR_ALIGN;
  QkArgs a = qk_args(dims, q, k, q_weight, k_weight, positions, inv_freq, eps);
  a.out[0] = q_out;
  a.out[1] = k_out;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launch_qk(a, dims, false, {}, s);
}

size_t mamba_qk_norm_rope_bwd_workspace_bytes(const mamba_qk_norm_rope_dims* dims) {
  if (check_qk(dims) != MAMBA_OK) return 0;
  return (size_t)qk_grid(dims).all * (size_t)dims->dim * sizeof(float);
}

int mamba_qk_norm_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                           const int64_t* positions, const double* inv_freq, float eps, const void* dq_out,
                           const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight,
                           const mamba_qk_norm_rope_dims* dims, void* workspace, size_t workspace_bytes,
                           void* stream) {
  int st = check_qk(dims);
  if (st != MAMBA_OK) return st;
  if (!dq_out || !dk_out || !dq || !dk || !dq_weight || !dk_weight) return MAMBA_ERR_NULL;
  if ((st = check_qk_inputs(dims, q, k, q_weight, k_weight, positions, inv_freq, eps)) != MAMBA_OK) return st;
  if (!aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return MAMBA_ERR_ALIGN;
  if (!workspace || workspace_bytes < mamba_qk_norm_rope_bwd_workspace_bytes(dims)) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 4)) return MAMBA_ERR_ALIGN;
  QkArgs a = qk_args(dims, q, k, q_weight, k_weight, positions, inv_freq, eps);
  a.dout[0] = dq_out;
  a.dout[1] = dk_out;
  a.out[0] = dq;
  a.out[1] = dk;
  a.part = static_cast<float*>(workspace);
  const QkGrid grid = qk_grid(dims);
  a.split = grid.split;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = launch_qk(a, dims, true, grid, s);
  if (st != MAMBA_OK) return st;
  hipLaunchKernelGGL(qk_fold_kernel, dim3((unsigned)((a.dim + kQkFoldCols - 1) / kQkFoldCols), 2), dim3(1024), 0, s,
                     a.part, dq_weight, dk_weight, (int)grid.split, (int)grid.all, a.dim);
  return launch_status();
}

}  // extern "C"
