// mamba_norm.hip -- the RMS norms around a block on gfx950, forward and gradients.
//
// gated norm (between the mixer and its output projection), per row and group of `dim` values:
//     h = y rsqrt(mean(y^2) + eps),  out = h w silu(z)                 (norm, then gate)
//     a = y silu(z),  h = a rsqrt(mean(a^2) + eps),  out = h w         (gate first)
// add norm (the join of two blocks), per row:
//     n = x, or x rsqrt(mean(x^2) + eps) post;  r = residual + scale n;
//     out = r rsqrt(mean(r^2) + eps) w
// with the RMS norm's gradient  d(h w) -> da = rs (dh - h mean(dh h)),  dh = dout w.
//
// All four are bound by memory: each input is read once into registers and each output written
// once.  A unit (one group of one row) belongs to a team of T lanes, T = 8..1024, that holds it as
// R vectors of 8 values per lane; sums and statistics are fp32, the gradients' fp64.  Vectors are read
// and written as 16-byte words at any address (rows of odd length start anywhere), the last one value by
// value.  The weights' gradients are sums over all units: a team keeps its columns' sums in registers over
// the units it visits, the teams of a workgroup add theirs in LDS, each workgroup writes one
// partial row, and a second launch adds the partial rows.  Every order is fixed: no atomics.
//
// Measured, 16384 rows, bf16 (a large copy reaches 4.9 to 5.4 TB/s):
//   gated norm, 40 groups of 128: 92 us forward (5.3 TB/s), 184 us gradients (4.5 TB/s) and 6 us their second
//   launch
//   add norm, 2560 wide, fp32 stream, norm after the block: 103 us forward (4.8 TB/s), 168 us gradients
//   (4.5 TB/s) and 9 us
// 256 rows of 40 groups, or one row of 768: 3 to 4 us, latency.
#include "mamba_common.h"
#include "mamba_grid.h"

namespace mamba {
namespace {

// threads of a workgroup of teams of T lanes: from two waves on a team is a workgroup
template <int T>
constexpr int kBlock = T >= 128 ? T : 256;
constexpr int64_t kNormMaxDim = 16384;     // 1024 lanes x 2 vectors x 8 values
constexpr int64_t kNormMaxUnits = 0x7fffffff;
// Workgroups of a gradient launch: enough to fill 256 CUs at the kernel's occupancy, few enough
// that the partial rows they leave stay small beside the inputs.
constexpr int64_t kNormBwdWG = 1024;

typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// 8 consecutive values from any element address
__device__ __forceinline__ void ld8(const uint16_t* p, float (&v)[8]) {
  const u32x4u w = *reinterpret_cast<const u32x4u*>(p);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack(w[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ void ld8(const float* p, float (&v)[8]) {
  const f32x4u a = *reinterpret_cast<const f32x4u*>(p), b = *reinterpret_cast<const f32x4u*>(p + 4);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = a[k];
    v[4 + k] = b[k];
  }
}
__device__ __forceinline__ void st8(uint16_t* p, const float (&v)[8]) {
  u32x4u w;
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = pack_bf16(make_float2(v[2 * k], v[2 * k + 1]));
  *reinterpret_cast<u32x4u*>(p) = w;
}
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  f32x4u a, b;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[k] = v[k];
    b[k] = v[4 + k];
  }
  *reinterpret_cast<f32x4u*>(p) = a;
  *reinterpret_cast<f32x4u*>(p + 4) = b;
}

// 8 values as they are stored (a row on its way takes half the registers of its values)
template <typename E>
struct RawVec;
template <>
struct RawVec<uint16_t> {
  u32x4u w;
  __device__ __forceinline__ void get(const uint16_t* p) { w = *reinterpret_cast<const u32x4u*>(p); }
  __device__ __forceinline__ void some(const uint16_t* p, int n) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (2 * k < n ? (uint32_t)p[2 * k] : 0u) | (2 * k + 1 < n ? (uint32_t)p[2 * k + 1] << 16 : 0u);
  }
  __device__ __forceinline__ float operator[](int k) const {
    return __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
  }
};
template <>
struct RawVec<float> {
  f32x4u a, b;
  __device__ __forceinline__ void get(const float* p) {
    a = *reinterpret_cast<const f32x4u*>(p);
    b = *reinterpret_cast<const f32x4u*>(p + 4);
  }
  __device__ __forceinline__ void some(const float* p, int n) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = k < n ? p[k] : 0.f;
      b[k] = 4 + k < n ? p[4 + k] : 0.f;
    }
  }
  __device__ __forceinline__ float operator[](int k) const { return k < 4 ? a[k & 3] : b[k & 3]; }
};

// A lane's R vectors of one unit: vector r covers columns 8 (l + r T) .. +7 of `dim`.
template <int T, int R>
struct Cols {
  int l, dim;
  template <typename E>
  __device__ __forceinline__ void load(const E* p, float (&v)[R][8], bool live = true) const {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = 8 * (l + r * T);
      if (live && c + 8 <= dim) {
        ld8(p + c, v[r]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[r][k] = live && c + k < dim ? ld_f32(p, c + k) : 0.f;
      }
    }
  }
  template <typename E>
  __device__ __forceinline__ void load(const E* p, RawVec<E> (&v)[R], bool live) const {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = 8 * (l + r * T);
      if (live && c + 8 <= dim)
        v[r].get(p + c);
      else
        v[r].some(p + c, live ? dim - c : 0);
    }
  }
  template <typename E>
  __device__ __forceinline__ void store(E* p, const float (&v)[R][8]) const {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = 8 * (l + r * T);
      if (c + 8 <= dim) {
        st8(p + c, v[r]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < dim) st_out(p, c + k, v[r][k]);
      }
    }
  }
};

template <int kCtrl>
__device__ __forceinline__ float dpp_any(float v) { return dpp_row<kCtrl>(v); }
template <int kCtrl>
__device__ __forceinline__ double dpp_any(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __float_as_uint(dpp_row<kCtrl>(__uint_as_float((uint32_t)b)));
  const uint32_t hi = __float_as_uint(dpp_row<kCtrl>(__uint_as_float((uint32_t)(b >> 32))));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum of v over the team, in every lane.  T > 64 goes through LDS; the two slots alternate so that
// one barrier per call is enough (a slot is written again only after the barrier of the next call).
template <int T, typename V>
struct TeamSum {
  V (*slot)[kBlock<T> / 64][2];
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void operator()(V (&v)[N]) {
    static_assert(N <= 2 && (T == 8 || T >= 16), "slots hold two sums");
    // inside rows of 16 lanes by DPP rotations (a team of 8: xor by mirrors), further by lane exchange
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (T >= 16) {
        v[i] += dpp_any<0x128>(v[i]);
        v[i] += dpp_any<0x124>(v[i]);
        v[i] += dpp_any<0x122>(v[i]);
        v[i] += dpp_any<0x121>(v[i]);
      } else {
        v[i] += dpp_any<0xb1>(v[i]);   // quad_perm 1,0,3,2
        v[i] += dpp_any<0x4e>(v[i]);   // quad_perm 2,3,0,1
        v[i] += dpp_any<0x141>(v[i]);  // half row mirrored: lane 7 - l
      }
      if constexpr (T >= 32) v[i] += __shfl_xor(v[i], 16);
      if constexpr (T >= 64) v[i] += __shfl_xor(v[i], 32);
    }
    if constexpr (T > 64) {
      const int w = threadIdx.x >> 6, first = w / (T / 64) * (T / 64);
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) slot[turn][w][i] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = slot[turn][first][i];
#pragma unroll
        for (int j = 1; j < T / 64; ++j) v[i] += slot[turn][first + j][i];
      }
      turn ^= 1;
    }
  }
};

// sigmoid(z); exp(-z) overflows to infinity and the reciprocal is then 0
__device__ __forceinline__ float sigmoid_f32(float z) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
}

// The gradients' statistics are 1 / (mean + eps) in fp64, and zero for a team without a unit, whose zeros would
// make them infinite where eps is zero and leave NaN in the weights' sums.  An eps below 3e-39 can take them out of
// fp32's range, and their root is then taken in fp64 too (always so, the gradients' launches took 3% longer).
__device__ __forceinline__ float root_f32(double v) {
  float r = sqrtf((float)v);
  if (__builtin_expect(!(v < 1e38), 0)) r = (float)sqrt(v);
  return r;
}

// dh - v m: what is left of dh when its part along v is taken out.  Next to nothing is left where a
// unit has few values or dh is nearly parallel to v, so that m comes from sums in fp64 and the difference
// is taken there (fp64 fused multiply-adds run at the rate of unpacked fp32 ones on this target).
__device__ __forceinline__ float minus(float dh, float v, double m) {
  return (float)fma(-(double)v, m, (double)dh);
}

// Adds the workgroup's per-team column sums and writes them as one row of partials.
template <int T, int R>
__device__ __forceinline__ void put_partial(const Cols<T, R>& cols, const float (&acc)[R][8],
                                            float* sum, float* row) {
  constexpr int kTeams = kBlock<T> / T;
  if constexpr (kTeams == 1) {
    cols.store(row, acc);
  } else {
    // teams add in turn; columns past dim hold zeros
    const int team = threadIdx.x / T;
    for (int t = 0; t < kTeams; ++t) {
      if (team == t)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = 8 * (cols.l + r * T) + k;
            sum[c] = (t ? sum[c] : 0.f) + acc[r][k];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < cols.dim; c += kBlock<T>) row[c] = sum[c];
    __syncthreads();
  }
}

// ------------------------------------------------------------------ gated norm

struct GatedArgs {
  const void* y;
  const void* z;       // NULL: no gate
  const float* w;
  const void* dout;    // gradients only
  void* out;           // forward: out; gradients: dy
  void* dz;
  float* part;         // (gridDim.y, gridDim.x, dim) partial weight gradients
  int64_t rows, y_stride, z_stride;
  int32_t groups, dim, gate_first, per_group;
  float eps;
};

// unit -> row and group.  With one weight per group a workgroup stays in its group (blockIdx.y),
// so that its weight sums are that group's; with a shared weight units are taken in memory order.
struct Unit {
  int64_t row;
  int32_t grp;
};
__device__ __forceinline__ Unit unit_of(const GatedArgs& a, uint32_t u) {
  if (a.per_group) return {u, (int32_t)blockIdx.y};
  const uint32_t row = u / (uint32_t)a.groups;
  return {row, (int32_t)(u - row * (uint32_t)a.groups)};
}

template <typename E, int T, int R>
__global__ __launch_bounds__(kBlock<T>) void gated_norm_kernel(GatedArgs a, uint32_t units) {
  __shared__ float slot[2][kBlock<T> / 64][2];
  TeamSum<T, float> team_sum{slot};
  const Cols<T, R> cols{(int)(threadIdx.x % T), a.dim};
  const uint64_t u = (uint64_t)wide_index() * (kBlock<T> / T) + threadIdx.x / T;
  const bool live = u < units;
  const Unit at = unit_of(a, live ? (uint32_t)u : 0);
  float y[R][8], z[R][8], w[R][8];
  cols.load(static_cast<const E*>(a.y) + at.row * a.y_stride + (int64_t)at.grp * a.dim, y, live);
  if (a.z)
    cols.load(static_cast<const E*>(a.z) + at.row * a.z_stride + (int64_t)at.grp * a.dim, z, live);
  cols.load(a.w + (a.per_group ? (int64_t)at.grp * a.dim : 0), w);
  float s[1] = {0.f};
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (a.z) {
        z[r][k] = silu_f32(z[r][k]);
        if (a.gate_first) y[r][k] *= z[r][k];
      }
      s[0] = fmaf(y[r][k], y[r][k], s[0]);
    }
  team_sum(s);
  const float rs = rsqrtf(s[0] / a.dim + a.eps);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[r][k] *= rs * w[r][k];
      if (a.z && !a.gate_first) y[r][k] *= z[r][k];
    }
  if (live)
    cols.store(static_cast<E*>(a.out) + (at.row * a.groups + at.grp) * (int64_t)a.dim, y);
}

template <typename E, int T, int R>
__global__ __launch_bounds__(kBlock<T>) void gated_norm_bwd_kernel(GatedArgs a, uint32_t units) {
  constexpr int kTeams = kBlock<T> / T;
  __shared__ double slot[2][kBlock<T> / 64][2];
  __shared__ float sum[kTeams > 1 ? 8 * T * R : 1];
  TeamSum<T, double> team_sum{slot};
  const Cols<T, R> cols{(int)(threadIdx.x % T), a.dim};
  float w[R][8], acc[R][8];
  cols.load(a.w + (a.per_group ? (int64_t)blockIdx.y * a.dim : 0), w);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[r][k] = 0.f;
  const double inv = 1.0 / a.dim;
  // every team runs the same number of turns (the reductions hold barriers); the next unit is on its way
  // while one is worked on
  RawVec<E> yn[R], zn[R], dn[R];
  auto fetch = [&](uint32_t base) {
    const uint32_t u = base + threadIdx.x / T;
    const bool live = u < units;
    const Unit at = unit_of(a, live ? u : 0);
    const int64_t grp = (int64_t)at.grp * a.dim;
    cols.load(static_cast<const E*>(a.y) + at.row * a.y_stride + grp, yn, live);
    cols.load(static_cast<const E*>(a.z) + at.row * a.z_stride + grp, zn, live && a.z);
    cols.load(static_cast<const E*>(a.dout) + at.row * a.groups * (int64_t)a.dim + grp, dn, live);
  };
  const uint32_t stride = gridDim.x * kTeams;
  fetch(blockIdx.x * kTeams);
  for (uint32_t base = blockIdx.x * kTeams; base < units; base += stride) {
    const uint32_t u = base + threadIdx.x / T;
    const bool live = u < units;
    const Unit at = unit_of(a, live ? u : 0);
    const int64_t packed = (at.row * a.groups + at.grp) * (int64_t)a.dim;
    float y[R][8], z[R][8], d[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y[r][k] = yn[r][k];
        z[r][k] = zn[r][k];
        d[r][k] = dn[r][k];
      }
    if (units - base > stride) fetch(base + stride);
    // v = the normed value (y, or y silu(z)); s = sum v^2, sum dh v
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float g = a.z ? silu_f32(z[r][k]) : 1.f;
        const float v = a.gate_first ? y[r][k] * g : y[r][k];
        const float dh = d[r][k] * w[r][k] * (a.gate_first ? 1.f : g);
        s[0] = fma((double)v, (double)v, s[0]);
        s[1] = fma((double)dh, (double)v, s[1]);
      }
    team_sum(s);
    const double r2 = live ? 1.0 / fma(s[0], inv, (double)a.eps) : 0.0, m = s[1] * r2 * inv;
    const float rs = root_f32(r2);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float sg = a.z ? sigmoid_f32(z[r][k]) : 1.f;
        const float g = a.z ? z[r][k] * sg : 1.f;
        const float slope = a.z ? sg * fmaf(z[r][k], 1.f - sg, 1.f) : 0.f;  // silu'(z)
        if (a.gate_first) {
          const float v = y[r][k] * g, da = rs * minus(d[r][k] * w[r][k], v, m);
          acc[r][k] = fmaf(d[r][k], v * rs, acc[r][k]);
          z[r][k] = da * y[r][k] * slope;
          y[r][k] = da * g;
        } else {
          const float h = y[r][k] * rs, dg = d[r][k] * g;
          acc[r][k] = fmaf(dg, h, acc[r][k]);
          z[r][k] = d[r][k] * h * w[r][k] * slope;
          y[r][k] = rs * minus(d[r][k] * w[r][k] * g, y[r][k], m);
        }
      }
    if (live) {
      cols.store(static_cast<E*>(a.out) + packed, y);
      if (a.z) cols.store(static_cast<E*>(a.dz) + packed, z);
    }
  }
  put_partial(cols, acc, sum,
              a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (int64_t)a.dim);
}

// ------------------------------------------------------------------ add norm

struct AddArgs {
  const void* x;
  const void* residual;  // NULL: zero
  const float* w;
  const float* scale;    // NULL: one
  const float* post;     // NULL: no norm of x
  const void* dout;      // gradients only
  const void* dres;      // NULL: zero
  void* out;             // forward: out; gradients: dx
  void* res_out;         // forward: r; gradients: dresidual (NULL: not written)
  float* part;           // (1 or 2, gridDim.x, dim): partials of dw and of sum(dr h)
  int64_t rows;
  int32_t dim;
  float eps;
};

template <typename E, typename S, int T, int R>
__global__ __launch_bounds__(kBlock<T>) void add_norm_kernel(AddArgs a) {
  __shared__ float slot[2][kBlock<T> / 64][2];
  TeamSum<T, float> team_sum{slot};
  const Cols<T, R> cols{(int)(threadIdx.x % T), a.dim};
  const int64_t row = (int64_t)wide_index() * (kBlock<T> / T) + threadIdx.x / T;
  const bool live = row < a.rows;
  const int64_t at = (live ? row : 0) * a.dim;
  float x[R][8], q[R][8], p[R][8];
  cols.load(static_cast<const E*>(a.x) + at, x, live);
  if (a.residual) cols.load(static_cast<const S*>(a.residual) + at, q, live);
  const float inv = 1.f / a.dim;
  if (a.post) {
    cols.load(a.post, p);
    float s[1] = {0.f};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] = fmaf(x[r][k], x[r][k], s[0]);
    team_sum(s);
    const float rs = rsqrtf(s[0] * inv + a.eps);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[r][k] *= rs * p[r][k];
  }
  if (a.scale) {
    cols.load(a.scale, p);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[r][k] *= p[r][k];
  }
  cols.load(a.w, p);
  float s[1] = {0.f};
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (a.residual) x[r][k] += q[r][k];
      s[0] = fmaf(x[r][k], x[r][k], s[0]);
    }
  if (live) cols.store(static_cast<S*>(a.res_out) + at, x);
  team_sum(s);
  const float rs = rsqrtf(s[0] * inv + a.eps);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) x[r][k] *= rs * p[r][k];
  if (live) cols.store(static_cast<E*>(a.out) + at, x);
}

// r is recomputed from x and the residual, so that the gradients are those of the unrounded r
// whatever type the residual stream is stored in.
template <typename E, typename S, int T, int R>
__global__ __launch_bounds__(kBlock<T>) void add_norm_bwd_kernel(AddArgs a) {
  constexpr int kTeams = kBlock<T> / T;
  __shared__ double slot[2][kBlock<T> / 64][2];
  __shared__ float sum[kTeams > 1 ? 8 * T * R : 1];
  TeamSum<T, double> team_sum{slot};
  const Cols<T, R> cols{(int)(threadIdx.x % T), a.dim};
  // per column, for all rows: w; p = scale post (the weight of the normed x in r); and the sums
  float w[R][8], p[R][8], aw[R][8], ah[R][8];
  cols.load(a.w, w);
  if (a.post) cols.load(a.post, p);
  if (a.scale) cols.load(a.scale, aw);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      p[r][k] = (a.post ? p[r][k] : 1.f) * (a.scale ? aw[r][k] : 1.f);
      aw[r][k] = ah[r][k] = 0.f;
    }
  const double inv = 1.0 / a.dim;
  const int64_t stride = (int64_t)gridDim.x * kTeams;
  // the next row is on its way while one is worked on
  RawVec<E> xn[R], dn[R];
  RawVec<S> qn[R], en[R];
  auto fetch = [&](int64_t base) {
    const int64_t row = base + threadIdx.x / T;
    const bool live = row < a.rows;
    const int64_t at = (live ? row : 0) * a.dim;
    cols.load(static_cast<const E*>(a.x) + at, xn, live);
    cols.load(static_cast<const S*>(a.residual) + at, qn, live && a.residual);
    cols.load(static_cast<const E*>(a.dout) + at, dn, live);
    cols.load(static_cast<const S*>(a.dres) + at, en, live && a.dres);
  };
  fetch((int64_t)blockIdx.x * kTeams);
  for (int64_t base = (int64_t)blockIdx.x * kTeams; base < a.rows; base += stride) {
    const int64_t row = base + threadIdx.x / T;
    const bool live = row < a.rows;
    const int64_t at = (live ? row : 0) * a.dim;
    float x[R][8], v[R][8], d[R][8], e[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[r][k] = xn[r][k];
        v[r][k] = qn[r][k];
        d[r][k] = dn[r][k];
        e[r][k] = en[r][k];
      }
    if (base + stride < a.rows) fetch(base + stride);
    double rx2 = 1.0;
    if (a.post) {
      double s[1] = {0.0};
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] = fma((double)x[r][k], (double)x[r][k], s[0]);
      team_sum(s);
      rx2 = live ? 1.0 / fma(s[0], inv, (double)a.eps) : 0.0;
    }
    const float rx = root_f32(rx2);  // the normed x is x rx
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[r][k] = fmaf(p[r][k], x[r][k] * rx, v[r][k]);  // r
        s[0] = fma((double)v[r][k], (double)v[r][k], s[0]);
        s[1] = fma((double)(d[r][k] * w[r][k]), (double)v[r][k], s[1]);
      }
    team_sum(s);
    const double r2 = live ? 1.0 / fma(s[0], inv, (double)a.eps) : 0.0, m = s[1] * r2 * inv;
    const float rs = root_f32(r2);
    // v = dr.  With h the normed x, dscale = sum(dr post h) and dpost = sum(dr scale h): the other factor is
    // constant per column, so that both come from one sum.
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        aw[r][k] = fmaf(d[r][k], v[r][k] * rs, aw[r][k]);
        v[r][k] = fmaf(rs, minus(d[r][k] * w[r][k], v[r][k], m), e[r][k]);
        ah[r][k] = fmaf(v[r][k], x[r][k] * rx, ah[r][k]);
      }
    if (live && a.res_out) cols.store(static_cast<S*>(a.res_out) + at, v);
    if (a.post) {
      double t[1] = {0.0};
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) t[0] = fma((double)(v[r][k] * p[r][k]), (double)x[r][k], t[0]);
      team_sum(t);
      const double mx = t[0] * rx2 * inv;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[r][k] = rx * minus(v[r][k] * p[r][k], x[r][k], mx);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[r][k] = v[r][k] * p[r][k];
    }
    if (live) cols.store(static_cast<E*>(a.out) + at, x);
  }
  const int64_t n = (int64_t)gridDim.x * a.dim;
  float* row = a.part + (int64_t)blockIdx.x * a.dim;
  put_partial(cols, aw, sum, row);
  if (a.scale || a.post) put_partial(cols, ah, sum, row + n);
}

// ------------------------------------------------------------------ partial rows -> gradients

struct FoldArgs {
  const float* part;  // (gridDim.y, nrows, dim)
  float* dw;          // vectors 0 .. groups-1, (groups, dim)
  float* a;           // vector `groups` times mul_a, (dim); NULL: not written
  float* b;           // the same times mul_b
  const float* mul_a;  // NULL: one
  const float* mul_b;
  int32_t nrows, dim, groups;
};

// Column sums of the partial rows: 64 columns per workgroup, its 16 waves each add every 16th row
// and the 16 sums are added in order.
__global__ __launch_bounds__(1024) void norm_fold_kernel(FoldArgs a) {
  __shared__ float s[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  const float* p = a.part + (int64_t)blockIdx.y * a.nrows * a.dim;
  float t = 0.f;
  if (c < a.dim) {
#pragma unroll 8
    for (int r = w; r < a.nrows; r += 16) t += p[(int64_t)r * a.dim + c];
  }
  s[w][threadIdx.x & 63] = t;
  __syncthreads();
  if (w == 0 && c < a.dim) {
    for (int i = 1; i < 16; ++i) t += s[i][threadIdx.x & 63];
    if ((int)blockIdx.y < a.groups) {
      a.dw[(int64_t)blockIdx.y * a.dim + c] = t;
    } else {
      if (a.a) a.a[c] = a.mul_a ? t * a.mul_a[c] : t;
      if (a.b) a.b[c] = a.mul_b ? t * a.mul_b[c] : t;
    }
  }
}

// ------------------------------------------------------------------ host

// The team of a unit of `dim` values: calls f.template operator()<T, R>().  One vector per lane, so that a
// gradient's rows (up to six values per column) leave room for many waves: 2560 values, gradients, 16384
// rows, bf16 with an fp32 stream: 168 us with 5 waves of one vector, 316 us with 2
// waves of three.  Teams are powers of two and, between them, three, five and ten waves: the widths of the models
// that the package's workloads come from (1536, 2560 and 5120).  Any other width takes the next larger team, up to
// half of whose lanes then have no column.
template <typename F>
int with_team(int64_t dim, F f) {
  if (dim <= 64) return f.template operator()<8, 1>();
  if (dim <= 128) return f.template operator()<16, 1>();
  if (dim <= 256) return f.template operator()<32, 1>();
  if (dim <= 512) return f.template operator()<64, 1>();
  if (dim <= 1024) return f.template operator()<128, 1>();
  if (dim <= 8 * 192) return f.template operator()<192, 1>();
  if (dim <= 2048) return f.template operator()<256, 1>();
  if (dim <= 8 * 320) return f.template operator()<320, 1>();
  if (dim <= 4096) return f.template operator()<512, 1>();
  if (dim <= 8 * 640) return f.template operator()<640, 1>();
  if (dim <= 8192) return f.template operator()<1024, 1>();
  return f.template operator()<1024, 2>();
}

struct Lanes {
  template <int T, int R>
  int operator()() const { return T; }
};
int team_lanes(int64_t dim) {
  return with_team(dim, Lanes{});
}

int check_eps(float eps) { return eps >= 0.f && eps < 3e38f ? MAMBA_OK : MAMBA_ERR_UNSUPPORTED; }

bool known_dtype(int32_t t) { return t == MAMBA_F32 || t == MAMBA_BF16; }
size_t elem_size(int32_t t) { return t == MAMBA_BF16 ? 2 : 4; }

int check_gated(const mamba_gated_norm_dims* d) {
  if (!d) return MAMBA_ERR_NULL;
  if (!known_dtype(d->io_dtype)) return MAMBA_ERR_DTYPE;
  if (d->rows < 1 || d->groups < 1 || d->dim < 1) return MAMBA_ERR_SHAPE;
  if (d->dim > kNormMaxDim || d->rows > kNormMaxUnits || d->groups > 65535 ||
      d->rows * d->groups > kNormMaxUnits)
    return MAMBA_ERR_SHAPE;
  if (d->weight_groups != 1 && d->weight_groups != d->groups) return MAMBA_ERR_SHAPE;
  const int64_t packed = d->groups * d->dim, lim = (int64_t)1 << 40;
  if ((d->y_stride && d->y_stride < packed) || (d->z_stride && d->z_stride < packed) ||
      d->y_stride > lim || d->z_stride > lim)
    return MAMBA_ERR_SHAPE;
  return MAMBA_OK;
}

int check_add(const mamba_add_norm_dims* d) {
  if (!d) return MAMBA_ERR_NULL;
  if (!known_dtype(d->io_dtype) || !known_dtype(d->res_dtype)) return MAMBA_ERR_DTYPE;
  if (d->rows < 1 || d->dim < 1 || d->dim > kNormMaxDim || d->rows > kNormMaxUnits)
    return MAMBA_ERR_SHAPE;
  // a residual stream narrower than the block's own type is not kept
  if (d->io_dtype == MAMBA_F32 && d->res_dtype != MAMBA_F32) return MAMBA_ERR_UNSUPPORTED;
  return MAMBA_OK;
}

GatedArgs gated_args(const mamba_gated_norm_dims* d, float eps) {
  GatedArgs a = {};
  a.rows = d->rows;
  a.groups = (int32_t)d->groups;
  a.dim = (int32_t)d->dim;
  a.y_stride = d->y_stride ? d->y_stride : d->groups * d->dim;
  a.z_stride = d->z_stride ? d->z_stride : d->groups * d->dim;
  a.gate_first = d->gate_first != 0;
  a.per_group = d->weight_groups > 1;
  a.eps = eps;
  return a;
}

// units of one blockIdx.y and the workgroups that a gradient launch gives them
uint32_t gated_units(const GatedArgs& a) {
  return (uint32_t)(a.per_group ? a.rows : a.rows * a.groups);
}
uint32_t bwd_wgs(int64_t units, int64_t dim, int64_t ny) {
  const int64_t teams = team_lanes(dim) >= 128 ? 1 : 256 / team_lanes(dim);
  const int64_t need = (units + teams - 1) / teams;
  return (uint32_t)std::min(need, std::max<int64_t>(1, kNormBwdWG / ny));
}

int launch_fold(const FoldArgs& f, int ny, hipStream_t s) {
  hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)((f.dim + 63) / 64), (unsigned)ny), dim3(1024),
                     0, s, f);
  return launch_status();
}

template <typename E>
struct GatedFwd {
  GatedArgs a;
  hipStream_t s;
  template <int T, int R>
  int operator()() const {
    const uint32_t units = gated_units(a), teams = kBlock<T> / T;
    hipLaunchKernelGGL((gated_norm_kernel<E, T, R>),
                       wide_grid((units + teams - 1) / teams, kBlock<T>, a.per_group ? a.groups : 1),
                       dim3(kBlock<T>), 0, s, a, units);
    return launch_status();
  }
};
template <typename E>
struct GatedBwd {
  GatedArgs a;
  hipStream_t s;
  uint32_t wgs;
  template <int T, int R>
  int operator()() const {
    hipLaunchKernelGGL((gated_norm_bwd_kernel<E, T, R>), dim3(wgs, a.per_group ? a.groups : 1),
                       dim3(kBlock<T>), 0, s, a, gated_units(a));
    return launch_status();
  }
};
template <typename E, typename S>
struct AddFwd {
  AddArgs a;
  hipStream_t s;
  template <int T, int R>
  int operator()() const {
    const int64_t teams = kBlock<T> / T;
    hipLaunchKernelGGL((add_norm_kernel<E, S, T, R>), wide_grid((a.rows + teams - 1) / teams, kBlock<T>),
                       dim3(kBlock<T>), 0, s, a);
    return launch_status();
  }
};
template <typename E, typename S>
struct AddBwd {
  AddArgs a;
  hipStream_t s;
  uint32_t wgs;
  template <int T, int R>
  int operator()() const {
    hipLaunchKernelGGL((add_norm_bwd_kernel<E, S, T, R>), dim3(wgs), dim3(kBlock<T>), 0, s, a);
    return launch_status();
  }
};

}  // namespace
}  // namespace mamba

using namespace mamba;

extern "C" {

int mamba_gated_norm_fwd(const void* y, const void* z, const float* weight, float eps, void* out,
                         const mamba_gated_norm_dims* dims, void* stream) {
  int st = check_gated(dims);
  if (st != MAMBA_OK) return st;
  if (!y || !weight || !out) return MAMBA_ERR_NULL;
  if ((st = check_eps(eps)) != MAMBA_OK) return st;
  const size_t es = elem_size(dims->io_dtype);
  if (!aligned(y, es) || (z && !aligned(z, es)) || !aligned(out, es) || !aligned(weight, 4))
    return MAMBA_ERR_ALIGN;
  GatedArgs a = gated_args(dims, eps);
  a.y = y;
  a.z = z;
  a.w = weight;
  a.out = out;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dims->io_dtype == MAMBA_BF16 ? with_team(dims->dim, GatedFwd<uint16_t>{a, s})
                                      : with_team(dims->dim, GatedFwd<float>{a, s});
}

size_t mamba_gated_norm_bwd_workspace_bytes(const mamba_gated_norm_dims* dims) {
  if (check_gated(dims) != MAMBA_OK) return 0;
  const GatedArgs a = gated_args(dims, 0.f);
  const int64_t ny = a.per_group ? a.groups : 1;
  return (size_t)ny * bwd_wgs(gated_units(a), a.dim, ny) * (size_t)a.dim * sizeof(float);
}

int mamba_gated_norm_bwd(const void* y, const void* z, const float* weight, float eps,
                         const void* dout, void* dy, void* dz, float* dweight,
                         const mamba_gated_norm_dims* dims, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int st = check_gated(dims);
  if (st != MAMBA_OK) return st;
  if (!y || !weight || !dout || !dy || !dweight || (z && !dz)) return MAMBA_ERR_NULL;
  if ((st = check_eps(eps)) != MAMBA_OK) return st;
  const size_t es = elem_size(dims->io_dtype);
  if (!aligned(y, es) || (z && (!aligned(z, es) || !aligned(dz, es))) || !aligned(dout, es) ||
      !aligned(dy, es) || !aligned(weight, 4) || !aligned(dweight, 4))
    return MAMBA_ERR_ALIGN;
  if (!workspace || workspace_bytes < mamba_gated_norm_bwd_workspace_bytes(dims))
    return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 4)) return MAMBA_ERR_ALIGN;
  GatedArgs a = gated_args(dims, eps);
  a.y = y;
  a.z = z;
  a.w = weight;
  a.dout = dout;
  a.out = dy;
  a.dz = dz;
  a.part = static_cast<float*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t ny = a.per_group ? a.groups : 1;
  const uint32_t wgs = bwd_wgs(gated_units(a), a.dim, ny);
  st = dims->io_dtype == MAMBA_BF16 ? with_team(dims->dim, GatedBwd<uint16_t>{a, s, wgs})
                                    : with_team(dims->dim, GatedBwd<float>{a, s, wgs});
  if (st != MAMBA_OK) return st;
  FoldArgs f = {};
  f.part = a.part;
  f.dw = dweight;
  f.nrows = (int32_t)wgs;
  f.dim = a.dim;
  f.groups = (int32_t)ny;
  return launch_fold(f, (int)ny, s);
}

int mamba_add_norm_fwd(const void* x, const void* residual, const float* weight, const float* scale,
                       const float* post_weight, float eps, void* out, void* residual_out,
                       const mamba_add_norm_dims* dims, void* stream) {
  int st = check_add(dims);
  if (st != MAMBA_OK) return st;
  if (!x || !weight || !out || !residual_out) return MAMBA_ERR_NULL;
  if ((st = check_eps(eps)) != MAMBA_OK) return st;
  const size_t es = elem_size(dims->io_dtype), rs = elem_size(dims->res_dtype);
  if (!aligned(x, es) || !aligned(out, es) || (residual && !aligned(residual, rs)) ||
      !aligned(residual_out, rs) || !aligned(weight, 4) || (scale && !aligned(scale, 4)) ||
      (post_weight && !aligned(post_weight, 4)))
    return MAMBA_ERR_ALIGN;
  AddArgs a = {};
  a.x = x;
  a.residual = residual;
  a.w = weight;
  a.scale = scale;
  a.post = post_weight;
  a.out = out;
  a.res_out = residual_out;
  a.rows = dims->rows;
  a.dim = (int32_t)dims->dim;
  a.eps = eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dims->io_dtype == MAMBA_F32) return with_team(dims->dim, AddFwd<float, float>{a, s});
  return dims->res_dtype == MAMBA_F32 ? with_team(dims->dim, AddFwd<uint16_t, float>{a, s})
                                      : with_team(dims->dim, AddFwd<uint16_t, uint16_t>{a, s});
}

size_t mamba_add_norm_bwd_workspace_bytes(const mamba_add_norm_dims* dims) {
  if (check_add(dims) != MAMBA_OK) return 0;
  return 2 * (size_t)bwd_wgs(dims->rows, dims->dim, 1) * (size_t)dims->dim * sizeof(float);
}

int mamba_add_norm_bwd(const void* x, const void* residual, const float* weight, const float* scale,
                       const float* post_weight, float eps, const void* dout,
                       const void* dresidual_out, void* dx, void* dresidual, float* dweight,
                       float* dscale, float* dpost_weight, const mamba_add_norm_dims* dims,
                       void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_add(dims);
  if (st != MAMBA_OK) return st;
  if (!x || !weight || !dout || !dx || !dweight || (scale && !dscale) ||
      (post_weight && !dpost_weight))
    return MAMBA_ERR_NULL;
  if ((st = check_eps(eps)) != MAMBA_OK) return st;
  const size_t es = elem_size(dims->io_dtype), rs = elem_size(dims->res_dtype);
  if (!aligned(x, es) || !aligned(dout, es) || !aligned(dx, es) ||
      (residual && !aligned(residual, rs)) || (dresidual_out && !aligned(dresidual_out, rs)) ||
      (dresidual && !aligned(dresidual, rs)) || !aligned(weight, 4) || !aligned(dweight, 4) ||
      (scale && (!aligned(scale, 4) || !aligned(dscale, 4))) ||
      (post_weight && (!aligned(post_weight, 4) || !aligned(dpost_weight, 4))))
    return MAMBA_ERR_ALIGN;
  if (!workspace || workspace_bytes < mamba_add_norm_bwd_workspace_bytes(dims))
    return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 4)) return MAMBA_ERR_ALIGN;
  AddArgs a = {};
  a.x = x;
  a.residual = residual;
  a.w = weight;
  a.scale = scale;
  a.post = post_weight;
  a.dout = dout;
  a.dres = dresidual_out;
  a.out = dx;
  a.res_out = dresidual;
  a.part = static_cast<float*>(workspace);
  a.rows = dims->rows;
  a.dim = (int32_t)dims->dim;
  a.eps = eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const uint32_t wgs = bwd_wgs(dims->rows, dims->dim, 1);
  if (dims->io_dtype == MAMBA_F32)
    st = with_team(dims->dim, AddBwd<float, float>{a, s, wgs});
  else if (dims->res_dtype == MAMBA_F32)
    st = with_team(dims->dim, AddBwd<uint16_t, float>{a, s, wgs});
  else
    st = with_team(dims->dim, AddBwd<uint16_t, uint16_t>{a, s, wgs});
  if (st != MAMBA_OK) return st;
  FoldArgs f = {};
  f.part = a.part;
  f.dw = dweight;
  f.a = scale ? dscale : nullptr;
  f.b = post_weight ? dpost_weight : nullptr;
  f.mul_a = post_weight;
  f.mul_b = scale;
  f.nrows = (int32_t)wgs;
  f.dim = a.dim;
  f.groups = 1;
  return launch_fold(f, scale || post_weight ? 2 : 1, s);
}

}  // extern "C"
