// ss_gnorm.hip -- group norm with an activation on channels-last tensors, forward and backward (gfx950).
//
// Per row b and group g over its positions and channels (N values):  n = (x - mean) / sqrt(var + eps),
// u = n weight + bias, y = u or u sigmoid(u).  Backward with du = dy act'(u), d = du weight:
// dx = (d - mean(d) - n mean(d n)) / std,  dweight = sum du n,  dbias = sum du.
//
// Mapping.  A block takes a tile of positions of one row by a slab of channels, its lanes along the
// channels (8 of them a lane where rows are 16-byte aligned, else one), so every access is whole lines.
// Tiles are reduced to sums per channel, a block per (row, group) joins them in f64, and a second walk
// over the tiles writes the result.
//
// Precision.  A tile's sums are taken around a value K of the channel near its middle, so that a mean far from
// zero costs no digits: the median of three positions inside the tile, so that no single position far out (a
// row's first, say) becomes K.  The joined mean is kept as f32 and what its rounding left.
#include <algorithm>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int kDepth = 4;      // positions a lane loads at once
constexpr int kSumLen = 64;    // positions a lane adds up at most

template <typename T, int V>
__device__ __forceinline__ void load_line(const T* __restrict__ p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f32(p[0]);
  } else if constexpr (sizeof(T) == 2) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_line(T* __restrict__ p, const float (&v)[V]) {
  if constexpr (V == 1) {
    store_one(p, v[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<u32x4*>(p) =
        u32x4{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])};
  } else {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// How a call is cut: `lanes` lanes of V channels beside each other (a power of two), kThreads / lanes
// teams that take turns at the positions, tiles of `span` positions.
struct Cut {
  int32_t shift;         // lanes = 1 << shift
  int64_t slabs, tiles, span;
};

// Where a block works.  Lanes behind the last channel are clamped to the last channels (`live` false).
template <int V>
struct Spot {
  int64_t b, tile, l0, end;  // positions [l0, end), all of them inside the row's length
  int64_t c;
  int team, teams, lane;
  bool live;
  __device__ __forceinline__ Spot(const GroupNormArgs& p, const Cut& k) {
    int64_t i = blockIdx.x;
    const int64_t slab = i % k.slabs;
    i /= k.slabs;
    tile = i % k.tiles;
    b = i / k.tiles;
    lane = threadIdx.x & ((1 << k.shift) - 1);
    team = threadIdx.x >> k.shift;
    teams = kThreads >> k.shift;
    c = ((slab << k.shift) + lane) * V;
    live = c < p.channels;
    if (!live) c = p.channels - V;
    l0 = tile * k.span;
    end = min(l0 + k.span, length(p, b));
  }
  static __device__ __forceinline__ int64_t length(const GroupNormArgs& p, int64_t b) {
    if (!p.lengths) return p.L;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : n > p.L ? p.L : n;
  }
};

__device__ __forceinline__ float sigmoid_of(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u * kLog2e));
}

// The sum of n values a lane over the teams of a block, per channel, in team order; team 0 has it.
template <int V, int NV>
__device__ __forceinline__ void team_sum(float (&s)[NV][V], float* lds, int lane, int team, int teams) {
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) lds[(k * V + e) * kThreads + threadIdx.x] = s[k][e];
  __syncthreads();
  if (team) return;
  const int lanes = kThreads / teams;
  for (int t = 1; t < teams; ++t)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s[k][e] += lds[(k * V + e) * kThreads + t * lanes + lane];
}

// ---------------------------------------------------------------------------------- forward

// part[b][tile][3][channels]: K, sum (x - K), sum (x - K)^2
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void gnorm_sums_kernel(GroupNormArgs p, Cut k, float* part) {
  __shared__ float lds[2 * V * kThreads];
  const Spot<V> at(p, k);
  const T* x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c;
  float K[V] = {}, s[2][V] = {};
  if (at.l0 < at.end) {
    const int64_t last = at.end - at.l0 - 1;
    float a[V], b[V], c[V];
    load_line<T, V>(x + (at.l0 + last / 4) * p.x.st, a);
    load_line<T, V>(x + (at.l0 + last / 2) * p.x.st, b);
    load_line<T, V>(x + (at.l0 + last - last / 4) * p.x.st, c);
#pragma unroll
    for (int e = 0; e < V; ++e) K[e] = __builtin_amdgcn_fmed3f(a[e], b[e], c[e]);
  }
  for (int64_t l = at.l0 + at.team; l < at.end; l += (int64_t)at.teams * kDepth) {
    float v[kDepth][V];
#pragma unroll
    for (int j = 0; j < kDepth; ++j) load_line<T, V>(x + min(l + (int64_t)j * at.teams, at.end - 1) * p.x.st, v[j]);
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      if (l + (int64_t)j * at.teams >= at.end) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = v[j][e] - K[e];
        s[0][e] += d;
        s[1][e] = fmaf(d, d, s[1][e]);
      }
    }
  }
  team_sum<V, 2>(s, lds, at.lane, at.team, at.teams);
  if (at.team || !at.live) return;
  float* to = part + (at.b * k.tiles + at.tile) * 3 * p.channels + at.c;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    to[e] = K[e];
    to[p.channels + e] = s[0][e];
    to[2 * p.channels + e] = s[1][e];
  }
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) s += lds[i];
  return s;
}

// stats[b][g] from the tiles' sums: the mean of the tiles' means, then their squares around it
__global__ __launch_bounds__(kThreads) void gnorm_join_kernel(GroupNormArgs p, Cut k, const float* part) {
  __shared__ double lds[kThreads / 64];
  const int64_t b = blockIdx.x / p.groups, g = blockIdx.x % p.groups;
  const int64_t size = p.channels / p.groups, len = Spot<1>::length(p, b);
  const int64_t tiles = (len + k.span - 1) / k.span, all = tiles * size;
  const float* from = part + b * k.tiles * 3 * p.channels + g * size;
  double sum = 0, sq = 0;
  for (int64_t i = threadIdx.x; i < all; i += kThreads) {
    const int64_t t = i / size;
    const float* q = from + t * 3 * p.channels + i % size;
    sum += (double)q[0] * (double)min(k.span, len - t * k.span) + (double)q[p.channels];
  }
  const double N = (double)len * (double)size;
  const double mean = N > 0 ? block_sum(sum, lds) / N : 0;
  for (int64_t i = threadIdx.x; i < all; i += kThreads) {
    const int64_t t = i / size;
    const float* q = from + t * 3 * p.channels + i % size;
    const double n = (double)min(k.span, len - t * k.span), d = (double)q[0] - mean, s = (double)q[p.channels];
    sq += (double)q[2 * p.channels] + d * (2 * s + n * d);
  }
  const double var = N > 0 ? fmax(block_sum(sq, lds), 0.) / N : 0;
  if (threadIdx.x) return;
  float* to = p.stats + b * p.s_sb + g * p.s_sg;
  to[0] = (float)mean;
  to[1] = (float)(mean - (double)(float)mean);
  to[2] = (float)(1.0 / sqrt(var + (double)p.eps));
}

template <typename TX, typename TY, int V, bool SILU>
__global__ __launch_bounds__(kThreads) void gnorm_apply_kernel(GroupNormArgs p, Cut k) {
  const Spot<V> at(p, k);
  const TX* x = static_cast<const TX*>(p.x.p) + at.b * p.x.sb + at.c;
  TY* y = static_cast<TY*>(p.y.p) + at.b * p.y.sb + at.c;
  const int64_t size = p.channels / p.groups, stop = min(at.l0 + k.span, p.L);
  float mean[V], low[V], scale[V], bias[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float* st = p.stats + at.b * p.s_sb + (at.c + e) / size * p.s_sg;
    mean[e] = st[0];
    low[e] = st[1];
    scale[e] = st[2] * p.weight[at.c + e];
    bias[e] = p.bias ? p.bias[at.c + e] : 0.f;
  }
  if (!at.live) return;
  for (int64_t l = at.l0 + at.team; l < stop; l += (int64_t)at.teams * kDepth) {
    float v[kDepth][V];
#pragma unroll
    for (int j = 0; j < kDepth; ++j)
      if (l + (int64_t)j * at.teams < at.end) load_line<TX, V>(x + (l + (int64_t)j * at.teams) * p.x.st, v[j]);
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      const int64_t t = l + (int64_t)j * at.teams;
      if (t >= stop) break;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u = fmaf((v[j][e] - mean[e]) - low[e], scale[e], bias[e]);
        v[j][e] = t < at.end ? (SILU ? u * sigmoid_of(u) : u) : 0.f;
      }
      store_line<TY, V>(y + t * p.y.st, v[j]);
    }
  }
}

// --------------------------------------------------------------------------------- backward

// What a lane knows of its channels: n = (x - mean - low) inv, u = n weight + bias
template <int V>
struct Params {
  float mean[V], low[V], inv[V], w[V], bias[V];
  __device__ __forceinline__ Params(const GroupNormArgs& p, int64_t b, int64_t c) {
    const int64_t size = p.channels / p.groups;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float* st = p.stats + b * p.s_sb + (c + e) / size * p.s_sg;
      mean[e] = st[0];
      low[e] = st[1];
      inv[e] = st[2];
      w[e] = p.weight[c + e];
      bias[e] = p.bias ? p.bias[c + e] : 0.f;
    }
  }
  // n and du from x and dy
  template <bool SILU>
  __device__ __forceinline__ void at(int e, float x, float dy, float* n, float* du) const {
    *n = ((x - mean[e]) - low[e]) * inv[e];
    *du = dy;
    if constexpr (SILU) {
      const float u = fmaf(*n, w[e], bias[e]), s = sigmoid_of(u);
      *du = dy * (s * fmaf(u, 1.0f - s, 1.0f));
    }
  }
};

// (d - mean(d) - n mean(d n)) / std.  d is rounded before the mean is taken from it, as it was in the mean:
// a group of one value then has the gradient 0, not the rounding of a product.
__device__ __forceinline__ float through_norm(float du, float w, float m0, float n, float m1, float inv) {
#pragma clang fp contract(off)
  const float d = du * w;
  return ((d - m0) - n * m1) * inv;
}

// part[b][tile][2][channels]: sum du, sum du n
template <typename TX, typename TY, int V, bool SILU>
__global__ __launch_bounds__(kThreads) void gnorm_bwd_sums_kernel(GroupNormArgs p, Cut k, float* part) {
  __shared__ float lds[2 * V * kThreads];
  const Spot<V> at(p, k);
  const TX* x = static_cast<const TX*>(p.x.p) + at.b * p.x.sb + at.c;
  const TY* dy = static_cast<const TY*>(p.dy.p) + at.b * p.dy.sb + at.c;
  const Params<V> q(p, at.b, at.c);
  float s[2][V] = {};
  for (int64_t l = at.l0 + at.team; l < at.end; l += (int64_t)at.teams * kDepth) {
    float v[kDepth][V], g[kDepth][V];
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      const int64_t t = min(l + (int64_t)j * at.teams, at.end - 1);
      load_line<TX, V>(x + t * p.x.st, v[j]);
      load_line<TY, V>(dy + t * p.dy.st, g[j]);
    }
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      if (l + (int64_t)j * at.teams >= at.end) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float n, du;
        q.template at<SILU>(e, v[j][e], g[j][e], &n, &du);
        s[0][e] += du;
        s[1][e] = fmaf(du, n, s[1][e]);
      }
    }
  }
  team_sum<V, 2>(s, lds, at.lane, at.team, at.teams);
  if (at.team || !at.live) return;
  float* to = part + (at.b * k.tiles + at.tile) * 2 * p.channels + at.c;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    to[e] = s[0][e];
    to[p.channels + e] = s[1][e];
  }
}

// rows[b][2][channels]: the row's sums per channel; means[b][g]: mean of d and of d n
__global__ __launch_bounds__(kThreads) void gnorm_bwd_join_kernel(GroupNormArgs p, Cut k, const float* part,
                                                                  float* rows, float* means) {
  __shared__ double lds[kThreads / 64];
  const int64_t b = blockIdx.x / p.groups, g = blockIdx.x % p.groups;
  const int64_t size = p.channels / p.groups, len = Spot<1>::length(p, b);
  const int64_t tiles = (len + k.span - 1) / k.span;
  double m0 = 0, m1 = 0;
  for (int64_t i = threadIdx.x; i < size; i += kThreads) {
    const int64_t c = g * size + i;
    double s0 = 0, s1 = 0;
    for (int64_t t = 0; t < tiles; ++t) {
      const float* q = part + (b * k.tiles + t) * 2 * p.channels + c;
      s0 += (double)q[0];
      s1 += (double)q[p.channels];
    }
    rows[b * 2 * p.channels + c] = (float)s0;
    rows[(b * 2 + 1) * p.channels + c] = (float)s1;
    m0 += s0 * (double)p.weight[c];
    m1 += s1 * (double)p.weight[c];
  }
  m0 = block_sum(m0, lds);
  m1 = block_sum(m1, lds);
  const double N = fmax((double)len * (double)size, 1.);
  if (threadIdx.x) return;
  means[(b * p.groups + g) * 2] = (float)(m0 / N);
  means[(b * p.groups + g) * 2 + 1] = (float)(m1 / N);
}

// dbias and dweight from the rows' sums, rows in order
__global__ __launch_bounds__(kThreads) void gnorm_params_kernel(GroupNormArgs p, const float* rows) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= 2 * p.channels) return;
  float* to = i < p.channels ? p.dbias : p.dweight;
  if (!to) return;
  double s = 0;
  for (int64_t b = 0; b < p.batch; ++b) s += (double)rows[b * 2 * p.channels + i];
  to[i % p.channels] = (float)s;
}

template <typename TX, typename TY, int V, bool SILU>
__global__ __launch_bounds__(kThreads) void gnorm_bwd_apply_kernel(GroupNormArgs p, Cut k, const float* means) {
  const Spot<V> at(p, k);
  const TX* x = static_cast<const TX*>(p.x.p) + at.b * p.x.sb + at.c;
  const TY* dy = static_cast<const TY*>(p.dy.p) + at.b * p.dy.sb + at.c;
  TX* dx = static_cast<TX*>(p.dx.p) + at.b * p.dx.sb + at.c;
  const int64_t size = p.channels / p.groups, stop = min(at.l0 + k.span, p.L);
  const Params<V> q(p, at.b, at.c);
  float m0[V], m1[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float* m = means + (at.b * p.groups + (at.c + e) / size) * 2;
    m0[e] = m[0];
    m1[e] = m[1];
  }
  if (!at.live) return;
  for (int64_t l = at.l0 + at.team; l < stop; l += (int64_t)at.teams * kDepth) {
    float v[kDepth][V], g[kDepth][V];
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      const int64_t t = l + (int64_t)j * at.teams;
      if (t >= at.end) continue;
      load_line<TX, V>(x + t * p.x.st, v[j]);
      load_line<TY, V>(dy + t * p.dy.st, g[j]);
    }
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      const int64_t t = l + (int64_t)j * at.teams;
      if (t >= stop) break;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float n, du;
        q.template at<SILU>(e, v[j][e], g[j][e], &n, &du);
        v[j][e] = t < at.end ? through_norm(du, q.w[e], m0[e], n, m1[e], q.inv[e]) : 0.f;
      }
      store_line<TX, V>(dx + t * p.dx.st, v[j]);
    }
  }
}

// ------------------------------------------------------------------------------------ launch

// The lanes beside each other: the power of two from 8 to 64 that leaves the fewest lanes without a
// channel.  Tiles: four blocks for each CU where the positions allow, at most kSumLen positions a lane.
Cut cut_of(int64_t batch, int64_t L, int64_t channels, bool vec) {
  const int64_t lines = vec ? channels / 8 : channels;
  Cut k{};
  int64_t least = INT64_MAX;
  for (int s = 6; s >= 3; --s) {
    const int64_t slabs = (lines + (1 << s) - 1) >> s, lanes = slabs << s;
    if (lanes < least) {
      least = lanes;
      k.shift = s;
      k.slabs = slabs;
    }
  }
  const int64_t teams = kThreads >> k.shift, step = teams * kDepth;
  const int64_t want = std::max<int64_t>(1, (int64_t)4 * cu_count() / std::max<int64_t>(1, batch * k.slabs));
  int64_t span = (L + want - 1) / want;
  span = std::min(std::max((span + step - 1) / step * step, step), teams * kSumLen);
  k.span = span;
  k.tiles = (L + span - 1) / span;
  return k;
}

#define SS_GN_Y(RUN, TX, V, S) \
  if (a.y_bf16) RUN(TX, bf16_t, V, S); else RUN(TX, float, V, S);
#define SS_GN_X(RUN, V, S) \
  if (a.x_bf16) { SS_GN_Y(RUN, bf16_t, V, S) } else { SS_GN_Y(RUN, float, V, S) }
#define SS_GN_ALL(RUN)                                                       \
  if (a.vec) {                                                               \
    if (a.silu) { SS_GN_X(RUN, 8, true) } else { SS_GN_X(RUN, 8, false) }    \
  } else {                                                                   \
    if (a.silu) { SS_GN_X(RUN, 1, true) } else { SS_GN_X(RUN, 1, false) }    \
  }

int64_t tiles_most(int64_t batch, int64_t L, int64_t channels) {
  const int64_t t = channels % 8 == 0 ? cut_of(batch, L, channels, true).tiles : 0;
  return std::max(t, cut_of(batch, L, channels, false).tiles);
}

int64_t blocks_of(int64_t batch, const Cut& k) { return batch * k.tiles * k.slabs; }

}  // namespace

int64_t gnorm_blocks(int64_t batch, int64_t L, int64_t channels) {
  const int64_t n = channels % 8 == 0 ? blocks_of(batch, cut_of(batch, L, channels, true)) : 0;
  return std::max(n, blocks_of(batch, cut_of(batch, L, channels, false)));
}

int64_t gnorm_workspace_floats(int64_t batch, int64_t L, int64_t channels, int32_t groups, bool backward) {
  const int64_t tiles = tiles_most(batch, L, channels);
  if (backward) return batch * 2 * channels * (tiles + 1) + batch * groups * 2;
  return batch * tiles * 3 * channels + batch * groups * 3;
}

hipError_t launch_gnorm_fwd(const GroupNormArgs& given, float* ws, hipStream_t s) {
  GroupNormArgs a = given;
  const Cut k = cut_of(a.batch, a.L, a.channels, a.vec);
  const dim3 grid((unsigned)blocks_of(a.batch, k)), block(kThreads);
  if (!a.stats) {
    a.stats = ws;
    a.s_sb = a.groups * 3;
    a.s_sg = 3;
  }
  float* part = ws + a.batch * a.groups * 3;
  if (grid.x > 0) {
    if (a.vec) {
      if (a.x_bf16) hipLaunchKernelGGL((gnorm_sums_kernel<bf16_t, 8>), grid, block, 0, s, a, k, part);
      else hipLaunchKernelGGL((gnorm_sums_kernel<float, 8>), grid, block, 0, s, a, k, part);
    } else {
      if (a.x_bf16) hipLaunchKernelGGL((gnorm_sums_kernel<bf16_t, 1>), grid, block, 0, s, a, k, part);
      else hipLaunchKernelGGL((gnorm_sums_kernel<float, 1>), grid, block, 0, s, a, k, part);
    }
  }
  hipLaunchKernelGGL(gnorm_join_kernel, dim3((unsigned)(a.batch * a.groups)), block, 0, s, a, k, part);
#define SS_RUN(TX, TY, V, S) hipLaunchKernelGGL((gnorm_apply_kernel<TX, TY, V, S>), grid, block, 0, s, a, k)
  if (grid.x > 0) { SS_GN_ALL(SS_RUN) }
#undef SS_RUN
  return hipGetLastError();
}

hipError_t launch_gnorm_bwd(const GroupNormArgs& a, float* ws, hipStream_t s) {
  const Cut k = cut_of(a.batch, a.L, a.channels, a.vec);
  const dim3 grid((unsigned)blocks_of(a.batch, k)), block(kThreads);
  float* means = ws;
  float* rows = ws + a.batch * a.groups * 2;
  float* part = rows + a.batch * 2 * a.channels;
  if (a.batch > 0) {
#define SS_RUN(TX, TY, V, S) hipLaunchKernelGGL((gnorm_bwd_sums_kernel<TX, TY, V, S>), grid, block, 0, s, a, k, part)
    if (grid.x > 0) { SS_GN_ALL(SS_RUN) }
#undef SS_RUN
    hipLaunchKernelGGL(gnorm_bwd_join_kernel, dim3((unsigned)(a.batch * a.groups)), block, 0, s, a, k, part, rows,
                       means);
#define SS_RUN(TX, TY, V, S) \
  hipLaunchKernelGGL((gnorm_bwd_apply_kernel<TX, TY, V, S>), grid, block, 0, s, a, k, means)
    if (grid.x > 0) { SS_GN_ALL(SS_RUN) }
#undef SS_RUN
  }
  if (a.dweight || a.dbias)
    hipLaunchKernelGGL(gnorm_params_kernel, dim3((unsigned)((2 * a.channels + kThreads - 1) / kThreads)), block, 0, s,
                       a, rows);
  return hipGetLastError();
}

}  // namespace ss
