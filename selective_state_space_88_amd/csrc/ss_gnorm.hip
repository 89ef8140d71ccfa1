// ss_gnorm.hip -- group norm with an activation on channels-last tensors, forward and backward (gfx950).
//
// Per row b and group g over its positions and channels (N values):  n = (x - mean) / sqrt(var + eps),
// u = n weight + bias, y = u or u sigmoid(u).  Backward with du = dy act'(u), d = du weight:
// dx = (d - mean(d) - n mean(d n)) / std,  dweight = sum du n,  dbias = sum du.
//
// Mapping.  A lane holds 16 bytes of x's channels where rows are aligned (else 8 bytes or one channel).
// Groups that fit a block's registers (resident kernels): a block holds one row's group, its lanes beside each
// other along the group's channels and then along the positions, reduces it there and writes the result, one
// launch and every tensor touched once.  Blocks of neighbouring groups, which share lines of memory, run on one
// die (group_of).
// Larger groups: a block takes a tile of positions of one row by a slab of channels; tiles are reduced to sums
// per channel, a block per (row, group) joins them in f64, and a second walk over the tiles writes the result.
//
// Measured (a large copy: 4.8 TB/s): 16 x 4096 x 512 in 32 groups with silu, bf16, forward 51 us (2.6 TB/s),
// backward 79 (2.5): blocks of 1024 threads fill a CU alone, so loads, sums and stores follow each other; two a CU
// (64 registers, 8 spilled) took 62 forward.  32 x 256 x 1280: forward 14 us, backward 24 (3.1 and 2.6 TB/s).
// 4 x 65536 x 256 (tiles): sums 39 us, join 6, result 49, the second read from the cache behind the L2s; backward
// 162.  Few groups or small ones are far from that: 1 x 65536 x 128 in one group 138 us, of which the join's one
// block takes 112; 65536 x 1 x 2048 in 32 groups 3.8 ms, a block for each group of 64 values, and backward 27 ms, 23
// of them in such blocks and 4.4 in gnorm_params_kernel, which adds a channel's rows up in one thread.
//
// Precision.  Resident kernels take the deviations around a first mean, and from their own mean the rest of it
// (corrected two-pass sums).  A tile's sums are taken around a value K of the channel near its middle, so that a mean far from
// zero costs no digits: the median of three positions inside the tile, so that no single position far out (a
// row's first, say) becomes K.  The joined mean is kept as f32 and what its rounding left.
#include <algorithm>
#include <type_traits>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int kDepth = 4;      // positions a lane loads at once
constexpr int kSumLen = 64;    // positions a lane adds up at most

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// V channels (1, 4 or 8) as they lie in memory
template <typename T, int V>
struct Line {
  static constexpr int kBytes = V * (int)sizeof(T);
  T one;
  static __device__ __forceinline__ Line load(const T* p) { return Line{*p}; }
  __device__ __forceinline__ void get(float (&v)[V]) const { v[0] = to_f32(one); }
};
template <int V>
struct Line<bf16_t, V> {
  typedef typename std::conditional<V == 8, u32x4, typename std::conditional<V == 4, u32x2, uint16_t>::type>::type word;
  word w;
  static __device__ __forceinline__ Line load(const bf16_t* p) { return Line{*reinterpret_cast<const word*>(p)}; }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (V == 1) {
      v[0] = bf16_lo(w);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
};
template <>
struct Line<float, 4> {
  f32x4 w;
  static __device__ __forceinline__ Line load(const float* p) { return Line{*reinterpret_cast<const f32x4*>(p)}; }
  __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
  }
};
template <>
struct Line<float, 8> {
  f32x4 w[2];
  static __device__ __forceinline__ Line load(const float* p) {
    const f32x4* q = reinterpret_cast<const f32x4*>(p);
    return Line{q[0], q[1]};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i / 4][i % 4];
  }
};

template <typename T, int V>
__device__ __forceinline__ void load_line(const T* __restrict__ p, float (&v)[V]) {
  Line<T, V>::load(p).get(v);
}

template <typename T, int V>
__device__ __forceinline__ void store_line(T* __restrict__ p, const float (&v)[V]) {
  if constexpr (V == 1) {
    store_one(p, v[0]);
  } else if constexpr (sizeof(T) == 2) {
    typename Line<T, V>::word w;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pk_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<typename Line<T, V>::word*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  }
}

// How a call is cut: `lanes` lanes of V channels beside each other (a power of two), kThreads / lanes
// teams that take turns at the positions.  A tile is every tiles-th run of `step` positions (one batch of all
// teams), so that the blocks that run together read a window that moves through memory as a whole.
struct Cut {
  int32_t shift;         // lanes = 1 << shift
  int64_t slabs, tiles, step;
  // tiles that have positions, and how many, in a row of len of them
  __host__ __device__ __forceinline__ int64_t used(int64_t len) const {
    const int64_t n = (len + step - 1) / step;
    return n < tiles ? n : tiles;
  }
  __device__ __forceinline__ int64_t count(int64_t tile, int64_t len) const {
    const int64_t round = tiles * step, left = len % round - tile * step;
    return len / round * step + (left < 0 ? 0 : left < step ? left : step);
  }
  // the tile's position number i
  __device__ __forceinline__ int64_t at(int64_t tile, int64_t i) const {
    return (i / step * tiles + tile) * step + i % step;
  }
};

// Where a block works.  Lanes behind the last channel are clamped to the last channels (`live` false).
template <int V>
struct Spot {
  int64_t b, tile, l0, end;  // the tile's first position, the row's length
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
    l0 = tile * k.step;
    end = length(p, b);
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

// the slope of u sigmoid(u)
__device__ __forceinline__ float silu_slope(float u) {
  const float s = sigmoid_of(u);
  return s * fmaf(u, 1.0f - s, 1.0f);
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
    // batches of kDepth positions, the next one on its way while one is added up
    const int64_t step = k.tiles * k.step;
    Line<T, V> now[kDepth], next[kDepth];
    const auto fetch = [&](int64_t l, Line<T, V>(&to)[kDepth]) {
#pragma unroll
      for (int j = 0; j < kDepth; ++j)
        to[j] = Line<T, V>::load(x + min(l + (int64_t)j * at.teams, at.end - 1) * p.x.st);
    };
    fetch(at.l0 + at.team, now);
    const int64_t last = k.count(at.tile, at.end) - 1;
    float a[V], b[V], c[V];
    load_line<T, V>(x + k.at(at.tile, last / 4) * p.x.st, a);
    load_line<T, V>(x + k.at(at.tile, last / 2) * p.x.st, b);
    load_line<T, V>(x + k.at(at.tile, last - last / 4) * p.x.st, c);
#pragma unroll
    for (int e = 0; e < V; ++e) K[e] = __builtin_amdgcn_fmed3f(a[e], b[e], c[e]);
    for (int64_t l = at.l0 + at.team; l < at.end; l += step) {
      if (l + step < at.end) fetch(l + step, next);
#pragma unroll
      for (int j = 0; j < kDepth; ++j) {
        if (l + (int64_t)j * at.teams >= at.end) continue;
        float v[V];
        now[j].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[e] - K[e];
          s[0][e] += d;
          s[1][e] = fmaf(d, d, s[1][e]);
        }
      }
#pragma unroll
      for (int j = 0; j < kDepth; ++j) now[j] = next[j];
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

// stats[b][g] from the tiles' sums, moved in f64 to the first tile's K of the group's first channel: a value of
// the group, so that the squares' sum and the mean's square differ in what is left of f64's digits
__global__ __launch_bounds__(kThreads) void gnorm_join_kernel(GroupNormArgs p, Cut k, const float* part) {
  __shared__ double lds[kThreads / 64];
  const int64_t b = blockIdx.x / p.groups, g = blockIdx.x % p.groups;
  const int64_t size = p.channels / p.groups, len = Spot<1>::length(p, b);
  const int64_t all = k.used(len) * size;
  const float* from = part + b * k.tiles * 3 * p.channels + g * size;
  const double K0 = all ? (double)from[0] : 0;
  double sum = 0, sq = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < all; i += kThreads) {
    const int64_t t = i / size;
    const float* q = from + t * 3 * p.channels + i % size;
    const double n = (double)k.count(t, len), d = (double)q[0] - K0, s = (double)q[p.channels];
    sum += s + n * d;
    sq += (double)q[2 * p.channels] + d * (2 * s + n * d);
  }
  sum = block_sum(sum, lds);
  sq = block_sum(sq, lds);
  if (threadIdx.x) return;
  const double N = fmax((double)len * (double)size, 1.);
  const double mean = K0 + sum / N, var = sq / N - (sum / N) * (sum / N);
  float* to = p.stats + b * p.s_sb + g * p.s_sg;
  to[0] = (float)mean;
  to[1] = (float)(mean - (double)(float)mean);
  to[2] = (float)(1.0 / sqrt((var < 0. ? 0. : var) + (double)p.eps));
}

template <typename TX, typename TY, int V, bool SILU>
__global__ __launch_bounds__(kThreads) void gnorm_apply_kernel(GroupNormArgs p, Cut k) {
  const Spot<V> at(p, k);
  const TX* x = static_cast<const TX*>(p.x.p) + at.b * p.x.sb + at.c;
  TY* y = static_cast<TY*>(p.y.p) + at.b * p.y.sb + at.c;
  const int64_t size = p.channels / p.groups, stop = p.L;
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
  for (int64_t l = at.l0 + at.team; l < stop; l += k.tiles * k.step) {
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
    *du = SILU ? dy * silu_slope(fmaf(*n, w[e], bias[e])) : dy;
  }
};

// The same for channels of one group, with t = x - mean in the place of n = t / std, which saves a product for
// each value.  What mean's rounding left is taken off for bf16 inputs too: their values are 2^-8 apart, but the
// deviation of a group that is nearly constant may be below 2^-25 of its mean, and the rounding as large as it.
template <int V>
struct GroupParams {
  float mean, low, inv, w[V], scale[V], bias[V];
  __device__ __forceinline__ GroupParams(const GroupNormArgs& p, float mean_, float low_, float inv_, int64_t c)
      : mean(mean_), low(low_), inv(inv_) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = p.weight[c + e];
      scale[e] = inv * w[e];
      bias[e] = p.bias ? p.bias[c + e] : 0.f;
    }
  }
  __device__ __forceinline__ float centred(float x) const { return (x - mean) - low; }
  __device__ __forceinline__ float u(int e, float t) const { return fmaf(t, scale[e], bias[e]); }
  template <bool SILU>
  __device__ __forceinline__ void at(int e, float x, float dy, float* t, float* du) const {
    *t = centred(x);
    *du = SILU ? dy * silu_slope(u(e, *t)) : dy;
  }
};

// s + a b with the product rounded on its own
__device__ __forceinline__ float add_product(float a, float b, float s) {
#pragma clang fp contract(off)
  return s + a * b;
}

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
  for (int64_t l = at.l0 + at.team; l < at.end; l += k.tiles * k.step) {
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
  const int64_t tiles = k.used(len);
  // 16 channels at a time, 16 threads to each one's tiles
  constexpr int kCols = 16, kTeams = kThreads / kCols;
  __shared__ double acc[2][kTeams][kCols];
  const int col = threadIdx.x % kCols, team = threadIdx.x / kCols;
  double m0 = 0, m1 = 0;
  for (int64_t i0 = 0; i0 < size; i0 += kCols) {
    const int64_t c = g * size + i0 + col;
    double s0 = 0, s1 = 0;
    if (i0 + col < size) {
#pragma unroll 4
      for (int64_t t = team; t < tiles; t += kTeams) {
        const float* q = part + (b * k.tiles + t) * 2 * p.channels + c;
        s0 += (double)q[0];
        s1 += (double)q[p.channels];
      }
    }
    acc[0][team][col] = s0;
    acc[1][team][col] = s1;
    __syncthreads();
    if (team == 0 && i0 + col < size) {
      s0 = s1 = 0;
#pragma unroll
      for (int t = 0; t < kTeams; ++t) {
        s0 += acc[0][t][col];
        s1 += acc[1][t][col];
      }
      rows[b * 2 * p.channels + c] = (float)s0;
      rows[(b * 2 + 1) * p.channels + c] = (float)s1;
      m0 += s0 * (double)p.weight[c];
      m1 += s1 * (double)p.weight[c];
    }
    __syncthreads();
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
#pragma unroll 8
  for (int64_t b = 0; b < p.batch; ++b) s += (double)rows[b * 2 * p.channels + i];
  to[i % p.channels] = (float)s;
}

template <typename TX, typename TY, int V, bool SILU>
__global__ __launch_bounds__(kThreads) void gnorm_bwd_apply_kernel(GroupNormArgs p, Cut k, const float* means) {
  const Spot<V> at(p, k);
  const TX* x = static_cast<const TX*>(p.x.p) + at.b * p.x.sb + at.c;
  const TY* dy = static_cast<const TY*>(p.dy.p) + at.b * p.dy.sb + at.c;
  TX* dx = static_cast<TX*>(p.dx.p) + at.b * p.dx.sb + at.c;
  const int64_t size = p.channels / p.groups, stop = p.L;
  const Params<V> q(p, at.b, at.c);
  float m0[V], m1[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float* m = means + (at.b * p.groups + (at.c + e) / size) * 2;
    m0[e] = m[0];
    m1[e] = m[1];
  }
  if (!at.live) return;
  for (int64_t l = at.l0 + at.team; l < stop; l += k.tiles * k.step) {
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

// ------------------------------------------------------------------------- resident groups

// Block i's (row, group): the blocks of one die (they go round the dies in turn) take neighbours.
constexpr int kDies = 8;
__device__ __forceinline__ int64_t group_of(int64_t all) {
  const int64_t each = (all + kDies - 1) / kDies;
  return (int64_t)(blockIdx.x % kDies) * each + blockIdx.x / kDies;
}

// A lane's place: line `part` of the group's channels, positions team, team + teams, ... (K of them at most);
// threads behind the last whole team have none.
template <int V, int THREADS>
struct Seat {
  int64_t b, g, c;
  int len, size, parts, part, team, teams;
  int mine, rows;        // the lane's positions inside the row's length, and inside the row
  __device__ __forceinline__ Seat(const GroupNormArgs& p, int64_t i) {
    b = i / p.groups;
    g = i % p.groups;
    size = (int)(p.channels / p.groups);
    parts = size / V;
    part = threadIdx.x % parts;
    team = threadIdx.x / parts;
    teams = THREADS / parts;
    c = g * size + part * V;
    len = (int)Spot<1>::length(p, b);
    const int over = team < teams ? teams - 1 - team : -INT32_MAX;
    mine = over < 0 ? 0 : (int)(((int64_t)len + over) / teams);
    rows = over < 0 ? 0 : (int)((p.L + over) / teams);
  }
};

// The sum of a block's values, in every thread
template <int THREADS>
__device__ __forceinline__ float whole_sum(float v, float* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) s += lds[i];
  return s;
}

template <typename TX, typename TY, int V, int THREADS, int K, bool SILU>
__global__ __launch_bounds__(THREADS) void gnorm_fwd_kernel(GroupNormArgs p) {
  __shared__ float lds[THREADS / 64];
  const int64_t all = p.batch * p.groups, i = group_of(all);
  if (i >= all) return;
  const Seat<V, THREADS> at(p, i);
  const TX* x = static_cast<const TX*>(p.x.p) + at.b * p.x.sb + at.c + at.team * p.x.st;
  Line<TX, V> raw[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < at.mine) raw[k] = Line<TX, V>::load(x + k * (at.teams * p.x.st));
  const float inv_n = 1.0f / fmaxf((float)at.len * (float)at.size, 1.0f);
  float s = 0.f, q = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < at.mine) {
      float v[V];
      raw[k].get(v);
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[e];
    }
  const float first = whole_sum<THREADS>(s, lds) * inv_n;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < at.mine) {
      float v[V];
      raw[k].get(v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = v[e] - first;
        s += d;
        q = fmaf(d, d, q);
      }
    }
  const float rest = whole_sum<THREADS>(s, lds) * inv_n;
  float var = fmaf(-rest, rest, whole_sum<THREADS>(q, lds) * inv_n);
  var = var < 0.f ? 0.f : var;  // a NaN stays
  const float mean = first + rest, low = rest - (mean - first), inv = 1.0f / sqrtf(var + p.eps);
  if (p.stats && threadIdx.x == 0) {
    float* to = p.stats + at.b * p.s_sb + at.g * p.s_sg;
    to[0] = mean;
    to[1] = low;
    to[2] = inv;
  }
  TY* y = static_cast<TY*>(p.y.p) + at.b * p.y.sb + at.c + at.team * p.y.st;
  const GroupParams<V> r(p, mean, low, inv, at.c);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k >= at.rows) continue;
    float v[V] = {};
    if (k < at.mine) {
      raw[k].get(v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u = r.u(e, r.centred(v[e]));
        v[e] = SILU ? u * sigmoid_of(u) : u;
      }
    }
    store_line<TY, V>(y + k * (at.teams * p.y.st), v);
  }
}

// rows[b][2][channels]: sum du and sum du n of the row, per channel
template <typename T, int V, int THREADS, int K, bool SILU>
__global__ __launch_bounds__(THREADS) void gnorm_bwd_kernel(GroupNormArgs p, float* rows) {
  constexpr int kRows = THREADS / 64;
  __shared__ float lds[2 * V * THREADS];
  __shared__ float means[kRows][2];
  const int64_t all = p.batch * p.groups, i = group_of(all);
  if (i >= all) return;
  const Seat<V, THREADS> at(p, i);
  const T* x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c + at.team * p.x.st;
  const T* dy = static_cast<const T*>(p.dy.p) + at.b * p.dy.sb + at.c + at.team * p.dy.st;
  Line<T, V> rx[K], rg[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < at.mine) {
      rx[k] = Line<T, V>::load(x + k * (at.teams * p.x.st));
      rg[k] = Line<T, V>::load(dy + k * (at.teams * p.dy.st));
    }
  const float* st = p.stats + at.b * p.s_sb + at.g * p.s_sg;
  const GroupParams<V> q(p, st[0], st[1], st[2], at.c);
  float s[2][V] = {};
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < at.mine) {
      float v[V], g[V];
      rx[k].get(v);
      rg[k].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float t, du;
        q.template at<SILU>(e, v[e], g[e], &t, &du);
        s[0][e] += du;
        s[1][e] = fmaf(du, t, s[1][e]);
      }
    }
  // a row of no positions adds nothing, though with eps = 0 its 1 / std is an infinity
  const float unit = at.len > 0 ? q.inv : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    lds[e * THREADS + threadIdx.x] = s[0][e];
    lds[(V + e) * THREADS + threadIdx.x] = s[1][e] * unit;
  }
  __syncthreads();
  // a wave to each sum of a channel over the teams
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float m[2] = {0.f, 0.f};
  for (int j = wave; j < at.size; j += kRows) {
    const int part = j / V, e = j % V;
    float t0 = 0.f, t1 = 0.f;
    for (int t = lane; t < at.teams; t += 64) {
      t0 += lds[e * THREADS + t * at.parts + part];
      t1 += lds[(V + e) * THREADS + t * at.parts + part];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      t0 += __shfl_xor(t0, o);
      t1 += __shfl_xor(t1, o);
    }
    const int64_t c = at.g * at.size + j;
    if (lane == 0) {
      rows[at.b * 2 * p.channels + c] = t0;
      rows[(at.b * 2 + 1) * p.channels + c] = t1;
    }
    const float wc = p.weight[c];
    m[0] = add_product(t0, wc, m[0]);
    m[1] = fmaf(t1, wc, m[1]);
  }
  if (lane == 0) {
    means[wave][0] = m[0];
    means[wave][1] = m[1];
  }
  __syncthreads();
  const float inv_n = 1.0f / fmaxf((float)at.len * (float)at.size, 1.0f);
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    m0 += means[k][0];
    m1 += means[k][1];
  }
  m0 *= inv_n;
  m1 *= inv_n * q.inv;  // times t, not n
  T* dx = static_cast<T*>(p.dx.p) + at.b * p.dx.sb + at.c + at.team * p.dx.st;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k >= at.rows) continue;
    float v[V] = {}, g[V];
    if (k < at.mine) {
      rx[k].get(v);
      rg[k].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float t, du;
        q.template at<SILU>(e, v[e], g[e], &t, &du);
        v[e] = through_norm(du, q.w[e], m0, t, m1, q.inv);
      }
    }
    store_line<T, V>(dx + k * (at.teams * p.dx.st), v);
  }
}

// ------------------------------------------------------------------------------------ launch

// The lanes beside each other: the power of two from 8 to 64 that leaves the fewest lanes without a
// channel.  Tiles: four blocks for each CU where the positions allow, at most kSumLen positions a lane.
Cut cut_of(int64_t batch, int64_t L, int64_t channels, int line) {
  const int64_t lines = (channels + line - 1) / line;
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
  const int64_t teams = kThreads >> k.shift;
  k.step = teams * kDepth;
  const int64_t want = std::max<int64_t>(1, (int64_t)4 * cu_count() / std::max<int64_t>(1, batch * k.slabs));
  const int64_t most = (L + k.step - 1) / k.step, least_tiles = (L + teams * kSumLen - 1) / (teams * kSumLen);
  k.tiles = std::min(most, std::max(want, least_tiles));
  return k;
}

// Threads and positions a lane for a group that stays in a block's registers (0: it does not)
struct Hold {
  int threads, k;
};
Hold hold_of(const GroupNormArgs& a, bool backward) {
  const int64_t size = a.channels / a.groups;
  if (a.line * (a.x_bf16 ? 2 : 4) != 16 || size % a.line || (backward && a.x_bf16 != a.y_bf16)) return {0, 0};
  for (const Hold h : {Hold{256, 2}, Hold{256, 8}, Hold{1024, 8}, Hold{1024, 16}}) {
    if (size / a.line > h.threads || (backward && h.k == 16)) continue;
    if ((h.threads / (size / a.line)) * h.k >= a.L) return h;
  }
  return {0, 0};
}

#define SS_GN_Y(RUN, TX, V, S) \
  if (a.y_bf16) RUN(TX, bf16_t, V, S); else RUN(TX, float, V, S);
#define SS_GN_X(RUN, V, S) \
  if (a.x_bf16) { SS_GN_Y(RUN, bf16_t, V, S) } else { SS_GN_Y(RUN, float, V, S) }
#define SS_GN_ALL(RUN)                                                       \
  if (a.line == 8) {                                                         \
    if (a.silu) { SS_GN_Y(RUN, bf16_t, 8, true) } else { SS_GN_Y(RUN, bf16_t, 8, false) }  \
  } else if (a.line == 4) {                                                  \
    if (a.silu) { SS_GN_X(RUN, 4, true) } else { SS_GN_X(RUN, 4, false) }    \
  } else {                                                                   \
    if (a.silu) { SS_GN_X(RUN, 1, true) } else { SS_GN_X(RUN, 1, false) }    \
  }

int64_t blocks_of(int64_t batch, const Cut& k) {
  if (batch * k.slabs > INT32_MAX) return batch * k.slabs;  // already too many, and the product might not fit
  return batch * k.slabs * k.tiles;
}

constexpr int kLines[] = {1, 4, 8};
int64_t tiles_most(int64_t batch, int64_t L, int64_t channels) {
  int64_t n = 0;
  for (const int line : kLines) n = std::max(n, cut_of(batch, L, channels, line).tiles);
  return n;
}

}  // namespace

int64_t gnorm_threads(const GroupNormArgs& a, bool backward) {
  const int64_t all = a.batch * a.groups;
  if (const Hold h = hold_of(a, backward); h.k) return (all + kDies - 1) / kDies * kDies * h.threads;
  return std::max(all, blocks_of(a.batch, cut_of(a.batch, a.L, a.channels, a.line))) * kThreads;
}

int64_t gnorm_workspace_floats(int64_t batch, int64_t L, int64_t channels, int32_t groups, bool backward) {
  const int64_t tiles = tiles_most(batch, L, channels);
  if (backward) return batch * 2 * channels * (tiles + 1) + batch * groups * 2;
  return batch * tiles * 3 * channels + batch * groups * 3;
}

hipError_t launch_gnorm_fwd(const GroupNormArgs& given, float* ws, hipStream_t s) {
  GroupNormArgs a = given;
  if (const Hold h = hold_of(a, false); h.k) {
    const dim3 grid((unsigned)((a.batch * a.groups + kDies - 1) / kDies * kDies));
#define SS_RUN(TX, TY, V, S)                                                                                      \
  do {                                                                                                            \
    if (h.k == 2) hipLaunchKernelGGL((gnorm_fwd_kernel<TX, TY, V, 256, 2, S>), grid, dim3(256), 0, s, a);         \
    else if (h.threads == 256) hipLaunchKernelGGL((gnorm_fwd_kernel<TX, TY, V, 256, 8, S>), grid, dim3(256), 0, s, a); \
    else if (h.k == 8) hipLaunchKernelGGL((gnorm_fwd_kernel<TX, TY, V, 1024, 8, S>), grid, dim3(1024), 0, s, a);  \
    else hipLaunchKernelGGL((gnorm_fwd_kernel<TX, TY, V, 1024, 16, S>), grid, dim3(1024), 0, s, a);               \
  } while (0)
    if (a.x_bf16) {
      if (a.silu) { SS_GN_Y(SS_RUN, bf16_t, 8, true) } else { SS_GN_Y(SS_RUN, bf16_t, 8, false) }
    } else {
      if (a.silu) { SS_GN_Y(SS_RUN, float, 4, true) } else { SS_GN_Y(SS_RUN, float, 4, false) }
    }
#undef SS_RUN
    return hipGetLastError();
  }
  const Cut k = cut_of(a.batch, a.L, a.channels, a.line);
  const dim3 grid((unsigned)blocks_of(a.batch, k)), block(kThreads);
  if (!a.stats) {
    a.stats = ws;
    a.s_sb = a.groups * 3;
    a.s_sg = 3;
  }
  float* part = ws + a.batch * a.groups * 3;
  if (grid.x > 0) {
    if (a.line == 8) hipLaunchKernelGGL((gnorm_sums_kernel<bf16_t, 8>), grid, block, 0, s, a, k, part);
    else if (a.line == 4 && a.x_bf16) hipLaunchKernelGGL((gnorm_sums_kernel<bf16_t, 4>), grid, block, 0, s, a, k, part);
    else if (a.line == 4) hipLaunchKernelGGL((gnorm_sums_kernel<float, 4>), grid, block, 0, s, a, k, part);
    else if (a.x_bf16) hipLaunchKernelGGL((gnorm_sums_kernel<bf16_t, 1>), grid, block, 0, s, a, k, part);
    else hipLaunchKernelGGL((gnorm_sums_kernel<float, 1>), grid, block, 0, s, a, k, part);
  }
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  hipLaunchKernelGGL(gnorm_join_kernel, dim3((unsigned)(a.batch * a.groups)), block, 0, s, a, k, part);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
#define SS_RUN(TX, TY, V, S) hipLaunchKernelGGL((gnorm_apply_kernel<TX, TY, V, S>), grid, block, 0, s, a, k)
  if (grid.x > 0) { SS_GN_ALL(SS_RUN) }
#undef SS_RUN
  return hipGetLastError();
}

hipError_t launch_gnorm_bwd(const GroupNormArgs& a, float* ws, hipStream_t s) {
  float* means = ws;
  float* rows = ws + a.batch * a.groups * 2;
  const dim3 block(kThreads);
  if (const Hold h = hold_of(a, true); a.batch > 0 && h.k) {
    const dim3 grid((unsigned)((a.batch * a.groups + kDies - 1) / kDies * kDies));
#define SS_RUN(T, V, S)                                                                                         \
  do {                                                                                                          \
    if (h.k == 2) hipLaunchKernelGGL((gnorm_bwd_kernel<T, V, 256, 2, S>), grid, dim3(256), 0, s, a, rows);      \
    else if (h.threads == 256) hipLaunchKernelGGL((gnorm_bwd_kernel<T, V, 256, 8, S>), grid, dim3(256), 0, s, a, rows); \
    else hipLaunchKernelGGL((gnorm_bwd_kernel<T, V, 1024, 8, S>), grid, dim3(1024), 0, s, a, rows);             \
  } while (0)
    if (a.x_bf16) {
      if (a.silu) SS_RUN(bf16_t, 8, true); else SS_RUN(bf16_t, 8, false);
    } else {
      if (a.silu) SS_RUN(float, 4, true); else SS_RUN(float, 4, false);
    }
#undef SS_RUN
  } else if (a.batch > 0) {
    const Cut k = cut_of(a.batch, a.L, a.channels, a.line);
    const dim3 grid((unsigned)blocks_of(a.batch, k));
    float* part = rows + a.batch * 2 * a.channels;
#define SS_RUN(TX, TY, V, S) hipLaunchKernelGGL((gnorm_bwd_sums_kernel<TX, TY, V, S>), grid, block, 0, s, a, k, part)
    if (grid.x > 0) { SS_GN_ALL(SS_RUN) }
#undef SS_RUN
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL(gnorm_bwd_join_kernel, dim3((unsigned)(a.batch * a.groups)), block, 0, s, a, k, part, rows,
                       means);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
#define SS_RUN(TX, TY, V, S) \
  hipLaunchKernelGGL((gnorm_bwd_apply_kernel<TX, TY, V, S>), grid, block, 0, s, a, k, means)
    if (grid.x > 0) { SS_GN_ALL(SS_RUN) }
#undef SS_RUN
  }
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (a.dweight || a.dbias)
    hipLaunchKernelGGL(gnorm_params_kernel, dim3((unsigned)((2 * a.channels + kThreads - 1) / kThreads)), block, 0, s,
                       a, rows);
  return hipGetLastError();
}

}  // namespace ss
