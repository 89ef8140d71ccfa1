// ss_norm.hip -- the norms before and after a block, forward and backward (gfx950).
//
// Before: sum = residual + alpha x, y = sum / sqrt(mean(sum^2) + eps) * weight.  After: the same
// norm over groups of channels of x silu(z), or of x with silu(z) on the result.  With n = t / rms
// and d the gradient at n, the gradient at t is (d - n mean(d n)) / rms, so the backward needs two
// sums per row, sum t^2 and sum d t, taken together in one pass over registers.
//
// Mapping.  Elementwise work on rows: HBM-bound.  A row (a group of a row) is held in the registers
// of TPR lanes, 8 consecutive channels per lane and step (one 16-byte access in bf16, two in f32),
// NV steps, so that each tensor is read and written once; TPR is 16 or 64 lanes of a wave for short
// rows, a block for long ones.  Sums are f32.  The weight's gradient is a column sum over rows: every
// lane keeps its channels' sums in registers over the rows its block walks, the blocks' partial sums
// go to the workspace, and a second kernel adds them in a fixed order (deterministic, no atomics).
// Measured (a large copy: 4.7 TB/s): 2 x 8192 rows of 5120 in bf16 with an f32 residual, forward 181 us,
// 5.5 TB/s, backward 270 us, 5.0 TB/s; 2 x 4096 rows of 32 groups of 128 with the gate, forward 39 us,
// 5.2 TB/s, backward 66 us, 5.1 TB/s.
#include <algorithm>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

constexpr int kBlock = 256;

template <typename T, bool VEC, int STEP = 1>
__device__ __forceinline__ void load8(const T* __restrict__ p, int n, float (&v)[8]) {
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 2) {
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
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i * STEP < n ? to_f32(p[i * STEP]) : 0.f;
  }
}

template <typename T, bool VEC, int STEP = 1>
__device__ __forceinline__ void store8(T* __restrict__ p, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<u32x4*>(p) =
          u32x4{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])};
    } else {
      *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * STEP < n) store_one(p + i * STEP, v[i]);
  }
}

// The first channel of a lane's step: 8 in a row, or (rows that are not aligned, element accesses) 8
// that are TPR apart, so that the lanes of an access are neighbours (5 x 325 rows of 11033, bf16 with an f32
// residual: 8 in a row took 146 us, this 68).
template <int TPR, bool VEC>
__device__ __forceinline__ int first_channel(int j, int lane) {
  return VEC ? (j * TPR + lane) * 8 : j * TPR * 8 + lane;
}

// The sums of N values over the TPR lanes of a row, in every lane.  Rows longer than a wave go
// through LDS (the whole block is one row then).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N]) {
#pragma unroll
  for (int m = (TPR < 64 ? TPR : 64) / 2; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __shared__ float part[W][N];
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the previous row's reads are done
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[w][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) s += part[k][i];
      v[i] = s;
    }
  }
}

// 1 / sqrt(x), once per row
__device__ __forceinline__ float inv_sqrt(float x) { return 1.0f / sqrtf(x); }

__device__ __forceinline__ float sigmoid_f32(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// Where row r (of batch * L) starts, in elements.
__device__ __forceinline__ int64_t row_at(const NormRows& t, int64_t b, int64_t l) { return b * t.sb + l * t.st; }

template <typename TX, typename TR, typename TY, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(TPR > kBlock ? TPR : kBlock) void addnorm_fwd_kernel(AddNormArgs p) {
  constexpr int kRows = TPR > kBlock ? 1 : kBlock / TPR;
  constexpr int kStep = VEC ? 1 : TPR;
  const int lane = threadIdx.x % TPR;
  const int64_t rows = p.batch * p.L;
  const int C = (int)p.channels;
  const float inv_c = 1.0f / (float)C;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + threadIdx.x / TPR;
    const bool live = r < rows;
    const int64_t b = live ? r / p.L : 0, l = live ? r % p.L : 0;
    const TX* x = static_cast<const TX*>(p.x.p) + row_at(p.x, b, l);
    const TR* res = static_cast<const TR*>(p.residual.p);
    if (res) res += row_at(p.residual, b, l);
    float t[NV][8], ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = 0.f;
      if (live && c < C) {
        float rv[8];
        load8<TX, VEC, kStep>(x + c, C - c, t[j]);
        if (res) {
          load8<TR, VEC, kStep>(res + c, C - c, rv);
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] = fmaf(p.alpha, t[j][i], rv[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] *= p.alpha;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(t[j][i], t[j][i], ss[0]);
    row_sum<TPR, 1>(ss);
    const float inv = inv_sqrt(fmaf(ss[0], inv_c, p.eps));
    TR* sum = static_cast<TR*>(p.sum.p);
    if (sum) sum += row_at(p.sum, b, l);
    TY* y = static_cast<TY*>(p.y.p) + row_at(p.y, b, l);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
      if (live && c < C) {
        if (sum) store8<TR, VEC, kStep>(sum + c, C - c, t[j]);
        float w[8];
        load8<float, VEC, kStep>(p.weight + c, C - c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = t[j][i] * inv * w[i];
        store8<TY, VEC, kStep>(y + c, C - c, w);
      }
    }
  }
}

// Partial column sums of a block: one row [channels of the group] of the workspace per block.  The
// block's TPR-lane teams hold the same channels; they are added through LDS, team by team.
template <int TPR, int NV, bool VEC>
__device__ __forceinline__ void store_partial(float (&dw)[NV][8], float* __restrict__ part, int C) {
  constexpr int kTeams = TPR >= kBlock ? 1 : kBlock / TPR;
  const int lane = threadIdx.x % TPR, team = threadIdx.x / TPR, kStep = VEC ? 1 : TPR;
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = first_channel<TPR, VEC>(j, lane) + i * kStep;
        if (c < C) part[c] = dw[j][i];
      }
  } else {
    __shared__ float acc[TPR * NV * 8];
    for (int k = 0; k < kTeams; ++k) {
      __syncthreads();
      if (team == k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = first_channel<TPR, VEC>(j, lane) + i * kStep;
            acc[c] = k ? acc[c] + dw[j][i] : dw[j][i];
          }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += kBlock) part[c] = acc[c];
  }
}

template <typename TY, typename TR, typename TX, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(TPR > kBlock ? TPR : kBlock) void addnorm_bwd_kernel(AddNormArgs p, float* part) {
  constexpr int kRows = TPR > kBlock ? 1 : kBlock / TPR;
  constexpr int kStep = VEC ? 1 : TPR;
  const int lane = threadIdx.x % TPR;
  const int64_t rows = p.batch * p.L;
  const int C = (int)p.channels;
  const float inv_c = 1.0f / (float)C;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = first_channel<TPR, VEC>(j, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[j][i] = dw[j][i] = 0.f;
    if (c < C) load8<float, VEC, kStep>(p.weight + c, C - c, w[j]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + threadIdx.x / TPR;
    const bool live = r < rows;
    const int64_t b = live ? r / p.L : 0, l = live ? r % p.L : 0;
    const TY* dy = static_cast<const TY*>(p.dy.p) + row_at(p.dy, b, l);
    const TR* sum = static_cast<const TR*>(p.sum.p) + row_at(p.sum, b, l);
    const TR* ds = static_cast<const TR*>(p.dsum.p);
    if (ds) ds += row_at(p.dsum, b, l);
    float t[NV][8], g[NV][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = g[j][i] = 0.f;
      if (live && c < C) {
        load8<TR, VEC, kStep>(sum + c, C - c, t[j]);
        load8<TY, VEC, kStep>(dy + c, C - c, g[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] = fmaf(t[j][i], t[j][i], s[0]);
        s[1] = fmaf(g[j][i] * w[j][i], t[j][i], s[1]);
      }
    row_sum<TPR, 2>(s);
    const float inv = inv_sqrt(fmaf(s[0], inv_c, p.eps));
    const float back = -(s[1] * inv_c) * inv * inv * inv;
    TR* dres = static_cast<TR*>(p.dres.p);
    if (dres) dres += row_at(p.dres, b, l);
    TX* dx = static_cast<TX*>(p.dx.p);
    if (dx) dx += row_at(p.dx, b, l);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
      if (live && c < C) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = fmaf(g[j][i] * w[j][i], inv, t[j][i] * back);
          dw[j][i] = fmaf(g[j][i], t[j][i] * inv, dw[j][i]);
        }
        if (ds) {
          float e[8];
          load8<TR, VEC, kStep>(ds + c, C - c, e);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] += e[i];
        }
        if (dres) store8<TR, VEC, kStep>(dres + c, C - c, d);
        if (dx) {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] *= p.alpha;
          store8<TX, VEC, kStep>(dx + c, C - c, d);
        }
      }
    }
  }
  if (part) store_partial<TPR, NV, VEC>(dw, part + (int64_t)blockIdx.x * C, C);
}

// ------------------------------------------------------------------ the norm after, with its gate

template <typename TX, typename TZ, typename TY, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(TPR > kBlock ? TPR : kBlock) void gatenorm_fwd_kernel(GateNormArgs p) {
  constexpr int kRows = TPR > kBlock ? 1 : kBlock / TPR;
  constexpr int kStep = VEC ? 1 : TPR;
  const int lane = threadIdx.x % TPR;
  const int64_t rows = p.batch * p.L * p.groups;
  const int C = (int)(p.channels / p.groups);
  const float inv_c = 1.0f / (float)C;
  const bool first = p.gate_first, gate = p.z.p != nullptr;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + threadIdx.x / TPR;
    const bool live = r < rows;
    const int64_t bl = live ? r / p.groups : 0, g0 = live ? (r % p.groups) * C : 0;
    const int64_t b = bl / p.L, l = bl % p.L;
    const TX* x = static_cast<const TX*>(p.x.p) + row_at(p.x, b, l) + g0;
    const TZ* z = gate ? static_cast<const TZ*>(p.z.p) + row_at(p.z, b, l) + g0 : nullptr;
    float t[NV][8], s[NV][8], ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = s[j][i] = 0.f;
      if (live && c < C) {
        load8<TX, VEC, kStep>(x + c, C - c, t[j]);
        if (gate) load8<TZ, VEC, kStep>(z + c, C - c, s[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (gate) s[j][i] *= sigmoid_f32(s[j][i]);
        if (first) t[j][i] *= s[j][i];
        ss[0] = fmaf(t[j][i], t[j][i], ss[0]);
      }
    row_sum<TPR, 1>(ss);
    const float inv = inv_sqrt(fmaf(ss[0], inv_c, p.eps));
    TY* y = static_cast<TY*>(p.y.p) + row_at(p.y, b, l) + g0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
      if (live && c < C) {
        float w[8];
        load8<float, VEC, kStep>(p.weight + g0 + c, C - c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = t[j][i] * inv * w[i];
          if (gate && !first) w[i] *= s[j][i];
        }
        store8<TY, VEC, kStep>(y + c, C - c, w);
      }
    }
  }
}

// Blocks walk the rows of one group (blockIdx.y), so that every lane keeps its channels.
template <typename TX, typename TZ, typename TY, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(TPR > kBlock ? TPR : kBlock) void gatenorm_bwd_kernel(GateNormArgs p, float* part) {
  constexpr int kRows = TPR > kBlock ? 1 : kBlock / TPR;
  constexpr int kStep = VEC ? 1 : TPR;
  const int lane = threadIdx.x % TPR;
  const int64_t rows = p.batch * p.L;
  const int C = (int)(p.channels / p.groups);
  const int64_t g0 = (int64_t)blockIdx.y * C;
  const float inv_c = 1.0f / (float)C;
  const bool first = p.gate_first, gate = p.z.p != nullptr;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = first_channel<TPR, VEC>(j, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[j][i] = dw[j][i] = 0.f;
    if (c < C) load8<float, VEC, kStep>(p.weight + g0 + c, C - c, w[j]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + threadIdx.x / TPR;
    const bool live = r < rows;
    const int64_t b = live ? r / p.L : 0, l = live ? r % p.L : 0;
    const TX* x = static_cast<const TX*>(p.x.p) + row_at(p.x, b, l) + g0;
    const TZ* z = gate ? static_cast<const TZ*>(p.z.p) + row_at(p.z, b, l) + g0 : nullptr;
    const TY* dy = static_cast<const TY*>(p.dy.p) + row_at(p.dy, b, l) + g0;
    float xv[NV][8], zv[NV][8], g[NV][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) xv[j][i] = zv[j][i] = g[j][i] = 0.f;
      if (live && c < C) {
        load8<TX, VEC, kStep>(x + c, C - c, xv[j]);
        load8<TY, VEC, kStep>(dy + c, C - c, g[j]);
        if (gate) load8<TZ, VEC, kStep>(z + c, C - c, zv[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = gate ? zv[j][i] * sigmoid_f32(zv[j][i]) : 1.f;
        const float t = first ? xv[j][i] * a : xv[j][i];
        const float d = first ? g[j][i] : g[j][i] * a;  // the gradient at norm(t) weight
        s[0] = fmaf(t, t, s[0]);
        s[1] = fmaf(d * w[j][i], t, s[1]);
      }
    row_sum<TPR, 2>(s);
    const float inv = inv_sqrt(fmaf(s[0], inv_c, p.eps));
    const float back = -(s[1] * inv_c) * inv * inv * inv;
    TX* dx = static_cast<TX*>(p.dx.p) + row_at(p.dx, b, l) + g0;
    TZ* dz = gate ? static_cast<TZ*>(p.dz.p) + row_at(p.dz, b, l) + g0 : nullptr;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = first_channel<TPR, VEC>(j, lane);
      if (live && c < C) {
        float ox[8], oz[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float zz = zv[j][i], sg = gate ? sigmoid_f32(zz) : 1.f, a = gate ? zz * sg : 1.f;
          const float slope = sg * fmaf(zz, 1.f - sg, 1.f);
          const float t = first ? xv[j][i] * a : xv[j][i];
          const float d = first ? g[j][i] : g[j][i] * a;
          const float dt = fmaf(d * w[j][i], inv, t * back);
          dw[j][i] = fmaf(d, t * inv, dw[j][i]);
          ox[i] = first ? dt * a : dt;
          oz[i] = (first ? dt * xv[j][i] : g[j][i] * (t * inv) * w[j][i]) * slope;
        }
        store8<TX, VEC, kStep>(dx + c, C - c, ox);
        if (gate) store8<TZ, VEC, kStep>(dz + c, C - c, oz);
      }
    }
  }
  if (part) store_partial<TPR, NV, VEC>(dw, part + (int64_t)blockIdx.x * p.channels + g0, C);
}

// dw[c] = sum over the blocks' partial rows, in a fixed order: 16 columns a block (64 bytes of a row),
// 64 teams that share the rows, eight loads in flight each, the teams' sums added through LDS.
constexpr int kSumCols = 16, kSumTeams = 64;
__global__ __launch_bounds__(kSumCols * kSumTeams) void column_sum_kernel(const float* __restrict__ part,
                                                                          float* __restrict__ dw, int64_t C, int64_t n) {
  __shared__ float acc[kSumTeams][kSumCols];
  const int lane = threadIdx.x % kSumCols, team = threadIdx.x / kSumCols;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + lane;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < C)
    for (int64_t r = team; r < n; r += 8 * kSumTeams)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r + k * kSumTeams < n) s[k] += part[(r + k * kSumTeams) * C + c];
  acc[team][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (team == 0 && c < C) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kSumTeams; ++k) v += acc[k][lane];
    dw[c] = v;
  }
}

// ------------------------------------------- any layout: channel or time innermost, per tensor

// A block takes TL = 8 TG tokens of one group; a thread holds 8 tokens of one channel, TG threads
// side by side along time, THREADS / TG channels a step.  A tensor with time innermost is read and
// written as it is (16 bytes of bf16, 32 of f32 a thread); one with channels innermost goes through
// an LDS tile, 16 bytes along the channels a thread.  x, z (and dy) are read twice, for the sums and
// for the result: a tile of 32 tokens, whose lines of 128 bytes (f32) are read whole, is larger than
// the registers and LDS of a CU, and narrower tiles that fit (8 or 16 tokens, read once) measured
// slower, 290 to 330 us against 243 at 2 x 5120 x 8192 (x in f32, z and y in bf16: 2.8 TB/s of the
// bytes that have to move, 4.8 of those that do).

struct Raw {
  u32x4 a, b;
};

// eight tokens of a channel with time innermost
template <bool VEC>
__device__ __forceinline__ Raw read_time(const NormRows& t, int64_t at, int n) {
  Raw r = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
  if (n <= 0) return r;
  if (VEC && n >= 8) {
    if (t.bf16) {
      r.a = *reinterpret_cast<const u32x4*>(static_cast<const bf16_t*>(t.p) + at);
    } else {
      r.a = *reinterpret_cast<const u32x4*>(static_cast<const float*>(t.p) + at);
      r.b = *reinterpret_cast<const u32x4*>(static_cast<const float*>(t.p) + at + 4);
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      const int64_t o = at + i * t.st;
      if (t.bf16) {
        const uint32_t x = static_cast<const bf16_t*>(t.p)[o].bits;
        r.a[i >> 1] |= x << (16 * (i & 1));
      } else if (i < 4) {
        r.a[i] = __float_as_uint(static_cast<const float*>(t.p)[o]);
      } else {
        r.b[i - 4] = __float_as_uint(static_cast<const float*>(t.p)[o]);
      }
    }
  return r;
}

__device__ __forceinline__ void widen(const Raw& r, bool bf16, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16 ? bf16_lo(r.a[i]) : __uint_as_float(i < 2 ? r.a[2 * i] : r.b[2 * i - 4]);
    v[2 * i + 1] = bf16 ? bf16_hi(r.a[i]) : __uint_as_float(i < 2 ? r.a[2 * i + 1] : r.b[2 * i - 3]);
  }
}

template <bool VEC>
__device__ __forceinline__ void write_time(const NormRows& t, int64_t at, int n, const float (&v)[8]) {
  if (VEC && n >= 8) {
    if (t.bf16) store8<bf16_t, true>(static_cast<bf16_t*>(t.p) + at, 8, v);
    else store8<float, true>(static_cast<float*>(t.p) + at, 8, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      if (t.bf16) store_one(static_cast<bf16_t*>(t.p) + at + i * t.st, v[i]);
      else static_cast<float*>(t.p)[at + i * t.st] = v[i];
    }
}

template <int THREADS, int TG, bool VEC>
struct Tile {
  static constexpr int kTokens = 8 * TG, kChannels = THREADS / TG;
  // pitch: the TG rows of a wave's read fall on different banks
  static constexpr int kPitch = kChannels + (TG == 4 ? 2 : 1);
  float (*lds)[kPitch];
  int64_t b, l0, c0;   // row, first token, first channel of the group
  int nt, C;           // tokens here, channels of the group
  int tg, ci;

  // the thread's tokens of channel step * kChannels + ci
  __device__ __forceinline__ void load(const NormRows& t, int step, bool time, float (&v)[8]) {
    int c = step * kChannels + ci;
    if (time) {
      // addresses of unrolled steps are made where they are used, not kept from the loop's start
      asm volatile("" : "+v"(c));
      const int n = c < C ? nt - 8 * tg : 0;
      widen(read_time<VEC>(t, b * t.sb + (l0 + 8 * tg) * t.st + (c0 + c) * t.sc, n), t.bf16, v);
      return;
    }
    __syncthreads();  // the tile's last readers are done
    constexpr int kPieces = kChannels / 4;
    for (int i = threadIdx.x; i < kTokens * kPieces; i += THREADS) {
      const int l = i / kPieces, k = i % kPieces * 4;
      const int left = l < nt ? C - (step * kChannels + k) : 0;
      const int64_t at = b * t.sb + (l0 + l) * t.st + c0 + step * kChannels + k;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (VEC && left >= 4) {
        if (t.bf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const bf16_t*>(t.p) + at);
          x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
        } else {
          const f32x4 w = *reinterpret_cast<const f32x4*>(static_cast<const float*>(t.p) + at);
          x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left)
            x[j] = t.bf16 ? to_f32(static_cast<const bf16_t*>(t.p)[at + j * t.sc])
                          : static_cast<const float*>(t.p)[at + j * t.sc];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) lds[l][k + j] = x[j];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lds[8 * tg + i][ci];
  }

  __device__ __forceinline__ void store(const NormRows& t, int step, bool time, const float (&v)[8]) {
    const int c = step * kChannels + ci;
    if (time) {
      const int n = c < C ? nt - 8 * tg : 0;
      write_time<VEC>(t, b * t.sb + (l0 + 8 * tg) * t.st + (c0 + c) * t.sc, n, v);
      return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) lds[8 * tg + i][ci] = v[i];
    __syncthreads();
    constexpr int kPieces = kChannels / 8;
    for (int i = threadIdx.x; i < kTokens * kPieces; i += THREADS) {
      const int l = i / kPieces, k = i % kPieces * 8;
      const int left = l < nt ? C - (step * kChannels + k) : 0;
      const int64_t at = b * t.sb + (l0 + l) * t.st + c0 + step * kChannels + k;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = lds[l][k + j];
      if (VEC && left >= 8) {
        if (t.bf16) store8<bf16_t, true>(static_cast<bf16_t*>(t.p) + at, 8, x);
        else store8<float, true>(static_cast<float*>(t.p) + at, 8, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) {
            if (t.bf16) store_one(static_cast<bf16_t*>(t.p) + at + j * t.sc, x[j]);
            else static_cast<float*>(t.p)[at + j * t.sc] = x[j];
          }
      }
    }
  }

  // sums over the group's channels for the thread's tokens, from every thread's own
  template <int N>
  __device__ __forceinline__ void token_sum(float (&s)[N][8], float (*red)[kTokens][N]) {
#pragma unroll
    for (int m = TG; m < 64; m <<= 1)
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[k][i] += __shfl_xor(s[k][i], m);
    __syncthreads();
    if ((threadIdx.x & 63) < TG)
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) red[threadIdx.x >> 6][8 * tg + i][k] = s[k][i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = 0.f;
        for (int w = 0; w < THREADS / 64; ++w) v += red[w][8 * tg + i][k];
        s[k][i] = v;
      }
  }
};

// whether a tensor is taken along time (else along channels)
__device__ __forceinline__ bool along_time(const NormRows& t) { return t.sc != 1; }

// the tile-th tile, with neighbours on one XCD
__device__ __forceinline__ int64_t xcd_order(int64_t i, int64_t n) {
  return n % 8 == 0 ? (i % 8) * (n / 8) + i / 8 : i;
}

template <int THREADS, int TG, bool VEC>
__global__ __launch_bounds__(THREADS) void gatenorm_any_fwd_kernel(GateNormArgs p, int64_t tiles) {
  typedef Tile<THREADS, TG, VEC> Tl;
  __shared__ float lds[Tl::kTokens][Tl::kPitch];
  __shared__ float red[THREADS / 64][Tl::kTokens][1];
  Tl t;
  t.lds = lds;
  t.tg = threadIdx.x % TG;
  t.ci = threadIdx.x / TG;
  t.C = (int)(p.channels / p.groups);
  const int64_t per_row = (p.L + Tl::kTokens - 1) / Tl::kTokens;
  const bool first = p.gate_first, gate = p.z.p != nullptr;
  const bool tx = along_time(p.x), tz = along_time(p.z), ty = along_time(p.y);
  const int steps = (t.C + Tl::kChannels - 1) / Tl::kChannels;
  for (int64_t i = blockIdx.x; i < tiles * p.groups; i += gridDim.x) {
    const int64_t k = xcd_order(i, tiles * p.groups), tile = k % tiles;
    t.c0 = k / tiles * t.C;
    t.b = tile / per_row;
    t.l0 = tile % per_row * Tl::kTokens;
    t.nt = (int)min((int64_t)Tl::kTokens, p.L - t.l0);
    float u[8], z[8], s[1][8], inv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0][e] = 0.f;
    for (int j = 0; j < steps; ++j) {
      t.load(p.x, j, tx, u);
      if (first) t.load(p.z, j, tz, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = first ? u[e] * z[e] * sigmoid_f32(z[e]) : u[e];
        s[0][e] = fmaf(v, v, s[0][e]);
      }
    }
    t.token_sum(s, red);
#pragma unroll
    for (int e = 0; e < 8; ++e) inv[e] = inv_sqrt(s[0][e] / (float)t.C + p.eps);
    for (int j = 0; j < steps; ++j) {
      t.load(p.x, j, tx, u);
      if (gate) t.load(p.z, j, tz, z);
      const int c = j * Tl::kChannels + t.ci;
      const float w = c < t.C ? p.weight[t.c0 + c] : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] *= inv[e] * w * (gate ? z[e] * sigmoid_f32(z[e]) : 1.f);
      t.store(p.y, j, ty, u);
    }
  }
}

template <int THREADS, int TG, bool VEC>
__global__ __launch_bounds__(THREADS) void gatenorm_any_bwd_kernel(GateNormArgs p, float* part, int64_t tiles) {
  typedef Tile<THREADS, TG, VEC> Tl;
  __shared__ float lds[Tl::kTokens][Tl::kPitch];
  __shared__ float red[THREADS / 64][Tl::kTokens][2];
  Tl t;
  t.lds = lds;
  t.tg = threadIdx.x % TG;
  t.ci = threadIdx.x / TG;
  t.C = (int)(p.channels / p.groups);
  t.c0 = (int64_t)blockIdx.y * t.C;
  const int64_t per_row = (p.L + Tl::kTokens - 1) / Tl::kTokens;
  const bool first = p.gate_first, gate = p.z.p != nullptr;
  const bool tx = along_time(p.x), tz = along_time(p.z), ty = along_time(p.dy);
  const bool tdx = along_time(p.dx), tdz = along_time(p.dz);
  const int steps = (t.C + Tl::kChannels - 1) / Tl::kChannels;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    t.b = tile / per_row;
    t.l0 = tile % per_row * Tl::kTokens;
    t.nt = (int)min((int64_t)Tl::kTokens, p.L - t.l0);
    float s[2][8], inv[8], back[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0][e] = s[1][e] = 0.f;
    for (int j = 0; j < steps; ++j) {
      const int c = j * Tl::kChannels + t.ci;
      const float w = c < t.C ? p.weight[t.c0 + c] : 0.f;
      float x[8], z[8], g[8];
      t.load(p.x, j, tx, x);
      t.load(p.dy, j, ty, g);
      if (gate) t.load(p.z, j, tz, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = gate ? z[e] * sigmoid_f32(z[e]) : 1.f;
        const float v = first ? x[e] * a : x[e], d = first ? g[e] : g[e] * a;
        s[0][e] = fmaf(v, v, s[0][e]);
        s[1][e] = fmaf(d * w, v, s[1][e]);
      }
    }
    t.token_sum(s, red);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // behind the last token: 0, since there 1 / sqrt(eps) may be infinite, and dw takes all eight
      inv[e] = 8 * t.tg + e < t.nt ? inv_sqrt(s[0][e] / (float)t.C + p.eps) : 0.f;
      back[e] = -(s[1][e] / (float)t.C) * inv[e] * inv[e] * inv[e];
    }
    for (int j = 0; j < steps; ++j) {
      const int c = j * Tl::kChannels + t.ci;
      const float w = c < t.C ? p.weight[t.c0 + c] : 0.f;
      float x[8], z[8], g[8], dw = 0.f;
      t.load(p.x, j, tx, x);
      t.load(p.dy, j, ty, g);
      if (gate) t.load(p.z, j, tz, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float sg = gate ? sigmoid_f32(z[e]) : 1.f, a = gate ? z[e] * sg : 1.f;
        const float v = first ? x[e] * a : x[e], d = first ? g[e] : g[e] * a;
        const float dt = fmaf(d * w, inv[e], v * back[e]);
        dw = fmaf(d, v * inv[e], dw);
        const float dz = (first ? dt * x[e] : g[e] * (v * inv[e]) * w) * sg * fmaf(gate ? z[e] : 0.f, 1.f - sg, 1.f);
        x[e] = first ? dt * a : dt;
        z[e] = dz;
      }
      t.store(p.dx, j, tdx, x);
      if (gate) t.store(p.dz, j, tdz, z);
      if (part) {
        // the block's sum for the channel, kept in the workspace from tile to tile
#pragma unroll
        for (int m = 1; m < TG; m <<= 1) dw += __shfl_xor(dw, m);
        if (t.tg == 0 && c < t.C) {
          float* at = part + (int64_t)blockIdx.x * p.channels + t.c0 + c;
          *at = tile == blockIdx.x ? dw : *at + dw;
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------ launch

// blocks of a persistent backward: their partial rows are the workspace
int64_t bwd_blocks(int64_t rows, int32_t groups) {
  const int64_t want = std::max<int64_t>(1, (int64_t)4 * cu_count() / groups);
  return std::min<int64_t>(rows, want);
}

// Lanes per row and steps of 8 channels per lane for rows of C channels: as few steps as hold the row,
// since a backward keeps four values a channel in registers (1024 lanes of 4 steps exceed them and
// spill: 5 x 325 rows of 11033, training, 385 us with 4 steps, 188 with 2).
struct Shape {
  int tpr, nv;
};
Shape shape_of(int64_t C, bool vec) {
  const int64_t n = (C + 7) / 8;
  if (vec) {
    if (n <= 16) return {16, 1};
    if (n <= 64) return {64, 1};
    if (n <= 128) return {64, 2};
    if (n <= 256) return {256, 1};
    if (n <= 512) return {256, 2};
    if (n <= 1024) return {256, 4};
  } else {
    if (n <= 64) return {64, 1};
    if (n <= 1024) return {256, 4};
  }
  if (n <= 2048) return {1024, 2};
  return {1024, 4};
}

#define SS_SHAPES(RUN)                                                                                   \
  if (vec) {                                                                                             \
    if (sh.tpr == 16) RUN(16, 1, true)                                                                   \
    else if (sh.tpr == 64 && sh.nv == 1) RUN(64, 1, true)                                                \
    else if (sh.tpr == 64) RUN(64, 2, true)                                                              \
    else if (sh.tpr == 256 && sh.nv == 1) RUN(256, 1, true)                                              \
    else if (sh.tpr == 256 && sh.nv == 2) RUN(256, 2, true)                                              \
    else if (sh.tpr == 256) RUN(256, 4, true)                                                            \
    else if (sh.nv == 2) RUN(1024, 2, true)                                                              \
    else RUN(1024, 4, true)                                                                              \
  } else {                                                                                               \
    if (sh.tpr == 64) RUN(64, 1, false)                                                                  \
    else if (sh.tpr == 256) RUN(256, 4, false)                                                           \
    else if (sh.nv == 2) RUN(1024, 2, false)                                                             \
    else RUN(1024, 4, false)                                                                             \
  }

dim3 block_of(Shape sh) { return dim3(sh.tpr > kBlock ? sh.tpr : kBlock); }
int64_t rows_of(Shape sh) { return sh.tpr > kBlock ? 1 : kBlock / sh.tpr; }

template <typename TX, typename TR, typename TY>
hipError_t addnorm_fwd_t(const AddNormArgs& a, hipStream_t s) {
  const bool vec = a.vec;
  const Shape sh = shape_of(a.channels, vec);
  const int64_t rows = a.batch * a.L, blocks = std::min<int64_t>((rows + rows_of(sh) - 1) / rows_of(sh), 1 << 20);
#define SS_RUN(T, N, V) hipLaunchKernelGGL((addnorm_fwd_kernel<TX, TR, TY, T, N, V>), dim3((unsigned)blocks), block_of(sh), 0, s, a);
  SS_SHAPES(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

template <typename TY, typename TR, typename TX>
hipError_t addnorm_bwd_t(const AddNormArgs& a, float* part, int64_t blocks, hipStream_t s) {
  const bool vec = a.vec;
  const Shape sh = shape_of(a.channels, vec);
#define SS_RUN(T, N, V) hipLaunchKernelGGL((addnorm_bwd_kernel<TY, TR, TX, T, N, V>), dim3((unsigned)blocks), block_of(sh), 0, s, a, part);
  SS_SHAPES(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

template <typename TX, typename TZ, typename TY>
hipError_t gatenorm_fwd_t(const GateNormArgs& a, hipStream_t s) {
  const bool vec = a.vec;
  const Shape sh = shape_of(a.channels / a.groups, vec);
  const int64_t rows = a.batch * a.L * a.groups;
  const int64_t blocks = std::min<int64_t>((rows + rows_of(sh) - 1) / rows_of(sh), 1 << 20);
#define SS_RUN(T, N, V) hipLaunchKernelGGL((gatenorm_fwd_kernel<TX, TZ, TY, T, N, V>), dim3((unsigned)blocks), block_of(sh), 0, s, a);
  SS_SHAPES(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

template <typename TX, typename TZ, typename TY>
hipError_t gatenorm_bwd_t(const GateNormArgs& a, float* part, int64_t blocks, hipStream_t s) {
  const bool vec = a.vec;
  const Shape sh = shape_of(a.channels / a.groups, vec);
  const dim3 grid((unsigned)blocks, (unsigned)a.groups);
#define SS_RUN(T, N, V) hipLaunchKernelGGL((gatenorm_bwd_kernel<TX, TZ, TY, T, N, V>), grid, block_of(sh), 0, s, a, part);
  SS_SHAPES(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

#define SS_TYPES(FN, X, Y, Z, ...)                                                                      \
  ((X) ? ((Y) ? ((Z) ? FN<bf16_t, bf16_t, bf16_t>(__VA_ARGS__) : FN<bf16_t, bf16_t, float>(__VA_ARGS__)) \
              : ((Z) ? FN<bf16_t, float, bf16_t>(__VA_ARGS__) : FN<bf16_t, float, float>(__VA_ARGS__)))  \
       : ((Y) ? ((Z) ? FN<float, bf16_t, bf16_t>(__VA_ARGS__) : FN<float, bf16_t, float>(__VA_ARGS__))   \
              : ((Z) ? FN<float, float, bf16_t>(__VA_ARGS__) : FN<float, float, float>(__VA_ARGS__))))

}  // namespace

hipError_t launch_column_sum(const float* part, float* out, int64_t C, int64_t n, hipStream_t s) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((C + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumTeams),
                     0, s, part, out, C, n);
  return hipGetLastError();
}

int64_t norm_workspace_floats(int64_t batch, int64_t L, int64_t channels, int32_t groups) {
  return bwd_blocks(batch * L, groups) * channels;
}

hipError_t launch_addnorm_fwd(const AddNormArgs& a, hipStream_t s) {
  const bool rb = a.residual.p ? a.residual.bf16 : a.sum.bf16;
  return SS_TYPES(addnorm_fwd_t, a.x.bf16, rb, a.y.bf16, a, s);
}

hipError_t launch_addnorm_bwd(const AddNormArgs& a, float* ws, hipStream_t s) {
  const int64_t blocks = bwd_blocks(a.batch * a.L, 1);
  float* part = a.dweight ? ws : nullptr;
  if (blocks > 0) {
    const bool xb = a.dx.p ? a.dx.bf16 : a.dy.bf16;
    const hipError_t e = SS_TYPES(addnorm_bwd_t, a.dy.bf16, a.sum.bf16, xb, a, part, blocks, s);
    if (e != hipSuccess) return e;
  }
  return a.dweight ? launch_column_sum(part, a.dweight, a.channels, blocks, s) : hipSuccess;
}

hipError_t launch_gatenorm_fwd(const GateNormArgs& a, hipStream_t s) {
  const bool zb = a.z.p ? a.z.bf16 : a.x.bf16;
  if (a.rows) return SS_TYPES(gatenorm_fwd_t, a.x.bf16, zb, a.y.bf16, a, s);
  // more than 256 channels: 32 tokens by 128 channels a step; fewer: 64 tokens by 32
  const int64_t C = a.channels / a.groups, tl = C > 256 ? 32 : 64;
  const int64_t tiles = a.batch * ((a.L + tl - 1) / tl);
  const dim3 grid((unsigned)std::min<int64_t>(tiles * a.groups, 1 << 21));
#define SS_ANY(TH, TG, V) hipLaunchKernelGGL((gatenorm_any_fwd_kernel<TH, TG, V>), grid, dim3(TH), 0, s, a, tiles)
  if (C <= 256) {
    if (a.any_vec) SS_ANY(256, 8, true); else SS_ANY(256, 8, false);
  } else {
    if (a.any_vec) SS_ANY(512, 4, true); else SS_ANY(512, 4, false);
  }
#undef SS_ANY
  return hipGetLastError();
}

hipError_t launch_gatenorm_bwd(const GateNormArgs& a, float* ws, hipStream_t s) {
  int64_t blocks = bwd_blocks(a.batch * a.L, a.groups);
  float* part = a.dweight ? ws : nullptr;
  if (blocks > 0) {
    hipError_t e;
    if (a.rows) {
      const bool zb = a.z.p ? a.z.bf16 : a.x.bf16;
      e = SS_TYPES(gatenorm_bwd_t, a.x.bf16, zb, a.dy.bf16, a, part, blocks, s);
    } else {
      const int64_t C = a.channels / a.groups, tl = C > 256 ? 32 : 64;
      const int64_t tiles = a.batch * ((a.L + tl - 1) / tl);
      blocks = std::min(blocks, tiles);
      const dim3 grid((unsigned)blocks, (unsigned)a.groups);
#define SS_ANY(TH, TG)                                                                                             \
  do {                                                                                                             \
    if (a.any_vec) hipLaunchKernelGGL((gatenorm_any_bwd_kernel<TH, TG, true>), grid, dim3(TH), 0, s, a, part, tiles); \
    else hipLaunchKernelGGL((gatenorm_any_bwd_kernel<TH, TG, false>), grid, dim3(TH), 0, s, a, part, tiles);       \
  } while (0)
      if (C > 256) SS_ANY(512, 4);
      else SS_ANY(256, 8);
#undef SS_ANY
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  return a.dweight ? launch_column_sum(part, a.dweight, a.channels, blocks, s) : hipSuccess;
}

}  // namespace ss
