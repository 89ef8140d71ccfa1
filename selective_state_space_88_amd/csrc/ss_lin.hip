// ss_lin.hip -- linear attention with one fixed decay per head (gfx950).
//
// The recurrence itself, token by token (see LinArgs for the three forms it serves): a block keeps a
// [D, 16] part of one head's state in registers, 16 lanes along d for each of 16 columns e.
#include <algorithm>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

constexpr int kMaxD = 256;

// lam = exp(log_decay); NaN stays NaN, -infinity gives 0
__device__ __forceinline__ float decay_of(float log_decay) { return expf(log_decay); }

template <typename T, typename TO>
__global__ __launch_bounds__(256) void lin_walk_kernel(LinArgs p) {
  const int dl = threadIdx.x & 15, el = threadIdx.x >> 4;
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / p.heads, h = bh % p.heads;
  const int e = blockIdx.y * 16 + el;
  const bool le = e < p.E;
  int64_t n = p.L;
  if (p.lengths) n = min(max((int64_t)p.lengths[b], (int64_t)0), p.L);
  const float lam = decay_of(p.log_decay[h]);
  float z[kMaxD / 16];
#pragma unroll
  for (int i = 0; i < kMaxD / 16; ++i) {
    const int d = dl + 16 * i;
    z[i] = p.z_in && le && d < p.D ? p.z_in[b * p.zi_sb + h * p.zi_sh + d * p.zi_sd + e * p.zi_se] : 0.f;
  }
  const T* A = static_cast<const T*>(p.a.p) + b * p.a.sb + h / p.a.share * p.a.sh;
  const T* B = static_cast<const T*>(p.b.p) + b * p.b.sb + h / p.b.share * p.b.sh;
  const T* C = static_cast<const T*>(p.c.p) + b * p.c.sb + h / p.c.share * p.c.sh;
  TO* O = static_cast<TO*>(p.o) + b * p.o_sb + h * p.o_sh;
  for (int64_t r = 0; r < n; ++r) {
    const int64_t t = p.reverse ? n - 1 - r : r;
    const float c = le ? to_f32(C[t * p.c.st + e]) * p.pair_scale : 0.f;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxD / 16; ++i) {
      const int d = dl + 16 * i;
      if (d < p.D) {
        const float x = p.e0 ? lam * z[i] : z[i];
        z[i] = fmaf(to_f32(B[t * p.b.st + d]), c, x);
        o = fmaf(to_f32(A[t * p.a.st + d]), z[i], o);
        if (!p.e0) z[i] *= lam;
      }
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) o += __shfl_xor(o, m);
    if (dl == 0 && le) store_one(O + t * p.o_st + e, o * p.out_scale);
  }
  for (int64_t t = n + dl; t < p.L; t += 16)
    if (le) store_one(O + t * p.o_st + e, 0.f);
  if (p.z_out && le)
#pragma unroll
    for (int i = 0; i < kMaxD / 16; ++i) {
      const int d = dl + 16 * i;
      if (d < p.D) p.z_out[b * p.zo_sb + h * p.zo_sh + d * p.zo_sd + e * p.zo_se] = z[i];
    }
}

__global__ __launch_bounds__(256) void head_sum_kernel(const float* __restrict__ src, void* dst, int64_t d_sb,
                                                       int64_t d_st, int64_t d_sh, int bf16, int64_t L, int heads,
                                                       int share, int D, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / D, d = i - row * D;
    const int64_t bl = row / heads, h = row - bl * heads;
    const int64_t b = bl / L, l = bl - b * L;
    const float* s = src + row * share * D + d;
    float v = 0.f;
    for (int k = 0; k < share; ++k) v += s[(int64_t)k * D];
    const int64_t at = b * d_sb + l * d_st + h * d_sh + d;
    if (bf16) store_one(static_cast<bf16_t*>(dst) + at, v);
    else static_cast<float*>(dst)[at] = v;
  }
}

// One token: a block takes 16 columns of one head's state.
template <typename T, typename TO>
__global__ __launch_bounds__(256) void lin_step_kernel(LinStepArgs p) {
  __shared__ float red[16][17];
  const int vl = threadIdx.x & 15, kl = threadIdx.x >> 4;
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / p.heads, h = bh % p.heads;
  const int e = blockIdx.y * 16 + vl;
  const bool le = e < p.V;
  const float lam = decay_of(p.log_decay[h]);
  const T* q = static_cast<const T*>(p.q.p) + b * p.q.sb + h / p.q.share * p.q.sh;
  const T* k = static_cast<const T*>(p.k.p) + b * p.k.sb + h / p.k.share * p.k.sh;
  const T* v = static_cast<const T*>(p.v.p) + b * p.v.sb + h / p.v.share * p.v.sh;
  const float* s = p.s + b * p.s_sb + h * p.s_sh + e;
  float* so = p.s_out + b * p.so_sb + h * p.so_sh + e;
  float acc = 0.f;
  if (le) {
    const float vv = to_f32(v[e]);
    for (int d = kl; d < p.K; d += 16) {
      const float x = fmaf(to_f32(k[d]), vv, lam * s[d * p.s_sk]);
      so[d * p.so_sk] = x;
      acc = fmaf(to_f32(q[d]), x, acc);
    }
  }
  red[kl][vl] = acc;
  __syncthreads();
  if (kl == 0 && le) {
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o += red[i][vl];
    store_one(static_cast<TO*>(p.o) + b * p.o_sb + h * p.o_sh + e, o * p.scale);
  }
}

}  // namespace

int64_t lin_workspace_floats(const LinArgs*, int) { return 0; }

hipError_t launch_lin(const LinArgs* a, int n, float*, hipStream_t s) {
  for (int i = 0; i < n; ++i) {
    const dim3 grid((unsigned)(a[i].batch * a[i].heads), (unsigned)((a[i].E + 15) / 16));
    if (!a[i].bf16) hipLaunchKernelGGL((lin_walk_kernel<float, float>), grid, dim3(256), 0, s, a[i]);
    else if (a[i].o_f32) hipLaunchKernelGGL((lin_walk_kernel<bf16_t, float>), grid, dim3(256), 0, s, a[i]);
    else hipLaunchKernelGGL((lin_walk_kernel<bf16_t, bf16_t>), grid, dim3(256), 0, s, a[i]);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_head_sum(const float* src, void* dst, int64_t d_sb, int64_t d_st, int64_t d_sh, int bf16,
                           int64_t batch, int64_t L, int32_t heads, int32_t share, int32_t D, hipStream_t s) {
  const int64_t total = batch * L * heads * D;
  if (total == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, 1 << 20);
  hipLaunchKernelGGL(head_sum_kernel, dim3((unsigned)blocks), dim3(256), 0, s, src, dst, d_sb, d_st, d_sh, bf16, L,
                     heads, share, D, total);
  return hipGetLastError();
}

hipError_t launch_lin_step(const LinStepArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.heads), (unsigned)((a.V + 15) / 16));
  if (a.in_bf16) {
    if (a.out_bf16) hipLaunchKernelGGL((lin_step_kernel<bf16_t, bf16_t>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((lin_step_kernel<bf16_t, float>), grid, dim3(256), 0, s, a);
  } else {
    if (a.out_bf16) hipLaunchKernelGGL((lin_step_kernel<float, bf16_t>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((lin_step_kernel<float, float>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace ss
