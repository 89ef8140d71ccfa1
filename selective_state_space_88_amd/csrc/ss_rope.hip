// ss_rope.hip -- rotary positions on one or two tensors (gfx950).
//
// out = (a cos t - b sin t, a sin t + b cos t) amp for every pair of a head's rotated features, the
// rest copied; t = position * inv_freq.  The turns t / 2 pi are formed in f64 with their whole part
// dropped before a product is rounded (rounded first it is off by position 2^-53 turns, 0.1 rad at
// 2^50), so a far position costs no precision; cos and sin of what is left are f32.
//
// Bound by HBM: every feature is read and written once.  The angle depends on the token and the pair
// only, so a thread takes one token and P pairs, computes their cos and sin once, and walks heads.
// P pairs are two 16-byte accesses (8 pairs in bf16, 4 in f32): (i, i + n) reads two places of the
// head, (2 i, 2 i + 1) one run.  Heads are split over threads only as far as that is needed to fill
// the chip (eight blocks a CU), since every split repeats the angles.  Measured on 2 x 8192 tokens, 32 and
// 8 heads of 128 in bf16: 75 us, 4.4 TB/s (a large copy: 4.7).
#include <algorithm>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr double kInv2Pi = 0.15915494309189535, kInv2PiLo = -9.839338337591243e-18;  // 1 / 2 pi, its rounding's rest

template <typename T, int P>
struct Run {
  T v[P];
};
template <>
struct Run<bf16_t, 8> {
  u32x4 v;
};
template <>
struct Run<float, 4> {
  f32x4 v;
};

__device__ __forceinline__ void widen(const Run<bf16_t, 8>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(r.v[i]);
    f[2 * i + 1] = bf16_hi(r.v[i]);
  }
}
__device__ __forceinline__ void widen(const Run<float, 4>& r, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = r.v[i];
}
template <typename T>
__device__ __forceinline__ void widen(const Run<T, 1>& r, float (&f)[1]) {
  f[0] = to_f32(r.v[0]);
}
__device__ __forceinline__ void narrow(const float (&f)[8], Run<bf16_t, 8>& r) {
  r.v = u32x4{pk_bf16(f[0], f[1]), pk_bf16(f[2], f[3]), pk_bf16(f[4], f[5]), pk_bf16(f[6], f[7])};
}
__device__ __forceinline__ void narrow(const float (&f)[4], Run<float, 4>& r) { r.v = f32x4{f[0], f[1], f[2], f[3]}; }
template <typename T>
__device__ __forceinline__ void narrow(const float (&f)[1], Run<T, 1>& r) {
  store_one(&r.v[0], f[0]);
}

// Unit u of a token: the P pairs from P u on (u < units_rot), or P features behind the rotated ones
// to copy.  Threads are (token, unit) pairs, blockIdx.y a split of the heads.
template <typename T, int P, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs p, int units_rot, int units, int64_t total) {
  typedef Run<T, P> R;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t tok = i / units;
    const int u = (int)(i - tok * units);
    const int64_t b = tok / p.L, l = tok - b * p.L;
    const bool rot = u < units_rot;
    float cs[P], sn[P];
    if (rot) {
      const int64_t pos = p.pos ? (int64_t)p.pos[b * p.p_sb + l * p.p_st] : p.pos0 + l;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        // position inv_freq / 2 pi with inv_freq / 2 pi in two parts; the first product's whole turns go
        // before it is rounded
        const double f = (double)p.inv_freq[u * P + k], f_hi = f * kInv2Pi, f_lo = fma(f, kInv2Pi, -f_hi) + f * kInv2PiLo;
        const double at = (double)pos, turns = fma(at, f_hi, -rint(at * f_hi)) + at * f_lo;
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[k] = c * p.amp;
        sn[k] = (p.inverse ? -s : s) * p.amp;
      }
    }
    // places of the two runs inside a head
    const int at0 = rot ? (INTER ? 2 * P * u : P * u) : 2 * p.n + P * (u - units_rot);
    const int at1 = INTER ? at0 + P : at0 + p.n;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const auto& t = p.t[k];
      if (!rot && !t.copy) continue;
      const T* x = static_cast<const T*>(t.x) + b * t.x_sb + l * t.x_st;
      T* out = static_cast<T*>(t.out) + b * t.o_sb + l * t.o_st;
#pragma unroll 4
      for (int h = blockIdx.y; h < t.heads; h += gridDim.y) {
        const T* xh = x + h * t.x_sh;
        T* oh = out + h * t.o_sh;
        if (!rot) {
          *reinterpret_cast<R*>(oh + at0) = *reinterpret_cast<const R*>(xh + at0);
          continue;
        }
        R r0 = *reinterpret_cast<const R*>(xh + at0), r1 = *reinterpret_cast<const R*>(xh + at1);
        float f[2][P], g[2][P];
        widen(r0, f[0]);
        widen(r1, f[1]);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          if constexpr (INTER) {
            const float a0 = f[(2 * e) / P][(2 * e) % P], b0 = f[(2 * e + 1) / P][(2 * e + 1) % P];
            g[(2 * e) / P][(2 * e) % P] = fmaf(a0, cs[e], -b0 * sn[e]);
            g[(2 * e + 1) / P][(2 * e + 1) % P] = fmaf(a0, sn[e], b0 * cs[e]);
          } else {
            g[0][e] = fmaf(f[0][e], cs[e], -f[1][e] * sn[e]);
            g[1][e] = fmaf(f[0][e], sn[e], f[1][e] * cs[e]);
          }
        }
        narrow(g[0], r0);
        narrow(g[1], r1);
        *reinterpret_cast<R*>(oh + at0) = r0;
        *reinterpret_cast<R*>(oh + at1) = r1;
      }
    }
  }
}

template <typename T, int P>
hipError_t launch_p(const RopeArgs& a, hipStream_t s) {
  const int units_rot = a.n / P;
  const bool copies = a.t[0].copy || a.t[1].copy;
  const int units = units_rot + (copies ? (a.dim - 2 * a.n) / P : 0);
  if (units == 0) return hipSuccess;
  const int64_t total = a.batch * a.L * units;
  const int64_t blocks = std::min<int64_t>((total + kThreads - 1) / kThreads, 1 << 22);
  const int heads = std::max(a.t[0].heads, a.t[1].heads);
  const int64_t splits = std::min<int64_t>(heads, std::max<int64_t>(1, 8 * cu_count() / blocks));
  const dim3 grid((unsigned)blocks, (unsigned)splits);
  if (a.interleaved)
    hipLaunchKernelGGL((rope_kernel<T, P, true>), grid, dim3(kThreads), 0, s, a, units_rot, units, total);
  else
    hipLaunchKernelGGL((rope_kernel<T, P, false>), grid, dim3(kThreads), 0, s, a, units_rot, units, total);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  const int wide = a.bf16 ? 8 : 4;
  const bool vec = a.vec && a.n % wide == 0 && (a.dim - 2 * a.n) % wide == 0;
  if (a.bf16) return vec ? launch_p<bf16_t, 8>(a, s) : launch_p<bf16_t, 1>(a, s);
  return vec ? launch_p<float, 4>(a, s) : launch_p<float, 1>(a, s);
}

}  // namespace ss
