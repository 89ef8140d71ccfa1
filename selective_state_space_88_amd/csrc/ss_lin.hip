// ss_lin.hip -- linear attention with one fixed decay per head, in its chunked matrix form (gfx950).
//
// Method.  Over a chunk of T tokens the recurrence (LinArgs: its three forms) is, with lam the
// head's decay, M_ij = lam^(i-j) for j <= i and Z [D, E] the state entering the chunk,
//   O  = (A B^T o M) C + diag(lam^(i + e0)) A Z        Z' = lam^T Z + B^T diag(lam^(T - j - e0)) C
// four dense products.  All powers of lam have exponents >= 0 and are taken directly, so neither a
// strong decay (down to 0) nor a long chunk overflows; lam^T enters as 1 + expm1(T g), added as
// Z + expm1 Z, so that a decay near 1 loses nothing in f32 over many chunks.
//
// Mapping.  A block of four waves takes one (row, head), a tile of columns of E and a segment of the
// row, and walks its chunks in order.  Wave w owns 16 NE of the columns and keeps Z for them in
// MFMA accumulators over the whole walk.  A 16x16 accumulator tile holds rows 4 g .. 4 g + 3 (g =
// lane / 16) of column lane % 16, so with the contraction index of every product put in the order
// (16 (2 k + e / 4) + 4 g + e % 4: slot e of lane group g in step k) Z is an operand straight from
// its accumulators; rows of A and B are read in that order as two pieces of four, and C and B^T
// (contraction over tokens) come from LDS through the transposing read, four tokens a lane.  The
// masked scores are formed transposed, so that a lane holds four neighbouring j of one i: they go to
// LDS as one piece and come back in the same order.  The products are taken as O^T, so that a lane
// holds four neighbouring columns of one token for its store.
//
// Types.  bf16 inputs run on v_mfma_f32_16x16x32_bf16: the inputs are exact operands; the masked
// scores and the copy of Z that A reads are rounded to bf16 (factors of a bf16 output: an error of
// its own last place); the weighted C of the state update is split in bf16 hi + lo, so Z keeps f32
// accuracy over any number of chunks.  f32 inputs run on v_mfma_f32_16x16x4_f32, nothing rounded.
//
// Few rows: the row is cut into segments.  A pre-pass of the same walk without the outputs forms
// each segment's own part of the state, a small kernel turns these into the states that the segments
// start from.
#include <algorithm>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kMaxD = 256;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// exponents are multiples of g log2 e; -infinity (no memory) becomes a number whose products with 0
// are 0 and whose powers are 0, NaN stays
__device__ __forceinline__ float log2_decay(float log_decay) {
  return log_decay < -1e30f ? -1e30f : log_decay * kLog2e;
}
__device__ __forceinline__ float power(float l2, int n) { return __builtin_amdgcn_exp2f(l2 * (float)n); }

// ---- per element type: an operand of 8 values a lane, and the product of two

template <typename T>
struct Mma;

template <>
struct Mma<bf16_t> {
  static constexpr int kChunk = 64;  // tokens
  typedef bf16x8 Frag;
  typedef u32x2 Four;
  static __device__ __forceinline__ Frag join(Four a, Four b) {
    return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
  }
  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Four narrow(const float (&v)[4]) {
    return u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
  }
};

template <>
struct Mma<float> {
  static constexpr int kChunk = 32;
  struct Frag {
    float v[8];
  };
  typedef f32x4 Four;
  static __device__ __forceinline__ Frag join(Four a, Four b) {
    return Frag{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Four narrow(const float (&v)[4]) { return f32x4{v[0], v[1], v[2], v[3]}; }
};

// ---- LDS tiles [rows][W] of T.  16-byte pieces of a row are permuted by the row, so that both the
// row reads (16 rows, one piece) and the transposing reads (8 rows, two pieces) meet every bank once.
template <typename T, int W>
__device__ __forceinline__ int place(int row, int col) {
  constexpr int kBytes = W * (int)sizeof(T), kPieces = kBytes / 16;
  constexpr int kRows = kBytes >= 256 ? 1 : 256 / kBytes;  // rows that share the 64 banks
  int f;
  if constexpr (sizeof(T) == 2)
    f = (((row / kRows) & (8 / kRows - 1)) << 1) | ((row >> 3) & 1);
  else
    f = (row / kRows) & (kPieces < 16 ? kPieces - 1 : 15);
  const int at = col * (int)sizeof(T);
  return row * kBytes + (((at >> 4) ^ f) << 4) + (at & 15);
}

// row `row` as an operand: the 8 values of step ks
template <typename T, int W>
__device__ __forceinline__ typename Mma<T>::Frag row_frag(const uint8_t* tile, int row, int ks, int g) {
  typedef typename Mma<T>::Four Four;
  const Four a = *reinterpret_cast<const Four*>(tile + place<T, W>(row, 32 * ks + 4 * g));
  const Four b = *reinterpret_cast<const Four*>(tile + place<T, W>(row, 32 * ks + 16 + 4 * g));
  return Mma<T>::join(a, b);
}

// column c0 + lane % 16 as an operand: the 8 rows (tokens) of step ks
template <typename T, int W>
__device__ __forceinline__ typename Mma<T>::Frag col_frag(const uint8_t* tile, int c0, int ks, int lane) {
  const int g = lane >> 4, q = lane & 15;
  if constexpr (sizeof(T) == 2) {
    u32x2 r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = place<T, W>(32 * ks + 16 * i + 4 * g + (q >> 2), c0 + 4 * (q & 3));
      r[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(tile + at)));
    }
    return Mma<T>::join(r[0], r[1]);
  } else {
    typename Mma<T>::Frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.v[e] = *reinterpret_cast<const float*>(tile + place<T, W>(32 * ks + 16 * (e >> 2) + 4 * g + (e & 3), c0 + q));
    return f;
  }
}

// ---- a chunk of rows on its way from HBM to LDS, in registers

template <typename T, int W, int ROWS, bool VEC>
struct Stage {
  static constexpr int kPer = 16 / (int)sizeof(T);  // values of a 16-byte piece
  static constexpr int kPieces = W / kPer;
  static constexpr int kN = (ROWS * kPieces + kThreads - 1) / kThreads;
  u32x4 v[kN];

  // rows r0 .. r0 + ROWS of the walk (token t at base + t step), those from `rows` on and the
  // columns from `cols` on as zero
  __device__ __forceinline__ void load(const T* base, int64_t step, int rows, int cols) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int id = i * kThreads + threadIdx.x;
      const int row = id / kPieces, c = id % kPieces * kPer;
      v[i] = u32x4{0, 0, 0, 0};
      if (row < rows && c < cols) {
        const T* p = base + row * step + c;
        if constexpr (VEC) {
          v[i] = *reinterpret_cast<const u32x4*>(p);
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            if constexpr (sizeof(T) == 2) {
              const uint32_t x = c + j < cols ? p[j].bits : 0u;
              v[i][j >> 1] |= x << (16 * (j & 1));
            } else {
              v[i][j] = c + j < cols ? __float_as_uint(p[j]) : 0u;
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ void store(uint8_t* tile) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int id = i * kThreads + threadIdx.x;
      const int row = id / kPieces, c = id % kPieces * kPer;
      if (ROWS * kPieces % kThreads == 0 || row < ROWS) *reinterpret_cast<u32x4*>(tile + place<T, W>(row, c)) = v[i];
    }
  }
};

// x = hi + lo in bf16 for eight values
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8& hi, bf16x8& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = pk_bf16(x[2 * j], x[2 * j + 1]);
    l[j] = pk_bf16(x[2 * j] - bf16_lo(h[j]), x[2 * j + 1] - bf16_hi(h[j]));
  }
  hi = __builtin_bit_cast(bf16x8, u32x4{h[0], h[1], h[2], h[3]});
  lo = __builtin_bit_cast(bf16x8, u32x4{l[0], l[1], l[2], l[3]});
}

// How a row is cut: segments of `len` tokens (a multiple of every chunk size).
struct Cut {
  int64_t len;
  int32_t n, etiles;
  float* z;  // [batch heads][n][D][E], n > 1: the states that the segments start from
};

// The state update of a chunk: acc[m][e] (rows 16 m .., columns of this wave) += B^T (w o C).
template <typename T, int D32, int NE>
__device__ __forceinline__ void update(f32x4 (&z)[2 * D32][NE], const uint8_t* sB, const uint8_t* sC,
                                       const float (&w)[Mma<T>::kChunk / 32][8], int wave, int lane) {
  constexpr int kKs = Mma<T>::kChunk / 32;
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    if constexpr (sizeof(T) == 2) {
      bf16x8 hi[NE], lo[NE];
#pragma unroll
      for (int n = 0; n < NE; ++n) {
        const u32x4 c = __builtin_bit_cast(u32x4, col_frag<T, 64 * NE>(sC, 16 * (wave * NE + n), ks, lane));
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = bf16_lo(c[e]) * w[ks][2 * e];
          x[2 * e + 1] = bf16_hi(c[e]) * w[ks][2 * e + 1];
        }
        split8(x, hi[n], lo[n]);
      }
#pragma unroll
      for (int m = 0; m < 2 * D32; ++m) {
        const bf16x8 b = col_frag<T, 32 * D32>(sB, 16 * m, ks, lane);
#pragma unroll
        for (int n = 0; n < NE; ++n) {
          z[m][n] = Mma<T>::mma(b, hi[n], z[m][n]);
          z[m][n] = Mma<T>::mma(b, lo[n], z[m][n]);
        }
      }
    } else {
      typename Mma<T>::Frag c[NE];
#pragma unroll
      for (int n = 0; n < NE; ++n) {
        c[n] = col_frag<T, 64 * NE>(sC, 16 * (wave * NE + n), ks, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[n].v[e] *= w[ks][e];
      }
#pragma unroll
      for (int m = 0; m < 2 * D32; ++m) {
        const typename Mma<T>::Frag b = col_frag<T, 32 * D32>(sB, 16 * m, ks, lane);
#pragma unroll
        for (int n = 0; n < NE; ++n) z[m][n] = Mma<T>::mma(b, c[n], z[m][n]);
      }
    }
  }
}

// OUT: the walk with outputs; else only the segment's own part of the state, from zero.
template <typename T, typename TO, int D32, int NE, bool VEC, bool OUT>
__global__ __launch_bounds__(kThreads, D32 == 8 || !VEC ? 1 : 2) void lin_kernel(LinArgs p, Cut cut) {
  constexpr int kT = Mma<T>::kChunk, kD = 32 * D32, kE = 64 * NE, kKs = kT / 32, kIt = kT / 16;
  typedef Mma<T> M;
  __shared__ __align__(16) uint8_t sA[OUT ? kT * kD * sizeof(T) : 16], sB[kT * kD * sizeof(T)], sC[kT * kE * sizeof(T)],
      sP[OUT ? kT * kT * sizeof(T) : 16];
  const int lane0 = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane0 >> 4, q = lane0 & 15;
  // neighbouring blocks (tiles of one head, heads of one segment: shared operands) on one XCD
  int64_t id = blockIdx.x;
  if (gridDim.x % 8 == 0) id = (id % 8) * (gridDim.x / 8) + id / 8;
  const int et = (int)(id % cut.etiles);
  id /= cut.etiles;
  const int h = (int)(id % p.heads);
  id /= p.heads;
  const int seg = (int)(id % cut.n);
  const int64_t b = id / cut.n, bh = b * p.heads + h;
  const int e0 = et * kE + wave * 16 * NE;  // this wave's first column

  int64_t len = p.L;
  if (p.lengths) len = min(max((int64_t)p.lengths[b], (int64_t)0), p.L);
  const int64_t r0 = seg * cut.len, r_end = min(r0 + cut.len, p.L), r1 = min(r_end, len);
  if (!OUT && r0 >= r1) return;  // no token: the segment's part is never read
  const float g_ln = p.log_decay[h], l2 = log2_decay(g_ln);

  f32x4 z[2 * D32][NE];
  float* zs = cut.n > 1 ? cut.z + (bh * cut.n + seg) * p.D * (int64_t)p.E : nullptr;
#pragma unroll
  for (int m = 0; m < 2 * D32; ++m)
#pragma unroll
    for (int n = 0; n < NE; ++n) {
      z[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int e = e0 + 16 * n + q;
      if (OUT && e < p.E && (zs || p.z_in))
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 16 * m + 4 * g + r;
          if (d < p.D)
            z[m][n][r] = zs ? zs[(int64_t)d * p.E + e]
                            : p.z_in[b * p.zi_sb + h * p.zi_sh + d * p.zi_sd + e * p.zi_se];
        }
    }

  const T* A = static_cast<const T*>(p.a.p) + b * p.a.sb + h / p.a.share * p.a.sh;
  const T* B = static_cast<const T*>(p.b.p) + b * p.b.sb + h / p.b.share * p.b.sh;
  const T* C = static_cast<const T*>(p.c.p) + b * p.c.sb + h / p.c.share * p.c.sh + et * kE;
  TO* O = static_cast<TO*>(p.o) + b * p.o_sb + h * p.o_sh;
  const int64_t t0 = p.reverse ? len - 1 : 0, dir = p.reverse ? -1 : 1;
  const int ecols = p.E - et * kE;

  Stage<T, kD, kT, VEC> a_in, b_in;
  Stage<T, kE, kT, VEC> c_in;
  auto fetch = [&](int64_t r) {
    const int rows = (int)min((int64_t)kT, r1 - r);
    const int64_t t = t0 + dir * r;
    if (OUT) a_in.load(A + t * p.a.st, dir * p.a.st, rows, p.D);
    b_in.load(B + t * p.b.st, dir * p.b.st, rows, p.D);
    c_in.load(C + t * p.c.st, dir * p.c.st, rows, ecols);
  };

  // weights of a chunk of n tokens: w on token j's part of the state, em on the state itself
  float w[kKs][8], em = 0.f;
  auto weights = [&](int n) {
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int left = n - p.e0 - (32 * ks + 16 * (e >> 2) + 4 * g + (e & 3));
        w[ks][e] = left >= 0 ? p.pair_scale * power(l2, left) : 0.f;
      }
    em = l2 <= -1e30f ? -1.f : expm1f(g_ln * (float)n);
  };
  float since[kIt];  // lam^(i + e0) of this lane's token in each tile
#pragma unroll
  for (int i = 0; i < kIt; ++i) since[i] = power(l2, 16 * i + q + p.e0);

  if (r0 < r1) fetch(r0);
  int cur = 0;
  for (int64_t r = r0; r < r1; r += kT) {
    // the LDS addresses are a few operations on the lane number: made anew in every chunk, since
    // kept over the loop they would push the state out of the registers
    int lane = lane0;
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4, q = lane & 15;
    const int n = (int)min((int64_t)kT, r1 - r);
    if (n != cur) weights(cur = n);
    if (OUT) a_in.store(sA);
    b_in.store(sB);
    c_in.store(sC);
    __syncthreads();
    if (r + kT < r1) fetch(r + kT);

    f32x4 o[kIt][NE];
    if constexpr (OUT) {
      // masked scores, transposed: tile (it, jt) with lane i = 16 it + q, rows j = 16 jt + 4 g + r
      const int it = kIt == 4 ? wave : wave >> 1;
      typename M::Frag qa[D32];
#pragma unroll
      for (int ks = 0; ks < D32; ++ks) qa[ks] = row_frag<T, kD>(sA, 16 * it + q, ks, g);
#pragma unroll
      for (int jj = 0; jj < (kIt == 4 ? 4 : 1); ++jj) {
        const int jt = kIt == 4 ? jj : wave & 1;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (jt <= it) {
          f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < D32; ++ks) s = M::mma(row_frag<T, kD>(sB, 16 * jt + q, ks, g), qa[ks], s);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int gap = 16 * (it - jt) + q - 4 * g - k;
            x[k] = gap >= 0 ? s[k] * (p.pair_scale * power(l2, gap)) : 0.f;
          }
        }
        *reinterpret_cast<typename M::Four*>(sP + place<T, kT>(16 * it + q, 16 * jt + 4 * g)) = M::narrow(x);
      }
      // A Z, rows scaled
#pragma unroll
      for (int i = 0; i < kIt; ++i)
#pragma unroll
        for (int ne = 0; ne < NE; ++ne) o[i][ne] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < D32; ++ks) {
        typename M::Frag zf[NE];
#pragma unroll
        for (int ne = 0; ne < NE; ++ne) {
          const f32x4 za = z[2 * ks][ne], zb = z[2 * ks + 1][ne];
          const float lo[4] = {za.x, za.y, za.z, za.w}, hi[4] = {zb.x, zb.y, zb.z, zb.w};
          zf[ne] = M::join(M::narrow(lo), M::narrow(hi));
        }
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const typename M::Frag a = row_frag<T, kD>(sA, 16 * i + q, ks, g);
#pragma unroll
          for (int ne = 0; ne < NE; ++ne) o[i][ne] = M::mma(zf[ne], a, o[i][ne]);
        }
      }
#pragma unroll
      for (int i = 0; i < kIt; ++i)
#pragma unroll
        for (int ne = 0; ne < NE; ++ne) o[i][ne] *= since[i];
      __syncthreads();
      // + P C
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        typename M::Frag c[NE];
#pragma unroll
        for (int ne = 0; ne < NE; ++ne) c[ne] = col_frag<T, kE>(sC, 16 * (wave * NE + ne), ks, lane);
#pragma unroll
        for (int i = 2 * ks; i < kIt; ++i) {
          const typename M::Frag s = row_frag<T, kT>(sP, 16 * i + q, ks, g);
#pragma unroll
          for (int ne = 0; ne < NE; ++ne) o[i][ne] = M::mma(c[ne], s, o[i][ne]);
        }
      }
    }
    // the state
#pragma unroll
    for (int m = 0; m < 2 * D32; ++m)
#pragma unroll
      for (int ne = 0; ne < NE; ++ne)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[m][ne][k] = fmaf(z[m][ne][k], em, z[m][ne][k]);
    update<T, D32, NE>(z, sB, sC, w, wave, lane);
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        if (16 * i + q >= n) continue;
        TO* row = O + (t0 + dir * (r + 16 * i + q)) * p.o_st;
#pragma unroll
        for (int ne = 0; ne < NE; ++ne) {
          const int e = e0 + 16 * ne + 4 * g;
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = o[i][ne][k] * p.out_scale;
          if constexpr (VEC) {
            if (e < p.E) *reinterpret_cast<typename Mma<TO>::Four*>(row + e) = Mma<TO>::narrow(x);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (e + k < p.E) store_one(row + e + k, x[k]);
          }
        }
      }
    }
    __syncthreads();
  }

  if constexpr (OUT) {
    // behind the row's length: zeros
    for (int64_t i = max(r0, len) * kE + threadIdx.x; i < r_end * kE; i += kThreads) {
      const int64_t t = i / kE;
      const int e = (int)(i - t * kE);
      if (e < ecols) store_one(O + t * p.o_st + et * kE + e, 0.f);
    }
  }
  // the end state: the row's own where its last token was taken here
  const bool last = OUT && (r1 == len && (r0 < len || (len == 0 && seg == 0)));
  float* zo = OUT ? (last ? p.z_out : nullptr) : zs;
  if (!zo) return;
  const int64_t sd = OUT ? p.zo_sd : p.E, se = OUT ? p.zo_se : 1;
  if (OUT) zo += b * p.zo_sb + h * p.zo_sh;
#pragma unroll
  for (int m = 0; m < 2 * D32; ++m)
#pragma unroll
    for (int ne = 0; ne < NE; ++ne) {
      const int e = e0 + 16 * ne + q;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int d = 16 * m + 4 * g + k;
        if (d < p.D && e < p.E) zo[d * sd + e * se] = z[m][ne][k];
      }
    }
}

// Each segment's own part of the state -> the state that it starts from.
__global__ __launch_bounds__(kThreads) void lin_join_kernel(LinArgs p, Cut cut) {
  const int64_t bh = blockIdx.x, b = bh / p.heads, h = bh % p.heads;
  const int i = blockIdx.y * kThreads + threadIdx.x;
  if (i >= p.D * p.E) return;
  const int d = i / p.E, e = i - d * p.E;
  int64_t len = p.L;
  if (p.lengths) len = min(max((int64_t)p.lengths[b], (int64_t)0), p.L);
  const float g = p.log_decay[h], l2 = log2_decay(g);
  float* zs = cut.z + bh * cut.n * p.D * (int64_t)p.E + i;
  const int64_t step = p.D * (int64_t)p.E;
  float run = p.z_in ? p.z_in[b * p.zi_sb + h * p.zi_sh + d * p.zi_sd + e * p.zi_se] : 0.f;
  const float whole = l2 <= -1e30f ? -1.f : expm1f(g * (float)cut.len);
  for (int s = 0; s < cut.n; ++s) {
    const float own = (s + 1) * cut.len < len ? zs[s * step] : 0.f;
    zs[s * step] = run;
    // only a whole segment has one behind it
    run = fmaf(run, whole, run) + own;
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

// One token.  Bound by HBM: the state is read and written once, 8 K V bytes a head against a few K of
// q, k and v.  A block takes 4 VL columns of one head's state, VL lanes of four columns (one if the
// rows are not aligned) by 256 / VL rows, and issues the loads of eight row steps before it uses the
// first, so that every lane keeps 128 bytes in flight; the columns' sums over k go through the wave
// and LDS.
template <typename T, typename TO, int VL, int PER>
__global__ __launch_bounds__(kThreads) void lin_step_kernel(LinStepArgs p) {
  constexpr int kRows = kThreads / VL, kDeep = 8;
  __shared__ float sq[kMaxD], sk[kMaxD], red[kWaves][VL * PER];
  const int vl = threadIdx.x % VL, row = threadIdx.x / VL;
  const int tiles = (p.V + VL * PER - 1) / (VL * PER);
  const int64_t bh = blockIdx.x / tiles, b = bh / p.heads, h = bh - b * p.heads;
  const int e = ((int)(blockIdx.x - bh * tiles) * VL + vl) * PER;
  const bool live = e < p.V;
  const T* q = static_cast<const T*>(p.q.p) + b * p.q.sb + h / p.q.share * p.q.sh;
  const T* k = static_cast<const T*>(p.k.p) + b * p.k.sb + h / p.k.share * p.k.sh;
  const T* v = static_cast<const T*>(p.v.p) + b * p.v.sb + h / p.v.share * p.v.sh;
  const float* s = p.s + b * p.s_sb + h * p.s_sh + e;
  float* so = p.s_out + b * p.so_sb + h * p.so_sh + e;
  float x[kDeep][PER];
  auto read = [&](int d0) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int d = d0 + i * kRows + row;
      if (live && d < p.K) {
        if constexpr (PER == 4) {
          const f32x4 r = *reinterpret_cast<const f32x4*>(s + d * p.s_sk);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = r[j];
        } else {
          x[i][0] = s[d * p.s_sk];
        }
      }
    }
  };
  read(0);
  if ((int)threadIdx.x < p.K) {
    sq[threadIdx.x] = to_f32(q[threadIdx.x]);
    sk[threadIdx.x] = to_f32(k[threadIdx.x]);
  }
  float vv[PER], acc[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    vv[j] = live ? to_f32(v[e + j]) : 0.f;
    acc[j] = 0.f;
  }
  // lam - 1: lam S is taken as S + (lam - 1) S, which a decay near 1 leaves exact to f32 over any
  // number of tokens
  const float em = expm1f(p.log_decay[h]);
  __syncthreads();
  for (int d0 = 0; d0 < p.K; d0 += kDeep * kRows) {
    if (d0) read(d0);
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int d = d0 + i * kRows + row;
      if (live && d < p.K) {
        const float kk = sk[d], qq = sq[d];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          x[i][j] = fmaf(kk, vv[j], fmaf(x[i][j], em, x[i][j]));
          acc[j] = fmaf(qq, x[i][j], acc[j]);
        }
        if constexpr (PER == 4) *reinterpret_cast<f32x4*>(so + d * p.so_sk) = f32x4{x[i][0], x[i][1], x[i][2], x[i][3]};
        else so[d * p.so_sk] = x[i][0];
      }
    }
  }
#pragma unroll
  for (int m = VL; m < 64; m <<= 1)
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] += __shfl_xor(acc[j], m);
  if ((threadIdx.x & 63) < VL)
#pragma unroll
    for (int j = 0; j < PER; ++j) red[threadIdx.x >> 6][vl * PER + j] = acc[j];
  __syncthreads();
  if ((int)threadIdx.x < VL * PER) {
    const int c = (int)(blockIdx.x - bh * tiles) * VL * PER + threadIdx.x;
    if (c < p.V) {
      const float o = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
      store_one(static_cast<TO*>(p.o) + b * p.o_sb + h * p.o_sh + c, o * p.scale);
    }
  }
}

// ------------------------------------------------------------------------------------ launch

int d32_of(int D) { return D <= 32 ? 1 : D <= 64 ? 2 : D <= 128 ? 4 : 8; }
// 128 columns a block (two tiles a wave) where they are there and the state of 256 rows does not
// fill the registers; f32 takes 64
int ne_of(const LinArgs& a) { return a.bf16 && a.E > 64 && a.D <= 128 ? 2 : 1; }

Cut cut_of(const LinArgs& a) {
  Cut c{};
  c.etiles = (a.E + 64 * ne_of(a) - 1) / (64 * ne_of(a));
  const int64_t blocks = a.batch * a.heads * c.etiles, slots = 2LL * cu_count();
  const int64_t chunks = (a.L + 63) / 64;
  // segments of at least 8 chunks; a segmented walk costs half as much again (the pre-pass), so the
  // count that ends first is taken: rounds of the chip times segment length
  int64_t best = 1, best_cost = 0;
  for (int64_t n = 1; n <= 256 && (n == 1 || chunks / n >= 8); ++n) {
    const int64_t per = (chunks + n - 1) / n;
    const int64_t cost = (blocks * n + slots - 1) / slots * per * (n == 1 ? 2 : 3);
    if (n == 1 || cost < best_cost) best = n, best_cost = cost;
  }
  c.len = std::max<int64_t>(1, (chunks + best - 1) / best) * 64;
  c.n = (int32_t)std::max<int64_t>(1, (a.L + c.len - 1) / c.len);
  return c;
}

int64_t cut_floats(const LinArgs& a, const Cut& c) {
  return c.n > 1 ? (a.batch * a.heads * c.n * a.D * (int64_t)a.E + 3) / 4 * 4 : 0;
}

template <typename T, typename TO, int D32, int NE>
hipError_t launch_shape(const LinArgs& a, const Cut& cut, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.heads * cut.n * cut.etiles)), block(kThreads);
  if (cut.n > 1) {
    if (a.vec) hipLaunchKernelGGL((lin_kernel<T, float, D32, NE, true, false>), grid, block, 0, s, a, cut);
    else hipLaunchKernelGGL((lin_kernel<T, float, D32, NE, false, false>), grid, block, 0, s, a, cut);
    const dim3 jg((unsigned)(a.batch * a.heads), (unsigned)((a.D * a.E + kThreads - 1) / kThreads));
    hipLaunchKernelGGL(lin_join_kernel, jg, block, 0, s, a, cut);
  }
  if (a.vec) hipLaunchKernelGGL((lin_kernel<T, TO, D32, NE, true, true>), grid, block, 0, s, a, cut);
  else hipLaunchKernelGGL((lin_kernel<T, TO, D32, NE, false, true>), grid, block, 0, s, a, cut);
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t launch_types(const LinArgs& a, const Cut& cut, hipStream_t s) {
  const int d = d32_of(a.D);
  if constexpr (sizeof(T) == 2) {
    if (ne_of(a) == 2) {
      if (d == 1) return launch_shape<T, TO, 1, 2>(a, cut, s);
      if (d == 2) return launch_shape<T, TO, 2, 2>(a, cut, s);
      return launch_shape<T, TO, 4, 2>(a, cut, s);
    }
  }
  if (d == 1) return launch_shape<T, TO, 1, 1>(a, cut, s);
  if (d == 2) return launch_shape<T, TO, 2, 1>(a, cut, s);
  if (d == 4) return launch_shape<T, TO, 4, 1>(a, cut, s);
  return launch_shape<T, TO, 8, 1>(a, cut, s);
}

}  // namespace

int64_t lin_workspace_floats(const LinArgs* a, int n) {
  // the passes run one after the other and share the place
  int64_t most = 0;
  for (int i = 0; i < n; ++i) most = std::max(most, cut_floats(a[i], cut_of(a[i])));
  return most;
}

hipError_t launch_lin(const LinArgs* a, int n, float* ws, hipStream_t s) {
  for (int i = 0; i < n; ++i) {
    Cut cut = cut_of(a[i]);
    cut.z = ws;
    const hipError_t e = !a[i].bf16     ? launch_types<float, float>(a[i], cut, s)
                         : a[i].o_f32 ? launch_types<bf16_t, float>(a[i], cut, s)
                                      : launch_types<bf16_t, bf16_t>(a[i], cut, s);
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

template <typename T, typename TO>
static hipError_t launch_step_types(const LinStepArgs& a, hipStream_t s) {
  const int64_t bh = a.batch * a.heads;
  // 128 columns a block where that gives every CU four blocks, else 32: more blocks, fewer rows each
  const bool wide = a.V > 32 && bh * ((a.V + 127) / 128) >= 4 * cu_count();
#define SS_STEP(VL, PER)                                                                                            \
  hipLaunchKernelGGL((lin_step_kernel<T, TO, VL, PER>), dim3((unsigned)(bh * ((a.V + VL * PER - 1) / (VL * PER)))), \
                     dim3(kThreads), 0, s, a)
  if (a.vec) {
    if (wide) SS_STEP(32, 4); else SS_STEP(8, 4);
  } else {
    SS_STEP(32, 1);
  }
#undef SS_STEP
  return hipGetLastError();
}

hipError_t launch_lin_step(const LinStepArgs& a, hipStream_t s) {
  if (a.in_bf16) return a.out_bf16 ? launch_step_types<bf16_t, bf16_t>(a, s) : launch_step_types<bf16_t, float>(a, s);
  return a.out_bf16 ? launch_step_types<float, bf16_t>(a, s) : launch_step_types<float, float>(a, s);
}

}  // namespace ss
