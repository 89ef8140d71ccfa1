// ss_lin.hip -- linear attention with one fixed decay per head, in its chunked matrix form (gfx950).
//
// Method.  Over a chunk of T tokens the recurrence (LinArgs: its three forms) is, with lam the
// head's decay, M_ij = lam^(i-j) for j <= i and Z [D, E] the state entering the chunk,
//   O  = (A B^T o M) C + diag(lam^(i + e0)) A Z        Z' = lam^T Z + B^T diag(lam^(T - j - e0)) C
// four dense products.  All powers of lam have exponents >= 0 and are taken directly, from a product
// T g held in two floats, so neither a strong decay (down to 0) nor a long chunk overflows or costs
// places.  From lam^T = 1/2 on it enters as Z + expm1(T g) Z, so that a decay near 1 loses nothing in
// f32 over many chunks; below as exp(T g) Z, since 1 + expm1 would leave an error of 2^-25 of the old
// state (T = 64: 0.7% of what remains of it at g = -0.2, all of it from -0.5 on).
//
// Mapping.  A block of four or eight waves takes one (row, head), 16 columns of E a wave and a
// segment of the row, and walks its chunks in order.  A wave keeps Z for its columns in MFMA
// accumulators over the whole walk.  A 16x16 accumulator tile holds rows 4 g .. 4 g + 3 (g =
// lane / 16) of column lane % 16, so with the contraction index of every product put in the order
// (16 (2 k + e / 4) + 4 g + e % 4: slot e of lane group g in step k) Z is an operand straight from
// its accumulators; rows of A and B are read in that order as two pieces of four, and C and B^T
// (contraction over tokens) come from LDS through the transposing read, four tokens a lane.  The
// masked scores are formed transposed, so that a lane holds four neighbouring j of one i: they go to
// LDS as one piece and come back in the same order.  The products are taken as O^T, so that a lane
// holds four neighbouring columns of one token for its store.
//
// Types.  bf16 inputs run on v_mfma_f32_16x16x32_bf16: the inputs are exact operands; the f32 factors
// (the masked scores, the Z that A reads, the weighted C of the state update) enter as three bf16 parts,
// 24 bits, so that nothing of f32 is lost, also where terms cancel.  (Two parts, 16 bits, took 12 to 17%
// less time and left up to 2^-16 of a term: more than the last place of a bf16 output where two terms
// nearly cancel.)  f32 inputs run on v_mfma_f32_16x16x4_f32, nothing rounded.
//
// Few rows: the row is cut into segments.  A pre-pass of the same walk without the outputs forms
// each segment's own part of the state, a small kernel turns these into the states that the segments
// start from.
//
// What bounds it.  For a chunk of one head with D = E = 128 a wave issues 119 MFMA, 570 other VALU and
// 153 LDS instructions; over the output walk the matrix pipe is busy 43% of the time, VALU issue 63%,
// LDS 36%, and no one of them alone bounds it: without the loads, the scores or the state update in
// turn (bf16, one part each) a walk of 118 us took 96, 99 and 100.  Four waves of 32 columns in place
// of eight of 16 (half the LDS reads) measured the same.  Measured: one row of 65536 tokens, 16 heads
// of 128 x 128, bf16, state out: 452 us, a third of it the segments' states, 2.4 TB/s of the bytes that
// have to move; 2 x 8192 tokens, 80 heads of 128 x 64 sharing q, k and v: 283 us (295 with a v for each
// head); f32 at 4 x 2048 tokens, 16 heads of 128 x 128: 180 us.
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

// exponents are multiples of g log2 e, held as hi + lo; -infinity (no memory) becomes a number whose
// products with 0 are 0 and whose powers are 0, NaN stays
struct Log2 {
  float hi, lo;
};
__device__ __forceinline__ Log2 log2_decay(float g) {
  if (g < -1e30f) return Log2{-1e30f, 0.f};
  const float hi = g * kLog2e;
  return Log2{hi, fmaf(g, kLog2e, -hi) + g * 1.92596303e-08f};  // log2 e: kLog2e and this
}
// a value that is the same in every lane, in a scalar register
__device__ __forceinline__ float uniform(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}
// lam^n, off by some 2^-23 of itself however strong the decay
__device__ __forceinline__ float power(Log2 l2, int n) {
  const float t = l2.hi * (float)n, e = fmaf(l2.hi, (float)n, -t) + l2.lo * (float)n;
  return __builtin_amdgcn_exp2f(t) * fmaf(e, kLn2, 1.f);
}

// A state through n tokens: from lam^n = 1/2 on z + by z with by = expm1(n g), else by z, by = exp(n g).
struct Fade {
  float by;
  bool near;
  __device__ __forceinline__ float operator()(float z) const { return near ? fmaf(z, by, z) : z * by; }
};
__device__ __forceinline__ Fade fade_of(float g, float n) {
  const float x = g * n, rest = fmaf(g, n, -x);
  if (x < -200.f) return Fade{0.f, false};  // no f32 number (-infinity too)
  if (x < -kLn2) {
    const float lam = expf(x);
    return Fade{fmaf(lam, rest, lam), false};
  }
  const float em = expm1f(x);
  return Fade{fmaf(1.f + em, rest, em), true};
}

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
  // s and 0 times every value of an operand: in some lane not 0 if one of them is not finite
  static __device__ __forceinline__ float times0(const Frag& c, float s) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{c[2 * e], c[2 * e + 1]}, bf16x2{}, s, false);
    return s;
  }
  // v as the sum of N parts
  template <int N>
  static __device__ __forceinline__ void split(const float (&v)[4], Four (&part)[N]) {
    float left[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      part[n] = narrow(left);
      left[0] -= bf16_lo(part[n].x);
      left[1] -= bf16_hi(part[n].x);
      left[2] -= bf16_lo(part[n].y);
      left[3] -= bf16_hi(part[n].y);
    }
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
  static __device__ __forceinline__ float times0(const Frag& c, float s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(c.v[e], 0.f, s);
    return s;
  }
  template <int N>
  static __device__ __forceinline__ void split(const float (&v)[4], Four (&part)[N]) {
    static_assert(N == 1, "f32 is its own only part");
    part[0] = narrow(v);
  }
};

// ---- LDS tiles [rows][W] of T.  16-byte pieces of a row are permuted by the row, so that both the
// row reads (16 rows, one piece) and the transposing reads (8 rows, two pieces) meet every bank once.
// The permutation is an XOR with bits of row % 16, so a lane's address for another step along the
// row is its first one XOR a constant, and for another 16 rows that plus a constant.
// Every 16 rows are followed by 16 bytes, so that the compiler cannot join the reads of two such
// groups in one ds_read2st64_b64: joined, the two conflict (measured: 12 cycles against 2 each).
template <typename T, int W>
constexpr int group16() {  // bytes of 16 rows
  return 16 * W * (int)sizeof(T) + 16;
}
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
  return row * kBytes + (row >> 4) * 16 + (((at >> 4) ^ f) << 4) + (at & 15);
}

// row 16 i + q as an operand: the 8 values of step ks; `at` = place(q, 4 g)
template <typename T, int W>
__device__ __forceinline__ typename Mma<T>::Frag row_frag(const uint8_t* tile, int at, int i, int ks) {
  typedef typename Mma<T>::Four Four;
  constexpr int kStep = 32 * (int)sizeof(T), kRows16 = group16<T, W>();
  const Four a = *reinterpret_cast<const Four*>(tile + (at ^ (ks * kStep)) + i * kRows16);
  const Four b = *reinterpret_cast<const Four*>(tile + (at ^ (ks * kStep + kStep / 2)) + i * kRows16);
  return Mma<T>::join(a, b);
}

// where a lane's part of column block 0 starts, for col_frag
template <typename T, int W>
__device__ __forceinline__ int col_at(int lane) {
  const int g = lane >> 4, q = lane & 15;
  return sizeof(T) == 2 ? place<T, W>(4 * g + (q >> 2), 4 * (q & 3)) : place<T, W>(4 * g, q);
}

// column 16 c + q as an operand: the 8 rows (tokens) of step ks
template <typename T, int W>
__device__ __forceinline__ typename Mma<T>::Frag col_frag(const uint8_t* tile, int at, int c, int ks) {
  constexpr int kBytes = W * (int)sizeof(T), kCols = 16 * (int)sizeof(T);
  if constexpr (sizeof(T) == 2) {
    u32x2 r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                           (lds_i16x4*)(tile + (at ^ (c * kCols)) + (2 * ks + i) * group16<T, W>())));
    return Mma<T>::join(r[0], r[1]);
  } else {
    // the rows 4 g + k of a step differ in the permutation by k / kRows
    constexpr int kRows = kBytes >= 256 ? 1 : 256 / kBytes;
    typename Mma<T>::Frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.v[e] = *reinterpret_cast<const float*>(tile + (at ^ (c * kCols) ^ (((e & 3) / kRows) << 4)) +
                                               (2 * ks + (e >> 2)) * group16<T, W>() + (e & 3) * kBytes);
    return f;
  }
}

// Buffer accesses: a base in scalar registers and 32-bit byte offsets; an offset of kNowhere is past
// the buffer's 2 GiB, where loads give 0 and stores do nothing (the address is not touched).
constexpr int kNowhere = (int)0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, kNowhere, 0x00027000);
}

// ---- a chunk of rows on its way from HBM to LDS, in registers

template <typename T, int W, int ROWS, int THREADS, bool VEC>
struct Stage {
  static constexpr int kPer = 16 / (int)sizeof(T);  // values of a 16-byte piece
  static constexpr int kPieces = W / kPer;
  static constexpr int kN = (ROWS * kPieces + THREADS - 1) / THREADS;
  static constexpr int kRowStep = THREADS / kPieces;
  u32x4 v[kN];
  int off;    // VEC: the thread's first piece, in bytes from the chunk's lowest row
  int more;   // and from there to its next one

  // step: elements from a row of the walk to the next, negative when the walk runs backwards
  __device__ __forceinline__ void init(int64_t step) {
    const int row = threadIdx.x / kPieces, c = threadIdx.x % kPieces * kPer;
    off = (int)(((step < 0 ? row - (ROWS - 1) : row) * step + c) * (int)sizeof(T));
    more = (int)(kRowStep * step * (int)sizeof(T));
  }
  // rows 0 .. ROWS of a chunk at `base`, those from `rows` on and the columns from `cols` on as zero
  __device__ __forceinline__ void load(const T* base, int64_t step, int rows, int cols) {
    const int row0 = threadIdx.x / kPieces, c = threadIdx.x % kPieces * kPer;
    if constexpr (VEC) {
      const __amdgpu_buffer_rsrc_t rs = buffer(step < 0 ? base + (ROWS - 1) * step : base);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        v[i] = __builtin_amdgcn_raw_buffer_load_b128(
            rs, row0 + i * kRowStep < rows && c < cols ? off + i * more : kNowhere, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int row = row0 + i * kRowStep;
        v[i] = u32x4{0, 0, 0, 0};
        if (row < rows && c < cols) {
          const T* p = base + row * step + c;
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
    const int row = threadIdx.x / kPieces, c = threadIdx.x % kPieces * kPer;
    constexpr bool kEven = kRowStep % 16 == 0;  // the next piece is the first one, some 16s of rows on
    const int at = place<T, W>(row, c);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int to = kEven ? at + i * (kRowStep / 16) * group16<T, W>() : place<T, W>(row + i * kRowStep, c);
      if (ROWS * kPieces % THREADS == 0 || row + i * kRowStep < ROWS) *reinterpret_cast<u32x4*>(tile + to) = v[i];
    }
  }
};

// Eight values as the sum of N bf16 parts, each the rounding of what the parts before it leave.
template <int N>
__device__ __forceinline__ void split8(float (&left)[8], bf16x8 (&part)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = pk_bf16(left[2 * j], left[2 * j + 1]);
      left[2 * j] -= bf16_lo(h[j]);
      left[2 * j + 1] -= bf16_hi(h[j]);
    }
    part[n] = __builtin_bit_cast(bf16x8, u32x4{h[0], h[1], h[2], h[3]});
  }
}

// How a row is cut: segments of `len` tokens (a multiple of every chunk size).
struct Cut {
  uint32_t len;
  int32_t n, etiles;
  float* z;  // n > 1: the states that the segments start from, D E floats for every [batch heads][n],
  int64_t z_sd, z_se;  // element (d, e) at d z_sd + e z_se
};

// The state update of a chunk: z[m] (rows 16 m .., this wave's 16 columns) += B^T (w o C), w_j at
// wt[j].  bf16 takes w o C in three parts.
template <typename T, int D32, int W>
__device__ __forceinline__ void update(f32x4 (&z)[2 * D32], const uint8_t* sB, const uint8_t* sC, const float* wt,
                                       int wave, int lane) {
  constexpr int kKs = Mma<T>::kChunk / 32, kM = 2;  // tiles whose operands are read together
  const int g = lane >> 4, b_at = col_at<T, 32 * D32>(lane), c_at = col_at<T, W>(lane);
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    const f32x4 w0 = *reinterpret_cast<const f32x4*>(wt + 32 * ks + 4 * g);
    const f32x4 w1 = *reinterpret_cast<const f32x4*>(wt + 32 * ks + 16 + 4 * g);
    const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    if constexpr (sizeof(T) == 2) {
      const u32x4 c = __builtin_bit_cast(u32x4, col_frag<T, W>(sC, c_at, wave, ks));
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(c[e]) * w[2 * e];
        x[2 * e + 1] = bf16_hi(c[e]) * w[2 * e + 1];
      }
      bf16x8 part[3];
      split8(x, part);
#pragma unroll
      for (int m0 = 0; m0 < 2 * D32; m0 += kM) {
        bf16x8 b[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m) b[m] = col_frag<T, 32 * D32>(sB, b_at, m0 + m, ks);
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
          for (int m = 0; m < kM; ++m) z[m0 + m] = Mma<T>::mma(b[m], part[k], z[m0 + m]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      typename Mma<T>::Frag c = col_frag<T, W>(sC, c_at, wave, ks);
#pragma unroll
      for (int e = 0; e < 8; ++e) c.v[e] *= w[e];
#pragma unroll
      for (int m = 0; m < 2 * D32; ++m) z[m] = Mma<T>::mma(col_frag<T, 32 * D32>(sB, b_at, m, ks), c, z[m]);
    }
  }
}

// waves per SIMD that the registers are held to
constexpr int lin_waves(bool bf16, int d32, int nw, bool vec) {
  return !vec || d32 == 8 ? (nw == 8 || (vec && !bf16) ? 2 : 1) : !bf16 ? 2 : nw == 8 ? 4 : 3;
}

// OUT: the walk with outputs; else only the segment's own part of the state, from zero.
template <typename T, typename TO, int D32, int NW, bool VEC, bool OUT>
__global__ __launch_bounds__(64 * NW, lin_waves(sizeof(T) == 2, D32, NW, VEC)) void lin_kernel(LinArgs p, Cut cut) {
  constexpr int kT = Mma<T>::kChunk, kD = 32 * D32, kE = 16 * NW, kKs = kT / 32, kIt = kT / 16;
  // bf16 parts of a score and of the state that A reads; in blocks of four waves the scores take A's
  // place in LDS (a barrier more, three blocks a CU instead of two)
  constexpr int kP = sizeof(T) == 2 ? 3 : 1;
  constexpr bool kOver = sizeof(T) == 2 && NW == 4;
  constexpr int kSizeD = kIt * group16<T, kD>(), kSizeE = kIt * group16<T, kE>(), kSizeP = kIt * group16<T, kT>();
  typedef Mma<T> M;
  // B, C, then A and the scores' planes (or both in one place, the larger's)
  constexpr int kScores = kP * kSizeP, kSizeA = kOver ? (kSizeD > kScores ? kSizeD : kScores) : kSizeD + kScores;
  __shared__ __align__(16) uint8_t lds[kSizeD + kSizeE + (OUT ? kSizeA : 0)];
  // pw[kT + i]: lam^i times the scales of a score for 0 <= i < kT, 0 for i < 0; sn[i]: lam^(i + e0)
  // out_scale; wt[j]: weight of token j in the state
  __shared__ __align__(16) float pw[OUT ? 2 * kT : 1], sn[OUT ? kT : 1], wt[kT];
  uint8_t *sB = lds, *sC = lds + kSizeD, *sA = sC + kSizeE, *sP = kOver ? sA : sA + kSizeD;
  const int lane0 = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring blocks (tiles of one head, heads of one segment: shared operands) on one XCD
  int64_t id = blockIdx.x;
  if (gridDim.x % 8 == 0) id = (id % 8) * (gridDim.x / 8) + id / 8;
  const int et = (int)(id % cut.etiles);
  id /= cut.etiles;
  const int h = (int)(id % p.heads);
  id /= p.heads;
  const int seg = (int)(id % cut.n);
  const int64_t b = id / cut.n, bh = b * p.heads + h;
  const int e0 = et * kE + wave * 16;  // this wave's first column

  // positions in the row are unsigned 32-bit numbers (L < 2^31), in scalar registers
  uint32_t len = (uint32_t)p.L;
  if (p.lengths) len = min((uint32_t)max(__builtin_amdgcn_readfirstlane(p.lengths[b]), 0), len);
  const uint32_t r0 = (uint32_t)seg * cut.len, r_end = min(r0 + cut.len, (uint32_t)p.L), r1 = min(r_end, len);
  if (!OUT && r0 >= r1) return;  // no token: the segment's part is never read
  // whether the row's last token is taken here: then this walk's end state is the row's
  const bool last = OUT && (r1 == len && (r0 < len || (len == 0 && seg == 0)));
  const float g_ln = uniform(p.log_decay[h]);
  Log2 l2 = log2_decay(g_ln);
  l2 = Log2{uniform(l2.hi), uniform(l2.lo)};

  f32x4 z[2 * D32];
  float* zs = cut.n > 1 ? cut.z + (bh * cut.n + seg) * p.D * (int64_t)p.E : nullptr;
  {
    const float* from = !OUT ? nullptr : zs ? zs : p.z_in;
    const int64_t sd = zs ? cut.z_sd : p.zi_sd, se = zs ? cut.z_se : p.zi_se;
    const int g = lane0 >> 4, e = e0 + (lane0 & 15);
    if (from && !zs) from += b * p.zi_sb + h * p.zi_sh;
#pragma unroll
    for (int m = 0; m < 2 * D32; ++m) {
      z[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (from && e < p.E)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 16 * m + 4 * g + r;
          if (d < p.D) z[m][r] = from[d * sd + e * se];
        }
    }
  }

  const T* A = static_cast<const T*>(p.a.p) + b * p.a.sb + h / p.a.share * p.a.sh;
  const T* B = static_cast<const T*>(p.b.p) + b * p.b.sb + h / p.b.share * p.b.sh;
  const T* C = static_cast<const T*>(p.c.p) + b * p.c.sb + h / p.c.share * p.c.sh + et * kE;
  TO* O = static_cast<TO*>(p.o) + b * p.o_sb + h * p.o_sh;
  const int64_t t0 = p.reverse ? (int64_t)len - 1 : 0, dir = p.reverse ? -1 : 1;
  const int ecols = p.E - et * kE;

  Stage<T, kD, kT, 64 * NW, VEC> a_in, b_in;
  Stage<T, kE, kT, 64 * NW, VEC> c_in;
  if constexpr (OUT) a_in.init(dir * p.a.st);
  b_in.init(dir * p.b.st);
  c_in.init(dir * p.c.st);
  auto fetch = [&](uint32_t r) {
    const int rows = (int)min((uint32_t)kT, r1 - r);
    const int64_t t = t0 + dir * r;
    if constexpr (OUT) a_in.load(A + t * p.a.st, dir * p.a.st, rows, p.D);
    b_in.load(B + t * p.b.st, dir * p.b.st, rows, p.D);
    c_in.load(C + t * p.c.st, dir * p.c.st, rows, ecols);
  };

  if constexpr (OUT)
    for (int i = threadIdx.x; i < 2 * kT; i += 64 * NW) {
      pw[i] = i < kT ? 0.f : p.pair_scale * p.out_scale * power(l2, i - kT);
      if (i < kT) sn[i] = p.out_scale * power(l2, i + p.e0);
    }
  if (r0 < r1) fetch(r0);
  int cur = 0;
  Fade fade{};
  for (uint32_t r = r0; r < r1; r += kT) {
    // the LDS addresses are a few operations on the lane number: made anew in every chunk, since
    // kept over the loop they would push the state out of the registers
    int lane = lane0;
    asm volatile("" : "+v"(lane));
    const int g = lane >> 4, q = lane & 15;
    const int n = (int)min((uint32_t)kT, r1 - r);
    if (n != cur) {
      // weights of a chunk of n tokens: of each token, and on the state itself
      cur = n;
      for (int j = threadIdx.x; j < kT; j += 64 * NW)
        wt[j] = n - p.e0 - j >= 0 ? p.pair_scale * power(l2, n - p.e0 - j) : 0.f;
      fade = fade_of(g_ln, (float)n);
      fade.by = uniform(fade.by);
      fade.near = __builtin_amdgcn_readfirstlane(fade.near);
    }
    if constexpr (OUT) a_in.store(sA);
    b_in.store(sB);
    c_in.store(sC);
    __syncthreads();
    if (r + kT < r1) fetch(r + kT);
    __builtin_amdgcn_sched_barrier(0);

    f32x4 o[OUT ? kIt : 1];
    if constexpr (OUT) {
      // masked scores, transposed: tile (it, jt) with lane i = 16 it + q, rows j = 16 jt + 4 g + r
      constexpr int kJ = kIt * kIt / NW;  // tiles a wave
      const int it = wave * kJ / kIt, j0 = wave * kJ % kIt;
      const int at = place<T, kD>(q, 4 * g);
      typename M::Four part[kJ][kP];
      {
        typename M::Frag qa[D32];
#pragma unroll
        for (int ks = 0; ks < D32; ++ks) qa[ks] = row_frag<T, kD>(sA + it * (kSizeD / kIt), at, 0, ks);
        const float* gap = pw + kT + 16 * it + q - 4 * g;
#pragma unroll
        for (int jj = 0; jj < kJ; ++jj) {
          const int jt = j0 + jj;
          float x[4] = {0.f, 0.f, 0.f, 0.f};
          if (jt <= it) {
            f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < D32; ++ks) s = M::mma(row_frag<T, kD>(sB + jt * (kSizeD / kIt), at, 0, ks), qa[ks], s);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = s[k] * gap[-16 * jt - k];
            // a later token's score may be infinite or NaN, which no weight of 0 takes out
            if (jt == it)
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = 4 * g + k <= q ? x[k] : 0.f;
          }
          M::split(x, part[jj]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      const int p_at = place<T, kT>(q, 4 * g);
      auto scores = [&]() {
#pragma unroll
        for (int jj = 0; jj < kJ; ++jj)
#pragma unroll
          for (int k = 0; k < kP; ++k)
            *reinterpret_cast<typename M::Four*>(sP + k * kSizeP + it * group16<T, kT>() +
                                                 (p_at ^ ((j0 + jj) * 16 * (int)sizeof(T)))) = part[jj][k];
      };
      if constexpr (!kOver) scores();
      // A Z, rows scaled; a wave in a run of MFMAs (here and in update) goes before those that stage: 1 to
      // 3% of a call's time (measured with two parts: 80 shared heads 244 -> 236 us, long prompt 412 -> 405)
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < kIt; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < D32; ++ks) {
        const f32x4 za = z[2 * ks], zb = z[2 * ks + 1];
        const float lo[4] = {za.x, za.y, za.z, za.w}, hi[4] = {zb.x, zb.y, zb.z, zb.w};
        typename M::Four pl[kP], ph[kP];
        M::split(lo, pl);
        M::split(hi, ph);
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const typename M::Frag a = row_frag<T, kD>(sA, at, i, ks);
#pragma unroll
          for (int k = 0; k < kP; ++k) o[i] = M::mma(M::join(pl[k], ph[k]), a, o[i]);
        }
        if (ks & 1) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const float since = sn[16 * i + q];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] *= since;
      }
      __builtin_amdgcn_s_setprio(0);
      if constexpr (kOver) {
        __syncthreads();  // A is read
        scores();
      }
      __syncthreads();
      // + P C.  The masked half of P is 0, but 0 times an infinity or a NaN is not: a wave whose columns
      // of C hold one adds its tokens one by one instead, each to the outputs from its own on.
      const int c_at = col_at<T, kE>(lane);
      float off = 0.f;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) off = M::times0(col_frag<T, kE>(sC, c_at, wave, ks), off);
      if (!__any(off != 0.f)) {
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
          const typename M::Frag c = col_frag<T, kE>(sC, c_at, wave, ks);
#pragma unroll
          for (int k = 0; k < kP; ++k)
#pragma unroll
            for (int i = 2 * ks; i < kIt; ++i) o[i] = M::mma(c, row_frag<T, kT>(sP + k * kSizeP, p_at, i, ks), o[i]);
        }
      } else {
#pragma clang loop unroll(disable)
        for (int j = 0; j < n; ++j) {
          float cj[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            cj[k] = to_f32(*reinterpret_cast<const T*>(sC + place<T, kE>(j, wave * 16 + 4 * g + k)));
#pragma unroll
          for (int i = 0; i < kIt; ++i) {
            float w = 0.f;
#pragma unroll
            for (int k = 0; k < kP; ++k)
              w += to_f32(*reinterpret_cast<const T*>(sP + k * kSizeP + place<T, kT>(16 * i + q, j)));
            if (j <= 16 * i + q)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i][k] = fmaf(w, cj[k], o[i][k]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (OUT) {
      const int e = e0 + 4 * g;
      // VEC: 32-bit offsets from the chunk's lowest row
      const int64_t low = t0 + dir * (p.reverse ? r + kT - 1 : r);
      const __amdgpu_buffer_rsrc_t rs = buffer(O + low * p.o_st);
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int row = 16 * i + q;
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = o[i][k];
        if constexpr (VEC) {
          const int up = p.reverse ? kT - 1 - row : row;
          const int at = row < n && e < p.E ? (up * (int)p.o_st + e) * (int)sizeof(TO) : kNowhere;
          if constexpr (sizeof(TO) == 2)
            __builtin_amdgcn_raw_buffer_store_b64(Mma<TO>::narrow(x), rs, at, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, Mma<TO>::narrow(x)), rs, at, 0, 0);
        } else if (row < n) {
          TO* to = O + (t0 + dir * (r + row)) * p.o_st + e;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (e + k < p.E) store_one(to + k, x[k]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // the state
    if (fade.near) {
#pragma unroll
      for (int m = 0; m < 2 * D32; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[m][k] = fmaf(z[m][k], fade.by, z[m][k]);
    } else {
#pragma unroll
      for (int m = 0; m < 2 * D32; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[m][k] *= fade.by;
    }
    __builtin_amdgcn_s_setprio(1);
    update<T, D32, kE>(z, sB, sC, wt, wave, lane);
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();
  }

  if constexpr (OUT) {
    // behind the row's length: zeros
    for (int64_t i = (int64_t)max(r0, len) * kE + threadIdx.x; i < (int64_t)r_end * kE; i += 64 * NW) {
      const int64_t t = i / kE;
      const int e = (int)(i - t * kE);
      if (e < ecols) store_one(O + t * p.o_st + et * kE + e, 0.f);
    }
  }
  float* zo = OUT ? (last ? p.z_out : nullptr) : zs;
  if (!zo) return;
  const int64_t sd = OUT ? p.zo_sd : cut.z_sd, se = OUT ? p.zo_se : cut.z_se;
  if (OUT) zo += b * p.zo_sb + h * p.zo_sh;
  const int g = lane0 >> 4, e = e0 + (lane0 & 15);
#pragma unroll
  for (int m = 0; m < 2 * D32; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = 16 * m + 4 * g + k;
      if (d < p.D && e < p.E) zo[d * sd + e * se] = z[m][k];
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
  float* zs = cut.z + bh * cut.n * p.D * (int64_t)p.E + i;
  const int64_t step = p.D * (int64_t)p.E;
  float run = p.z_in ? p.z_in[b * p.zi_sb + h * p.zi_sh + d * p.zi_sd + e * p.zi_se] : 0.f;
  const Fade whole = fade_of(p.log_decay[h], (float)cut.len);
  for (int s0 = 0; s0 < cut.n; s0 += 8) {
    float own[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) own[k] = (int64_t)(s0 + k + 1) * cut.len < len ? zs[(s0 + k) * step] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (s0 + k >= cut.n) break;
      zs[(s0 + k) * step] = run;
      // only a whole segment has one behind it
      run = whole(run) + own[k];
    }
  }
}

// The gradient of a shared head: PER neighbouring features a thread, the sharing heads' f32 gradients
// added in order.  Bound by HBM.
template <int PER>
__global__ __launch_bounds__(kThreads) void head_sum_kernel(const float* __restrict__ src, void* dst, int64_t d_sb,
                                                            int64_t d_st, int64_t d_sh, int bf16, int64_t L, int heads,
                                                            int share, int D, int64_t total) {
  const int per_row = D / PER;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / per_row;
    const int d = (int)(i - row * per_row) * PER;
    const int64_t bl = row / heads, h = row - bl * heads;
    const int64_t b = bl / L, l = bl - b * L;
    const float* s = src + row * share * D + d;
    float v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < share; ++k) {
      if constexpr (PER == 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(s + (int64_t)k * D);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += x[j];
      } else {
        v[0] += s[(int64_t)k * D];
      }
    }
    const int64_t at = b * d_sb + l * d_st + h * d_sh + d;
    if constexpr (PER == 4) {
      if (bf16) *reinterpret_cast<u32x2*>(static_cast<bf16_t*>(dst) + at) = Mma<bf16_t>::narrow(v);
      else *reinterpret_cast<f32x4*>(static_cast<float*>(dst) + at) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
      if (bf16) store_one(static_cast<bf16_t*>(dst) + at, v[0]);
      else static_cast<float*>(dst)[at] = v[0];
    }
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
  const Fade fade = fade_of(p.log_decay[h], 1.f);
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
          x[i][j] = fmaf(kk, vv[j], fade(x[i][j]));
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
// eight waves, 128 columns a block, where there are more than 64
int nw_of(const LinArgs& a) { return a.bf16 && a.E > 64 ? 8 : 4; }

Cut cut_of(const LinArgs& a) {
  Cut c{};
  c.etiles = (a.E + 16 * nw_of(a) - 1) / (16 * nw_of(a));
  const int64_t blocks = a.batch * a.heads * c.etiles, cus = cu_count();
  const int64_t chunks = (a.L + 63) / 64;
  // The time of a walk is its chunks times the blocks that share a CU, at least two (of eight waves;
  // three of four): fewer wait more than they work.  Cutting a row repeats half of it (the segments'
  // parts of the state), costs two launches (about two chunk times) and moves every segment's state
  // four times, at about 10 MB a chunk time.
  double best_cost = 0;
  int64_t best = 1;
  for (int64_t n = 1; n <= std::min<int64_t>(256, std::max<int64_t>(1, chunks)); ++n) {
    const int64_t per = (chunks + n - 1) / n, on_cu = std::max<int64_t>(nw_of(a) == 8 ? 2 : 3, (blocks * n + cus - 1) / cus);
    const double walk = (double)per * on_cu;
    const double cost =
        n == 1 ? walk : 1.5 * walk + 4 + (double)(a.batch * a.heads * n) * a.D * a.E * 16 / 10e6;
    if (n == 1 || cost < best_cost) best = n, best_cost = cost;
  }
  c.len = (uint32_t)(std::max<int64_t>(1, (chunks + best - 1) / best) * 64);
  c.n = (int32_t)std::max<int64_t>(1, (a.L + c.len - 1) / c.len);
  return c;
}

int64_t cut_floats(const LinArgs& a, const Cut& c) {
  return c.n > 1 ? (a.batch * a.heads * c.n * a.D * (int64_t)a.E + 3) / 4 * 4 : 0;
}

template <typename T, typename TO, int D32, int NW>
hipError_t launch_shape(const LinArgs& a, const Cut& cut, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.heads * cut.n * cut.etiles)), block(64 * NW);
  // the vector path's byte offsets within a chunk are below 2^31
  const int64_t far = ((int64_t)1 << 31) / 4 / (Mma<T>::kChunk + 1);
  const bool vec = a.vec && a.a.st < far && a.b.st < far && a.c.st < far && a.o_st < far;
  if (cut.n > 1 && !a.z_before) {
    if (vec) hipLaunchKernelGGL((lin_kernel<T, float, D32, NW, true, false>), grid, block, 0, s, a, cut);
    else hipLaunchKernelGGL((lin_kernel<T, float, D32, NW, false, false>), grid, block, 0, s, a, cut);
    const dim3 jg((unsigned)(a.batch * a.heads), (unsigned)((a.D * a.E + kThreads - 1) / kThreads));
    hipLaunchKernelGGL(lin_join_kernel, jg, dim3(kThreads), 0, s, a, cut);
  }
  if (vec) hipLaunchKernelGGL((lin_kernel<T, TO, D32, NW, true, true>), grid, block, 0, s, a, cut);
  else hipLaunchKernelGGL((lin_kernel<T, TO, D32, NW, false, true>), grid, block, 0, s, a, cut);
  return hipGetLastError();
}

template <typename T, typename TO, int NW>
hipError_t launch_depth(const LinArgs& a, const Cut& cut, hipStream_t s) {
  switch (d32_of(a.D)) {
    case 1: return launch_shape<T, TO, 1, NW>(a, cut, s);
    case 2: return launch_shape<T, TO, 2, NW>(a, cut, s);
    case 4: return launch_shape<T, TO, 4, NW>(a, cut, s);
    default: return launch_shape<T, TO, 8, NW>(a, cut, s);
  }
}

template <typename T, typename TO>
hipError_t launch_types(const LinArgs& a, const Cut& cut, hipStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (nw_of(a) == 8) return launch_depth<T, TO, 8>(a, cut, s);
  return launch_depth<T, TO, 4>(a, cut, s);
}

hipError_t launch_head_sum(const LinArgs& a, const HeadSum& h, hipStream_t s) {
  const float* src = static_cast<const float*>(a.o);
  // four features a thread where the source's rows (dense) and the destination's allow it
  const bool vec = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(h.dst) % 16 == 0 && h.sb % 4 == 0 && h.st % 4 == 0 && h.sh % 4 == 0;
  const int heads = a.heads / h.share;
  const int64_t total = a.batch * a.L * heads * (vec ? a.E / 4 : a.E);
  if (total == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((total + kThreads - 1) / kThreads, 1 << 20));
  if (vec)
    hipLaunchKernelGGL((head_sum_kernel<4>), grid, dim3(kThreads), 0, s, src, h.dst, h.sb, h.st, h.sh, a.bf16, a.L,
                       heads, h.share, a.E, total);
  else
    hipLaunchKernelGGL((head_sum_kernel<1>), grid, dim3(kThreads), 0, s, src, h.dst, h.sb, h.st, h.sh, a.bf16, a.L,
                       heads, h.share, a.E, total);
  return hipGetLastError();
}

}  // namespace

int64_t lin_workspace_floats(const LinArgs* a, int n) {
  // the passes run one after the other and share the place
  int64_t most = 0;
  for (int i = 0; i < n; ++i) most = std::max(most, cut_floats(a[i], cut_of(a[i])));
  return most;
}

hipError_t launch_lin(const LinArgs* a, const HeadSum* sums, int n, float* ws, hipStream_t s) {
  Cut cut;
  for (int i = 0; i < n; ++i) {
    if (a[i].z_before) {
      // the states of the pass before, transposed, by its cut
      cut.etiles = cut_of(a[i]).etiles;
      cut.z_sd = 1;
      cut.z_se = a[i].D;
    } else {
      cut = cut_of(a[i]);
      cut.z = ws;
      cut.z_sd = a[i].E;
      cut.z_se = 1;
    }
    const hipError_t e = !a[i].bf16     ? launch_types<float, float>(a[i], cut, s)
                         : a[i].o_f32 ? launch_types<bf16_t, float>(a[i], cut, s)
                                      : launch_types<bf16_t, bf16_t>(a[i], cut, s);
    if (e != hipSuccess) return e;
    if (sums && sums[i].share > 1) {
      const hipError_t e2 = launch_head_sum(a[i], sums[i], s);
      if (e2 != hipSuccess) return e2;
    }
  }
  return hipSuccess;
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
