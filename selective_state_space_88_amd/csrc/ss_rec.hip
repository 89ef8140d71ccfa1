// ss_rec.hip -- the gated linear recurrence on channels-last tensors, forward, backward and single
// tokens (gfx950).
//
//   h_t = a_t h_{t-1} + w(a_t) s_t x_t,   a = sigmoid(g) or exp(-rate sigmoid(g)),   s = sigmoid(i) or 1,
//   w = 1, 1 - a or sqrt(1 - a^2);   G_t = dh_t + a_{t+1} G_{t+1} is the gradient at h_t.
//
// Mapping.  A wave holds kTokens consecutive tokens of 64 lanes' channels (two bf16 channels or one f32 a
// lane, 256 bytes of a row an access), so that a token's flags are the same for all lanes and the scan
// over a lane's tokens is plain code.  The waves of a block hold consecutive pieces of one row: each
// reduces its own piece to (decay A, end state from zero), they exchange these through LDS, and each
// walks its piece again from its true start.
//
// Precision.  All arithmetic is f32.  1 - a is formed without cancellation (sigmoid(-g), or -expm1), and
// a piece's decay enters the next one as H - (1 - A) H + h where A >= 1/2, with 1 - A accumulated on its
// own: A itself, rounded to 24 bits in every token, would shift a memory of n tokens by n 2^-25.  Below
// 1/2 it enters as A H + h, which keeps what a strong decay leaves of a large state.
#include <algorithm>

#include "ss_device.h"
#include "ss_launch.h"

namespace ss {
namespace {

// VC channels of a lane as they lie in memory
template <typename T, int VC>
struct Word;
template <>
struct Word<float, 1> {
  typedef float raw;
  static __device__ __forceinline__ float get(raw r, int) { return r; }
  static __device__ __forceinline__ raw put(const float (&v)[1]) { return v[0]; }
};
template <>
struct Word<bf16_t, 1> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(raw r, int) { return bf16_lo(r); }
  static __device__ __forceinline__ raw put(const float (&v)[1]) { return (uint16_t)f32_to_bf16_bits(v[0]); }
};
template <>
struct Word<bf16_t, 2> {
  typedef uint32_t raw;
  static __device__ __forceinline__ float get(raw r, int k) { return k ? bf16_hi(r) : bf16_lo(r); }
  static __device__ __forceinline__ raw put(const float (&v)[2]) { return pk_bf16(v[0], v[1]); }
};

// sigmoid(z) and 1 - sigmoid(z), each to f32 relative accuracy.  The exponent is capped at 2^126, where
// both are still normal numbers and a NaN passes.
__device__ __forceinline__ void sigmoids(float z, float* s, float* left) {
  float t = -z * kLog2e;
  t = t > 126.f ? 126.f : t;
  const float e = __builtin_amdgcn_exp2f(t);
  *s = __builtin_amdgcn_rcpf(1.0f + e);
  *left = e * *s;
}

// The decay a and 1 - a from the gate's sigmoid sg, its complement and the channel's -rate.
// 1 - e^l is its Taylor polynomial -l (1 + l/2 + ... + l^5/720) for |l| < 1/4 (next term: 5e-8 of it),
// where the difference would cancel; a = 1 - (1 - a) there.
template <bool RATE>
__device__ __forceinline__ void decay_of(float sg, float left, float nrate, float* a, float* m) {
  if constexpr (RATE) {
    const float l = nrate * sg;
    float q = 1.f / 720.f;
    q = fmaf(q, l, 1.f / 120.f);
    q = fmaf(q, l, 1.f / 24.f);
    q = fmaf(q, l, 1.f / 6.f);
    q = fmaf(q, l, 0.5f);
    q = fmaf(q, l, 1.f);
    q *= -l;
    const float e = __builtin_amdgcn_exp2f(l * kLog2e);
    const bool near = l > -0.25f;
    *m = near ? q : 1.0f - e;
    *a = near ? 1.0f - q : e;
  } else {
    *a = sg;
    *m = left;
  }
}

template <int MIX>
__device__ __forceinline__ float share_of(float m) {
  if constexpr (MIX == 1) return m;
  if constexpr (MIX == 2) return __builtin_amdgcn_sqrtf(m * (2.0f - m));
  return 1.0f;
}

// A piece of a row as a step on the state that enters it: H -> A H + h, kept as one word t for A (A itself
// below 1/2, else -(1 - A), told apart by the sign bit) and h.  A = 0 exactly takes nothing over.
struct Piece {
  float t, h;
};
__device__ __forceinline__ float piece_word(float A, float M) { return A < 0.5f ? A : -M; }
__device__ __forceinline__ float step_over(float t, float h, float H) {
  const bool near = __float_as_int(t) < 0;
  const float r = fmaf(t, H, h) + (near ? H : 0.f);
  return __float_as_int(t) == 0 ? h : r;
}

constexpr int kFwdTokens = 16, kFwdWaves = 8;
constexpr int kBwdTokens = 8, kBwdWaves = 8;  // an even number of waves: two share a mark

// Where a block works: the row, the lane's first channel (clamped so that every lane's loads are in
// bounds; `live` says whether they are its own)
template <int VC>
struct Place {
  int64_t b;
  int64_t c;
  bool live;
  __device__ __forceinline__ Place(const RecArgs& p, int64_t block) {
    const int64_t slabs = (p.channels + 64 * VC - 1) / (64 * VC);
    b = block / slabs;
    c = (block % slabs) * (64 * VC) + (int64_t)(threadIdx.x & 63) * VC;
    live = c < p.channels;
    if (!live) c = p.channels - VC;
  }
};

__device__ __forceinline__ int64_t row_length(const RecArgs& p, int64_t b) {
  if (!p.lengths) return p.L;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// The loads of n <= N tokens from t0 on (the last one again behind them)
template <typename T, int VC, int N>
__device__ __forceinline__ void load_tokens(const RecRows& r, const Place<VC>& at, int64_t t0, int n,
                                            typename Word<T, VC>::raw (&v)[N]) {
  const T* q = static_cast<const T*>(r.p) + at.b * r.sb + at.c;
#pragma unroll
  for (int j = 0; j < N; ++j)
    v[j] = *reinterpret_cast<const typename Word<T, VC>::raw*>(q + (t0 + (j < n ? j : n - 1)) * r.st);
}

template <typename T, int VC>
__device__ __forceinline__ void store_token(const RecRows& r, const Place<VC>& at, int64_t t, const float (&v)[VC]) {
  T* q = static_cast<T*>(r.p) + at.b * r.sb + at.c + t * r.st;
  if (at.live) *reinterpret_cast<typename Word<T, VC>::raw*>(q) = Word<T, VC>::put(v);
}

// bit j: token t0 + j starts from an empty state
template <int N>
__device__ __forceinline__ uint32_t start_bits(const RecArgs& p, int64_t b, int64_t t0, int n) {
  if (!p.starts) return 0;
  const int lane = threadIdx.x & 63;
  bool s = false;
  if (lane < n) s = p.starts[b * p.starts_sb + (t0 + lane) * p.starts_st] != 0;
  return (uint32_t)__ballot(s);
}

// ---------------------------------------------------------------------------------- forward

template <typename T, int VC, bool RATE, int MIX>
__global__ __launch_bounds__(64 * kFwdWaves) void rec_fwd_kernel(RecArgs p) {
  constexpr int N = kFwdTokens;
  typedef Word<T, VC> W;
  __shared__ Piece pieces[2][kFwdWaves][64 * VC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const Place<VC> at(p, blockIdx.x);
  const int64_t len = row_length(p, at.b);
  float nrate[VC], H[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    nrate[k] = RATE ? -p.rate[at.c + k] : 0.f;
    H[k] = p.s_in ? p.s_in[at.b * p.si_sb + at.c + k] : 0.f;
  }
  int turn = 0;
  for (int64_t t0 = 0; t0 < p.L; t0 += (int64_t)waves * N, turn ^= 1) {
    const int64_t tw = t0 + wave * N;
    const int n = (int)max((int64_t)0, min((int64_t)N, len - tw));
    float a[N][VC], in[N][VC], A[VC], M[VC], hl[VC];
    uint32_t starts = 0;
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      A[k] = 1.f;
      M[k] = hl[k] = 0.f;
    }
    if (n > 0) {
      typename W::raw x[N], g[N], gi[N];
      load_tokens<T, VC, N>(p.x, at, tw, n, x);
      load_tokens<T, VC, N>(p.g, at, tw, n, g);
      if (p.i.p) load_tokens<T, VC, N>(p.i, at, tw, n, gi);
      starts = start_bits<N>(p, at.b, tw, n);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j >= n) continue;
        const bool fresh = starts >> j & 1;
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          float sg, left, m;
          sigmoids(W::get(g[j], k), &sg, &left);
          decay_of<RATE>(sg, left, nrate[k], &a[j][k], &m);
          float v = W::get(x[j], k) * share_of<MIX>(m);
          if (p.i.p) {
            float s, sl;
            sigmoids(W::get(gi[j], k), &s, &sl);
            v *= s;
          }
          in[j][k] = v;
          if (fresh) {
            A[k] = 0.f;
            M[k] = 1.f;
            hl[k] = v;
          } else {
            A[k] *= a[j][k];
            M[k] += fmaf(-m, M[k], m);
            hl[k] = fmaf(a[j][k], hl[k], v);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < VC; ++k) pieces[turn][wave][lane * VC + k] = Piece{piece_word(A[k], M[k]), hl[k]};
    __syncthreads();  // the other buffer's readers passed here one turn ago
    const int busy = (int)max((int64_t)0, min((int64_t)waves, (len - t0 + N - 1) / N));
    float S[VC];
#pragma unroll
    for (int k = 0; k < VC; ++k) S[k] = H[k];
    for (int v = 0; v < busy; ++v) {
      if (v == wave)
#pragma unroll
        for (int k = 0; k < VC; ++k) S[k] = H[k];
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        const Piece q = pieces[turn][v][lane * VC + k];
        H[k] = step_over(q.t, q.h, H[k]);
      }
    }
    if (wave >= busy)
#pragma unroll
      for (int k = 0; k < VC; ++k) S[k] = H[k];
    if (tw >= p.L) continue;
    if (p.marks && at.live) {
      float* mk = p.marks + at.b * p.mk_sb + (tw / kRecMark) * p.mk_st + at.c;
#pragma unroll
      for (int k = 0; k < VC; ++k) mk[k] = S[k];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j < n) {
#pragma unroll
        for (int k = 0; k < VC; ++k) S[k] = starts >> j & 1 ? in[j][k] : fmaf(a[j][k], S[k], in[j][k]);
        store_token<T, VC>(p.h, at, tw + j, S);
      } else if (tw + j < p.L) {
        const float zero[VC] = {};
        store_token<T, VC>(p.h, at, tw + j, zero);
      }
    }
  }
  if (p.s_out && wave == 0 && at.live)
#pragma unroll
    for (int k = 0; k < VC; ++k) p.s_out[at.b * p.so_sb + at.c + k] = H[k];
}

// --------------------------------------------------------------------------------- backward

// The gradients of one token and channel: what the reverse walk knows is G, the state before the token
// (0 where it starts afresh), the decay a and the share w.
template <bool RATE, int MIX>
struct Grad {
  float dx, dg, di, dr;
  __device__ __forceinline__ Grad(float G, float hp, float a, float w, float x, float g, float i, bool has_i,
                                  float nrate) {
    float sg, left, s = 1.f, sl = 0.f;
    sigmoids(g, &sg, &left);
    if (has_i) sigmoids(i, &s, &sl);
    const float ds = G * w;
    dx = ds * s;
    di = ds * x * (s * sl);
    const float sx = s * x;
    float to_a = hp;
    if constexpr (MIX == 1) to_a -= sx;
    // the slope of sqrt(1 - a^2) is -a / w; at w = 0 (a = 1: the gate is shut) it is taken as 0
    if constexpr (MIX == 2) to_a -= w > 0.f ? sx * a * __builtin_amdgcn_rcpf(w) : 0.f;
    to_a *= G * a;
    if constexpr (RATE) {
      dr = -to_a * sg;
      dg = to_a * nrate * (sg * left);
    } else {
      dr = 0.f;
      dg = to_a * left;
    }
  }
};

template <typename T, int VC, bool RATE, int MIX>
__global__ __launch_bounds__(64 * kBwdWaves) void rec_bwd_kernel(RecArgs p, float* part) {
  constexpr int N = kBwdTokens;
  typedef Word<T, VC> W;
  __shared__ float word[2][kBwdWaves][64 * VC], ahead[2][kBwdWaves][64 * VC], back[2][kBwdWaves][64 * VC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const Place<VC> at(p, blockIdx.x);
  const int64_t len = row_length(p, at.b);
  float nrate[VC], D[VC], dr[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    nrate[k] = RATE ? -p.rate[at.c + k] : 0.f;
    D[k] = p.s_in ? p.s_in[at.b * p.si_sb + at.c + k] : 0.f;
    dr[k] = 0.f;
  }
  const int64_t span = (int64_t)waves * N;
  int turn = 0;
  for (int64_t t0 = (p.L - 1) / span * span; t0 >= 0 && p.L > 0; t0 -= span, turn ^= 1) {
    const int64_t tw = t0 + wave * N;
    const int n = (int)max((int64_t)0, min((int64_t)N, len - tw));
    typename W::raw x[N], g[N], gi[N], dh[N];
    float a[N][VC], w[N][VC], in[N][VC], A[VC], M[VC], hl[VC], dl[VC], S[VC];
    uint32_t starts = 0;
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      A[k] = 1.f;
      M[k] = hl[k] = dl[k] = S[k] = 0.f;
    }
    if (n > 0) {
      load_tokens<T, VC, N>(p.x, at, tw, n, x);
      load_tokens<T, VC, N>(p.g, at, tw, n, g);
      load_tokens<T, VC, N>(p.dh, at, tw, n, dh);
      if (p.i.p) load_tokens<T, VC, N>(p.i, at, tw, n, gi);
      const float* mk = p.marks + at.b * p.mk_sb + (tw / kRecMark) * p.mk_st + at.c;
#pragma unroll
      for (int k = 0; k < VC; ++k) S[k] = mk[k];
      starts = start_bits<N>(p, at.b, tw, n);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j >= n) continue;
        const bool fresh = starts >> j & 1;
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          float sg, left, m;
          sigmoids(W::get(g[j], k), &sg, &left);
          decay_of<RATE>(sg, left, nrate[k], &a[j][k], &m);
          w[j][k] = share_of<MIX>(m);
          float v = W::get(x[j], k) * w[j][k];
          if (p.i.p) {
            float s, sl;
            sigmoids(W::get(gi[j], k), &s, &sl);
            v *= s;
          }
          in[j][k] = v;
          if (fresh) {
            A[k] = 0.f;
            M[k] = 1.f;
            hl[k] = v;
          } else {
            A[k] *= a[j][k];
            M[k] += fmaf(-m, M[k], m);
            hl[k] = fmaf(a[j][k], hl[k], v);
          }
        }
      }
#pragma unroll
      for (int j = N - 1; j >= 0; --j) {
        if (j >= n) continue;
#pragma unroll
        for (int k = 0; k < VC; ++k)
          dl[k] = starts >> j & 1 ? 0.f : a[j][k] * (W::get(dh[j], k) + dl[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      word[turn][wave][lane * VC + k] = piece_word(A[k], M[k]);
      ahead[turn][wave][lane * VC + k] = hl[k];
      back[turn][wave][lane * VC + k] = dl[k];
    }
    __syncthreads();  // the other buffer's readers passed here one turn ago
    const int busy = (int)max((int64_t)0, min((int64_t)waves, (len - t0 + N - 1) / N));
    float C[VC];
#pragma unroll
    for (int k = 0; k < VC; ++k) C[k] = D[k];
    for (int v = busy - 1; v >= 0; --v) {
      if (v == wave)
#pragma unroll
        for (int k = 0; k < VC; ++k) C[k] = D[k];
#pragma unroll
      for (int k = 0; k < VC; ++k)
        D[k] = step_over(word[turn][v][lane * VC + k], back[turn][v][lane * VC + k], D[k]);
    }
    if (n > 0) {
      // the state before the piece: the mark, or one piece behind it
      if ((tw % kRecMark) != 0)
#pragma unroll
        for (int k = 0; k < VC; ++k)
          S[k] = step_over(word[turn][wave - 1][lane * VC + k], ahead[turn][wave - 1][lane * VC + k], S[k]);
      // `in` becomes the state before each token
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j >= n) continue;
        const bool fresh = starts >> j & 1;
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          const float v = in[j][k];
          in[j][k] = fresh ? 0.f : S[k];
          S[k] = fresh ? v : fmaf(a[j][k], S[k], v);
        }
      }
    }
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
      float dx[VC] = {}, dg[VC] = {}, di[VC] = {};
      if (j < n) {
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          const float G = W::get(dh[j], k) + C[k];
          const Grad<RATE, MIX> r(G, in[j][k], a[j][k], w[j][k], W::get(x[j], k), W::get(g[j], k),
                                  p.i.p ? W::get(gi[j], k) : 0.f, p.i.p != nullptr, nrate[k]);
          dx[k] = r.dx;
          dg[k] = r.dg;
          di[k] = r.di;
          if constexpr (RATE) dr[k] += r.dr;
          C[k] = starts >> j & 1 ? 0.f : a[j][k] * G;
        }
      }
      if (tw + j < p.L) {
        store_token<T, VC>(p.dx, at, tw + j, dx);
        store_token<T, VC>(p.dg, at, tw + j, dg);
        if (p.i.p) store_token<T, VC>(p.di, at, tw + j, di);
      }
    }
  }
  if (p.s_out && wave == 0 && at.live)
#pragma unroll
    for (int k = 0; k < VC; ++k) p.s_out[at.b * p.so_sb + at.c + k] = D[k];
  if constexpr (RATE) {
    if (part) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < VC; ++k) word[0][wave][lane * VC + k] = dr[k];
      __syncthreads();
      if (wave == 0 && at.live)
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          float s = 0.f;
          for (int v = 0; v < waves; ++v) s += word[0][v][lane * VC + k];
          part[at.b * p.channels + at.c + k] = s;
        }
    }
  }
}

// ------------------------------------------------------------------------------ single tokens

template <typename T, int VC, bool RATE, int MIX>
__global__ __launch_bounds__(256) void rec_step_kernel(RecArgs p) {
  typedef Word<T, VC> W;
  const int64_t per = p.channels / VC, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= p.batch * per) return;
  const int64_t b = e / per, c = e % per * VC;
  auto load = [&](const RecRows& r) {
    return *reinterpret_cast<const typename W::raw*>(static_cast<const T*>(r.p) + b * r.sb + c);
  };
  const typename W::raw x = load(p.x), g = load(p.g), gi = p.i.p ? load(p.i) : typename W::raw();
  float h[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) h[k] = p.s_in[b * p.si_sb + c + k];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    float sg, left, a, m;
    sigmoids(W::get(g, k), &sg, &left);
    decay_of<RATE>(sg, left, RATE ? -p.rate[c + k] : 0.f, &a, &m);
    float v = W::get(x, k) * share_of<MIX>(m);
    if (p.i.p) {
      float s, sl;
      sigmoids(W::get(gi, k), &s, &sl);
      v *= s;
    }
    h[k] = step_over(piece_word(a, m), v, h[k]);
  }
#pragma unroll
  for (int k = 0; k < VC; ++k) p.s_out[b * p.so_sb + c + k] = h[k];
  *reinterpret_cast<typename W::raw*>(static_cast<T*>(p.h.p) + b * p.h.sb + c) = W::put(h);
}

// ------------------------------------------------------------------------------------ launch

int channels_of(const RecArgs& a) { return a.bf16 && a.pairs ? 2 : 1; }  // a lane's

// waves of a block: as many pieces of n tokens as a row has, at most `most`, at least `least`
int waves_for(int64_t L, int n, int least, int most) {
  int w = least;
  while (w < most && (int64_t)w * n < L) w *= 2;
  return w;
}

#define SS_REC_MIXES(RUN, T, VC, R)       \
  if (a.mix == 0) RUN(T, VC, R, 0);       \
  else if (a.mix == 1) RUN(T, VC, R, 1);  \
  else RUN(T, VC, R, 2);
#define SS_REC_RATES(RUN, T, VC)          \
  if (a.rate) { SS_REC_MIXES(RUN, T, VC, true) } else { SS_REC_MIXES(RUN, T, VC, false) }
#define SS_REC_ALL(RUN)                                        \
  if (!a.bf16) { SS_REC_RATES(RUN, float, 1) }                 \
  else if (a.pairs) { SS_REC_RATES(RUN, bf16_t, 2) }           \
  else { SS_REC_RATES(RUN, bf16_t, 1) }

int64_t slabs_of(const RecArgs& a) {
  const int64_t per = 64 * channels_of(a);
  return (a.channels + per - 1) / per;
}

}  // namespace

int64_t rec_blocks(int64_t batch, int64_t L, int64_t channels) { return batch * ((channels + 63) / 64); }

int64_t rec_workspace_floats(int64_t batch, int64_t L, int64_t channels, bool backward) {
  return backward && L > 0 ? batch * channels : 0;
}

hipError_t launch_rec_fwd(const RecArgs& a, float* ws, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * slabs_of(a))), block(64 * waves_for(a.L, kFwdTokens, 1, kFwdWaves));
#define SS_RUN(T, VC, R, M) hipLaunchKernelGGL((rec_fwd_kernel<T, VC, R, M>), grid, block, 0, s, a)
  SS_REC_ALL(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

hipError_t launch_rec_bwd(const RecArgs& a, float* ws, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * slabs_of(a))), block(64 * waves_for(a.L, kBwdTokens, 2, kBwdWaves));
  float* part = a.drate && a.L > 0 ? ws : nullptr;
#define SS_RUN(T, VC, R, M) hipLaunchKernelGGL((rec_bwd_kernel<T, VC, R, M>), grid, block, 0, s, a, part)
  if (a.batch > 0) { SS_REC_ALL(SS_RUN) }
#undef SS_RUN
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.drate) return e;
  return launch_column_sum(part, a.drate, a.channels, part ? a.batch : 0, s);
}

hipError_t launch_rec_step(const RecArgs& a, hipStream_t s) {
  const int64_t lanes = a.batch * (a.channels / channels_of(a));
  const dim3 grid((unsigned)((lanes + 255) / 256)), block(256);
#define SS_RUN(T, VC, R, M) hipLaunchKernelGGL((rec_step_kernel<T, VC, R, M>), grid, block, 0, s, a)
  SS_REC_ALL(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

}  // namespace ss
