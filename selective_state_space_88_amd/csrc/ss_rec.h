// ss_rec.h -- the gated linear recurrence on channels-last tensors, forward, backward and single
// tokens (gfx950).
//
//   h_t = a_t h_{t-1} + w(a_t) s_t x_t,   a = sigmoid(g) or exp(-rate sigmoid(g)),   s = sigmoid(i) or 1,
//   w = 1, 1 - a or sqrt(1 - a^2);   G_t = dh_t + a_{t+1} G_{t+1} is the gradient at h_t.
//
// Mapping.  A wave holds 16 (backward: 8) consecutive tokens of 64 lanes' channels (two bf16 channels or one
// f32 a lane, 256 bytes of a row an access), so that a token's flags are the same for all lanes and the scan
// over a lane's tokens is plain code.  The waves of a block hold consecutive pieces of one chunk of a row:
// each reduces its own piece to (decay A, end state from zero), they exchange these through LDS, and each
// walks its piece again from its true start, out of registers: every input is read once.
//
// Chunks of a row run in parallel and pass the state on through memory (see Link): a chunk publishes its
// own (A, end state) at once, and takes what comes before it from the state at the last boundary of
// kGroup chunks and the chunks since, always joined in the same order, so that results do not depend on
// timing.  Groups hand the state on one after the other, kGroup chunks at a time.
// Chunks are handed out by a counter in the order of their dependence, so what a chunk waits for belongs to
// blocks that already run, and every wait is bounded besides.
//
// Measured, calls behind each other (a large copy: 4.8 TB/s): 2 x 8192 x 5120, bf16 with both gates, unit share:
// 159 us, 4.2 TB/s; one row of 262144 x 512: 243 us, 4.4 TB/s; forward and backward of 2 x 4096 x 5120: 260 us,
// 3.6 TB/s (forward 90, backward 170; with starts 98 and 199, of 5119 channels 127 and 294).  About 46 VALU
// operations an element forward, 101 backward, a sixth of them transcendental, take two thirds of that time; a
// chunk lives 17 us, of which it waits 1 for its number and 3.6 for its neighbours,
// two blocks a CU.  Other shapes measured slower: 4 or 16 waves a block (290 and 306 us for the training step at
// a time when 8 took 269), pieces of 8 tokens forward (114 us against 105), groups of 32 chunks (176 us against
// 166 for the prompt), persistent blocks that load a chunk ahead (493 us for the training step: a chunk held as
// the next one holds up its chain).
//
// Precision.  All arithmetic is f32.  1 - a is formed without cancellation (sigmoid(-g), or -expm1), and
// a piece's decay enters the next one as H - (1 - A) H + h where A >= 1/2, with 1 - A accumulated on its
// own: A itself, rounded to 24 bits in every token, would shift a memory of n tokens by n 2^-25.  Below
// 1/2 it enters as A H + h, which keeps what a strong decay leaves of a large state.
#pragma once

#include <stdlib.h>

#include <algorithm>

#include "../../include/ss_scan.h"
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

// The same word, as one that the compiler knows nothing of: what was formed from it before is formed again, not
// kept in registers until here
template <typename R>
__device__ __forceinline__ R opaque(R r) {
  if constexpr (sizeof(R) == 2) {
    uint32_t u = r;
    asm("" : "+v"(u));
    return (R)u;
  } else {
    asm("" : "+v"(r));
    return r;
  }
}

__device__ __forceinline__ float sigmoid_f32(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// sigmoid(z) and 1 - sigmoid(z), each to f32 relative accuracy.  The exponent is capped at 2^126, where
// both are still normal numbers and a NaN passes.
__device__ __forceinline__ void sigmoids(float z, float* s, float* left) {
  float t = -z * kLog2e;
  t = t > 126.f ? 126.f : t;
  const float e = __builtin_amdgcn_exp2f(t);
  *s = __builtin_amdgcn_rcpf(1.0f + e);
  *left = e * *s;
}

// 1 - e^l for -1/4 < l <= 0, where the difference would cancel: the Taylor polynomial
// -l (1 + l/2 + ... + l^5/720), whose next term is 5e-8 of it.
constexpr float kNear = -0.25f;
__device__ __forceinline__ float near_one(float l) {
  float q = 1.f / 720.f;
  q = fmaf(q, l, 1.f / 120.f);
  q = fmaf(q, l, 1.f / 24.f);
  q = fmaf(q, l, 1.f / 6.f);
  q = fmaf(q, l, 0.5f);
  q = fmaf(q, l, 1.f);
  return q * -l;
}
// e^l and 1 - e^l
__device__ __forceinline__ void exps(float l, float* a, float* m) {
  *a = __builtin_amdgcn_exp2f(l * kLog2e);
  const float q = near_one(l);
  *m = l > kNear ? q : 1.0f - *a;
}

// The decay a, 1 - a and (with a rate) log a of one gate
template <bool RATE>
__device__ __forceinline__ void decay_of(float g, float nrate, float* a, float* m, float* l) {
  if constexpr (RATE) {
    *l = nrate * sigmoid_f32(g);
    exps(*l, a, m);
  } else {
    sigmoids(g, a, m);
  }
}

template <int MIX>
__device__ __forceinline__ float share_of(float m) {
  if constexpr (MIX == 1) return m;
  if constexpr (MIX == 2) return __builtin_amdgcn_sqrtf(m * (2.0f - m));
  return 1.0f;
}

// A piece of a row as a step on the state that enters it: H -> A H + h, kept as one word t for A (A itself
// below 1/2, else -(1 - A), and 1 where that is 0, so that all of H passes, infinities too) and h.  A piece with
// a start takes nothing over, NaN neither: kCut, which stays -0 in products.  A decay that has come to 0 is no
// cut: 0 H + h is a NaN where H is an infinity or NaN.
struct Piece {
  float t, h;
  __device__ __forceinline__ bool cut() const { return __float_as_int(t) == INT32_MIN; }
};
constexpr float kAll = 1.f, kCut = -0.f;
__device__ __forceinline__ float piece_word(float A, float M) { return A < 0.5f ? A : M == 0.f ? kAll : -M; }

// The decay of the tokens so far: (A, 1 - A) multiplied up, or, where log a is at hand, its sum
template <bool RATE>
struct Passed {
  float u = RATE ? 0.f : 1.f, v = 0.f;
  __device__ __forceinline__ void add(float a, float m, float l) {
    if constexpr (RATE) {
      u += l;
    } else {
      u *= a;
      v += fmaf(-m, v, m);
    }
  }
  __device__ __forceinline__ float word() const {
    if constexpr (!RATE) return piece_word(u, v);
    float A, M;
    exps(u, &A, &M);
    return piece_word(A, M);
  }
};
__device__ __forceinline__ float step_over(Piece q, float H) {
  return (q.cut() ? q.h : fmaf(q.t, H, q.h)) + (q.t < 0.f ? H : 0.f);
}
// p, then q
__device__ __forceinline__ Piece join(Piece p, Piece q) {
  if (q.cut()) return q;
  const bool np = p.t < 0.f, nq = q.t < 0.f;
  const float A = np ? 1.f + p.t : p.t, M = np ? -p.t : 1.f - p.t;
  const float B = nq ? 1.f + q.t : q.t, N = nq ? -q.t : 1.f - q.t;
  return Piece{piece_word(A * B, fmaf(N, A, M)), step_over(q, p.h)};
}

constexpr int kWaves = 8;   // of a block whose row has several chunks
constexpr int kGroup = 16;  // chunks from one handed-over state to the next

// The chain of a row's chunks through memory.  Words start as all ones; a published word is never that (a NaN
// is written with other bits), so that a word is its own flag and needs no ordering.  What is stored and
// loaded as atomics of device scope passes the L2s of the chip's dies.
struct Chain {
  uint32_t* counter;     // hands out the chunks; nullptr: every row is one chunk.  Then, 16 bytes on, the
                         // address of the word to set when a wait has reached its limit
  uint64_t* pieces;      // [chains][chunks][lanes' channels]: (t, h)
  uint32_t* states;      // [chains][groups][lanes' channels]: the state before a group, from the second on
  uint32_t chunks, chains, limit;
  __device__ __forceinline__ int* error() const { return *reinterpret_cast<int* const*>(counter + 4); }
};

__device__ __forceinline__ uint32_t not_ones(float v) {
  const uint32_t u = __float_as_uint(v);
  return u == 0xffffffffu ? 0x7fc00000u : u;
}

// A block's place in its chain.  The waves share the channels; the lanes of a wave are kTeams teams
// that share a channel's pieces, the block's own and those of the chunks before it, and join them by shuffles,
// in order.
template <int VC>
struct Link {
  static constexpr int kOwn = 64 * VC / kWaves, kTeams = 64 / kOwn;
  const Chain& ch;
  uint32_t at, slot;     // the chunk's place in its chain; the lane's channel in the slab
  int team;
  uint64_t* pieces;
  uint32_t* states;
  __device__ __forceinline__ Link(const Chain& c, uint32_t chain, uint32_t place, int wave) : ch(c), at(place) {
    slot = wave * kOwn + (threadIdx.x & (kOwn - 1));
    team = (threadIdx.x & 63) / kOwn;
    pieces = c.pieces + (int64_t)chain * c.chunks * (64 * VC);
    states = c.states + (int64_t)chain * ((c.chunks + kGroup - 1) / kGroup) * (64 * VC);
  }
  // the teams' pieces joined, the first team's first; every team has the result
  __device__ __forceinline__ Piece join_teams(Piece q) const {
#pragma unroll
    for (int m = kOwn; m < 64; m <<= 1) {
      const Piece o{__shfl_xor(q.t, m), __shfl_xor(q.h, m)};
      q = threadIdx.x & m ? join(o, q) : join(q, o);
    }
    return q;
  }
  // Poll `load` until every lane has what it asked for, or the limit is reached
  template <typename F>
  __device__ __forceinline__ void wait(F load) const {
    for (uint32_t polls = 0; !__all(load()); ++polls) {
      if (polls >= ch.limit) {
        if ((threadIdx.x & 63) == 0) atomicOr(ch.error(), 1);
        return;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
  // the chunks before this one in its group, joined
  __device__ __forceinline__ Piece before() const {
    constexpr int kEach = kGroup / kTeams;
    const uint32_t group = at / kGroup * kGroup, n = at - group;
    Piece r{kAll, 0.f};
    if (n == 0) return r;
    uint64_t q[kEach];
    wait([&] {
      bool ready = true;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const uint32_t k = min((uint32_t)(team * kEach + j), n - 1);
        q[j] = __hip_atomic_load(pieces + (int64_t)(group + k) * (64 * VC) + slot, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
        ready &= (uint32_t)(q[j] >> 32) != 0xffffffffu;
      }
      return ready;
    });
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if ((uint32_t)(team * kEach + j) < n) {
        const Piece v{__uint_as_float((uint32_t)q[j]), __uint_as_float((uint32_t)(q[j] >> 32))};
        r = j ? join(r, v) : v;
      }
    return join_teams(r);
  }
  // Publishes the chunk and writes the state before it to `entry`.  own(v): the block's piece v of the lane's
  // channel, in the chain's order; first: the chain's first state there.
  template <typename F>
  __device__ __forceinline__ void enter(F own, float first, float* entry) const {
    const bool hand_over = at % kGroup == kGroup - 1 && at + 1 < ch.chunks;
    Piece all = own(team * (kWaves / kTeams));
#pragma unroll
    for (int v = 1; v < kWaves / kTeams; ++v) all = join(all, own(team * (kWaves / kTeams) + v));
    all = join_teams(all);
    if (!hand_over && team == 0)
      __hip_atomic_store(pieces + (int64_t)at * (64 * VC) + slot,
                         (uint64_t)not_ones(all.h) << 32 | __float_as_uint(all.t), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    const Piece r = before();
    uint32_t st = __float_as_uint(first);
    if (at >= kGroup)
      wait([&] {
        st = __hip_atomic_load(states + (int64_t)(at / kGroup) * (64 * VC) + slot, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        return st != 0xffffffffu;
      });
    const float H = step_over(r, __uint_as_float(st));
    if (team == 0) {
      if (hand_over)
        __hip_atomic_store(states + (int64_t)((at + 1) / kGroup) * (64 * VC) + slot, not_ones(step_over(all, H)),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      entry[slot] = H;
    }
  }
};

// Which chunk this block takes: chain and place, in the order of the counter
__device__ __forceinline__ void take_chunk(const Chain& ch, uint32_t* chain, uint32_t* place) {
  *chain = blockIdx.x;
  *place = 0;
  if (ch.chunks <= 1) return;
  __shared__ uint32_t turn;
  if (threadIdx.x == 0) turn = atomicAdd(ch.counter, 1u);
  __syncthreads();
  const uint32_t i = __builtin_amdgcn_readfirstlane(turn);
  *chain = i % ch.chains;
  *place = i / ch.chains;
}

constexpr int kFwdTokens = 16;  // of a piece
constexpr int kBwdTokens = 8;   // two pieces share a mark
static_assert(kFwdTokens == kRecMark && 2 * kBwdTokens == kRecMark && kRecMark == SS_REC_MARK, "marks");

// Where a block works: the row, the slab's first channel and the lane's place in it (clamped so that every
// lane's loads are in bounds; `live` says whether they are its own).  Everything but the place is the same
// for the whole block, which keeps addresses in scalar registers.
template <typename T, int VC>
struct Place {
  int64_t b, c0, c;
  uint32_t off, bytes;   // in channels; in bytes of T
  bool live;
  __device__ __forceinline__ Place(const RecArgs& p, uint32_t block) {
    const uint32_t slabs = (uint32_t)((p.channels + 64 * VC - 1) / (64 * VC));
    b = block / slabs;
    c0 = (int64_t)(block % slabs) * (64 * VC);
    off = (threadIdx.x & 63) * VC;
    live = c0 + off < p.channels;
    if (!live) off = (uint32_t)(p.channels - VC - c0);
    c = c0 + off;
    bytes = off * sizeof(T);
  }
};

// the chain's first state in the slab's channel `slot` (clamped likewise)
template <typename T, int VC>
__device__ __forceinline__ float first_state(const RecArgs& p, const Place<T, VC>& at, uint32_t slot) {
  return p.s_in ? p.s_in[at.b * p.si_sb + min(at.c0 + slot, p.channels - 1)] : 0.f;
}

__device__ __forceinline__ int64_t row_length(const RecArgs& p, int64_t b) {
  if (!p.lengths) return p.L;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// A word of a row: `row` is the same for the block, the lane adds its bytes
template <typename T, int VC>
__device__ __forceinline__ typename Word<T, VC>::raw* word_at(const T* row, const Place<T, VC>& at) {
  const char* q = reinterpret_cast<const char*>(row) + at.bytes;
  return reinterpret_cast<typename Word<T, VC>::raw*>(const_cast<char*>(q));
}

// The loads of n <= N tokens of R tensors from t0 on (the last token again behind them), token by token, so
// that the first can be worked on while the others are on their way
template <typename T, int VC, bool PLAIN, int N, int R>
__device__ __forceinline__ void load_tokens(const RecRows* const (&r)[R], const Place<T, VC>& at, int64_t t0, int n,
                                            typename Word<T, VC>::raw (&v)[R][N]) {
  const T* q[R];
#pragma unroll
  for (int i = 0; i < R; ++i) q[i] = static_cast<const T*>(r[i]->p) + at.b * r[i]->sb + at.c0 + t0 * r[i]->st;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      v[i][j] = *word_at<T, VC>(q[i], at);
      if (PLAIN || j + 1 < n) q[i] += r[i]->st;
    }
}

template <typename T, int VC>
__device__ __forceinline__ void store_token(const RecRows& r, const Place<T, VC>& at, int64_t t, const float (&v)[VC]) {
  const T* q = static_cast<const T*>(r.p) + at.b * r.sb + at.c0 + t * r.st;
  if (at.live) *word_at<T, VC>(q, at) = Word<T, VC>::put(v);
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

// The lane's -rate
template <bool RATE, typename T, int VC>
__device__ __forceinline__ void load_rates(const RecArgs& p, const Place<T, VC>& at, float (&nrate)[VC]) {
#pragma unroll
  for (int k = 0; k < VC; ++k) nrate[k] = RATE ? -p.rate[at.c + k] : 0.f;
}

// A piece's tokens from their inputs: every token's a and b = w s x, the piece's word and end state from zero;
// with KEEP the shares w too.  Four tokens at a time, since work further ahead only takes registers.  What a
// token's place does to it (n, starts; nothing if PLAIN) is the same for the whole wave: selects, no branches.
template <typename T, int VC, int N, bool RATE, int MIX, bool GATE, bool KEEP, bool PLAIN>
__device__ __forceinline__ void read_piece(const typename Word<T, VC>::raw (&x)[N], const typename Word<T, VC>::raw (&g)[N],
                                           const typename Word<T, VC>::raw (&gi)[N], int n, uint32_t starts,
                                           const float (&nrate)[VC], float (&a)[N][VC], float (&b)[N][VC],
                                           float (&w)[KEEP ? N : 1][VC], float (&word)[VC], float (&end)[VC]) {
  typedef Word<T, VC> W;
  Passed<RATE> passed[VC];
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const bool fresh = !PLAIN && (starts >> t & 1), pad = !PLAIN && t >= n;
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      float m, l = 0.f;
      decay_of<RATE>(W::get(g[t], k), nrate[k], &a[t][k], &m, &l);
      const float share = share_of<MIX>(m);
      float v = W::get(x[t], k) * share;
      if constexpr (GATE) v *= sigmoid_f32(W::get(gi[t], k));
      // behind the last token: a state passes as it is
      a[t][k] = pad ? 1.f : a[t][k];
      b[t][k] = v = pad ? 0.f : v;
      if constexpr (KEEP) w[t][k] = share;
      passed[k].add(a[t][k], pad ? 0.f : m, pad ? 0.f : l);
      end[k] = fresh ? v : fmaf(a[t][k], end[k], v);
    }
    if (t % 4 == 3) __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int k = 0; k < VC; ++k) word[k] = !PLAIN && starts ? kCut : passed[k].word();
}

// ------------------------------------------------------------------------------------ launch

int channels_of(const RecArgs& a) { return a.bf16 && a.pairs ? 2 : 1; }  // a lane's

// waves of a block: as many pieces of n tokens as a row has, at most `most`, at least `least`
int waves_for(int64_t L, int n, int least, int most) {
  int w = least;
  while (w < most && (int64_t)w * n < L) w *= 2;
  return w;
}

#define SS_REC_GATES(RUN, T, VC, R, M) \
  if (a.i.p) RUN(T, VC, R, M, true); else RUN(T, VC, R, M, false);
#define SS_REC_MIXES(RUN, T, VC, R)                         \
  if (a.mix == 0) { SS_REC_GATES(RUN, T, VC, R, 0) }        \
  else if (a.mix == 1) { SS_REC_GATES(RUN, T, VC, R, 1) }   \
  else { SS_REC_GATES(RUN, T, VC, R, 2) }
#define SS_REC_RATES(RUN, T, VC)          \
  if (a.rate) { SS_REC_MIXES(RUN, T, VC, true) } else { SS_REC_MIXES(RUN, T, VC, false) }
#define SS_REC_ALL(RUN)                                        \
  if (!a.bf16) { SS_REC_RATES(RUN, float, 1) }                 \
  else if (a.pairs) { SS_REC_RATES(RUN, bf16_t, 2) }           \
  else { SS_REC_RATES(RUN, bf16_t, 1) }
// The same with whether every piece of n tokens is whole (rows of single bf16 channels go without the form)
#define SS_REC_PIECES(RUN, n)                                                       \
  const bool whole = !a.lengths && !a.starts && a.L % (n) == 0;                     \
  if (!a.bf16) {                                                                    \
    if (whole) { SS_REC_RATES(RUN##_PLAIN, float, 1) } else { SS_REC_RATES(RUN, float, 1) }  \
  } else if (a.pairs) {                                                             \
    if (whole) { SS_REC_RATES(RUN##_PLAIN, bf16_t, 2) } else { SS_REC_RATES(RUN, bf16_t, 2) } \
  } else { SS_REC_RATES(RUN, bf16_t, 1) }

int64_t slabs_of(const RecArgs& a) {
  const int64_t per = 64 * channels_of(a);
  return (a.channels + per - 1) / per;
}

int fwd_waves(int64_t L) { return waves_for(L, kFwdTokens, 1, kWaves); }
int bwd_waves(int64_t L) { return waves_for(L, kBwdTokens, 2, kWaves); }

// chunks of a row (one at least: a row of no tokens still passes its state on)
int64_t chunks_of(int64_t L, bool backward) {
  const int64_t span = backward ? bwd_waves(L) * kBwdTokens : fwd_waves(L) * kFwdTokens;
  return std::max<int64_t>(1, (L + span - 1) / span);
}

constexpr int64_t kCounterWords = 64;  // the counter's own lines

// 4-byte words of a chain over `lanes` channels (every row's, rounded up to whole waves)
int64_t chain_words(int64_t lanes, int64_t chunks) {
  if (chunks <= 1) return 0;
  const int64_t words = kCounterWords + lanes * (2 * chunks + (chunks + kGroup - 1) / kGroup);
  return (words + 3) / 4 * 4;
}

// the counter 0 and the error's address behind it, every word all ones
__global__ __launch_bounds__(256) void chain_clear_kernel(u32x4* words, int64_t n, uint64_t error) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const uint32_t v = i < kCounterWords / 4 ? 0u : 0xffffffffu;
    words[i] = i == 1 ? u32x4{(uint32_t)error, (uint32_t)(error >> 32), 0u, 0u} : u32x4{v, v, v, v};
  }
}

// Polls of a wait, about a microsecond each; SS_SPIN_LIMIT in the environment lowers it for tests.
uint32_t wait_limit() {
  if (const char* e = getenv("SS_SPIN_LIMIT")) return (uint32_t)strtoul(e, nullptr, 10);
  return 1u << 22;
}

// The chain of a call, its words cleared on the stream
hipError_t make_chain(const RecArgs& a, bool backward, float* ws, hipStream_t s, Chain* to) {
  Chain& ch = *to = Chain{};
  ch.chunks = (uint32_t)chunks_of(a.L, backward);
  ch.chains = (uint32_t)(a.batch * slabs_of(a));
  if (ch.chunks <= 1) return hipSuccess;
  int* error = nullptr;
  if (const hipError_t e = spin_error_word(&error); e != hipSuccess) return e;
  const int64_t lanes = (int64_t)ch.chains * 64 * channels_of(a);
  ch.counter = reinterpret_cast<uint32_t*>(ws);
  ch.pieces = reinterpret_cast<uint64_t*>(ws + kCounterWords);
  ch.states = reinterpret_cast<uint32_t*>(ws + kCounterWords + 2 * lanes * ch.chunks);
  ch.limit = wait_limit();
  const int64_t n = chain_words(lanes, ch.chunks) / 4;
  hipLaunchKernelGGL(chain_clear_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4 * cu_count())), dim3(256), 0,
                     s, reinterpret_cast<u32x4*>(ws), n, (uint64_t)reinterpret_cast<uintptr_t>(error));
  return hipGetLastError();
}

}  // namespace
}  // namespace ss
