// ss_rec_bwd.hip -- the gated linear recurrence's gradients.  See ss_rec.h.
#include <type_traits>

#include "ss_rec.h"

namespace ss {
namespace {

// --------------------------------------------------------------------------------- backward

// The gradients of one token and channel: what the reverse walk knows is G, the state before the token
// (0 where it starts afresh), the decay a and the share w.
template <bool RATE, int MIX, bool GATE>
struct Grad {
  float dx, dg, di, dr;
  __device__ __forceinline__ Grad(float G, float hp, float a, float w, float x, float g, float i, float nrate) {
    float sg, left, s = 1.f, sl = 0.f;
    sigmoids(g, &sg, &left);
    if constexpr (GATE) sigmoids(i, &s, &sl);
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

template <typename T, int VC, bool RATE, int MIX, bool GATE, bool PLAIN>
__global__ __launch_bounds__(64 * kWaves, 4) void rec_bwd_kernel(RecArgs p, Chain ch, float* part) {
  constexpr int N = kBwdTokens;
  typedef Word<T, VC> W;
  __shared__ float word[kWaves][64 * VC], ahead[kWaves][64 * VC], back[kWaves][64 * VC], entry[64 * VC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  uint32_t chain, place;
  take_chunk(ch, &chain, &place);
  const Place<T, VC> at(p, chain);
  const int64_t len = row_length(p, at.b);
  const uint32_t chunk = ch.chunks - 1 - place;  // the gradient walks from the last chunk to the first
  const int64_t t0 = (int64_t)chunk * waves * N, tw = t0 + wave * N;
  const int n = (int)max((int64_t)0, min((int64_t)N, len - tw));
  typename W::raw raws[GATE ? 4 : 3][N];
  auto &x = raws[0], &g = raws[1], &dh = raws[2], &gi = raws[GATE ? 3 : 0];
  float nrate[VC], mark[VC], dr[VC] = {};
  uint32_t starts = 0;
  if (n > 0) {
    if constexpr (GATE) load_tokens<T, VC, PLAIN, N>({&p.x, &p.g, &p.dh, &p.i}, at, tw, n, raws);
    else load_tokens<T, VC, PLAIN, N>({&p.x, &p.g, &p.dh}, at, tw, n, raws);
    const float* mk = p.marks + at.b * p.mk_sb + (tw / kRecMark) * p.mk_st + at.c0;
#pragma unroll
    for (int k = 0; k < VC; ++k) mark[k] = mk[at.off + k];
    if constexpr (!PLAIN) starts = start_bits<N>(p, at.b, tw, n);
  }
  load_rates<RATE, T, VC>(p, at, nrate);
  float a[N][VC], w[N][VC], in[N][VC], head[VC], end[VC], dl[VC], D[VC], S[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    head[k] = kAll;
    end[k] = dl[k] = 0.f;
    S[k] = mark[k];
    D[k] = p.s_in ? p.s_in[at.b * p.si_sb + at.c + k] : 0.f;
  }
  if (n > 0) {
    read_piece<T, VC, N, RATE, MIX, GATE, true, PLAIN>(x, g, gi, n, starts, nrate, a, in, w, head, end);
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
      if (!PLAIN && j >= n) continue;
#pragma unroll
      for (int k = 0; k < VC; ++k)
        dl[k] = !PLAIN && (starts >> j & 1) ? 0.f : a[j][k] * (W::get(dh[j], k) + dl[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    word[wave][lane * VC + k] = head[k];
    ahead[wave][lane * VC + k] = end[k];
    back[wave][lane * VC + k] = dl[k];
  }
  __syncthreads();
  if (ch.chunks > 1) {
    const Link<VC> link(ch, chain, place, wave);
    link.enter([&](int u) { return Piece{word[kWaves - 1 - u][link.slot], back[kWaves - 1 - u][link.slot]}; },
               first_state(p, at, link.slot), entry);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VC; ++k) D[k] = entry[lane * VC + k];
  }
  for (int u = waves - 1; u > wave; --u)
#pragma unroll
    for (int k = 0; k < VC; ++k) D[k] = step_over(Piece{word[u][lane * VC + k], back[u][lane * VC + k]}, D[k]);
  if (p.s_out && wave == 0 && chunk == 0 && at.live)
#pragma unroll
    for (int k = 0; k < VC; ++k) p.s_out[at.b * p.so_sb + at.c + k] = step_over(Piece{head[k], dl[k]}, D[k]);
  // the state before the piece: the mark, or one piece behind it
  if (n > 0 && tw % kRecMark != 0)
#pragma unroll
    for (int k = 0; k < VC; ++k)
      S[k] = step_over(Piece{word[wave - 1][lane * VC + k], ahead[wave - 1][lane * VC + k]}, S[k]);
  // With masks too, most pieces are whole and without starts: without an input gate those take a walk without
  // selects (1 x 16384 x 1536, leak: 88 -> 82 us); with one, the second walk's registers cost more than it saves
  // (rate and unit share with starts, bf16: 1 x 16384 x 1536 133 -> 139 us, 2 x 4096 x 5120 199 -> 203; padded rows
  // of 3 x 1031 x 1537, f32: 35 -> 37)
  constexpr bool kTwoWalks = !PLAIN && !GATE;
  const auto walk = [&](auto is_whole) {
    constexpr bool whole = decltype(is_whole)::value;
    // `in` becomes the state before each token
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!whole && j >= n) continue;
      const bool fresh = !whole && (starts >> j & 1);
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        const float b = in[j][k];
        in[j][k] = fresh ? 0.f : S[k];
        S[k] = fresh ? b : fmaf(a[j][k], S[k], b);
      }
    }
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
      float dx[VC] = {}, dg[VC] = {}, di[VC] = {};
      if (whole || j < n) {
        const auto word_of = [](typename W::raw r) { return kTwoWalks ? r : opaque(r); };
        const typename W::raw xj = word_of(x[j]), gj = word_of(g[j]), ij = word_of(gi[j]), dj = word_of(dh[j]);
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          const float G = W::get(dj, k) + D[k];
          const Grad<RATE, MIX, GATE> r(G, in[j][k], a[j][k], w[j][k], W::get(xj, k), W::get(gj, k), W::get(ij, k),
                                        nrate[k]);
          dx[k] = r.dx;
          dg[k] = r.dg;
          di[k] = r.di;
          if constexpr (RATE) dr[k] += r.dr;
          D[k] = !whole && (starts >> j & 1) ? 0.f : a[j][k] * G;
        }
      }
      if (whole || tw + j < p.L) {
        store_token<T, VC>(p.dx, at, tw + j, dx);
        store_token<T, VC>(p.dg, at, tw + j, dg);
        if constexpr (GATE) store_token<T, VC>(p.di, at, tw + j, di);
      }
      if (!kTwoWalks && j % 2 == 0) __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (tw < p.L) {
    if constexpr (!kTwoWalks) walk(std::bool_constant<PLAIN>());
    else if (n == N && !starts) walk(std::true_type());
    else walk(std::false_type());
  }
  if constexpr (RATE) {
    if (part) {
      __syncthreads();  // the pieces have been read
#pragma unroll
      for (int k = 0; k < VC; ++k) word[wave][lane * VC + k] = dr[k];
      __syncthreads();
      if (wave == 0 && at.live)
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          float s = 0.f;
          for (int v = 0; v < waves; ++v) s += word[v][lane * VC + k];
          part[(at.b * ch.chunks + chunk) * p.channels + at.c + k] = s;
        }
    }
  }
}

}  // namespace

hipError_t launch_rec_bwd(const RecArgs& a, float* ws, hipStream_t s) {
  int64_t rows = 0;
  float* part = nullptr;
  if (a.batch > 0) {
    Chain ch;
    if (const hipError_t e = make_chain(a, true, ws, s, &ch); e != hipSuccess) return e;
    const dim3 grid(ch.chains * ch.chunks), block(64 * bwd_waves(a.L));
    if (a.drate && a.L > 0) {
      rows = a.batch * ch.chunks;
      part = ws + chain_words((int64_t)ch.chains * 64 * channels_of(a), ch.chunks);
    }
#define SS_RUN(T, VC, R, M, G) hipLaunchKernelGGL((rec_bwd_kernel<T, VC, R, M, G, false>), grid, block, 0, s, a, ch, part)
#define SS_RUN_PLAIN(T, VC, R, M, G) \
  hipLaunchKernelGGL((rec_bwd_kernel<T, VC, R, M, G, true>), grid, block, 0, s, a, ch, part)
    SS_REC_PIECES(SS_RUN, kBwdTokens)
#undef SS_RUN
#undef SS_RUN_PLAIN
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.drate) return e;
  return launch_column_sum(part, a.drate, a.channels, rows, s);
}

}  // namespace ss
