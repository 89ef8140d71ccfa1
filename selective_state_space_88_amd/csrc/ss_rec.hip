// ss_rec.hip -- the gated linear recurrence: forward and single tokens.  See ss_rec.h.
#include "ss_rec.h"

namespace ss {
namespace {

// PLAIN: every piece is whole or empty and no token starts afresh (no lengths, no starts, L a multiple of the
// piece), which saves the selects of each token
template <typename T, int VC, bool RATE, int MIX, bool GATE, bool PLAIN>
__global__ __launch_bounds__(64 * kWaves, 4) void rec_fwd_kernel(RecArgs p, Chain ch) {
  constexpr int N = kFwdTokens;
  typedef Word<T, VC> W;
  __shared__ Piece pieces[kWaves][64 * VC];
  __shared__ float entry[64 * VC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  uint32_t chain, place;
  take_chunk(ch, &chain, &place);
  const Place<T, VC> at(p, chain);
  const int64_t len = row_length(p, at.b);
  const int64_t t0 = (int64_t)place * waves * N, tw = t0 + wave * N;
  const int n = (int)max((int64_t)0, min((int64_t)N, len - tw));
  typename W::raw v[GATE ? 3 : 2][N];
  float nrate[VC];
  uint32_t starts = 0;
  if (n > 0) {
    if constexpr (GATE) load_tokens<T, VC, PLAIN, N>({&p.x, &p.g, &p.i}, at, tw, n, v);
    else load_tokens<T, VC, PLAIN, N>({&p.x, &p.g}, at, tw, n, v);
    if constexpr (!PLAIN) starts = start_bits<N>(p, at.b, tw, n);
  }
  load_rates<RATE, T, VC>(p, at, nrate);
  float a[N][VC], in[N][VC], none[1][VC], word[VC], end[VC], S[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    word[k] = kAll;
    end[k] = 0.f;
    S[k] = p.s_in ? p.s_in[at.b * p.si_sb + at.c + k] : 0.f;
  }
  if (n > 0)
    read_piece<T, VC, N, RATE, MIX, GATE, false, PLAIN>(v[0], v[1], v[GATE ? 2 : 0], n, starts, nrate, a, in,
                                                        none, word, end);
#pragma unroll
  for (int k = 0; k < VC; ++k) pieces[wave][lane * VC + k] = Piece{word[k], end[k]};
  __syncthreads();
  if (ch.chunks > 1) {
    const Link<VC> link(ch, chain, place, wave);
    link.enter([&](int u) { return pieces[u][link.slot]; }, first_state(p, at, link.slot), entry);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VC; ++k) S[k] = entry[lane * VC + k];
  }
  for (int u = 0; u < wave; ++u)
#pragma unroll
    for (int k = 0; k < VC; ++k) S[k] = step_over(pieces[u][lane * VC + k], S[k]);
  if (p.s_out && wave == waves - 1 && place + 1 == ch.chunks && at.live)
#pragma unroll
    for (int k = 0; k < VC; ++k) p.s_out[at.b * p.so_sb + at.c + k] = step_over(Piece{word[k], end[k]}, S[k]);
  if (tw >= p.L) return;
  if (p.marks && at.live) {
    float* mk = p.marks + at.b * p.mk_sb + (tw / kRecMark) * p.mk_st + at.c0;
#pragma unroll
    for (int k = 0; k < VC; ++k) mk[at.off + k] = S[k];
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float h[VC];
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      S[k] = !PLAIN && (starts >> j & 1) ? in[j][k] : fmaf(a[j][k], S[k], in[j][k]);
      h[k] = PLAIN || j < n ? S[k] : 0.f;
    }
    if (PLAIN || tw + j < p.L) store_token<T, VC>(p.h, at, tw + j, h);
  }
}

// ------------------------------------------------------------------------------ single tokens

template <typename T, int VC, bool RATE, int MIX, bool GATE>
__global__ __launch_bounds__(256) void rec_step_kernel(RecArgs p) {
  typedef Word<T, VC> W;
  const int64_t per = p.channels / VC, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= p.batch * per) return;
  const int64_t b = e / per, c = e % per * VC;
  auto load = [&](const RecRows& r) {
    return *reinterpret_cast<const typename W::raw*>(static_cast<const T*>(r.p) + b * r.sb + c);
  };
  const typename W::raw x = load(p.x), g = load(p.g), gi = GATE ? load(p.i) : typename W::raw();
  float h[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) h[k] = p.s_in[b * p.si_sb + c + k];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    float a, m, l;
    decay_of<RATE>(W::get(g, k), RATE ? -p.rate[c + k] : 0.f, &a, &m, &l);
    float v = W::get(x, k) * share_of<MIX>(m);
    if constexpr (GATE) v *= sigmoid_f32(W::get(gi, k));
    h[k] = step_over(Piece{piece_word(a, m), v}, h[k]);
  }
#pragma unroll
  for (int k = 0; k < VC; ++k) p.s_out[b * p.so_sb + c + k] = h[k];
  *reinterpret_cast<typename W::raw*>(static_cast<T*>(p.h.p) + b * p.h.sb + c) = W::put(h);
}

}  // namespace

int64_t rec_threads(int64_t batch, int64_t L, int64_t channels, int each, RecPass pass) {
  if (pass == RecPass::step) return (batch * (channels / each) + 255) / 256 * 256;
  const bool backward = pass == RecPass::backward;
  const int64_t per = 64 * each, threads = batch * ((channels + per - 1) / per) * 64;  // of one wave a chain
  if (threads > UINT32_MAX) return threads;  // already too many, and the product might not fit
  return threads * chunks_of(L, backward) * (backward ? bwd_waves(L) : fwd_waves(L));
}

int64_t rec_workspace_floats(int64_t batch, int64_t L, int64_t channels, bool backward) {
  const int64_t chunks = chunks_of(L, backward);
  const int64_t words = chain_words(batch * ((channels + 127) / 128 * 128), chunks);  // the most of any path
  return words + (backward && L > 0 ? batch * chunks * channels : 0);
}

hipError_t launch_rec_fwd(const RecArgs& a, float* ws, hipStream_t s) {
  Chain ch;
  if (const hipError_t e = make_chain(a, false, ws, s, &ch); e != hipSuccess) return e;
  const dim3 grid(ch.chains * ch.chunks), block(64 * fwd_waves(a.L));
#define SS_RUN(T, VC, R, M, G) hipLaunchKernelGGL((rec_fwd_kernel<T, VC, R, M, G, false>), grid, block, 0, s, a, ch)
#define SS_RUN_PLAIN(T, VC, R, M, G) hipLaunchKernelGGL((rec_fwd_kernel<T, VC, R, M, G, true>), grid, block, 0, s, a, ch)
  SS_REC_PIECES(SS_RUN, kFwdTokens)
#undef SS_RUN
#undef SS_RUN_PLAIN
  return hipGetLastError();
}

hipError_t launch_rec_step(const RecArgs& a, hipStream_t s) {
  const int64_t lanes = a.batch * (a.channels / channels_of(a));
  const dim3 grid((unsigned)((lanes + 255) / 256)), block(256);
#define SS_RUN(T, VC, R, M, G) hipLaunchKernelGGL((rec_step_kernel<T, VC, R, M, G>), grid, block, 0, s, a)
  SS_REC_ALL(SS_RUN)
#undef SS_RUN
  return hipGetLastError();
}

}  // namespace ss
