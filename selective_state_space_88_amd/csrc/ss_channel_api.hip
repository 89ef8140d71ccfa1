// ss_channel_api.hip -- C ABI of the operators on channels-last tensors beside the scan: the gated linear
// recurrence and the group norm with an activation.  See include/ss_scan.h.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "../../include/ss_scan.h"
#include "ss_host.h"
#include "ss_launch.h"

using namespace ss::host;

namespace {

constexpr int64_t kMaxBatch = 1 << 20, kMaxChannels = 1 << 24, kMaxThreads = UINT32_MAX;  // threads: of a launch

ss::RecRows rows_of(const ss_tensor* t) {
  if (!present(t)) return ss::RecRows{};
  return ss::RecRows{t->data, t->stride[0], t->ndim > 2 ? t->stride[1] : 0};
}

int check_lengths(const ss_tensor* lengths, int64_t Bt) {
  if (!present(lengths)) return SS_OK;
  const int rc = check_i32(lengths, 1, &Bt);
  if (rc) return rc;
  return lengths->stride[0] != 1 && Bt > 1 ? SS_ERR_STRIDE : SS_OK;
}

// an f32 tensor, read or (out) written
int check_f32(const ss_tensor* t, int ndim, const int64_t* shape, bool out) {
  const int rc = out ? check_out(t, ndim, shape) : check_in(t, ndim, shape);
  if (rc) return rc;
  return t->dtype == SS_F32 ? SS_OK : SS_ERR_DTYPE;
}

// a vector [channels] f32 of stride 1
int check_row(const ss_tensor* t, int64_t C) {
  const int rc = check_vector(t, C);
  if (rc) return rc;
  return t->stride[0] != 1 && C > 1 ? SS_ERR_STRIDE : SS_OK;
}

// every row starts at a multiple of `bytes`
bool aligned_to(const ss_tensor* t, int64_t bytes) {
  if (!present(t)) return true;
  if (reinterpret_cast<uintptr_t>(t->data) % bytes) return false;
  for (int i = 0; i + 1 < t->ndim; ++i)
    if (t->shape[i] > 1 && (t->stride[i] * esize(t->dtype)) % bytes) return false;
  return true;
}

// ------------------------------------------------------------------- gated linear recurrence

// sizes that no alignment of the rows makes too large for a launch
int rec_sizes(int64_t Bt, int64_t L, int64_t C, bool bf16, ss::RecPass pass) {
  if (Bt < 0 || L < 0 || C < 1) return SS_ERR_SHAPE;
  if (Bt > kMaxBatch || L > INT32_MAX || C > kMaxChannels) return SS_ERR_UNSUPPORTED;
  return ss::rec_threads(Bt, L, C, bf16 && C % 2 == 0 ? 2 : 1, pass) > kMaxThreads ? SS_ERR_UNSUPPORTED : SS_OK;
}

// the same for the call's own rows
int rec_launches(const ss::RecArgs& a, ss::RecPass pass) {
  const int64_t n = ss::rec_threads(a.batch, a.L, a.channels, a.pairs ? 2 : 1, pass);
  return n > kMaxThreads ? SS_ERR_UNSUPPORTED : SS_OK;
}

// what the forward, the backward (of [batch, L, channels]) and the step (of [batch, channels]) check alike
int rec_common(const ss_tensor* x, const ss_tensor* g, const ss_tensor* i, const ss_tensor* rate, uint32_t flags,
               ss::RecPass pass, ss::RecArgs* a) {
  if (!x || !g) return SS_ERR_NULL;
  const int ndim = pass == ss::RecPass::step ? 2 : 3;
  if ((flags & ~(SS_REC_LEAK | SS_REC_UNIT)) || flags == (SS_REC_LEAK | SS_REC_UNIT)) return SS_ERR_FLAGS;
  int rc;
  if ((rc = check_basic(x, ndim)) || (rc = check_in(g, ndim, x->shape)) ||
      (given(i) && (rc = check_in(i, ndim, x->shape))))
    return rc;
  if (g->dtype != x->dtype || (given(i) && i->dtype != x->dtype)) return SS_ERR_DTYPE;
  a->batch = x->shape[0];
  a->L = ndim == 3 ? x->shape[1] : 1;
  a->channels = x->shape[ndim - 1];
  if ((rc = rec_sizes(a->batch, a->L, a->channels, x->dtype == SS_BF16, pass))) return rc;
  if (present(rate) && (rc = check_row(rate, a->channels))) return rc;
  a->x = rows_of(x);
  a->g = rows_of(g);
  a->i = rows_of(i);
  a->rate = present(rate) ? static_cast<const float*>(rate->data) : nullptr;
  a->mix = flags & SS_REC_LEAK ? 1 : flags & SS_REC_UNIT ? 2 : 0;
  a->bf16 = x->dtype == SS_BF16;
  a->pairs = a->bf16 && a->channels % 2 == 0 && aligned_to(x, 4) && aligned_to(g, 4) && aligned_to(i, 4);
  return SS_OK;
}

int rec_masks(const ss_tensor* lengths, const ss_tensor* starts, ss::RecArgs* a) {
  int rc;
  if ((rc = check_lengths(lengths, a->batch))) return rc;
  const int64_t shape[2] = {a->batch, a->L};
  if (present(starts)) {
    if ((rc = check_i32(starts, 2, shape))) return rc;
    a->starts = static_cast<const int32_t*>(starts->data);
    a->starts_sb = starts->stride[0];
    a->starts_st = starts->stride[1];
  }
  a->lengths = present(lengths) ? static_cast<const int32_t*>(lengths->data) : nullptr;
  return SS_OK;
}

void rec_states(const ss_tensor* in, ss_tensor* out, ss::RecArgs* a) {
  if (present(in)) {
    a->s_in = static_cast<const float*>(in->data);
    a->si_sb = in->stride[0];
  }
  if (present(out)) {
    a->s_out = static_cast<float*>(out->data);
    a->so_sb = out->stride[0];
  }
}

// --------------------------------------------------------------------------------- group norm

// sizes that x's type and the rows' alignment may make small enough for a launch
int gnorm_sizes(int64_t Bt, int64_t L, int64_t C, int64_t groups, bool backward) {
  if (Bt < 0 || L < 0 || C < 1 || groups < 1 || C % groups) return SS_ERR_SHAPE;
  if (Bt > kMaxBatch || L > INT32_MAX || C > kMaxChannels) return SS_ERR_UNSUPPORTED;
  ss::GroupNormArgs a{};
  a.batch = Bt;
  a.L = L;
  a.channels = C;
  a.groups = (int32_t)groups;
  for (const int bf16 : {0, 1})
    for (const int line : {1, 4, 8}) {
      if (C % line || (line == 8 && !bf16)) continue;
      a.x_bf16 = a.y_bf16 = bf16;
      a.line = line;
      if (ss::gnorm_threads(a, backward) <= kMaxThreads) return SS_OK;
    }
  return SS_ERR_UNSUPPORTED;
}

// Channels of an access: 16 bytes of x, else 8 bytes of bf16, else one; every tensor's rows start at a
// multiple of as many of its own elements (of 16 bytes where they are more)
int gnorm_line(const ss_tensor* x, const ss_tensor* t, const ss_tensor* u) {
  const int64_t C = x->shape[2];
  for (const int line : {8, 4}) {
    if ((line == 8 && x->dtype != SS_BF16) || C % line) continue;
    const auto fits = [&](const ss_tensor* v) { return aligned_to(v, std::min<int64_t>(16, line * esize(v->dtype))); };
    if (fits(x) && fits(t) && fits(u)) return line;
  }
  return 1;
}

// what the forward and the backward check alike; `y`: y or dy
int gnorm_common(const ss_tensor* x, const ss_tensor* weight, const ss_tensor* bias, int32_t groups, float eps,
                 uint32_t flags, const ss_tensor* lengths, const ss_tensor* y, bool y_out, ss::GroupNormArgs* a) {
  if (!x || !weight || !y) return SS_ERR_NULL;
  if (flags & ~SS_NORM_SILU) return SS_ERR_FLAGS;
  int rc;
  if ((rc = check_basic(x, 3)) || (rc = y_out ? check_out(y, 3, x->shape) : check_in(y, 3, x->shape))) return rc;
  a->batch = x->shape[0];
  a->L = x->shape[1];
  a->channels = x->shape[2];
  a->groups = groups;
  if ((rc = gnorm_sizes(a->batch, a->L, a->channels, groups, !y_out))) return rc;
  if ((rc = check_row(weight, a->channels)) || (present(bias) && (rc = check_row(bias, a->channels))) ||
      (rc = check_lengths(lengths, a->batch)))
    return rc;
  if (!(eps >= 0.f)) return SS_ERR_UNSUPPORTED;
  a->eps = eps;
  a->silu = (flags & SS_NORM_SILU) != 0;
  a->x = rows_of(x);
  a->weight = static_cast<const float*>(weight->data);
  a->bias = present(bias) ? static_cast<const float*>(bias->data) : nullptr;
  a->lengths = present(lengths) ? static_cast<const int32_t*>(lengths->data) : nullptr;
  a->x_bf16 = x->dtype == SS_BF16;
  a->y_bf16 = y->dtype == SS_BF16;
  a->line = gnorm_line(x, x, y);
  return SS_OK;
}

void gnorm_stats(const ss_tensor* stats, ss::GroupNormArgs* a) {
  if (!present(stats)) return;
  a->stats = static_cast<float*>(stats->data);
  a->s_sb = stats->stride[0];
  a->s_sg = stats->stride[1];
}

}  // namespace

extern "C" {

int64_t ss_gatedrec_workspace(int64_t batch, int64_t L, int64_t channels, int32_t dtype, int32_t backward) {
  if (dtype != SS_F32 && dtype != SS_BF16) return SS_ERR_DTYPE;
  const int rc = rec_sizes(batch, L, channels, dtype == SS_BF16,
                           backward ? ss::RecPass::backward : ss::RecPass::forward);
  return rc ? rc : ss::rec_workspace_floats(batch, L, channels, backward != 0);
}

int ss_gatedrec_fwd(const ss_tensor* x, const ss_tensor* g, const ss_tensor* i, const ss_tensor* rate, uint32_t flags,
                    const ss_tensor* lengths, const ss_tensor* starts, const ss_tensor* s_init, ss_tensor* s_final,
                    ss_tensor* marks, ss_tensor* h, const ss_tensor* ws, void* stream) {
  if (!h) return SS_ERR_NULL;
  ss::RecArgs a{};
  int rc;
  if ((rc = rec_common(x, g, i, rate, flags, ss::RecPass::forward, &a)) || (rc = rec_masks(lengths, starts, &a)))
    return rc;
  const int64_t state[2] = {a.batch, a.channels}, mk[3] = {a.batch, (a.L + SS_REC_MARK - 1) / SS_REC_MARK, a.channels};
  if ((rc = check_out(h, 3, x->shape))) return rc;
  if (h->dtype != x->dtype) return SS_ERR_DTYPE;
  if (present(s_init) && (rc = check_f32(s_init, 2, state, false))) return rc;
  if (present(s_final) && (rc = check_f32(s_final, 2, state, true))) return rc;
  if (present(marks) && (rc = check_f32(marks, 3, mk, true))) return rc;
  const ss_tensor* ts[] = {x, g, i, rate, lengths, starts, s_init, s_final, marks, h};
  if (any_shares(h, ts, 10, 9) || (present(s_final) && any_shares(s_final, ts, 10, 7)) ||
      (present(marks) && any_shares(marks, ts, 10, 8)))
    return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 10))) return rc;
  if (a.batch == 0 || (a.L == 0 && !present(s_final))) return SS_OK;
  if (a.L > 0 && (!x->data || !g->data || !h->data)) return SS_ERR_NULL;
  a.h = rows_of(h);
  a.pairs = a.pairs && aligned_to(h, 4);
  if ((rc = rec_launches(a, ss::RecPass::forward))) return rc;
  rec_states(s_init, s_final, &a);
  if (present(marks)) {
    a.marks = static_cast<float*>(marks->data);
    a.mk_sb = marks->stride[0];
    a.mk_st = marks->stride[1];
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(ss::rec_workspace_floats(a.batch, a.L, a.channels, false), &wp))) return rc;
  return done(ss::launch_rec_fwd(a, wp, s));
}

int ss_gatedrec_bwd(const ss_tensor* x, const ss_tensor* g, const ss_tensor* i, const ss_tensor* rate, uint32_t flags,
                    const ss_tensor* lengths, const ss_tensor* starts, const ss_tensor* marks, const ss_tensor* dh,
                    const ss_tensor* ds_final, ss_tensor* dx, ss_tensor* dg, ss_tensor* di, ss_tensor* drate,
                    ss_tensor* ds_init, const ss_tensor* ws, void* stream) {
  if (!marks || !dh || !dx || !dg) return SS_ERR_NULL;
  ss::RecArgs a{};
  int rc;
  if ((rc = rec_common(x, g, i, rate, flags, ss::RecPass::backward, &a)) || (rc = rec_masks(lengths, starts, &a)))
    return rc;
  const bool gi = given(i), dr = present(drate);
  if (gi != given(di)) return SS_ERR_NULL;  // di exactly when i is given
  if (dr && !present(rate)) return SS_ERR_NULL;
  const int64_t state[2] = {a.batch, a.channels}, mk[3] = {a.batch, (a.L + SS_REC_MARK - 1) / SS_REC_MARK, a.channels};
  if ((rc = check_in(dh, 3, x->shape)) || (rc = check_out(dx, 3, x->shape)) || (rc = check_out(dg, 3, x->shape)) ||
      (gi && (rc = check_out(di, 3, x->shape))) || (rc = check_f32(marks, 3, mk, false)))
    return rc;
  if (dh->dtype != x->dtype || dx->dtype != x->dtype || dg->dtype != x->dtype || (gi && di->dtype != x->dtype))
    return SS_ERR_DTYPE;
  if (present(ds_final) && (rc = check_f32(ds_final, 2, state, false))) return rc;
  if (present(ds_init) && (rc = check_f32(ds_init, 2, state, true))) return rc;
  if (dr && (rc = check_row(drate, a.channels))) return rc;
  const ss_tensor* ts[] = {x, g, i, rate, lengths, starts, marks, dh, ds_final, dx, dg, di, drate, ds_init};
  if (any_shares(dx, ts, 14, 9) || any_shares(dg, ts, 14, 10) || (gi && any_shares(di, ts, 14, 11)) ||
      (dr && any_shares(drate, ts, 14, 12)) || (present(ds_init) && any_shares(ds_init, ts, 14, 13)))
    return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 14))) return rc;
  const bool some = a.batch > 0 && a.L > 0;
  if (!some && !dr && (a.batch == 0 || !present(ds_init))) return SS_OK;
  if (some && (!x->data || !g->data || !dh->data || !marks->data || !dx->data || !dg->data || (gi && !di->data)))
    return SS_ERR_NULL;
  a.dh = rows_of(dh);
  a.dx = rows_of(dx);
  a.dg = rows_of(dg);
  a.di = rows_of(di);
  a.pairs = a.pairs && aligned_to(dh, 4) && aligned_to(dx, 4) && aligned_to(dg, 4) && aligned_to(di, 4);
  if ((rc = rec_launches(a, ss::RecPass::backward))) return rc;
  rec_states(ds_final, ds_init, &a);
  a.marks = static_cast<float*>(marks->data);
  a.mk_sb = marks->stride[0];
  a.mk_st = marks->stride[1];
  a.drate = dr ? static_cast<float*>(drate->data) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(ss::rec_workspace_floats(a.batch, a.L, a.channels, true), &wp))) return rc;
  return done(ss::launch_rec_bwd(a, wp, s));
}

int ss_gatedrec_step(const ss_tensor* x, const ss_tensor* g, const ss_tensor* i, const ss_tensor* rate, uint32_t flags,
                     const ss_tensor* s, ss_tensor* s_out, ss_tensor* h, void* stream) {
  if (!s || !s_out || !h) return SS_ERR_NULL;
  ss::RecArgs a{};
  int rc;
  if ((rc = rec_common(x, g, i, rate, flags, ss::RecPass::step, &a))) return rc;
  if ((rc = check_out(h, 2, x->shape)) || (rc = check_f32(s, 2, x->shape, false)) ||
      (rc = check_f32(s_out, 2, x->shape, true)))
    return rc;
  if (h->dtype != x->dtype) return SS_ERR_DTYPE;
  const ss_tensor* ts[] = {x, g, i, rate, s, s_out, h};
  const ss_tensor* but_s[] = {x, g, i, rate, h};
  if (any_shares(h, ts, 7, 6)) return SS_ERR_ALIAS;
  if (same_view(s, s_out) ? any_shares(s_out, but_s, 5) : any_shares(s_out, ts, 7, 5)) return SS_ERR_ALIAS;
  if (a.batch == 0) return SS_OK;
  if (!x->data || !g->data || !s->data || !s_out->data || !h->data) return SS_ERR_NULL;
  a.h = rows_of(h);
  a.pairs = a.pairs && aligned_to(h, 4);
  if ((rc = rec_launches(a, ss::RecPass::step))) return rc;
  rec_states(s, s_out, &a);
  return done(ss::launch_rec_step(a, static_cast<hipStream_t>(stream)));
}

int64_t ss_groupnorm_workspace(int64_t batch, int64_t L, int64_t channels, int32_t groups, int32_t backward) {
  const int rc = gnorm_sizes(batch, L, channels, groups, backward != 0);
  return rc ? rc : ss::gnorm_workspace_floats(batch, L, channels, groups, backward != 0);
}

int ss_groupnorm_fwd(const ss_tensor* x, const ss_tensor* weight, const ss_tensor* bias, int32_t groups, float eps,
                     uint32_t flags, const ss_tensor* lengths, ss_tensor* stats, ss_tensor* y, const ss_tensor* ws,
                     void* stream) {
  ss::GroupNormArgs a{};
  int rc;
  if ((rc = gnorm_common(x, weight, bias, groups, eps, flags, lengths, y, true, &a))) return rc;
  const int64_t st[3] = {a.batch, groups, 3};
  if (present(stats) && (rc = check_f32(stats, 3, st, true))) return rc;
  const ss_tensor* ts[] = {x, weight, bias, lengths, stats, y};
  if (any_shares(y, ts, 6, 5) || (present(stats) && any_shares(stats, ts, 6, 4))) return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 6))) return rc;
  if (a.batch == 0 || (a.L == 0 && !present(stats))) return SS_OK;
  if (!weight->data || (a.L > 0 && (!x->data || !y->data))) return SS_ERR_NULL;
  if (ss::gnorm_threads(a, false) > kMaxThreads) return SS_ERR_UNSUPPORTED;
  a.y = rows_of(y);
  gnorm_stats(stats, &a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(ss::gnorm_workspace_floats(a.batch, a.L, a.channels, groups, false), &wp))) return rc;
  return done(ss::launch_gnorm_fwd(a, wp, s));
}

int ss_groupnorm_bwd(const ss_tensor* dy, const ss_tensor* x, const ss_tensor* weight, const ss_tensor* bias,
                     const ss_tensor* stats, int32_t groups, uint32_t flags, const ss_tensor* lengths, ss_tensor* dx,
                     ss_tensor* dweight, ss_tensor* dbias, const ss_tensor* ws, void* stream) {
  if (!stats || !dx) return SS_ERR_NULL;
  ss::GroupNormArgs a{};
  int rc;
  if ((rc = gnorm_common(x, weight, bias, groups, 0.f, flags, lengths, dy, false, &a))) return rc;
  const int64_t st[3] = {a.batch, groups, 3};
  const bool dw = present(dweight), db = present(dbias);
  if ((rc = check_f32(stats, 3, st, false)) || (rc = check_out(dx, 3, x->shape)) ||
      (dw && (rc = check_row(dweight, a.channels))) || (db && (rc = check_row(dbias, a.channels))))
    return rc;
  if (dx->dtype != x->dtype) return SS_ERR_DTYPE;
  const ss_tensor* ts[] = {dy, x, weight, bias, stats, lengths, dx, dweight, dbias};
  if (any_shares(dx, ts, 9, 6) || (dw && any_shares(dweight, ts, 9, 7)) || (db && any_shares(dbias, ts, 9, 8)))
    return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 9))) return rc;
  const bool some = a.batch > 0 && a.L > 0;
  if (!some && !dw && !db) return SS_OK;
  // stats are read for every row there is, of no positions too
  if (!weight->data || (a.batch > 0 && !stats->data)) return SS_ERR_NULL;
  if (some && (!dy->data || !x->data || !dx->data)) return SS_ERR_NULL;
  a.dy = rows_of(dy);
  a.dx = rows_of(dx);
  a.line = gnorm_line(x, dy, dx);
  if (ss::gnorm_threads(a, true) > kMaxThreads) return SS_ERR_UNSUPPORTED;
  gnorm_stats(stats, &a);
  a.dweight = dw ? static_cast<float*>(dweight->data) : nullptr;
  a.dbias = db ? static_cast<float*>(dbias->data) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(ss::gnorm_workspace_floats(a.batch, a.L, a.channels, groups, true), &wp))) return rc;
  return done(ss::launch_gnorm_bwd(a, wp, s));
}

}  // extern "C"
