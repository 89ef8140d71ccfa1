// ss_block_api.hip -- C ABI of the operators around and beside the scan: linear attention with a
// decay per head, rotary positions, the norms before and after a block.  See include/ss_scan.h.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "../../include/ss_scan.h"
#include "ss_host.h"
#include "ss_launch.h"

using namespace ss::host;

namespace {

// ------------------------------------------------------------------------ linear attention

constexpr int64_t kMaxHeadDim = 256, kMaxRows = 1 << 20;  // K and V; batch * heads

int lin_sizes(int64_t Bt, int64_t L, int64_t H, int64_t Hq, int64_t Hk, int64_t Hv, int64_t K, int64_t V) {
  if (Bt < 0 || L < 0 || H < 1 || Hq < 1 || Hk < 1 || Hv < 1) return SS_ERR_SHAPE;
  if (H % Hq || H % Hk || H % Hv) return SS_ERR_SHAPE;
  if (K < 1 || V < 1 || K > kMaxHeadDim || V > kMaxHeadDim) return SS_ERR_UNSUPPORTED;
  if (L > INT32_MAX || H > kMaxRows || Bt > kMaxRows || Bt * H > kMaxRows) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

ss::HeadRows head_rows(const ss_tensor* t, int64_t heads) {
  return ss::HeadRows{t->data, t->stride[0], t->stride[1], t->stride[2], (int32_t)(heads / t->shape[2])};
}

bool rows16(const ss_tensor* t) {
  const int64_t per = 16 / esize(t->dtype);
  return aligned16(t) && t->shape[t->ndim - 1] % per == 0;
}

struct LinCall {
  int64_t Bt, L, H, K, V;
  bool bf16;
  ss::HeadRows q, k, v;
  const float* log_decay;
  const int32_t* lengths;
  float scale;
  bool vec;
};

// what the forward and the backward check alike
int lin_common(const ss_tensor* q, const ss_tensor* k, const ss_tensor* v, const ss_tensor* log_decay, float scale,
               const ss_tensor* lengths, LinCall* c) {
  if (!q || !k || !v || !log_decay) return SS_ERR_NULL;
  int rc;
  if ((rc = check_basic(q, 4)) || (rc = check_basic(k, 4)) || (rc = check_basic(v, 4)) ||
      (rc = check_basic(log_decay, 1)))
    return rc;
  if (k->dtype != q->dtype || v->dtype != q->dtype || log_decay->dtype != SS_F32) return SS_ERR_DTYPE;
  c->Bt = q->shape[0];
  c->L = q->shape[1];
  c->K = q->shape[3];
  c->V = v->shape[3];
  c->H = log_decay->shape[0];
  if (k->shape[0] != c->Bt || v->shape[0] != c->Bt || k->shape[1] != c->L || v->shape[1] != c->L ||
      k->shape[3] != c->K)
    return SS_ERR_SHAPE;
  if ((rc = lin_sizes(c->Bt, c->L, c->H, q->shape[2], k->shape[2], v->shape[2], c->K, c->V))) return rc;
  if (lengths && lengths->data && (rc = check_i32(lengths, 1, &c->Bt))) return rc;
  if (present(lengths) && lengths->stride[0] != 1 && c->Bt > 1) return SS_ERR_STRIDE;
  c->bf16 = q->dtype == SS_BF16;
  c->q = head_rows(q, c->H);
  c->k = head_rows(k, c->H);
  c->v = head_rows(v, c->H);
  c->log_decay = static_cast<const float*>(log_decay->data);
  c->lengths = present(lengths) ? static_cast<const int32_t*>(lengths->data) : nullptr;
  c->scale = scale;
  c->vec = rows16(q) && rows16(k) && rows16(v);
  return SS_OK;
}

int check_lin_state(const ss_tensor* s, const LinCall& c, bool out) {
  const int64_t shape[4] = {c.Bt, c.H, c.K, c.V};
  const int rc = out ? check_out(s, 4, shape) : check_in(s, 4, shape);
  if (rc) return rc;
  return s->dtype == SS_F32 ? SS_OK : SS_ERR_DTYPE;
}

ss::LinArgs lin_args(const LinCall& c) {
  ss::LinArgs a{};
  a.log_decay = c.log_decay;
  a.lengths = c.lengths;
  a.batch = c.Bt;
  a.L = c.L;
  a.heads = (int32_t)c.H;
  a.bf16 = c.bf16;
  a.pair_scale = 1.f;
  a.out_scale = 1.f;
  return a;
}

void set_z_in(ss::LinArgs& a, const ss_tensor* s, bool transposed) {
  if (!present(s)) return;
  a.z_in = static_cast<const float*>(s->data);
  a.zi_sb = s->stride[0];
  a.zi_sh = s->stride[1];
  a.zi_sd = transposed ? 1 : s->stride[2];
  a.zi_se = transposed ? s->stride[2] : 1;
}

void set_z_out(ss::LinArgs& a, const ss_tensor* s) {
  if (!present(s)) return;
  a.z_out = static_cast<float*>(s->data);
  a.zo_sb = s->stride[0];
  a.zo_sh = s->stride[1];
  a.zo_sd = s->stride[2];
  a.zo_se = 1;
}

void set_o(ss::LinArgs& a, void* o, int64_t sb, int64_t st, int64_t sh, bool f32) {
  a.o = o;
  a.o_sb = sb;
  a.o_st = st;
  a.o_sh = sh;
  a.o_f32 = f32;
}

ss::LinArgs lin_forward(const LinCall& c, const ss_tensor* s_init, ss_tensor* s_final, ss_tensor* o) {
  ss::LinArgs a = lin_args(c);
  a.a = c.q;
  a.b = c.k;
  a.c = c.v;
  a.D = (int32_t)c.K;
  a.E = (int32_t)c.V;
  a.out_scale = c.scale;
  a.e0 = 1;
  set_z_in(a, s_init, false);
  set_z_out(a, s_final);
  if (o) set_o(a, o->data, o->stride[0], o->stride[1], o->stride[2], !c.bf16);
  a.vec = c.vec && (!o || rows16(o));
  return a;
}

// The three passes of the backward.  dq is the forward's form on (d_o, v, k) with the state
// transposed; dv and dk run from the last token back, on (k, q, d_o) and (v, d_o, q), and carry
// the same state, dk its transpose.
struct LinBackward {
  ss::LinArgs pass[3];  // dq, dv, dk
  int64_t sum_floats;   // the largest per-head gradient of shared heads
};

// floats of the per-head gradient of a tensor whose heads are shared
int64_t head_floats(const LinCall& c, int32_t share, int64_t dim) { return share > 1 ? c.Bt * c.L * c.H * dim : 0; }

LinBackward lin_backward(const LinCall& c, const ss_tensor* s_init, const ss_tensor* d_o, const ss_tensor* ds_final,
                         ss_tensor* dq, ss_tensor* dk, ss_tensor* dv, ss_tensor* ds_init) {
  LinBackward r;
  for (ss::LinArgs& a : r.pass) a = lin_args(c);
  const ss::HeadRows g = d_o ? head_rows(d_o, c.H) : ss::HeadRows{};
  ss::LinArgs &pq = r.pass[0], &pv = r.pass[1], &pk = r.pass[2];
  pq.a = g, pq.b = c.v, pq.c = c.k;
  pk.a = c.v, pk.b = g, pk.c = c.q;
  pv.a = c.k, pv.b = c.q, pv.c = g;
  pq.D = pk.D = pv.E = (int32_t)c.V;
  pq.E = pk.E = pv.D = (int32_t)c.K;
  pq.out_scale = c.scale;
  pq.e0 = 1;
  pk.pair_scale = pv.pair_scale = c.scale;
  pk.reverse = pv.reverse = 1;
  pk.z_before = 1;
  set_z_in(pq, s_init, true);
  set_z_in(pk, ds_final, true);
  set_z_in(pv, ds_final, false);
  set_z_out(pv, ds_init);
  ss_tensor* outs[3] = {dq, dv, dk};
  for (int i = 0; i < 3; ++i)
    if (outs[i]) set_o(r.pass[i], outs[i]->data, outs[i]->stride[0], outs[i]->stride[1], outs[i]->stride[2], !c.bf16);
  r.sum_floats = std::max(head_floats(c, std::max(c.q.share, c.k.share), c.K), head_floats(c, c.v.share, c.V));
  return r;
}

// ------------------------------------------------------------------------------------ norms

int check_rows(const ss_tensor* t, const int64_t* shape, bool out, bool time_too) {
  if (t->ndim != 3) return SS_ERR_SHAPE;
  if (t->dtype != SS_F32 && t->dtype != SS_BF16) return SS_ERR_DTYPE;
  for (int i = 0; i < 3; ++i) {
    if (t->shape[i] != shape[i]) return SS_ERR_SHAPE;
    if (t->stride[i] < 0) return SS_ERR_STRIDE;
  }
  const bool channel = t->stride[2] == 1 || t->shape[2] <= 1, time = t->stride[1] == 1 || t->shape[1] <= 1;
  if (!channel && !(time_too && time)) return SS_ERR_STRIDE;
  return out && folds(t) ? SS_ERR_STRIDE : SS_OK;
}

ss::NormRows norm_rows(const ss_tensor* t) {
  if (!given(t)) return ss::NormRows{};
  return ss::NormRows{t->data, t->stride[0], t->stride[1], t->stride[2], t->dtype == SS_BF16};
}

bool channel_inner(const ss_tensor* t) { return !given(t) || t->stride[2] == 1 || t->shape[2] <= 1; }

bool norm_vec(const ss_tensor* t) {
  if (!given(t)) return true;
  return aligned16(t);
}

// the same for a tensor whose innermost dimension is the channels or the time: every line of 8
// elements from a multiple of 8 on is 16-byte aligned
bool line_vec(const ss_tensor* t, int64_t group) {
  if (!given(t)) return true;
  if (reinterpret_cast<uintptr_t>(t->data) % 16) return false;
  const int64_t es = esize(t->dtype);
  const bool channel = channel_inner(t);
  const int outer = channel ? 1 : 2;
  if (channel && (group * es) % 16) return false;
  return (t->shape[0] <= 1 || (t->stride[0] * es) % 16 == 0) &&
         (t->shape[outer] <= 1 || (t->stride[outer] * es) % 16 == 0);
}

int norm_sizes(int64_t Bt, int64_t L, int64_t C, int64_t groups) {
  if (Bt < 0 || L < 0 || C < 1 || groups < 1 || C % groups) return SS_ERR_SHAPE;
  if (C / groups > 32768) return SS_ERR_UNSUPPORTED;
  if (Bt > 0 && L > (((int64_t)1 << 31) - 1) / Bt) return SS_ERR_UNSUPPORTED;
  if (groups > 65535 || C > (1 << 24)) return SS_ERR_UNSUPPORTED;  // sizes of launches
  return SS_OK;
}

}  // namespace

extern "C" {

int64_t ss_linattn_workspace(int64_t batch, int64_t L, int64_t heads, int64_t heads_q, int64_t heads_k,
                             int64_t heads_v, int64_t K, int64_t V, int32_t dtype, int32_t backward) {
  if (dtype != SS_F32 && dtype != SS_BF16) return SS_ERR_DTYPE;
  const int rc = lin_sizes(batch, L, heads, heads_q, heads_k, heads_v, K, V);
  if (rc) return rc;
  LinCall c{};
  c.Bt = batch;
  c.L = L;
  c.H = heads;
  c.K = K;
  c.V = V;
  c.bf16 = dtype == SS_BF16;
  c.q.share = (int32_t)(heads / heads_q);
  c.k.share = (int32_t)(heads / heads_k);
  c.v.share = (int32_t)(heads / heads_v);
  if (!backward) {
    const ss::LinArgs a = lin_forward(c, nullptr, nullptr, nullptr);
    return ss::lin_workspace_floats(&a, 1);
  }
  const LinBackward r = lin_backward(c, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  return ss::lin_workspace_floats(r.pass, 3) + r.sum_floats;
}

int ss_linattn_fwd(const ss_tensor* q, const ss_tensor* k, const ss_tensor* v, const ss_tensor* log_decay,
                   float scale, const ss_tensor* lengths, const ss_tensor* s_init, ss_tensor* s_final,
                   ss_tensor* o, const ss_tensor* ws, void* stream) {
  if (!o) return SS_ERR_NULL;
  LinCall c;
  int rc;
  if ((rc = lin_common(q, k, v, log_decay, scale, lengths, &c))) return rc;
  const int64_t so[4] = {c.Bt, c.L, c.H, c.V};
  if ((rc = check_out(o, 4, so))) return rc;
  if (o->dtype != q->dtype) return SS_ERR_DTYPE;
  if (present(s_init) && (rc = check_lin_state(s_init, c, false))) return rc;
  if (present(s_final) && (rc = check_lin_state(s_final, c, true))) return rc;
  const ss_tensor* ts[] = {q, k, v, log_decay, lengths, s_init, s_final, o};
  if (any_shares(o, ts, 8, 7) || (present(s_final) && any_shares(s_final, ts, 8, 6))) return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 8))) return rc;
  if (c.Bt == 0 || (c.L == 0 && !present(s_final))) return SS_OK;
  if (!log_decay->data || (c.L > 0 && (!q->data || !k->data || !v->data || !o->data))) return SS_ERR_NULL;
  if (log_decay->stride[0] != 1 && c.H > 1) return SS_ERR_STRIDE;
  const ss::LinArgs a = lin_forward(c, s_init, s_final, o);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(ss::lin_workspace_floats(&a, 1), &wp))) return rc;
  return done(ss::launch_lin(&a, nullptr, 1, wp, s));
}

int ss_linattn_bwd(const ss_tensor* q, const ss_tensor* k, const ss_tensor* v, const ss_tensor* log_decay,
                   float scale, const ss_tensor* lengths, const ss_tensor* s_init, const ss_tensor* d_o,
                   const ss_tensor* ds_final, ss_tensor* dq, ss_tensor* dk, ss_tensor* dv, ss_tensor* ds_init,
                   const ss_tensor* ws, void* stream) {
  if (!d_o || !dq || !dk || !dv) return SS_ERR_NULL;
  LinCall c;
  int rc;
  if ((rc = lin_common(q, k, v, log_decay, scale, lengths, &c))) return rc;
  const int64_t so[4] = {c.Bt, c.L, c.H, c.V};
  if ((rc = check_in(d_o, 4, so)) || (rc = check_out(dq, 4, q->shape)) || (rc = check_out(dk, 4, k->shape)) ||
      (rc = check_out(dv, 4, v->shape)))
    return rc;
  if (d_o->dtype != q->dtype || dq->dtype != q->dtype || dk->dtype != q->dtype || dv->dtype != q->dtype)
    return SS_ERR_DTYPE;
  if (present(s_init) && (rc = check_lin_state(s_init, c, false))) return rc;
  if (present(ds_final) && (rc = check_lin_state(ds_final, c, false))) return rc;
  if (present(ds_init) && (rc = check_lin_state(ds_init, c, true))) return rc;
  const ss_tensor* ts[] = {q, k, v, log_decay, lengths, s_init, d_o, ds_final, dq, dk, dv, ds_init};
  if (any_shares(dq, ts, 12, 8) || any_shares(dk, ts, 12, 9) || any_shares(dv, ts, 12, 10) ||
      (present(ds_init) && any_shares(ds_init, ts, 12, 11)))
    return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 12))) return rc;
  if (c.Bt == 0 || (c.L == 0 && !present(ds_init))) return SS_OK;
  if (!log_decay->data) return SS_ERR_NULL;
  if (c.L > 0 && (!q->data || !k->data || !v->data || !d_o->data || !dq->data || !dk->data || !dv->data))
    return SS_ERR_NULL;
  if (log_decay->stride[0] != 1 && c.H > 1) return SS_ERR_STRIDE;
  LinBackward r = lin_backward(c, s_init, d_o, ds_final, dq, dk, dv, ds_init);
  ss_tensor* outs[3] = {dq, dv, dk};
  const int32_t share[3] = {c.q.share, c.v.share, c.k.share};
  for (int i = 0; i < 3; ++i) r.pass[i].vec = c.vec && rows16(d_o) && (share[i] > 1 || rows16(outs[i]));
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(ss::lin_workspace_floats(r.pass, 3) + r.sum_floats, &wp))) return rc;
  // the per-head gradients of shared heads go to the workspace first (behind the passes' own part,
  // a multiple of four floats: aligned rows wherever the head size allows) and are summed from there
  // before the next pass, which writes in the same place: half the memory, and read while it is cached
  float* per_head = wp + ss::lin_workspace_floats(r.pass, 3);
  ss::HeadSum sums[3] = {};
  for (int i = 0; i < 3; ++i) {
    const int64_t dim = r.pass[i].E;
    if (share[i] <= 1) continue;
    sums[i] = ss::HeadSum{outs[i]->data, outs[i]->stride[0], outs[i]->stride[1], outs[i]->stride[2], share[i]};
    set_o(r.pass[i], per_head, c.L * c.H * dim, c.H * dim, dim, true);
  }
  return done(ss::launch_lin(r.pass, sums, 3, wp, s));
}

int ss_linattn_step(const ss_tensor* q, const ss_tensor* k, const ss_tensor* v, const ss_tensor* log_decay,
                    float scale, const ss_tensor* st, ss_tensor* s_out, ss_tensor* o, void* stream) {
  if (!q || !k || !v || !log_decay || !st || !s_out || !o) return SS_ERR_NULL;
  int rc;
  if ((rc = check_basic(q, 3)) || (rc = check_basic(k, 3)) || (rc = check_basic(v, 3)) ||
      (rc = check_basic(log_decay, 1)))
    return rc;
  if (k->dtype != q->dtype || v->dtype != q->dtype || log_decay->dtype != SS_F32) return SS_ERR_DTYPE;
  LinCall c{};
  c.Bt = q->shape[0];
  c.K = q->shape[2];
  c.V = v->shape[2];
  c.H = log_decay->shape[0];
  if (k->shape[0] != c.Bt || v->shape[0] != c.Bt || k->shape[2] != c.K) return SS_ERR_SHAPE;
  if ((rc = lin_sizes(c.Bt, 1, c.H, q->shape[1], k->shape[1], v->shape[1], c.K, c.V))) return rc;
  const int64_t so[3] = {c.Bt, c.H, c.V};
  if ((rc = check_out(o, 3, so)) || (rc = check_lin_state(st, c, false)) || (rc = check_lin_state(s_out, c, true)))
    return rc;
  const ss_tensor* ts[] = {q, k, v, log_decay, st, s_out, o};
  const ss_tensor* but_s[] = {q, k, v, log_decay, o};
  if (any_shares(o, ts, 7, 6)) return SS_ERR_ALIAS;
  if (same_view(st, s_out) ? any_shares(s_out, but_s, 5) : any_shares(s_out, ts, 7, 5)) return SS_ERR_ALIAS;
  if (c.Bt == 0) return SS_OK;
  if (!q->data || !k->data || !v->data || !log_decay->data || !st->data || !s_out->data || !o->data)
    return SS_ERR_NULL;
  if (log_decay->stride[0] != 1 && c.H > 1) return SS_ERR_STRIDE;
  ss::LinStepArgs a{};
  auto rows = [&](const ss_tensor* t) {
    return ss::HeadRows{t->data, t->stride[0], 0, t->stride[1], (int32_t)(c.H / t->shape[1])};
  };
  a.q = rows(q);
  a.k = rows(k);
  a.v = rows(v);
  a.log_decay = static_cast<const float*>(log_decay->data);
  a.s = static_cast<const float*>(st->data);
  a.s_out = static_cast<float*>(s_out->data);
  a.o = o->data;
  a.s_sb = st->stride[0];
  a.s_sh = st->stride[1];
  a.s_sk = st->stride[2];
  a.so_sb = s_out->stride[0];
  a.so_sh = s_out->stride[1];
  a.so_sk = s_out->stride[2];
  a.o_sb = o->stride[0];
  a.o_sh = o->stride[1];
  a.scale = scale;
  a.batch = c.Bt;
  a.heads = (int32_t)c.H;
  a.K = (int32_t)c.K;
  a.V = (int32_t)c.V;
  a.in_bf16 = q->dtype == SS_BF16;
  a.out_bf16 = o->dtype == SS_BF16;
  a.vec = rows16(st) && rows16(s_out);
  return done(ss::launch_lin_step(a, static_cast<hipStream_t>(stream)));
}

int ss_rope(const ss_tensor* x, const ss_tensor* x2, const ss_tensor* pos, int64_t pos0, const ss_tensor* inv_freq,
            float amp, uint32_t flags, ss_tensor* out, ss_tensor* out2, void* stream) {
  if (!x || !inv_freq || !out) return SS_ERR_NULL;
  if (flags & ~(SS_ROPE_INTERLEAVED | SS_ROPE_INVERSE)) return SS_ERR_FLAGS;
  if (given(x2) != given(out2)) return SS_ERR_NULL;
  const bool two = given(x2);
  int rc;
  if ((rc = check_basic(x, 4)) || (rc = check_basic(inv_freq, 1)) || (rc = check_out(out, 4, x->shape))) return rc;
  if (two && ((rc = check_basic(x2, 4)) || (rc = check_out(out2, 4, x2->shape)))) return rc;
  if (inv_freq->dtype != SS_F32 || out->dtype != x->dtype) return SS_ERR_DTYPE;
  if (two && (x2->dtype != x->dtype || out2->dtype != x->dtype)) return SS_ERR_DTYPE;
  const int64_t Bt = x->shape[0], L = x->shape[1], D = x->shape[3], n = inv_freq->shape[0];
  if (two && (x2->shape[0] != Bt || x2->shape[1] != L || x2->shape[3] != D)) return SS_ERR_SHAPE;
  if (2 * n > D) return SS_ERR_SHAPE;
  const int64_t H = x->shape[2], H2 = two ? x2->shape[2] : 0;
  if (D > 65536 || H > 65535 || H2 > 65535) return SS_ERR_UNSUPPORTED;
  if (Bt > 0 && L > (((int64_t)1 << 31) - 1) / Bt) return SS_ERR_UNSUPPORTED;
  const int64_t ps[2] = {Bt, L};
  if (present(pos) && (rc = check_i32(pos, 2, ps))) return rc;
  const ss_tensor* others[] = {x2, pos, inv_freq, out2};
  const ss_tensor* others2[] = {x, pos, inv_freq, out};
  if (any_shares(out, others, 4) || (!same_view(x, out) && shares(out, x))) return SS_ERR_ALIAS;
  if (two && (any_shares(out2, others2, 4) || (!same_view(x2, out2) && shares(out2, x2)))) return SS_ERR_ALIAS;
  if (Bt * L == 0 || D == 0 || H + H2 == 0) return SS_OK;
  if (!present(pos) && (pos0 < -((int64_t)1 << 50) || pos0 > ((int64_t)1 << 50))) return SS_ERR_UNSUPPORTED;
  if ((H > 0 && (!x->data || !out->data)) || (H2 > 0 && (!x2->data || !out2->data)) || (n > 0 && !inv_freq->data))
    return SS_ERR_NULL;
  if (inv_freq->stride[0] != 1 && n > 1) return SS_ERR_STRIDE;
  ss::RopeArgs a{};
  auto put = [&](int i, const ss_tensor* in, ss_tensor* to) {
    a.t[i].x = in->data;
    a.t[i].out = to->data;
    a.t[i].x_sb = in->stride[0];
    a.t[i].x_st = in->stride[1];
    a.t[i].x_sh = in->stride[2];
    a.t[i].o_sb = to->stride[0];
    a.t[i].o_st = to->stride[1];
    a.t[i].o_sh = to->stride[2];
    a.t[i].heads = (int32_t)in->shape[2];
    a.t[i].copy = !same_view(in, to);
  };
  put(0, x, out);
  if (two) put(1, x2, out2);
  if (present(pos)) {
    a.pos = static_cast<const int32_t*>(pos->data);
    a.p_sb = pos->stride[0];
    a.p_st = pos->stride[1];
  }
  a.pos0 = pos0;
  a.inv_freq = static_cast<const float*>(inv_freq->data);
  a.amp = amp;
  a.batch = Bt;
  a.L = L;
  a.n = (int32_t)n;
  a.dim = (int32_t)D;
  a.interleaved = (flags & SS_ROPE_INTERLEAVED) != 0;
  a.inverse = (flags & SS_ROPE_INVERSE) != 0;
  a.bf16 = x->dtype == SS_BF16;
  a.vec = aligned16(x) && aligned16(out) && (!two || (aligned16(x2) && aligned16(out2)));
  return done(ss::launch_rope(a, static_cast<hipStream_t>(stream)));
}

int64_t ss_norm_workspace(int64_t batch, int64_t L, int64_t channels, int32_t groups) {
  const int rc = norm_sizes(batch, L, channels, groups);
  return rc ? rc : ss::norm_workspace_floats(batch, L, channels, groups);
}

int ss_addnorm_fwd(const ss_tensor* x, const ss_tensor* residual, const ss_tensor* weight, float alpha, float eps,
                   ss_tensor* sum, ss_tensor* y, void* stream) {
  if (!x || !weight || !y) return SS_ERR_NULL;
  const bool res = given(residual), out = given(sum);
  int rc;
  if (x->ndim != 3) return SS_ERR_SHAPE;
  const int64_t* shape = x->shape;
  if ((rc = check_rows(x, shape, false, false)) || (rc = check_rows(y, shape, true, false)) ||
      (res && (rc = check_rows(residual, shape, false, false))) ||
      (out && (rc = check_rows(sum, shape, true, false))))
    return rc;
  const int64_t Bt = shape[0], L = shape[1], C = shape[2];
  if ((rc = check_vector(weight, C)) || (rc = norm_sizes(Bt, L, C, 1))) return rc;
  if (res && out && residual->dtype != sum->dtype) return SS_ERR_DTYPE;
  if (!(eps >= 0.f)) return SS_ERR_UNSUPPORTED;
  const ss_tensor* ts[] = {x, residual, weight, sum, y};
  const ss_tensor* but_res[] = {x, weight, y};
  if (any_shares(y, ts, 5, 4)) return SS_ERR_ALIAS;
  if (out && (res && same_view(residual, sum) ? any_shares(sum, but_res, 3) : any_shares(sum, ts, 5, 3)))
    return SS_ERR_ALIAS;
  if (Bt * L == 0) return SS_OK;
  if (!x->data || !y->data || !weight->data) return SS_ERR_NULL;
  if (weight->stride[0] != 1 && C > 1) return SS_ERR_STRIDE;
  ss::AddNormArgs a{};
  a.x = norm_rows(x);
  a.residual = norm_rows(residual);
  a.sum = norm_rows(sum);
  a.y = norm_rows(y);
  a.weight = static_cast<const float*>(weight->data);
  a.alpha = alpha;
  a.eps = eps;
  a.batch = Bt;
  a.L = L;
  a.channels = C;
  a.vec = C % 8 == 0 && norm_vec(x) && norm_vec(residual) && norm_vec(sum) && norm_vec(y) && aligned16(weight);
  return done(ss::launch_addnorm_fwd(a, static_cast<hipStream_t>(stream)));
}

int ss_addnorm_bwd(const ss_tensor* dy, const ss_tensor* dsum, const ss_tensor* sum, const ss_tensor* weight,
                   float alpha, float eps, ss_tensor* dresidual, ss_tensor* dx, ss_tensor* dweight,
                   const ss_tensor* ws, void* stream) {
  if (!dy || !sum || !weight) return SS_ERR_NULL;
  const bool ds = given(dsum), dr = given(dresidual), dxx = given(dx), dw = given(dweight);
  int rc;
  if (sum->ndim != 3) return SS_ERR_SHAPE;
  const int64_t* shape = sum->shape;
  if ((rc = check_rows(sum, shape, false, false)) || (rc = check_rows(dy, shape, false, false)) ||
      (ds && (rc = check_rows(dsum, shape, false, false))) || (dr && (rc = check_rows(dresidual, shape, true, false))) ||
      (dxx && (rc = check_rows(dx, shape, true, false))))
    return rc;
  const int64_t Bt = shape[0], L = shape[1], C = shape[2];
  if ((rc = check_vector(weight, C)) || (dw && (rc = check_vector(dweight, C))) || (rc = norm_sizes(Bt, L, C, 1)))
    return rc;
  if ((ds && dsum->dtype != sum->dtype) || (dr && dresidual->dtype != sum->dtype)) return SS_ERR_DTYPE;
  if (!(eps >= 0.f)) return SS_ERR_UNSUPPORTED;
  const ss_tensor* ts[] = {dy, dsum, sum, weight, dresidual, dx, dweight};
  const ss_tensor* but_dsum[] = {dy, sum, weight, dx, dweight};
  if (dr && (ds && same_view(dsum, dresidual) ? any_shares(dresidual, but_dsum, 5) : any_shares(dresidual, ts, 7, 4)))
    return SS_ERR_ALIAS;
  if ((dxx && any_shares(dx, ts, 7, 5)) || (dw && any_shares(dweight, ts, 7, 6))) return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 7))) return rc;
  if (C > 1 && (weight->stride[0] != 1 || (dw && dweight->stride[0] != 1))) return SS_ERR_STRIDE;
  if (!(dr || dxx || dw)) return SS_OK;
  if (!weight->data || (dw && !dweight->data)) return SS_ERR_NULL;
  if (Bt * L > 0 && (!dy->data || !sum->data)) return SS_ERR_NULL;
  ss::AddNormArgs a{};
  a.dy = norm_rows(dy);
  a.dsum = norm_rows(dsum);
  a.sum = norm_rows(sum);
  a.dres = norm_rows(dresidual);
  a.dx = norm_rows(dx);
  a.weight = static_cast<const float*>(weight->data);
  a.dweight = dw ? static_cast<float*>(dweight->data) : nullptr;
  a.alpha = alpha;
  a.eps = eps;
  a.batch = Bt;
  a.L = L;
  a.channels = C;
  a.vec = C % 8 == 0 && norm_vec(dy) && norm_vec(dsum) && norm_vec(sum) && norm_vec(dresidual) && norm_vec(dx) &&
          aligned16(weight);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(dw ? ss::norm_workspace_floats(Bt, L, C, 1) : 0, &wp))) return rc;
  return done(ss::launch_addnorm_bwd(a, wp, s));
}

}  // extern "C"

namespace {

// what ss_gatenorm_fwd and _bwd check alike; `out`: y or dy
int gate_common(const ss_tensor* x, const ss_tensor* z, const ss_tensor* weight, int32_t groups, float eps,
                uint32_t flags, const ss_tensor* y, bool y_out, ss::GateNormArgs* a) {
  if (!x || !weight || !y) return SS_ERR_NULL;
  if (flags & ~SS_NORM_GATE_FIRST) return SS_ERR_FLAGS;
  int rc;
  if (x->ndim != 3) return SS_ERR_SHAPE;
  const int64_t* shape = x->shape;
  if ((rc = check_rows(x, shape, false, true)) || (rc = check_rows(y, shape, y_out, true)) ||
      (given(z) && (rc = check_rows(z, shape, false, true))))
    return rc;
  if ((rc = check_vector(weight, shape[2])) || (rc = norm_sizes(shape[0], shape[1], shape[2], groups))) return rc;
  if (weight->stride[0] != 1 && shape[2] > 1) return SS_ERR_STRIDE;
  if (!(eps >= 0.f)) return SS_ERR_UNSUPPORTED;
  a->x = norm_rows(x);
  a->z = norm_rows(z);
  a->weight = static_cast<const float*>(weight->data);
  a->eps = eps;
  a->batch = shape[0];
  a->L = shape[1];
  a->channels = shape[2];
  a->groups = groups;
  a->gate_first = given(z) && (flags & SS_NORM_GATE_FIRST);
  a->rows = channel_inner(x) && channel_inner(z) && channel_inner(y);
  const int64_t group = shape[2] / groups;
  a->any_vec = line_vec(x, group) && line_vec(z, group) && line_vec(y, group);
  a->vec = group % 8 == 0 && norm_vec(x) && norm_vec(z) && norm_vec(y) && aligned16(weight);
  return SS_OK;
}

}  // namespace

extern "C" {

int ss_gatenorm_fwd(const ss_tensor* x, const ss_tensor* z, const ss_tensor* weight, int32_t groups, float eps,
                    uint32_t flags, ss_tensor* y, void* stream) {
  ss::GateNormArgs a{};
  int rc;
  if ((rc = gate_common(x, z, weight, groups, eps, flags, y, true, &a))) return rc;
  const ss_tensor* ts[] = {x, z, weight};
  if (any_shares(y, ts, 3)) return SS_ERR_ALIAS;
  if (a.batch * a.L == 0) return SS_OK;
  if (!x->data || !weight->data || !y->data || (given(z) && !z->data)) return SS_ERR_NULL;
  a.y = norm_rows(y);
  return done(ss::launch_gatenorm_fwd(a, static_cast<hipStream_t>(stream)));
}

int ss_gatenorm_bwd(const ss_tensor* dy, const ss_tensor* x, const ss_tensor* z, const ss_tensor* weight,
                    int32_t groups, float eps, uint32_t flags, ss_tensor* dx, ss_tensor* dz, ss_tensor* dweight,
                    const ss_tensor* ws, void* stream) {
  if (!dx) return SS_ERR_NULL;
  ss::GateNormArgs a{};
  int rc;
  if ((rc = gate_common(x, z, weight, groups, eps, flags, dy, false, &a))) return rc;
  const bool gz = given(z), dw = given(dweight);
  if (gz != given(dz)) return SS_ERR_NULL;  // dz exactly when z is given
  if ((rc = check_rows(dx, x->shape, true, true)) || (gz && (rc = check_rows(dz, x->shape, true, true))) ||
      (dw && (rc = check_vector(dweight, a.channels))))
    return rc;
  if (dx->dtype != x->dtype || (gz && dz->dtype != z->dtype)) return SS_ERR_DTYPE;
  if (dw && dweight->stride[0] != 1 && a.channels > 1) return SS_ERR_STRIDE;
  const ss_tensor* ts[] = {dy, x, z, weight, dx, dz, dweight};
  if (any_shares(dx, ts, 7, 4) || (gz && any_shares(dz, ts, 7, 5)) || (dw && any_shares(dweight, ts, 7, 6)))
    return SS_ERR_ALIAS;
  if ((rc = check_ws(ws, ts, 7))) return rc;
  const bool some = a.batch * a.L > 0;
  if (!some && !dw) return SS_OK;
  if (!weight->data || (dw && !dweight->data)) return SS_ERR_NULL;
  if (some && (!dy->data || !x->data || !dx->data || (gz && (!z->data || !dz->data)))) return SS_ERR_NULL;
  a.dy = norm_rows(dy);
  a.dx = norm_rows(dx);
  a.dz = norm_rows(dz);
  a.dweight = dw ? static_cast<float*>(dweight->data) : nullptr;
  a.rows = a.rows && channel_inner(dx) && channel_inner(dz);
  a.any_vec = a.any_vec && line_vec(dx, a.channels / groups) && line_vec(dz, a.channels / groups);
  a.vec = a.vec && norm_vec(dx) && norm_vec(dz);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w(ws, s);
  float* wp;
  if ((rc = w.get(dw ? ss::norm_workspace_floats(a.batch, a.L, a.channels, groups) : 0, &wp))) return rc;
  return done(ss::launch_gatenorm_bwd(a, wp, s));
}

}  // extern "C"
