// The C ABI's entry points of the decayed linear attention, the rotary positions and the layer
// norm (include/kata.h).  As in kata_api.cpp, every call validates its arguments on the host,
// checks the device, enqueues its kernels on the caller's stream and returns.
#include <hip/hip_runtime.h>

#include <string>

#include "api.h"
#include "decay.h"
#include "kata.h"
#include "layer.h"
#include "layer_plan.h"
#include "plan.h"

using kata::check_device;
using kata::clear_error;
using kata::launch_status;
using kata::set_error;
using kata::Timed;

namespace {

// Strides for the kernels; an axis of one entry is never stepped along.
void copy3(long long (&to)[3], const int64_t from[3]) {
  for (int i = 0; i < 3; ++i) to[i] = from[i];
}

kata_status need_aligned(const void* p, size_t bytes, const char* name) {
  if (reinterpret_cast<uintptr_t>(p) % bytes)
    return set_error(KATA_ERR_INVALID_ARGUMENT,
                     std::string(name) + " is not " + std::to_string(bytes) + "-byte aligned");
  return KATA_OK;
}

struct Named {
  const void* p;
  const int64_t* st;
  const char* name;
};

// Problem, tensors, decays and offsets.
enum class Form { forward, backward, tokens };
kata_status check_decay(const kata_decay_problem* pr, Form form, const Named* ts, int n,
                        const float* log_decay, const int32_t* cu) {
  std::string why;
  kata_status s = form == Form::tokens ? kata::validate_decay_decode(pr, &why)
                                       : kata::validate_decay(pr, form == Form::backward, &why);
  if (s != KATA_OK) return set_error(s, why);
  const size_t es = kata::elem_size(pr->dtype);
  const int64_t sizes[3] = {pr->packed ? 1 : pr->n_seq, pr->T, pr->H};
  for (int i = 0; i < n; ++i)
    if ((s = kata::validate_rows(ts[i].p, ts[i].st, sizes, es, ts[i].name, &why)) != KATA_OK)
      return set_error(s, why);
  if (!log_decay) return set_error(KATA_ERR_INVALID_ARGUMENT, "log_decay is null");
  if (pr->packed && !cu) return set_error(KATA_ERR_INVALID_ARGUMENT, "cu_seqlens is null");
  if ((s = need_aligned(log_decay, 4, "log_decay")) != KATA_OK) return s;
  return need_aligned(cu, 4, "cu_seqlens");
}

kata_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return set_error(KATA_ERR_WORKSPACE, "workspace needs " + std::to_string(need) +
                                             " bytes, got " + std::to_string(have));
  return need ? need_aligned(ws, 256, "workspace") : KATA_OK;
}

kata::DecayArgs decay_args(const kata_decay_problem* pr, const kata::DecayPlan& p,
                           const float* log_decay, const int32_t* cu, int n_roles) {
  kata::DecayArgs a{};
  a.log_decay = log_decay;
  a.cu = cu;
  a.n_roles = n_roles;
  a.n_seq = pr->n_seq;
  a.H = pr->H;
  a.T = pr->T;
  a.packed = pr->packed;
  a.zero_tail = pr->zero_tail;
  a.L = p.L;
  a.n_seg = p.n_seg;
  a.n_slots = p.n_slots;
  a.scan = p.scan;
  a.join = p.join;
  a.stream = p.stream;
  return a;
}

// The kernels number their workgroups in 32 bits (grid_rows in device.h takes fewer than 2^31).
kata_status check_grid(const kata::DecayPlan& p) {
  if (p.groups >= int64_t(1) << 31)
    return set_error(KATA_ERR_UNSUPPORTED, "too many sequences and heads for one launch");
  return KATA_OK;
}

// Whether states are written where others are read.
bool states_overlap(const kata_decay_problem* pr, const float* written, const float* read) {
  const uintptr_t w = uintptr_t(written), r = uintptr_t(read);
  const uintptr_t n = uintptr_t(pr->n_seq) * pr->H * pr->dk * pr->dv * 4;
  return w && r && w < r + n && r < w + n;
}

kata_status run_decay(kata::DecayArgs& a, const kata::DecayPlan& p, bool bf16, bool exact_state,
                      hipStream_t st, const char* what) {
  hipError_t e = hipSuccess;
  if (p.scan) {
    {
      Timed t(KATA_K_CHUNK_STATE, st);
      e = kata::launch_decay_chunks(a, bf16, exact_state, true, st);
    }
    if (e != hipSuccess) return launch_status(e, what);
    if (!a.join) {
      Timed t(KATA_K_SCAN, st);
      e = kata::launch_decay_scan(a, st);
      if (e != hipSuccess) return launch_status(e, what);
    }
  }
  Timed t(a.n_roles > 1 ? KATA_K_BWD : KATA_K_CHUNK_OUTPUT, st);
  return launch_status(kata::launch_decay_chunks(a, bf16, exact_state, false, st), what);
}

}  // namespace

extern "C" {

size_t kata_fwd_decay_workspace_size(const kata_decay_problem* pr) {
  if (kata::validate_decay(pr, false, nullptr) != KATA_OK) return 0;
  return kata::plan_decay(pr, 1).role_bytes;
}

kata_status kata_fwd_decay(const kata_decay_problem* pr, const void* q, const void* k,
                           const void* v, const float* log_decay, const int32_t* cu_seqlens,
                           const float* initial_state, void* o, float* final_state,
                           void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  if (!pr) return set_error(KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  const Named ts[] = {{q, pr->sq, "q"}, {k, pr->sk, "k"}, {v, pr->sv, "v"}, {o, pr->so, "o"}};
  kata_status s = check_decay(pr, Form::forward, ts, 4, log_decay, cu_seqlens);
  if (s != KATA_OK) return s;
  if ((s = need_aligned(initial_state, 16, "initial_state")) != KATA_OK) return s;
  if ((s = need_aligned(final_state, 16, "final_state")) != KATA_OK) return s;
  const kata::DecayPlan p = kata::plan_decay(pr, 1);
  if ((s = check_workspace(workspace, ws_bytes, p.role_bytes)) != KATA_OK) return s;
  if ((s = check_grid(p)) != KATA_OK) return s;
  if (final_state != initial_state && states_overlap(pr, final_state, initial_state))
    return set_error(KATA_ERR_INVALID_ARGUMENT, "final_state overlaps initial_state without being it");
  if ((s = check_device()) != KATA_OK) return s;
  kata::DecayArgs a = decay_args(pr, p, log_decay, cu_seqlens, 1);
  kata::DecayRole& r = a.role[0];
  r.a = q; r.b = k; r.c = v; r.out = o;
  copy3(r.sa, pr->sq); copy3(r.sb, pr->sk); copy3(r.sc, pr->sv); copy3(r.so, pr->so);
  r.init = initial_state;
  r.fin = final_state;
  // one array: the walk's workgroups would read a sequence's initial state at different times, the scan
  // reads it once
  if (initial_state && initial_state == final_state) a.join = 0;
  r.states = static_cast<float*>(workspace);
  r.dk = pr->dk; r.dv = pr->dv;
  r.out_scale = pr->scale; r.kv_scale = 1.f;
  return run_decay(a, p, pr->dtype == KATA_BF16, final_state != nullptr,
                   reinterpret_cast<hipStream_t>(stream), "decayed attention");
}

size_t kata_bwd_decay_workspace_size(const kata_decay_problem* pr) {
  if (kata::validate_decay(pr, true, nullptr) != KATA_OK) return 0;
  return 3 * kata::plan_decay(pr, 3).role_bytes;
}

kata_status kata_bwd_decay(const kata_decay_problem* pr, const void* q, const void* k,
                           const void* v, const void* dO, const float* log_decay,
                           const int32_t* cu_seqlens, const float* initial_state,
                           const float* dfinal_state, void* dq, void* dk, void* dv,
                           float* dinitial_state, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  if (!pr) return set_error(KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  const int64_t H = pr->H, T = pr->T;
  const int64_t gk[3] = {T * H * pr->dk, H * pr->dk, pr->dk}, gv[3] = {T * H * pr->dv, H * pr->dv, pr->dv};
  const Named ts[] = {{q, pr->sq, "q"},  {k, pr->sk, "k"}, {v, pr->sv, "v"}, {dO, pr->sdo, "dO"},
                      {dq, gk, "dq"},    {dk, gk, "dk"},   {dv, gv, "dv"}};
  kata_status s = check_decay(pr, Form::backward, ts, 7, log_decay, cu_seqlens);
  if (s != KATA_OK) return s;
  if ((s = need_aligned(initial_state, 16, "initial_state")) != KATA_OK) return s;
  if ((s = need_aligned(dfinal_state, 16, "dfinal_state")) != KATA_OK) return s;
  if ((s = need_aligned(dinitial_state, 16, "dinitial_state")) != KATA_OK) return s;
  const kata::DecayPlan p = kata::plan_decay(pr, 3);
  if ((s = check_workspace(workspace, ws_bytes, 3 * p.role_bytes)) != KATA_OK) return s;
  if ((s = check_grid(p)) != KATA_OK) return s;
  if (states_overlap(pr, dinitial_state, initial_state) || states_overlap(pr, dinitial_state, dfinal_state))
    return set_error(KATA_ERR_INVALID_ARGUMENT, "dinitial_state overlaps initial_state or dfinal_state");
  if ((s = check_device()) != KATA_OK) return s;
  kata::DecayArgs a = decay_args(pr, p, log_decay, cu_seqlens, 3);
  char* ws = static_cast<char*>(workspace);
  auto role = [&](int i, const void* ra, const int64_t* sa, const void* rb, const int64_t* sb,
                  const void* rc, const int64_t* sc, void* out, const int64_t* so, int wk, int wv) {
    kata::DecayRole& r = a.role[i];
    r.a = ra; r.b = rb; r.c = rc; r.out = out;
    copy3(r.sa, sa); copy3(r.sb, sb); copy3(r.sc, sc); copy3(r.so, so);
    r.dk = wk; r.dv = wv;
    r.states = reinterpret_cast<float*>(ws + i * p.role_bytes);
    r.out_scale = r.kv_scale = 1.f;
    return &r;
  };
  // dq_t = scale ( g^(t+1) S_0 dO_t + sum_{s<=t} g^(t-s) (dO_t . v_s) k_s )
  kata::DecayRole* r = role(0, dO, pr->sdo, v, pr->sv, k, pr->sk, dq, gk, pr->dv, pr->dk);
  r->out_scale = pr->scale;
  r->init = initial_state;
  r->init_trans = 1;
  // dk_s = g^(T-1-s) dS_T v_s + scale sum_{t>=s} g^(t-s) (v_s . dO_t) q_t
  r = role(1, v, pr->sv, dO, pr->sdo, q, pr->sq, dk, gk, pr->dv, pr->dk);
  r->rev = 1;
  r->kv_scale = pr->scale;
  r->init = dfinal_state;
  r->init_trans = 1;
  // dv_s = g^(T-1-s) dS_T^T k_s + scale sum_{t>=s} g^(t-s) (k_s . q_t) dO_t, and behind the first
  // token dS_0 = g^T dS_T + scale sum_t g^(t+1) q_t dO_t^T
  r = role(2, k, pr->sk, q, pr->sq, dO, pr->sdo, dv, gv, pr->dk, pr->dv);
  r->rev = 1;
  r->kv_scale = pr->scale;
  r->init = dfinal_state;
  r->fin = dinitial_state;
  return run_decay(a, p, pr->dtype == KATA_BF16, dinitial_state != nullptr,
                   reinterpret_cast<hipStream_t>(stream), "decayed attention backward");
}

kata_status kata_decode_decay(const kata_decay_problem* pr, const void* q, const void* k,
                              const void* v, const float* log_decay, float* state, void* o,
                              void* stream) {
  clear_error();
  if (!pr) return set_error(KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  const Named ts[] = {{q, pr->sq, "q"}, {k, pr->sk, "k"}, {v, pr->sv, "v"}, {o, pr->so, "o"}};
  kata_status s = check_decay(pr, Form::tokens, ts, 4, log_decay, nullptr);
  if (s != KATA_OK) return s;
  if (!state) return set_error(KATA_ERR_INVALID_ARGUMENT, "state is null");
  if ((s = need_aligned(state, 16, "state")) != KATA_OK) return s;
  if ((s = check_device()) != KATA_OK) return s;
  long long sq[3], sk[3], sv[3], so[3];
  copy3(sq, pr->sq); copy3(sk, pr->sk); copy3(sv, pr->sv); copy3(so, pr->so);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Timed t(KATA_K_DECODE, st);
  return launch_status(kata::launch_decay_decode(pr->dtype == KATA_BF16, pr->n_seq, pr->T, pr->H,
                                                 pr->dk, pr->dv, sq, sk, sv, so, q, k, v, log_decay,
                                                 pr->scale, state, o, st),
                       "decayed attention decode");
}

static kata_status run_rotary(const kata_rotary_problem* pr, const void* q, const void* k,
                              const double* rates, const void* positions, const int32_t* axes,
                              int32_t n_axes, int64_t pos_a, void* out_q, void* out_k, void* stream) {
  std::string why;
  kata_status s = kata::validate_rotary(pr, &why);
  if (s != KATA_OK) return set_error(s, why);
  if (!q || !out_q) return set_error(KATA_ERR_INVALID_ARGUMENT, "q or its output is null");
  if (pr->Hk && (!k || !out_k)) return set_error(KATA_ERR_INVALID_ARGUMENT, "k or its output is null");
  if (pr->rot && !rates) return set_error(KATA_ERR_INVALID_ARGUMENT, "rates is null");
  const size_t es = kata::elem_size(pr->dtype);
  const void* ptrs[4] = {q, out_q, k, out_k};
  const int64_t* sts[4] = {pr->sq, pr->soq, pr->sk, pr->sok};
  const char* names[4] = {"q", "out q", "k", "out k"};
  const int64_t sizes[4][3] = {{pr->B, pr->T, pr->H}, {pr->B, pr->T, pr->H},
                               {pr->B, pr->T, pr->Hk}, {pr->B, pr->T, pr->Hk}};
  bool aligned = true;
  for (int i = 0; i < (pr->Hk ? 4 : 2); ++i) {
    if ((s = need_aligned(ptrs[i], es, names[i])) != KATA_OK) return s;
    aligned &= reinterpret_cast<uintptr_t>(ptrs[i]) % 16 == 0;
    for (int j = 0; j < 3; ++j) aligned &= sizes[i][j] == 1 || sts[i][j] * (int64_t)es % 16 == 0;
  }
  if ((s = need_aligned(rates, 8, "rates")) != KATA_OK) return s;
  if ((s = need_aligned(positions, pr->pos64 ? 8 : 4, "positions")) != KATA_OK) return s;
  if ((s = check_device()) != KATA_OK) return s;
  kata::RotaryArgs a{};
  a.q = q; a.k = k; a.oq = out_q; a.ok = out_k;
  a.rates = rates;
  a.positions = positions;
  a.axes = axes; a.n_axes = n_axes; a.pos_a = pos_a;
  a.pos_b = pr->pos_b; a.pos_t = pr->pos_t; a.offset = pr->offset;
  copy3(a.sq, pr->sq); copy3(a.sk, pr->sk); copy3(a.soq, pr->soq); copy3(a.sok, pr->sok);
  a.B = pr->B; a.T = pr->T; a.H = pr->H; a.Hk = pr->Hk; a.D = pr->D; a.rot = pr->rot;
  a.pos64 = pr->pos64; a.inverse = pr->inverse;
  a.magnitude = pr->magnitude;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Timed t(KATA_K_ROTARY, st);
  return launch_status(kata::launch_rotary(a, pr->dtype == KATA_BF16, aligned, pr->interleaved != 0, st),
                       "rotary positions");
}

kata_status kata_rotary(const kata_rotary_problem* pr, const void* q, const void* k,
                        const double* rates, const void* positions, void* out_q, void* out_k,
                        void* stream) {
  clear_error();
  return run_rotary(pr, q, k, rates, positions, nullptr, 1, 0, out_q, out_k, stream);
}

// Positions of several axes.
static kata_status check_axes(const void* positions, const int32_t* axes, int32_t n_axes, int64_t pos_a) {
  if (!positions || !axes) return set_error(KATA_ERR_INVALID_ARGUMENT, "positions or axes is null");
  if (n_axes < 1 || pos_a < 0)
    return set_error(KATA_ERR_INVALID_ARGUMENT, "n_axes must be >= 1, the axes' stride not negative");
  return need_aligned(axes, 4, "axes");
}

kata_status kata_rotary_axes(const kata_rotary_problem* pr, const void* q, const void* k,
                             const double* rates, const void* positions, const int32_t* axes,
                             int32_t n_axes, int64_t pos_a, void* out_q, void* out_k, void* stream) {
  clear_error();
  const kata_status s = check_axes(positions, axes, n_axes, pos_a);
  return s != KATA_OK ? s : run_rotary(pr, q, k, rates, positions, axes, n_axes, pos_a, out_q, out_k, stream);
}

// dq, dk: null in the forward pass.
static kata_status run_qk_norm(const kata_qk_norm_problem* pr, const void* dq, const void* dk, const void* q,
                               const void* k, const void* q_weight, const void* k_weight, const double* rates,
                               const void* positions, const int32_t* axes, void* out_q, void* out_k,
                               void* dq_weight, void* dk_weight, float* part, hipStream_t st, const char* what) {
  const bool backward = dq != nullptr;
  if (!q || !out_q) return set_error(KATA_ERR_INVALID_ARGUMENT, "q or its output is null");
  if (pr->Hk && (!k || !out_k || (backward && !dk)))
    return set_error(KATA_ERR_INVALID_ARGUMENT, "k, its output or its gradient is null");
  kata_status s;
  if (pr->rot) {
    if (!rates) return set_error(KATA_ERR_INVALID_ARGUMENT, "rates is null");
    if (axes && (s = check_axes(positions, axes, pr->n_axes, pr->pos_a)) != KATA_OK) return s;
    if ((s = need_aligned(rates, 8, "rates")) != KATA_OK) return s;
    if ((s = need_aligned(positions, pr->pos64 ? 8 : 4, "positions")) != KATA_OK) return s;
  }
  const size_t es = kata::elem_size(pr->dtype), ew = kata::elem_size(pr->w_dtype);
  const void* ptrs[6] = {q, out_q, dq, k, out_k, dk};
  const int64_t* sts[6] = {pr->sq, pr->soq, pr->sdq, pr->sk, pr->sok, pr->sdk};
  const char* names[6] = {"q", "out q", "dq", "k", "out k", "dk"};
  bool aligned = true;
  for (int i = 0; i < (pr->Hk ? 6 : 3); ++i) {
    if (!ptrs[i]) continue;                         // gradients of a forward pass
    if ((s = need_aligned(ptrs[i], es, names[i])) != KATA_OK) return s;
    aligned &= reinterpret_cast<uintptr_t>(ptrs[i]) % 16 == 0;
    const int64_t sizes[3] = {pr->B, pr->T, i < 3 ? pr->H : pr->Hk};
    for (int j = 0; j < 3; ++j) aligned &= sizes[j] == 1 || sts[i][j] * (int64_t)es % 16 == 0;
  }
  const void* weights[4] = {q_weight, k_weight, dq_weight, dk_weight};
  for (const void* w : weights)
    if ((s = need_aligned(w, ew, "a weight or its gradient")) != KATA_OK) return s;
  if ((s = check_device()) != KATA_OK) return s;
  kata::QkNormArgs a{};
  a.q = q; a.k = k; a.dq = dq; a.dk = dk; a.wq = q_weight; a.wk = k_weight;
  a.oq = out_q; a.ok = out_k; a.dwq = dq_weight; a.dwk = dk_weight;
  a.part = part;
  a.rates = rates; a.positions = positions; a.axes = axes;
  a.pos_a = pr->pos_a; a.pos_b = pr->pos_b; a.pos_t = pr->pos_t; a.offset = pr->offset;
  copy3(a.sq, pr->sq); copy3(a.sk, pr->sk); copy3(a.soq, pr->soq); copy3(a.sok, pr->sok);
  copy3(a.sdq, pr->sdq); copy3(a.sdk, pr->sdk);
  a.B = pr->B; a.T = pr->T; a.H = pr->H; a.Hk = pr->Hk; a.D = pr->D; a.rot = pr->rot;
  a.pos64 = pr->pos64; a.inverse = backward; a.n_axes = pr->n_axes; a.w_bf16 = pr->w_dtype == KATA_BF16;
  a.magnitude = pr->magnitude; a.eps = pr->eps; a.count = pr->l2 ? 1.f : (float)pr->D;
  Timed t(KATA_K_NORM, st);
  return launch_status(kata::launch_qk_norm(a, pr->dtype == KATA_BF16, aligned, pr->interleaved != 0, backward, st), what);
}

kata_status kata_fwd_qk_norm(const kata_qk_norm_problem* pr, const void* q, const void* k,
                             const void* q_weight, const void* k_weight, const double* rates,
                             const void* positions, const int32_t* axes, void* out_q, void* out_k,
                             void* stream) {
  clear_error();
  std::string why;
  const kata_status s = kata::validate_qk_norm(pr, false, &why);
  if (s != KATA_OK) return set_error(s, why);
  return run_qk_norm(pr, nullptr, nullptr, q, k, q_weight, k_weight, rates, positions, axes, out_q, out_k, nullptr,
                     nullptr, nullptr, reinterpret_cast<hipStream_t>(stream), "norm of queries and keys");
}

size_t kata_bwd_qk_norm_workspace_size(const kata_qk_norm_problem* pr) {
  return kata::validate_qk_norm(pr, true, nullptr) == KATA_OK ? size_t(kata::kQkNormBlocks) * 2 * pr->D * 4 : 0;
}

kata_status kata_bwd_qk_norm(const kata_qk_norm_problem* pr, const void* dq, const void* dk, const void* q,
                             const void* k, const void* q_weight, const void* k_weight,
                             const double* rates, const void* positions, const int32_t* axes, void* dq_in,
                             void* dk_in, void* dq_weight, void* dk_weight, void* workspace,
                             size_t ws_bytes, void* stream) {
  clear_error();
  std::string why;
  kata_status s = kata::validate_qk_norm(pr, true, &why);
  if (s != KATA_OK) return set_error(s, why);
  if (!dq) return set_error(KATA_ERR_INVALID_ARGUMENT, "dq is null");
  const bool sums = dq_weight || dk_weight;
  if (sums && (s = check_workspace(workspace, ws_bytes, kata_bwd_qk_norm_workspace_size(pr))) != KATA_OK) return s;
  return run_qk_norm(pr, dq, dk, q, k, q_weight, k_weight, rates, positions, axes, dq_in, dk_in, dq_weight, dk_weight,
                     sums ? static_cast<float*>(workspace) : nullptr, reinterpret_cast<hipStream_t>(stream),
                     "norm of queries and keys backward");
}

static kata_status check_norm(const kata_norm_problem* pr, bool backward) {
  std::string why;
  kata_status s = kata::validate_norm(pr, backward, &why);
  return s == KATA_OK ? s : set_error(s, why);
}

kata_status kata_fwd_layer_norm(const kata_norm_problem* pr, const void* x, const void* weight,
                                const void* bias, void* y, float* mean, float* rstd, void* stream) {
  clear_error();
  kata_status s = check_norm(pr, false);
  if (s != KATA_OK) return s;
  if (!x || !y) return set_error(KATA_ERR_INVALID_ARGUMENT, "x or y is null");
  if (!mean != !rstd) return set_error(KATA_ERR_INVALID_ARGUMENT, "mean and rstd go together");
  const size_t es = kata::elem_size(pr->dtype), ew = kata::elem_size(pr->w_dtype);
  if ((s = need_aligned(x, es, "x")) != KATA_OK || (s = need_aligned(y, es, "y")) != KATA_OK ||
      (s = need_aligned(weight, ew, "weight")) != KATA_OK ||
      (s = need_aligned(bias, ew, "bias")) != KATA_OK ||
      (s = need_aligned(mean, 4, "mean")) != KATA_OK || (s = need_aligned(rstd, 4, "rstd")) != KATA_OK)
    return s;
  if ((s = check_device()) != KATA_OK) return s;
  kata::NormArgs a{};
  a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
  a.rows = pr->rows; a.sx = pr->sx; a.sy = pr->sy;
  a.N = pr->N; a.w_bf16 = pr->w_dtype == KATA_BF16; a.eps = pr->eps;
  const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % 16) == 0 &&
                       (pr->rows == 1 || ((pr->sx | pr->sy) * (int64_t)es) % 16 == 0);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Timed t(KATA_K_NORM, st);
  return launch_status(kata::launch_norm_fwd(a, pr->dtype == KATA_BF16, aligned, st), "layer norm");
}

size_t kata_bwd_layer_norm_workspace_size(const kata_norm_problem* pr) {
  return kata::validate_norm(pr, true, nullptr) == KATA_OK ? kata::norm_workspace_bytes(pr) : 0;
}

kata_status kata_bwd_layer_norm(const kata_norm_problem* pr, const void* dy, const void* x,
                                const void* weight, const float* mean, const float* rstd, void* dx,
                                void* dweight, void* dbias, void* workspace, size_t ws_bytes,
                                void* stream) {
  clear_error();
  kata_status s = check_norm(pr, true);
  if (s != KATA_OK) return s;
  if (!dy || !x || !mean || !rstd)
    return set_error(KATA_ERR_INVALID_ARGUMENT, "dy, x, mean or rstd is null");
  if (!dx && !dweight && !dbias) return set_error(KATA_ERR_INVALID_ARGUMENT, "no gradient is asked for");
  const size_t es = kata::elem_size(pr->dtype), ew = kata::elem_size(pr->w_dtype);
  if ((s = need_aligned(x, es, "x")) != KATA_OK || (s = need_aligned(dy, es, "dy")) != KATA_OK ||
      (s = need_aligned(dx, es, "dx")) != KATA_OK ||
      (s = need_aligned(weight, ew, "weight")) != KATA_OK ||
      (s = need_aligned(dweight, ew, "dweight")) != KATA_OK ||
      (s = need_aligned(dbias, ew, "dbias")) != KATA_OK ||
      (s = need_aligned(mean, 4, "mean")) != KATA_OK || (s = need_aligned(rstd, 4, "rstd")) != KATA_OK)
    return s;
  const bool sums = dweight || dbias;
  if (sums && (s = check_workspace(workspace, ws_bytes, kata::norm_workspace_bytes(pr))) != KATA_OK)
    return s;
  if ((s = check_device()) != KATA_OK) return s;
  kata::NormArgs a{};
  a.x = x; a.dy = dy; a.w = weight; a.dx = dx; a.dw = dweight; a.db = dbias;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.rows = pr->rows; a.sx = pr->sx; a.sdy = pr->sdy; a.sdx = pr->sdx;
  a.N = pr->N; a.w_bf16 = pr->w_dtype == KATA_BF16; a.eps = pr->eps;
  const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy) |
                         reinterpret_cast<uintptr_t>(dx)) % 16) == 0 &&
                       (pr->rows == 1 || ((pr->sx | pr->sdy | pr->sdx) * (int64_t)es) % 16 == 0);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Timed t(KATA_K_NORM, st);
  return launch_status(kata::launch_norm_bwd(a, pr->dtype == KATA_BF16, aligned, st), "layer norm backward");
}

}  // extern "C"
