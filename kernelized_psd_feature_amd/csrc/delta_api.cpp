// The C ABI's entry points of the gated delta rule (include/kata.h).  As in kata_api.cpp, every call validates
// its arguments on the host, checks the device, enqueues its kernels on the caller's stream and returns.
#include <hip/hip_runtime.h>

#include <string>

#include "api.h"
#include "delta.h"
#include "delta_plan.h"
#include "kata.h"
#include "layer_plan.h"
#include "plan.h"

using kata::check_device;
using kata::clear_error;
using kata::launch_status;
using kata::set_error;
using kata::Timed;

namespace {

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
  int heads;
};

enum class Form { forward, backward, tokens };
kata_status check_delta(const kata_delta_problem* pr, Form form, const Named* ts, int n, const void* beta,
                        const float* log_decay, const int32_t* cu) {
  std::string why;
  kata_status s = form == Form::tokens ? kata::validate_delta_decode(pr, &why)
                                       : kata::validate_delta(pr, form == Form::backward, &why);
  if (s != KATA_OK) return set_error(s, why);
  const size_t es = kata::elem_size(pr->dtype);
  for (int i = 0; i < n; ++i) {
    const int64_t sizes[3] = {pr->packed ? 1 : pr->n_seq, pr->T, ts[i].heads ? pr->Hk : pr->H};
    if ((s = kata::validate_rows(ts[i].p, ts[i].st, sizes, es, ts[i].name, &why)) != KATA_OK)
      return set_error(s, why);
  }
  if (!beta) return set_error(KATA_ERR_INVALID_ARGUMENT, "beta is null");
  if (pr->packed && !cu) return set_error(KATA_ERR_INVALID_ARGUMENT, "cu_seqlens is null");
  if ((s = need_aligned(beta, es, "beta")) != KATA_OK) return s;
  if ((s = need_aligned(log_decay, 4, "log_decay")) != KATA_OK) return s;
  return need_aligned(cu, 4, "cu_seqlens");
}

kata_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return set_error(KATA_ERR_WORKSPACE, "workspace needs " + std::to_string(need) +
                                             " bytes, got " + std::to_string(have));
  return need ? need_aligned(ws, 256, "workspace") : KATA_OK;
}

// The kernels number their workgroups in 32 bits (grid_rows in device.h takes fewer than 2^31).
kata_status check_grid(const kata::DeltaPlan& p) {
  if (p.groups >= int64_t(1) << 31)
    return set_error(KATA_ERR_UNSUPPORTED, "too many sequences and heads for one launch");
  return KATA_OK;
}

// Whether states are written where others are read.
bool states_overlap(const kata_delta_problem* pr, const float* written, const float* read) {
  const uintptr_t w = uintptr_t(written), r = uintptr_t(read);
  const uintptr_t n = uintptr_t(pr->n_seq) * pr->H * pr->dk * pr->dv * 4;
  return w && r && w < r + n && r < w + n;
}

kata::DeltaArgs delta_args(const kata_delta_problem* pr, const void* q, const void* k, const void* v,
                           const void* beta, const float* log_decay, const int32_t* cu) {
  kata::DeltaArgs a{};
  a.m.cu = cu;
  a.m.packed = pr->packed; a.m.n_seq = pr->n_seq; a.m.T = pr->T;
  a.m.H = pr->H; a.m.Hk = pr->Hk; a.m.dk = pr->dk; a.m.dv = pr->dv;
  a.q = q; a.k = k; a.v = v; a.beta = beta; a.log_decay = log_decay;
  copy3(a.sq, pr->sq); copy3(a.sk, pr->sk); copy3(a.sv, pr->sv); copy3(a.so, pr->so);
  copy3(a.sdo, pr->sdo); copy3(a.sb, pr->sbeta); copy3(a.sl, pr->sdecay);
  a.scale = pr->scale;
  a.zero_tail = pr->zero_tail;
  return a;
}

void place(kata::DeltaArgs& a, const kata::DeltaPlan& p, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  a.m.L = p.L; a.m.n_seg = p.n_seg; a.m.n_chunks = p.n_chunks;
  a.m.n_slots = p.n_slots; a.m.c_slots = p.c_slots;
  a.vec = reinterpret_cast<float*>(ws + p.vec);
  a.inv = reinterpret_cast<float*>(ws + p.inv);
  a.sums = reinterpret_cast<float*>(ws + p.sums);
  a.trans = reinterpret_cast<float*>(ws + p.trans);
  a.rsums = reinterpret_cast<float*>(ws + p.rsums);
  a.cstates = reinterpret_cast<float*>(ws + p.cstates);
  a.rstates = reinterpret_cast<float*>(ws + p.rstates);
  a.u = reinterpret_cast<float*>(ws + p.u);
  a.x = reinterpret_cast<float*>(ws + p.x);
  a.fstates = reinterpret_cast<float*>(ws + p.fstates);
}

// Inverses, and the segments' entry states.
kata_status run_before(const kata::DeltaArgs& a, bool bf16, bool backward, hipStream_t st, const char* what) {
  {
    Timed t(KATA_K_CHUNK_STATE, st);
    hipError_t e = kata::launch_delta_prep(a, bf16, st);
    if (e == hipSuccess && a.m.n_seg > 1)
      e = backward ? kata::launch_delta_bwd_walk(a, bf16, true, st) : kata::launch_delta_segments(a, bf16, st);
    if (e != hipSuccess) return launch_status(e, what);
  }
  if (a.m.n_seg < 2) return KATA_OK;
  Timed t(KATA_K_SCAN, st);
  return launch_status(kata::launch_delta_join(a, backward, st), what);
}

}  // namespace

extern "C" {

size_t kata_fwd_delta_workspace_size(const kata_delta_problem* pr) {
  if (kata::validate_delta(pr, false, nullptr) != KATA_OK) return 0;
  return kata::plan_delta(pr, false).bytes;
}

kata_status kata_fwd_delta(const kata_delta_problem* pr, const void* q, const void* k, const void* v,
                           const void* beta, const float* log_decay, const int32_t* cu_seqlens,
                           const float* initial_state, void* o, float* final_state, void* workspace,
                           size_t ws_bytes, void* stream) {
  clear_error();
  if (!pr) return set_error(KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  const Named ts[] = {{q, pr->sq, "q", 1}, {k, pr->sk, "k", 1}, {v, pr->sv, "v", 0}, {o, pr->so, "o", 0}};
  kata_status s = check_delta(pr, Form::forward, ts, 4, beta, log_decay, cu_seqlens);
  if (s != KATA_OK) return s;
  if ((s = need_aligned(initial_state, 16, "initial_state")) != KATA_OK) return s;
  if ((s = need_aligned(final_state, 16, "final_state")) != KATA_OK) return s;
  const kata::DeltaPlan p = kata::plan_delta(pr, false);
  if ((s = check_grid(p)) != KATA_OK) return s;
  if ((s = check_workspace(workspace, ws_bytes, p.bytes)) != KATA_OK) return s;
  if (states_overlap(pr, final_state, initial_state))
    return set_error(KATA_ERR_INVALID_ARGUMENT, "final_state overlaps initial_state");
  if ((s = check_device()) != KATA_OK) return s;
  kata::DeltaArgs a = delta_args(pr, q, k, v, beta, log_decay, cu_seqlens);
  place(a, p, workspace);
  a.o = o;
  a.init = initial_state;
  a.fin = final_state;
  const bool bf16 = pr->dtype == KATA_BF16;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if ((s = run_before(a, bf16, false, st, "gated delta rule")) != KATA_OK) return s;
  Timed t(KATA_K_CHUNK_OUTPUT, st);
  return launch_status(kata::launch_delta_walk(a, bf16, st), "gated delta rule");
}

size_t kata_bwd_delta_workspace_size(const kata_delta_problem* pr) {
  if (kata::validate_delta(pr, true, nullptr) != KATA_OK) return 0;
  return kata::plan_delta(pr, true).bytes;
}

kata_status kata_bwd_delta(const kata_delta_problem* pr, const void* q, const void* k, const void* v,
                           const void* beta, const float* log_decay, const void* dO, const int32_t* cu_seqlens,
                           const float* initial_state, const float* dfinal_state, void* dq, void* dk, void* dv,
                           void* dbeta, float* dlog_decay, float* dinitial_state, void* workspace,
                           size_t ws_bytes, void* stream) {
  clear_error();
  if (!pr) return set_error(KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  const int64_t T = pr->T, H = pr->H, Hk = pr->Hk;
  const int64_t gk[3] = {T * Hk * pr->dk, Hk * pr->dk, pr->dk}, gv[3] = {T * H * pr->dv, H * pr->dv, pr->dv};
  const Named ts[] = {{q, pr->sq, "q", 1}, {k, pr->sk, "k", 1}, {v, pr->sv, "v", 0}, {dO, pr->sdo, "dO", 0},
                      {dq, gk, "dq", 1},   {dk, gk, "dk", 1},   {dv, gv, "dv", 0}};
  kata_status s = check_delta(pr, Form::backward, ts, 7, beta, log_decay, cu_seqlens);
  if (s != KATA_OK) return s;
  if (!dbeta) return set_error(KATA_ERR_INVALID_ARGUMENT, "dbeta is null");
  if ((s = need_aligned(dbeta, kata::elem_size(pr->dtype), "dbeta")) != KATA_OK) return s;
  if ((s = need_aligned(dlog_decay, 4, "dlog_decay")) != KATA_OK) return s;
  if ((s = need_aligned(initial_state, 16, "initial_state")) != KATA_OK) return s;
  if ((s = need_aligned(dfinal_state, 16, "dfinal_state")) != KATA_OK) return s;
  if ((s = need_aligned(dinitial_state, 16, "dinitial_state")) != KATA_OK) return s;
  const kata::DeltaPlan p = kata::plan_delta(pr, true);
  if ((s = check_grid(p)) != KATA_OK) return s;
  if ((s = check_workspace(workspace, ws_bytes, p.bytes)) != KATA_OK) return s;
  if (states_overlap(pr, dinitial_state, initial_state) || states_overlap(pr, dinitial_state, dfinal_state))
    return set_error(KATA_ERR_INVALID_ARGUMENT, "dinitial_state overlaps initial_state or dfinal_state");
  if ((s = check_device()) != KATA_OK) return s;
  kata::DeltaArgs a = delta_args(pr, q, k, v, beta, log_decay, cu_seqlens);
  place(a, p, workspace);
  a.dO = dO;
  a.init = initial_state;
  a.dfin = dfinal_state;
  a.dinit = dinitial_state;
  if (!dfinal_state || pr->dtype != KATA_BF16) a.fstates = nullptr;     // (fp32: the gradients do not read them)
  if (p.by_heads) {
    a.pq = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.pq);
    a.pk = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.pk);
  }
  a.dq = dq; a.dk = dk; a.dv = dv; a.dbeta = dbeta; a.dlog = dlog_decay;
  const bool bf16 = pr->dtype == KATA_BF16;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const char* what = "gated delta rule backward";
  if ((s = run_before(a, bf16, true, st, what)) != KATA_OK) return s;
  Timed t(KATA_K_BWD, st);
  hipError_t e = kata::launch_delta_bwd_walk(a, bf16, false, st);
  if (e == hipSuccess) e = kata::launch_delta_grads(a, bf16, st);
  return launch_status(e, what);
}

kata_status kata_decode_delta(const kata_delta_problem* pr, const void* q, const void* k, const void* v,
                              const void* beta, const float* log_decay, float* state, void* o, void* stream) {
  clear_error();
  if (!pr) return set_error(KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  const Named ts[] = {{q, pr->sq, "q", 1}, {k, pr->sk, "k", 1}, {v, pr->sv, "v", 0}, {o, pr->so, "o", 0}};
  kata_status s = check_delta(pr, Form::tokens, ts, 4, beta, log_decay, nullptr);
  if (s != KATA_OK) return s;
  if (!state) return set_error(KATA_ERR_INVALID_ARGUMENT, "state is null");
  if ((s = need_aligned(state, 16, "state")) != KATA_OK) return s;
  if ((s = check_device()) != KATA_OK) return s;
  kata::DeltaArgs a = delta_args(pr, q, k, v, beta, log_decay, nullptr);
  a.o = o;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Timed t(KATA_K_DECODE, st);
  return launch_status(kata::launch_delta_decode(a, pr->dtype == KATA_BF16, state, st), "gated delta rule decode");
}

}  // extern "C"
