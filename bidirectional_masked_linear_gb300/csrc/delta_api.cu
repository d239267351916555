// delta_api.cu -- the C ABI of the delta rule's operators declared in
// include/lion.h: argument checks, workspaces and the launches.
#include <initializer_list>

#include "api_check.h"
#include "lion_internal.h"

namespace {

using namespace lion::api;

constexpr long long kMaxWidth = LION_SSM_MAX_EXTENT;   // of a token's heads

// Whether a result's memory begins where none of these do: what other CTAs still read, or write as well.
bool apart(const void* out, std::initializer_list<const void*> others) {
  for (const void* x : others)
    if (out == x) return false;
  return true;
}

// d, rot, Hq and Hk as lion_qknorm_args has them.
lion_status qknorm_sizes(int B, int L, int Hq, int Hk, int d, int rot, int norm, int interleaved, float eps,
                         int dtype) {
  if (B < 1 || L < 1 || Hq < 1 || Hk < 1 || d < 1 || rot < 0 || rot > d || !flag(interleaved) || !(eps >= 0.f) ||
      (norm != LION_QKNORM_L2 && norm != LION_QKNORM_RMS) || !dtype_ok(dtype))
    return LION_ERR_INVALID_ARG;
  if (d % 8 || d > LION_QKNORM_MAX_D || rot % 8 || (long long)Hq + Hk > kMaxWidth / d || L > LION_SSM_MAX_EXTENT)
    return LION_ERR_UNSUPPORTED;
  return LION_OK;
}

template <typename Args>
lion_status qknorm_check(const Args& a) {
  const lion_status st =
      qknorm_sizes(a.B, a.L, a.Hq, a.Hk, a.d, a.rot, a.norm, a.interleaved, a.eps, a.dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a.dtype);
  if (!stride_ok(a.q_token, (long long)a.Hq * a.d) || !stride_ok(a.k_token, (long long)a.Hk * a.d) ||
      !ptr.need(a.q, es) || !ptr.need(a.k, es) || !ptr.maybe(a.q_weight, 4) || !ptr.maybe(a.k_weight, 4) ||
      !ptr.maybe(a.freqs, 4) || (a.rot > 0) != (a.freqs != nullptr) || !ptr.maybe(a.positions, 4))
    return LION_ERR_INVALID_ARG;
  return st;
}

lion_status delta_sizes(int B, int L, int Hk, int Hv, int dk, int dv, float scale, int dtype) {
  if (B < 1 || L < 1 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || dk < 1 || dv < 1 || !(scale - scale == 0.f) ||
      !dtype_ok(dtype))
    return LION_ERR_INVALID_ARG;
  if (dk % 8 || dv % 8 || dk > LION_DELTA_MAX_D || dv > LION_DELTA_MAX_D) return LION_ERR_UNSUPPORTED;
  if (L > LION_SSM_MAX_EXTENT || Hk > kMaxWidth / dk || Hv > kMaxWidth / dv) return LION_ERR_UNSUPPORTED;
  // a warp for 32 tokens of a head, and CTAs for 32 columns of one, on one grid axis
  if ((long long)B * Hv > kMaxGrid / 4 / ((long long)L / 32 + 1)) return LION_ERR_UNSUPPORTED;
  return LION_OK;
}

template <typename Args>
lion_status delta_check(const Args& a) {
  lion_status st = delta_sizes(a.B, a.L, a.Hk, a.Hv, a.dk, a.dv, a.scale, a.dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a.dtype);
  const long long qk = (long long)a.Hk * a.dk;
  if (!flag(a.reverse) || !stride_ok(a.q_token, qk) || !stride_ok(a.k_token, qk) ||
      !stride_ok(a.v_token, (long long)a.Hv * a.dv) || !stride_ok(a.g_token, a.Hv) || !stride_ok(a.beta_token, a.Hv) ||
      !ptr.need(a.q, es) || !ptr.need(a.k, es) || !ptr.need(a.v, es) || !ptr.need(a.g, es) || !ptr.need(a.beta, es) ||
      !ptr.maybe(a.h0, 16) || !ptr.maybe(a.lengths, 4) || !ptr.maybe(a.saved, 256))
    return LION_ERR_INVALID_ARG;
  return st;
}

}  // namespace

extern "C" {

lion_status lion_qknorm_fwd(const lion_qknorm_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = qknorm_check(*a);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->q_out, es) || !ptr.need(a->k_out, es) || !apart(a->q_out, {a->q, a->k, a->k_out}) ||
      !apart(a->k_out, {a->q, a->k}))   // heads of a token that are still to be read
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return from_cuda(lion::launch_qknorm_fwd(*a, a->stream));
}

size_t lion_qknorm_bwd_workspace_bytes(int B, int L, int Hq, int Hk, int d, int weights) {
  if (!weights || qknorm_sizes(B, L, Hq, Hk, d, 0, 0, 0, 0.f, 0) != LION_OK) return 0;
  return lion::qknorm_bwd_workspace_bytes(B, L, Hq, Hk, d);
}

lion_status lion_qknorm_bwd(const lion_qknorm_bwd_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = qknorm_check(*a);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->dq_out, es) || !ptr.need(a->dk_out, es) || !ptr.need(a->dq, es) || !ptr.need(a->dk, es) ||
      !apart(a->dq, {a->q, a->k, a->dq_out, a->dk_out, a->dk}) || !apart(a->dk, {a->q, a->k, a->dq_out, a->dk_out}) ||
      !ptr.maybe(a->dq_weight, 4) || !ptr.maybe(a->dk_weight, 4) || (a->dq_weight && !a->q_weight) ||
      (a->dk_weight && !a->k_weight))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  const bool weights = a->dq_weight || a->dk_weight;
  return with_workspace(a->workspace, a->workspace_bytes,
                        weights ? lion::qknorm_bwd_workspace_bytes(a->B, a->L, a->Hq, a->Hk, a->d) : 0, a->stream,
                        [&](void* ws) { return lion::launch_qknorm_bwd(*a, ws, a->stream); });
}

size_t lion_delta_saved_bytes(int B, int L, int Hk, int Hv, int dk, int dv, int dtype) {
  if (delta_sizes(B, L, Hk, Hv, dk, dv, 1.f, dtype) != LION_OK) return 0;
  return lion::delta_saved_bytes(B, L, Hv, dk, dv, dtype);
}

size_t lion_delta_workspace_bytes(int B, int L, int Hk, int Hv, int dk, int dv, int dtype, int save) {
  if (delta_sizes(B, L, Hk, Hv, dk, dv, 1.f, dtype) != LION_OK) return 0;
  return lion::delta_workspace_bytes(B, L, Hv, dk, dv, dtype, save != 0);
}

lion_status lion_delta_fwd(const lion_delta_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = delta_check(*a);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  if (!ptr.need(a->out, esize(a->dtype)) || !ptr.maybe(a->h_out, 16) || (a->h0 && a->h_out == a->h0) ||
      !apart(a->out, {a->q, a->k, a->v}))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return with_workspace(a->workspace, a->workspace_bytes,
                        lion::delta_workspace_bytes(a->B, a->L, a->Hv, a->dk, a->dv, a->dtype, a->saved != nullptr),
                        a->stream, [&](void* ws) { return lion::launch_delta_fwd(*a, ws, a->stream); });
}

size_t lion_delta_bwd_workspace_bytes(int B, int L, int Hk, int Hv, int dk, int dv, int dtype, int have_saved) {
  if (delta_sizes(B, L, Hk, Hv, dk, dv, 1.f, dtype) != LION_OK) return 0;
  return lion::delta_bwd_workspace_bytes(B, L, Hk, Hv, dk, dv, dtype, have_saved != 0);
}

lion_status lion_delta_bwd(const lion_delta_bwd_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = delta_check(*a);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->dout, es) || !ptr.need(a->dq, es) || !ptr.need(a->dk_out, es) || !ptr.need(a->dv_out, es) ||
      !ptr.need(a->dg, es) || !ptr.need(a->dbeta, es) || !ptr.maybe(a->dh0, 16) ||
      !apart(a->dv_out, {a->dout, a->q, a->k, a->dq, a->dk_out}) ||   // dR, read with these by the last launch but one
      !apart(a->dq, {a->dout, a->q, a->k, a->dk_out}) || !apart(a->dk_out, {a->dout, a->q, a->k}) ||
      !apart(a->dg, {a->g, a->beta, a->dbeta}) || !apart(a->dbeta, {a->g, a->beta}))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return with_workspace(
      a->workspace, a->workspace_bytes,
      lion::delta_bwd_workspace_bytes(a->B, a->L, a->Hk, a->Hv, a->dk, a->dv, a->dtype, a->saved != nullptr), a->stream,
      [&](void* ws) { return lion::launch_delta_bwd(*a, ws, a->stream); });
}

lion_status lion_delta_step(const lion_delta_step_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = delta_sizes(a->B, 1, a->Hk, a->Hv, a->dk, a->dv, a->scale, a->dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->h, 16) || !ptr.need(a->q, es) || !ptr.need(a->k, es) || !ptr.need(a->v, es) ||
      !ptr.need(a->g, es) || !ptr.need(a->beta, es) || !ptr.need(a->out, es) ||
      !apart(a->out, {a->q, a->k, a->g, a->beta}))   // a CTA writes 32 columns, each reads all of q and k
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return from_cuda(lion::launch_delta_step(*a, a->stream));
}

}  // extern "C"
