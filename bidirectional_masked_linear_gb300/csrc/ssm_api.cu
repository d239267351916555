// ssm_api.cu -- the C ABI of the state space block declared in include/lion.h:
// argument checks, workspaces and the launches.
#include <stdint.h>

#include "../../include/lion.h"
#include "lion_internal.h"
#include "ssm_check.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks of a call's pointers: aligned to `a` bytes and memory that the current device's kernels can use.
class Pointers {
 public:
  Pointers() {
    if (cudaGetDevice(&device_) != cudaSuccess) cudaGetLastError();   // no device: no pointer passes
  }
  bool need(const void* p, size_t a) const { return p && aligned(p, a) && usable(p); }
  bool maybe(const void* p, size_t a) const { return !p || need(p, a); }

 private:
  bool usable(const void* p) const {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    return lion::usable_on(at, device_);
  }
  int device_ = -1;
};
bool dtype_ok(int t) { return t == LION_DTYPE_BF16 || t == LION_DTYPE_FP32; }
size_t esize(int t) { return t == LION_DTYPE_BF16 ? 2 : 4; }
bool flag(int v) { return v == 0 || v == 1; }
bool stride_ok(long long ld, long long width) { return ld == 0 || ld >= width; }

constexpr long long kMaxGrid = 0x7fffffffLL;
// A token's or channel's index plus a tile's, run's, segment's or block's extent stays an int.
constexpr int kMaxExtent = LION_SSM_MAX_EXTENT;

lion_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return LION_OK;
  if (e == cudaErrorMemoryAllocation) return LION_ERR_NO_MEMORY;
  return LION_ERR_CUDA;
}

// Runs `go(workspace)` on the caller's workspace or on a stream-ordered one.
template <typename F>
lion_status with_workspace(void* ws, size_t ws_bytes, size_t want, cudaStream_t s, F go) {
  if (want == 0) return from_cuda(go(nullptr));
  if (ws) {
    if (!Pointers().need(ws, 256) || ws_bytes < want) return LION_ERR_INVALID_ARG;
    return from_cuda(go(ws));
  }
  cudaError_t e = cudaMallocAsync(&ws, want, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return from_cuda(e);
  }
  e = go(ws);
  const cudaError_t f = cudaFreeAsync(ws, s);
  return from_cuda(e != cudaSuccess ? e : f);
}

lion_status norm_sizes(int rows, int cols, long long x_row, int dtype) {
  if (rows < 1 || cols < 1 || !dtype_ok(dtype) || !stride_ok(x_row, cols)) return LION_ERR_INVALID_ARG;
  return cols > LION_LAYERNORM_MAX_COLS ? LION_ERR_UNSUPPORTED : LION_OK;
}

lion_status conv_sizes(int B, int L, int D, int K, int act, int reverse, int dtype, long long x_token) {
  if (B < 1 || L < 1 || D < 1 || K < 1 || !dtype_ok(dtype) || !flag(reverse) || !stride_ok(x_token, D) ||
      (act != LION_ACT_NONE && act != LION_ACT_SILU))
    return LION_ERR_INVALID_ARG;
  if (K < 2 || K > 4 || L > kMaxExtent || D > kMaxExtent) return LION_ERR_UNSUPPORTED;
  // a CTA for 128 vectors of four channels of a run of tokens, on one grid axis
  const long long runs = (long long)B * (L / 5 + 1);
  if (runs > kMaxGrid || runs > kMaxGrid / (((long long)D + 3) / 4) * 128) return LION_ERR_UNSUPPORTED;
  return LION_OK;
}

lion_status scan_sizes(int B, int L, int D, int N, int G, int softplus, int reverse, int dtype) {
  if (B < 1 || L < 1 || D < 1 || N < 1 || G < 1 || D % G != 0 || !flag(softplus) || !flag(reverse) || !dtype_ok(dtype))
    return LION_ERR_INVALID_ARG;
  if (N != 8 && N != 16 && N != 32 && N != 64) return LION_ERR_UNSUPPORTED;
  if (L > kMaxExtent || D > kMaxExtent || (long long)G * N > kMaxExtent) return LION_ERR_UNSUPPORTED;
  // CTAs on one grid axis, with as many segments as a sequence can have
  if ((long long)B * G > kMaxGrid / ((long long)D / G + 1) / ((long long)L / 64 + 1)) return LION_ERR_UNSUPPORTED;
  return LION_OK;
}

}  // namespace

extern "C" {

lion_status lion_layernorm_fwd(const lion_layernorm_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = norm_sizes(a->rows, a->cols, a->x_row, a->dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->x, es) || !ptr.need(a->weight, 4) || !ptr.maybe(a->bias, 4) || !ptr.need(a->y, es) ||
      !ptr.maybe(a->mean, 4) || !ptr.maybe(a->rstd, 4) || !a->mean != !a->rstd || !(a->eps >= 0.f))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return from_cuda(lion::launch_layernorm_fwd(*a, a->stream));
}

size_t lion_layernorm_bwd_workspace_bytes(int rows, int cols) {
  if (rows < 1 || cols < 1 || cols > LION_LAYERNORM_MAX_COLS) return 0;
  return lion::layernorm_bwd_workspace_bytes(rows, cols);
}

lion_status lion_layernorm_bwd(const lion_layernorm_bwd_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = norm_sizes(a->rows, a->cols, a->x_row, a->dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->dy, es) || !ptr.need(a->x, es) || !ptr.need(a->weight, 4) || !ptr.need(a->mean, 4) ||
      !ptr.need(a->rstd, 4) || !ptr.need(a->dx, es) || !ptr.need(a->dweight, 4) || !ptr.maybe(a->dbias, 4))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return with_workspace(a->workspace, a->workspace_bytes, lion::layernorm_bwd_workspace_bytes(a->rows, a->cols),
                        a->stream, [&](void* ws) { return lion::launch_layernorm_bwd(*a, ws, a->stream); });
}

lion_status lion_conv_fwd(const lion_conv_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = conv_sizes(a->B, a->L, a->D, a->K, a->act, a->reverse, a->dtype, a->x_token);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->x, es) || !ptr.need(a->weight, 4) || !ptr.maybe(a->bias, 4) || !ptr.maybe(a->state, es) ||
      !ptr.maybe(a->lengths, 4) || !ptr.need(a->y, es) || !ptr.maybe(a->state_out, es) ||
      (a->state && a->state_out == a->state) || a->y == a->x)   // other runs still read these
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return from_cuda(lion::launch_conv_fwd(*a, a->stream));
}

size_t lion_conv_bwd_workspace_bytes(int B, int L, int D, int K) {
  if (conv_sizes(B, L, D, K, 0, 0, 0, 0) != LION_OK) return 0;
  return lion::conv_bwd_workspace_bytes(B, L, D, K);
}

lion_status lion_conv_bwd(const lion_conv_bwd_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = conv_sizes(a->B, a->L, a->D, a->K, a->act, a->reverse, a->dtype, a->x_token);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->dy, es) || !ptr.need(a->x, es) || !ptr.need(a->weight, 4) || !ptr.maybe(a->bias, 4) ||
      !ptr.maybe(a->state, es) || !ptr.maybe(a->lengths, 4) || !ptr.need(a->dx, es) || !ptr.need(a->dweight, 4) ||
      !ptr.maybe(a->dbias, 4) || !ptr.maybe(a->dstate, es) || a->dx == a->x || a->dx == a->dy)
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return with_workspace(a->workspace, a->workspace_bytes, lion::conv_bwd_workspace_bytes(a->B, a->L, a->D, a->K),
                        a->stream, [&](void* ws) { return lion::launch_conv_bwd(*a, ws, a->stream); });
}

lion_status lion_conv_step(const void* x, void* state, const float* weight, const float* bias, void* y, int B, int D,
                           int K, int act, int dtype, cudaStream_t stream) {
  const lion_status st = conv_sizes(B, 1, D, K, act, 0, dtype, 0);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(dtype);
  if (!ptr.need(x, es) || !ptr.need(state, es) || !ptr.need(weight, 4) || !ptr.maybe(bias, 4) || !ptr.need(y, es))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return from_cuda(lion::launch_conv_step(x, state, weight, bias, y, B, D, K, act, dtype, stream));
}

size_t lion_scan_workspace_bytes(int B, int L, int D, int N, int G) {
  if (scan_sizes(B, L, D, N, G, 0, 0, 0) != LION_OK) return 0;
  return lion::scan_workspace_bytes(B, L, D, N, G);
}

lion_status lion_scan_fwd(const lion_scan_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = scan_sizes(a->B, a->L, a->D, a->N, a->G, a->dt_softplus, a->reverse, a->dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  const long long gn = (long long)a->G * a->N;
  if (!stride_ok(a->u_token, a->D) || !stride_ok(a->dt_token, a->D) || !stride_ok(a->z_token, a->D) ||
      !stride_ok(a->b_token, gn) || !stride_ok(a->c_token, gn))
    return LION_ERR_INVALID_ARG;
  if (!ptr.need(a->u, es) || !ptr.need(a->dt, es) || !ptr.need(a->A, 16) || !ptr.need(a->Bm, es) ||
      !ptr.need(a->Cm, es) || !ptr.maybe(a->Dskip, 4) || !ptr.maybe(a->z, es) || !ptr.maybe(a->dt_bias, 4) ||
      !ptr.maybe(a->h0, 16) || !ptr.maybe(a->lengths, 4) || !ptr.need(a->out, es) || !ptr.maybe(a->h_out, 16) ||
      !ptr.maybe(a->states, 16))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return with_workspace(a->workspace, a->workspace_bytes, lion::scan_workspace_bytes(a->B, a->L, a->D, a->N, a->G),
                        a->stream, [&](void* ws) { return lion::launch_scan_fwd(*a, ws, a->stream); });
}

size_t lion_scan_bwd_workspace_bytes(int B, int L, int D, int N, int G, int have_states) {
  if (scan_sizes(B, L, D, N, G, 0, 0, 0) != LION_OK) return 0;
  return lion::scan_bwd_workspace_bytes(B, L, D, N, G, have_states != 0);
}

lion_status lion_scan_bwd(const lion_scan_bwd_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  const lion_status st = scan_sizes(a->B, a->L, a->D, a->N, a->G, a->dt_softplus, a->reverse, a->dtype);
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  const long long gn = (long long)a->G * a->N;
  if (!stride_ok(a->u_token, a->D) || !stride_ok(a->dt_token, a->D) || !stride_ok(a->z_token, a->D) ||
      !stride_ok(a->b_token, gn) || !stride_ok(a->c_token, gn))
    return LION_ERR_INVALID_ARG;
  if (!ptr.need(a->dout, es) || !ptr.need(a->u, es) || !ptr.need(a->dt, es) || !ptr.need(a->A, 16) ||
      !ptr.need(a->Bm, es) || !ptr.need(a->Cm, es) || !ptr.maybe(a->Dskip, 4) || !ptr.maybe(a->z, es) ||
      !ptr.maybe(a->dt_bias, 4) || !ptr.maybe(a->h0, 16) || !ptr.maybe(a->lengths, 4) || !ptr.maybe(a->states, 16) ||
      !ptr.need(a->du, es) || !ptr.need(a->ddt, es) || !ptr.need(a->dA, 16) || !ptr.need(a->dB, es) ||
      !ptr.need(a->dC, es) || !ptr.maybe(a->dDskip, 4) || !ptr.maybe(a->dz, es) || !a->z != !a->dz ||
      !ptr.maybe(a->ddt_bias, 4) || !ptr.maybe(a->dh0, 16))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return with_workspace(a->workspace, a->workspace_bytes,
                        lion::scan_bwd_workspace_bytes(a->B, a->L, a->D, a->N, a->G, a->states != nullptr), a->stream,
                        [&](void* ws) { return lion::launch_scan_bwd(*a, ws, a->stream); });
}

lion_status lion_scan_step(const lion_scan_step_args* a) {
  if (!a) return LION_ERR_INVALID_ARG;
  lion_status st = scan_sizes(a->B, 1, a->D, a->N, a->G, a->dt_softplus, 0, a->dtype);
  if (st == LION_OK && a->B > 2 * 65535) st = LION_ERR_UNSUPPORTED;   // two sequences a CTA on a grid's second axis
  if (st == LION_ERR_INVALID_ARG) return st;
  const Pointers ptr;
  const size_t es = esize(a->dtype);
  if (!ptr.need(a->h, 16) || !ptr.need(a->u, es) || !ptr.need(a->dt, es) || !ptr.need(a->A, 16) ||
      !ptr.need(a->Bm, es) || !ptr.need(a->Cm, es) || !ptr.maybe(a->Dskip, 4) || !ptr.maybe(a->z, es) ||
      !ptr.maybe(a->dt_bias, 4) || !ptr.need(a->out, es))
    return LION_ERR_INVALID_ARG;
  if (st != LION_OK) return st;
  return from_cuda(lion::launch_scan_step(*a, a->stream));
}

}  // extern "C"
