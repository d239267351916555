// ssm_conv.cu -- the short causal depthwise convolution along the tokens, its
// gradients and its one-token step.
//
//   p_i = bias + sum_{j<K} w[K-1-j] x_{i-j},  y_i = act(p_i)
//   dx_i = sum_{j<K} w[K-1-j] dp_{i+j},  dp = dy act'(p)
//   dw[K-1-j] = sum_{b,i} dp_i x_{i-j},  dbias = sum_{b,i} dp_i
// with i the order in which tokens are walked.  2 K operations a value: bound
// by HBM.  A thread walks a run of tokens for eight channels with the window
// in registers, so an input is read once plus K-1 tokens before each run (and
// behind it, for the gradients), which the neighbouring runs' reads leave in
// the caches; a warp reads 32 x 8 adjacent channels.
#include "lion_internal.h"
#include "ssm_common.cuh"

namespace lion {
namespace {

struct ConvP {
  const void* x;
  const void* dy;
  const float* weight;
  const float* bias;
  const void* state;
  const int* lengths;
  void* out;          // y, or dx
  void* state_out;    // or dstate
  float* part;        // [parts][D*K | D]
  long long x_ld;
  int B, L, D;
  int act, reverse;
  int nvec, runs;     // channel vectors; runs of tokens a sequence
  bool x_wide, o_wide, s_wide;
};

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int L) {
  return lengths ? min(max(lengths[b], 0), L) : L;
}

constexpr int kRun = 16;

template <int K>
__device__ __forceinline__ void load_taps(const float* weight, int c0, int n, float (&w)[K][8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][e] = e < n ? weight[(size_t)(c0 + e) * K + k] : 0.f;
}

// The input processed i-th (i < 0: from the state; 0 where there is none).
template <typename T, int K>
__device__ __forceinline__ void load_at(const ConvP& p, int b, int len, int i, int c0, int n, float (&v)[8]) {
  if (i >= 0 && i < len) {
    const int t = p.reverse ? len - 1 - i : i;
    load8(static_cast<const T*>(p.x) + ((long long)b * p.L + t) * p.x_ld + c0, n, p.x_wide, v);
  } else if (i < 0 && i >= -(K - 1) && p.state) {
    load8(static_cast<const T*>(p.state) + ((long long)b * (K - 1) + K - 1 + i) * p.D + c0, n, p.s_wide, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(128) conv_fwd_kernel(ConvP p) {
  const long long item = (long long)blockIdx.x * 128 + threadIdx.x;
  const long long line = item / p.nvec;
  const int c0 = 8 * (int)(item - line * p.nvec), n = p.D - c0;
  const int b = (int)(line / p.runs), i0 = (int)(line - (long long)b * p.runs) * kRun;
  if (b >= p.B) return;
  const int len = clamp_len(p.lengths, b, p.L);
  const int i1 = min(i0 + kRun, p.L);
  float w[K][8], bias[8], win[K][8];
  load_taps<K>(p.weight, c0, n, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = p.bias && e < n ? p.bias[c0 + e] : 0.f;
#pragma unroll
  for (int k = 1; k < K; ++k) load_at<T, K>(p, b, len, i0 - K + k, c0, n, win[k]);
  T* y = static_cast<T*>(p.out);
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
#pragma unroll
    for (int k = 0; k + 1 < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) win[k][e] = win[k + 1][e];
    load_at<T, K>(p, b, len, i, c0, n, win[K - 1]);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a = bias[e];
#pragma unroll
      for (int k = 0; k < K; ++k) a = fmaf(w[k][e], win[k][e], a);
      o[e] = i < len ? (p.act ? a * sigmoid(a) : a) : 0.f;
    }
    // tokens past the length are not part of the walk: each is written as it lies
    const int t = p.reverse && i < len ? len - 1 - i : i;
    store8(y + ((long long)b * p.L + t) * p.D + c0, n, p.o_wide, o);
  }
  if (p.state_out && i0 == 0) {
    T* st = static_cast<T*>(p.state_out) + (long long)b * (K - 1) * p.D + c0;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      float v[8];
      load_at<T, K>(p, b, len, len - (K - 1) + k, c0, n, v);
      store8(st + (long long)k * p.D, n, p.s_wide, v);
    }
  }
}

// One CTA: 32 channel vectors (lanes) x 8 rows of runs.  Each thread keeps its
// channels' share of dweight and dbias over all the runs it walks.
template <typename T, int K>
__global__ void __launch_bounds__(256) conv_bwd_kernel(ConvP p) {
  __shared__ float sh[8][32][8];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int vec = blockIdx.x * 32 + lane, c0 = 8 * vec, n = p.D - c0;
  const bool live = n > 0;
  float w[K][8], bias[8], dw[K][8], db[8];
  load_taps<K>(p.weight, c0, live ? n : 0, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bias[e] = p.bias && e < n ? p.bias[c0 + e] : 0.f;
    db[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][e] = 0.f;
  }
  const long long lines = (long long)p.B * p.runs;
  for (long long line = (long long)blockIdx.y * 8 + r; live && line < lines; line += (long long)gridDim.y * 8) {
    const int b = (int)(line / p.runs), i0 = (int)(line - (long long)b * p.runs) * kRun;
    const int len = clamp_len(p.lengths, b, p.L);
    const int i1 = min(i0 + kRun, p.L);
    // win[k] = x_{i-K+1+k}; dp[k] = dp_{i-K+1+k}
    float win[K][8], dp[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) dp[k][e] = 0.f;
#pragma unroll
    for (int k = 1; k < K; ++k) load_at<T, K>(p, b, len, i0 - K + k, c0, n, win[k]);
    // the state's gradient takes the sums that end before the first token
    const bool head = i0 == 0 && p.state_out;
    for (int i = i0; i < i1 + K - 1; ++i) {
#pragma unroll
      for (int k = 0; k + 1 < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          win[k][e] = win[k + 1][e];
          dp[k][e] = dp[k + 1][e];
        }
      load_at<T, K>(p, b, len, i, c0, n, win[K - 1]);
      const bool real = i < len;
      float g[8];
      if (real) {
        const int t = p.reverse ? len - 1 - i : i;
        load8(static_cast<const T*>(p.dy) + ((long long)b * p.L + t) * p.D + c0, n, p.o_wide, g);
      }
      const bool mine = i < i1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float d = 0.f;
        if (real) {
          d = g[e];
          if (p.act) {
            float a = bias[e];
#pragma unroll
            for (int k = 0; k < K; ++k) a = fmaf(w[k][e], win[k][e], a);
            const float sg = sigmoid(a);
            d *= sg * fmaf(a, 1.f - sg, 1.f);
          }
          if (mine) {
            db[e] += d;
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][e] = fmaf(d, win[k][e], dw[k][e]);
          }
        }
        dp[K - 1][e] = d;
      }
      // dx_m for m = i - K + 1 is complete: sum_j w[K-1-j] dp_{m+j}
      const int m = i - K + 1;
      if (m < i0 && !(head && m < 0)) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) a = fmaf(w[K - 1 - j][e], dp[j][e], a);
        o[e] = m < len ? a : 0.f;
      }
      if (m < 0) {
        store8(static_cast<T*>(p.state_out) + ((long long)b * (K - 1) + K - 1 + m) * p.D + c0, n, p.s_wide, o);
      } else {
        const int t = p.reverse && m < len ? len - 1 - m : m;
        store8(static_cast<T*>(p.out) + ((long long)b * p.L + t) * p.D + c0, n, p.o_wide, o);
      }
    }
  }
  float* part = p.part + (size_t)blockIdx.y * p.D * (K + 1);
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[r][lane][e] = k < K ? dw[k < K ? k : 0][e] : db[e];
    __syncthreads();
    // thread (lane, r): channel c0 + r
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += sh[q][lane][r];
    const int c = c0 + r;
    if (c < p.D) {
      if (k < K) part[(size_t)c * K + k] = s;
      else part[(size_t)p.D * K + c] = s;
    }
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(128) conv_step_kernel(const T* x, T* state, const float* weight, const float* bias,
                                                        T* y, int B, int D, int act) {
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
  if (i >= (long long)B * D) return;
  const int b = (int)(i / D), c = (int)(i - (long long)b * D);
  T* st = state + (long long)b * (K - 1) * D + c;
  T win[K];
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) win[k] = st[(long long)k * D];
  win[K - 1] = x[i];
  float a = bias ? bias[c] : 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) a = fmaf(weight[(size_t)c * K + k], to_f32(win[k]), a);
  y[i] = from_f32<T>(act ? a * sigmoid(a) : a);
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) st[(long long)k * D] = win[k + 1];
}

#define LION_CONV_DISPATCH(RUN, dtype, K, ...)                                                     \
  (dtype == DT_BF16 ? (K == 2   ? RUN<__nv_bfloat16, 2>(__VA_ARGS__)                               \
                       : K == 3 ? RUN<__nv_bfloat16, 3>(__VA_ARGS__)                               \
                                : RUN<__nv_bfloat16, 4>(__VA_ARGS__))                              \
                    : (K == 2   ? RUN<float, 2>(__VA_ARGS__)                                       \
                       : K == 3 ? RUN<float, 3>(__VA_ARGS__)                                       \
                                : RUN<float, 4>(__VA_ARGS__)))

template <typename T, int K>
cudaError_t run_fwd(const ConvP& p, cudaStream_t s) {
  const long long items = (long long)p.B * p.runs * p.nvec;
  conv_fwd_kernel<T, K><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int K>
cudaError_t run_bwd(const ConvP& p, int parts, cudaStream_t s) {
  conv_bwd_kernel<T, K><<<dim3((p.nvec + 31) / 32, parts), 256, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int K>
cudaError_t run_step(const void* x, void* state, const float* weight, const float* bias, void* y, int B, int D,
                     int act, cudaStream_t s) {
  const long long n = (long long)B * D;
  conv_step_kernel<T, K><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(
      static_cast<const T*>(x), static_cast<T*>(state), weight, bias, static_cast<T*>(y), B, D, act);
  return cudaGetLastError();
}

// CTAs along the runs: enough to fill the SMs twice with the channels' CTAs.
int conv_parts(int B, int L, int D) {
  const long long lines = (long long)B * ((L + kRun - 1) / kRun);
  const int across = (D + 255) / 256;
  const long long want = (lines + 7) / 8, most = (4 * kSmCount + across - 1) / across;
  return (int)(want < most ? want : most);
}

}  // namespace

size_t conv_bwd_workspace_bytes(int B, int L, int D, int K) {
  return sizeof(float) * (size_t)conv_parts(B, L, D) * D * (K + 1);
}

cudaError_t launch_conv_fwd(const lion_conv_args& a, cudaStream_t s) {
  ConvP p = {};
  p.x = a.x;
  p.weight = a.weight;
  p.bias = a.bias;
  p.state = a.state;
  p.lengths = a.lengths;
  p.out = a.y;
  p.state_out = a.state_out;
  p.x_ld = a.x_token ? a.x_token : a.D;
  p.B = a.B;
  p.L = a.L;
  p.D = a.D;
  p.act = a.act;
  p.reverse = a.reverse;
  p.nvec = (a.D + 7) / 8;
  p.runs = (a.L + kRun - 1) / kRun;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.x_wide = rows_wide(a.x, p.x_ld, es);
  p.o_wide = rows_wide(a.y, a.D, es);
  p.s_wide = rows_wide(a.state, a.D, es) && rows_wide(a.state_out, a.D, es);
  return LION_CONV_DISPATCH(run_fwd, a.dtype, a.K, p, s);
}

cudaError_t launch_conv_bwd(const lion_conv_bwd_args& a, void* ws, cudaStream_t s) {
  ConvP p = {};
  p.x = a.x;
  p.dy = a.dy;
  p.weight = a.weight;
  p.bias = a.bias;
  p.state = a.state;
  p.lengths = a.lengths;
  p.out = a.dx;
  p.state_out = a.dstate;
  p.part = static_cast<float*>(ws);
  p.x_ld = a.x_token ? a.x_token : a.D;
  p.B = a.B;
  p.L = a.L;
  p.D = a.D;
  p.act = a.act;
  p.reverse = a.reverse;
  p.nvec = (a.D + 7) / 8;
  p.runs = (a.L + kRun - 1) / kRun;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.x_wide = rows_wide(a.x, p.x_ld, es);
  p.o_wide = rows_wide(a.dx, a.D, es) && rows_wide(a.dy, a.D, es);
  p.s_wide = rows_wide(a.state, a.D, es) && rows_wide(a.dstate, a.D, es);
  const int parts = conv_parts(a.B, a.L, a.D);
  cudaError_t e = LION_CONV_DISPATCH(run_bwd, a.dtype, a.K, p, parts, s);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(p.part, parts, (long long)a.D * (a.K + 1), (long long)a.D * a.K, a.dweight, a.D, a.dbias, 0, nullptr, s);
}

cudaError_t launch_conv_step(const void* x, void* state, const float* weight, const float* bias, void* y, int B, int D,
                             int K, int act, int dtype, cudaStream_t s) {
  return LION_CONV_DISPATCH(run_step, dtype, K, x, state, weight, bias, y, B, D, act, s);
}

}  // namespace lion
