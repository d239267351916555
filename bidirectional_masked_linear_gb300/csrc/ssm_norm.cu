// ssm_norm.cu -- layer norm over rows, its gradients, and the fixed-order sum
// of partials that the block's parameter gradients share.
//
// Bound by HBM: the forward reads x and writes y, the gradients read x and dy
// and write dx.  A row stays in its threads' registers between the sums and
// the outputs, so each is read once: one warp a row up to 1024 values (no
// barrier, shuffles only), one CTA above.  The mean is taken first and the
// variance from the centred values, which loses nothing when the mean is far
// from 0.
#include "lion_internal.h"
#include "ssm_common.cuh"

namespace lion {
namespace {

struct NormP {
  const void* x;
  const void* dy;
  const float* weight;
  const float* bias;
  void* out;          // y, or dx
  float* mean;
  float* rstd;
  float* part;        // [CTAs][2][cols]
  long long x_row;
  int rows, cols;
  float eps;
  bool x_wide, o_wide, w_wide;
};

// Sum of v over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (TPR == 32) return v;
  constexpr int NW = TPR / 32;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[w];
  return s;
}

template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) layernorm_fwd_kernel(NormP p) {
  __shared__ float red[32];
  constexpr int RPC = TPR == 32 ? 4 : 1;
  const int r = TPR == 32 ? threadIdx.x >> 5 : 0, lane = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
  const long long row = (long long)blockIdx.x * RPC + r;
  if (row >= p.rows) return;   // whole warps; a CTA of one row never
  const T* x = static_cast<const T*>(p.x) + row * p.x_row;
  const float inv = 1.f / p.cols;
  float v[NV][8], s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (lane + j * TPR);
    load8(x + c, max(0, p.cols - c), p.x_wide, v[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[j][e];
  }
  const float mean = row_sum<TPR>(s, red) * inv;
  s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = p.cols - 8 * (lane + j * TPR);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[j][e] = e < n ? v[j][e] - mean : 0.f;
      s = fmaf(v[j][e], v[j][e], s);
    }
  }
  const float rstd = 1.f / sqrtf(row_sum<TPR>(s, red) * inv + p.eps);
  if (p.mean && lane == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.out) + row * p.cols;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (lane + j * TPR), n = p.cols - c;
    if (n <= 0) break;
    float w[8], b[8];
    load8(p.weight + c, n, p.w_wide, w);
    if (p.bias) load8(p.bias + c, n, p.w_wide, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = p.bias ? fmaf(v[j][e] * rstd, w[e], b[e]) : v[j][e] * rstd * w[e];
    store8(y + c, n, p.o_wide, v[j]);
  }
}

// dx, and the CTA's share of dweight and dbias: each thread keeps the same
// columns for every row it takes and adds them up in registers.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) layernorm_bwd_kernel(NormP p) {
  __shared__ float red[32];
  extern __shared__ float sp[];   // [4][2][cols] for the warp form
  constexpr int RPC = TPR == 32 ? 4 : 1;
  const int r = TPR == 32 ? threadIdx.x >> 5 : 0, lane = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
  const float inv = 1.f / p.cols;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.f;
  for (long long row = (long long)blockIdx.x * RPC + r; row < p.rows; row += (long long)gridDim.x * RPC) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_row;
    const T* dy = static_cast<const T*>(p.dy) + row * p.cols;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float v[NV][8], g[NV][8], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (lane + j * TPR), n = max(0, p.cols - c);
      load8(x + c, n, p.x_wide, v[j]);
      load8(dy + c, n, p.o_wide, g[j]);
      float w[8];
      load8(p.weight + c, n, p.w_wide, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[j][e] = e < n ? (v[j][e] - mean) * rstd : 0.f;
        dw[j][e] = fmaf(g[j][e], v[j][e], dw[j][e]);
        db[j][e] += g[j][e];
        g[j][e] *= w[e];
        s1 += g[j][e];
        s2 = fmaf(g[j][e], v[j][e], s2);
      }
    }
    s1 = row_sum<TPR>(s1, red) * inv;
    s2 = row_sum<TPR>(s2, red) * inv;
    T* dx = static_cast<T*>(p.out) + row * p.cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (lane + j * TPR), n = p.cols - c;
      if (n <= 0) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = rstd * (g[j][e] - fmaf(v[j][e], s2, s1));
      store8(dx + c, n, p.o_wide, v[j]);
    }
  }
  float* part = p.part + (size_t)blockIdx.x * 2 * p.cols;
  if (TPR == 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (lane + j * TPR);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < p.cols) {
          sp[(2 * r) * p.cols + c + e] = dw[j][e];
          sp[(2 * r + 1) * p.cols + c + e] = db[j][e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.cols; c += 128)
      part[c] = (sp[c] + sp[2 * p.cols + c]) + (sp[4 * p.cols + c] + sp[6 * p.cols + c]);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (lane + j * TPR);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < p.cols) {
          part[c + e] = dw[j][e];
          part[p.cols + c + e] = db[j][e];
        }
    }
  }
}

template <typename T, int TPR, int NV>
cudaError_t run_fwd(const NormP& p, cudaStream_t s) {
  constexpr int RPC = TPR == 32 ? 4 : 1;
  layernorm_fwd_kernel<T, TPR, NV><<<(unsigned)((p.rows + RPC - 1) / RPC), TPR == 32 ? 128 : TPR, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int TPR, int NV>
cudaError_t run_bwd(const NormP& p, int ctas, cudaStream_t s) {
  layernorm_bwd_kernel<T, TPR, NV>
      <<<ctas, TPR == 32 ? 128 : TPR, TPR == 32 ? sizeof(float) * 8 * p.cols : 0, s>>>(p);
  return cudaGetLastError();
}

// The row's threads and vectors by its length.
#define LION_NORM_DISPATCH(RUN, T, ...)                                   \
  (p.cols <= 256     ? RUN<T, 32, 1>(__VA_ARGS__)                         \
   : p.cols <= 512   ? RUN<T, 32, 2>(__VA_ARGS__)                         \
   : p.cols <= 768   ? RUN<T, 32, 3>(__VA_ARGS__)                         \
   : p.cols <= 1024  ? RUN<T, 32, 4>(__VA_ARGS__)                         \
   : p.cols <= 2048  ? RUN<T, 256, 1>(__VA_ARGS__)                        \
   : p.cols <= 4096  ? RUN<T, 256, 2>(__VA_ARGS__)                        \
   : p.cols <= 8192  ? RUN<T, 512, 2>(__VA_ARGS__)                        \
                     : RUN<T, 512, 4>(__VA_ARGS__))

constexpr int kNormMaxCtas = 4 * kSmCount;
int norm_ctas(int rows, int cols) {
  const long long per = cols <= 1024 ? 4 : 1;
  const long long want = (rows + per - 1) / per;
  return (int)(want < kNormMaxCtas ? want : kNormMaxCtas);
}

// part[p * stride + i] summed over p: 8 threads an element, each every eighth p.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* part, int P, long long stride, long long n1,
                                                        float* out1, long long n2, float* out2, long long n3, float* out3) {
  __shared__ float sh[8][33];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const long long n = n1 + n2 + n3, i = (long long)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (i < n)
    for (int q = r; q < P; q += 8) s += part[q * stride + i];
  sh[r][lane] = s;
  __syncthreads();
  if (r == 0 && i < n) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sh[k][lane];
    if (i < n1) {
      if (out1) out1[i] = s;
    } else if (i < n1 + n2) {
      if (out2) out2[i - n1] = s;
    } else if (out3) {
      out3[i - n1 - n2] = s;
    }
  }
}

}  // namespace

cudaError_t launch_sum_parts(const float* part, int P, long long stride, long long n1, float* out1, long long n2, float* out2,
                             long long n3, float* out3, cudaStream_t s) {
  const long long n = n1 + n2 + n3;
  sum_parts_kernel<<<(unsigned)((n + 31) / 32), 256, 0, s>>>(part, P, stride, n1, out1, n2, out2, n3, out3);
  return cudaGetLastError();
}

cudaError_t launch_layernorm_fwd(const lion_layernorm_args& a, cudaStream_t s) {
  NormP p = {};
  p.x = a.x;
  p.weight = a.weight;
  p.bias = a.bias;
  p.out = a.y;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.x_row = a.x_row ? a.x_row : a.cols;
  p.rows = a.rows;
  p.cols = a.cols;
  p.eps = a.eps;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.x_wide = rows_wide(a.x, p.x_row, es);
  p.o_wide = rows_wide(a.y, a.cols, es);
  p.w_wide = rows_wide(a.weight, 0, 4) && rows_wide(a.bias, 0, 4);
  return a.dtype == DT_BF16 ? LION_NORM_DISPATCH(run_fwd, __nv_bfloat16, p, s) : LION_NORM_DISPATCH(run_fwd, float, p, s);
}

size_t layernorm_bwd_workspace_bytes(int rows, int cols) {
  return sizeof(float) * 2 * (size_t)norm_ctas(rows, cols) * cols;
}

cudaError_t launch_layernorm_bwd(const lion_layernorm_bwd_args& a, void* ws, cudaStream_t s) {
  NormP p = {};
  p.x = a.x;
  p.dy = a.dy;
  p.weight = a.weight;
  p.mean = const_cast<float*>(a.mean);
  p.rstd = const_cast<float*>(a.rstd);
  p.out = a.dx;
  p.part = static_cast<float*>(ws);
  p.x_row = a.x_row ? a.x_row : a.cols;
  p.rows = a.rows;
  p.cols = a.cols;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.x_wide = rows_wide(a.x, p.x_row, es);
  p.o_wide = rows_wide(a.dx, a.cols, es) && rows_wide(a.dy, a.cols, es);
  p.w_wide = rows_wide(a.weight, 0, 4);
  const int ctas = norm_ctas(a.rows, a.cols);
  cudaError_t e = a.dtype == DT_BF16 ? LION_NORM_DISPATCH(run_bwd, __nv_bfloat16, p, ctas, s)
                                     : LION_NORM_DISPATCH(run_bwd, float, p, ctas, s);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(p.part, ctas, 2LL * a.cols, a.cols, a.dweight, a.cols, a.dbias, 0, nullptr, s);
}

}  // namespace lion
