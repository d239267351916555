// ssm_norm.cu -- layer norm over rows, its gradients, and the fixed-order sum
// of partials that the block's parameter gradients share.
//
// Bound by HBM: the forward reads x and writes y, the gradients read x and dy
// and write dx.  A row stays in its threads' registers between the sums and
// the outputs, so each is read once.  Forward: one warp a row up to 1024 values
// (no barrier, shuffles only), one CTA above.  The mean is taken first and the
// variance from the centred values, which loses nothing when the mean is far
// from 0.  Measured at 48674 x 768 fp32: 50 us forward (6.0 TB/s, 90% of a
// copy's), 82 us for the gradients (5.5 TB/s) and 5 for the sum of their
// parameters' parts (a warp a row there: 113 + 8).
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

// Eight raw elements as they lie in memory, read ahead of their use.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool wide) {
    if (wide && n >= 8) {
      r = *reinterpret_cast<const uint4*>(p);
    } else {
      unsigned short h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = e < n ? reinterpret_cast<const unsigned short*>(p)[e] : 0;
      r = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(r, v); }
};
template <>
struct Raw8<float> {
  float f[8];
  __device__ __forceinline__ void load(const float* p, int n, bool wide) { load8(p, n, wide, f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e];
  }
};

// dx, and the CTA's share of dweight and dbias.  A row is shared by NW warps,
// eight columns a thread (NV times over), so that a thread's sums for its
// columns and the next row, read ahead, fit few registers and many rows are
// under way; RS rows at a time in a CTA, each with a barrier of its own.
template <typename T, int NW, int NV, int RS>
__global__ void __launch_bounds__(32 * NW * RS) layernorm_bwd_kernel(NormP p) {
  constexpr int TPR = 32 * NW;
  constexpr bool kAhead = NV <= 2;   // the next row is read ahead where it fits the registers
  __shared__ float2 red[RS][2][NW];
  extern __shared__ float sp[];   // [RS][2][cols] where RS > 1
  const int rs = threadIdx.x / TPR, tid = threadIdx.x % TPR, lane = tid & 31;
  const float inv = 1.f / p.cols;
  float dw[NV][8], db[NV][8], w[NV][8];
  int n[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    n[j] = max(0, p.cols - 8 * (tid + j * TPR));
    load8(p.weight + 8 * (tid + j * TPR), n[j], p.w_wide, w[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  const long long hop = (long long)gridDim.x * RS;
  long long row = (long long)blockIdx.x * RS + rs;
  const T* x = static_cast<const T*>(p.x) + row * p.x_row + 8 * tid;
  const T* dy = static_cast<const T*>(p.dy) + row * p.cols + 8 * tid;
  T* dx = static_cast<T*>(p.out) + row * p.cols + 8 * tid;
  Raw8<T> rx[NV], ry[NV];
  float mean = 0.f, rstd = 0.f;
  auto read = [&](long long r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rx[j].load(x + 8 * j * TPR, n[j], p.x_wide);
      ry[j].load(dy + 8 * j * TPR, n[j], p.o_wide);
    }
    mean = p.mean[r];
    rstd = p.rstd[r];
    x += hop * p.x_row;
    dy += hop * p.cols;
  };
  if (kAhead && row < p.rows) read(row);
  for (int turn = 0; row < p.rows; row += hop, turn ^= 1) {
    if (!kAhead) read(row);
    float v[NV][8], g[NV][8], s1 = 0.f, s2 = 0.f;
    const float rs_now = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rx[j].get(v[j]);
      ry[j].get(g[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[j][e] = e < n[j] ? (v[j][e] - mean) * rs_now : 0.f;
        dw[j][e] = fmaf(g[j][e], v[j][e], dw[j][e]);
        db[j][e] += g[j][e];
        g[j][e] *= w[j][e];
        s1 += g[j][e];
        s2 = fmaf(g[j][e], v[j][e], s2);
      }
    }
    if (kAhead && row + hop < p.rows) read(row + hop);
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (NW > 1) {
      if (lane == 0) red[rs][turn][tid >> 5] = make_float2(s1, s2);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + rs), "n"(TPR) : "memory");
      s1 = s2 = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        const float2 t = red[rs][turn][q];
        s1 += t.x;
        s2 += t.y;
      }
    }
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (n[j] <= 0) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = rs_now * (g[j][e] - fmaf(v[j][e], s2, s1));
      store8(dx + 8 * j * TPR, n[j], p.o_wide, v[j]);
    }
    dx += hop * p.cols;
  }
  float* part = p.part + (size_t)blockIdx.x * 2 * p.cols;
  float* mine = RS > 1 ? sp + rs * 2 * p.cols : part;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (tid + j * TPR);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n[j]) {
        mine[c + e] = dw[j][e];
        mine[p.cols + c + e] = db[j][e];
      }
  }
  if (RS > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.cols; c += TPR * RS) {
      float s = sp[c];
#pragma unroll
      for (int q = 1; q < RS; ++q) s += sp[q * 2 * p.cols + c];
      part[c] = s;
    }
  }
}

template <typename T, int TPR, int NV>
cudaError_t run_fwd(const NormP& p, cudaStream_t s) {
  constexpr int RPC = TPR == 32 ? 4 : 1;
  layernorm_fwd_kernel<T, TPR, NV><<<(unsigned)(((long long)p.rows + RPC - 1) / RPC), TPR == 32 ? 128 : TPR, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int NW, int NV, int RS>
cudaError_t run_bwd(const NormP& p, int ctas, cudaStream_t s) {
  layernorm_bwd_kernel<T, NW, NV, RS>
      <<<ctas, 32 * NW * RS, RS > 1 ? sizeof(float) * RS * 2 * p.cols : 0, s>>>(p);
  return cudaGetLastError();
}

// The row's threads and vectors by its length.  The gradients' registers hold
// two vectors a thread: of four (above 8192 columns) some 100 words a thread
// spill, and 8 of float32's two.
template <typename T>
cudaError_t run_fwd_any(const NormP& p, cudaStream_t s) {
  return p.cols <= 256    ? run_fwd<T, 32, 1>(p, s)
         : p.cols <= 512  ? run_fwd<T, 32, 2>(p, s)
         : p.cols <= 768  ? run_fwd<T, 32, 3>(p, s)
         : p.cols <= 1024 ? run_fwd<T, 32, 4>(p, s)
         : p.cols <= 2048 ? run_fwd<T, 256, 1>(p, s)
         : p.cols <= 4096 ? run_fwd<T, 256, 2>(p, s)
         : p.cols <= 8192 ? run_fwd<T, 512, 2>(p, s)
                          : run_fwd<T, 512, 4>(p, s);
}
template <typename T>
cudaError_t run_bwd_any(const NormP& p, int ctas, cudaStream_t s) {
  return p.cols <= 256    ? run_bwd<T, 1, 1, 8>(p, ctas, s)
         : p.cols <= 512  ? run_bwd<T, 2, 1, 4>(p, ctas, s)
         : p.cols <= 768  ? run_bwd<T, 3, 1, 4>(p, ctas, s)
         : p.cols <= 1024 ? run_bwd<T, 4, 1, 4>(p, ctas, s)
         : p.cols <= 2048 ? run_bwd<T, 8, 1, 1>(p, ctas, s)
         : p.cols <= 4096 ? run_bwd<T, 16, 1, 1>(p, ctas, s)
         : p.cols <= 8192 ? run_bwd<T, 16, 2, 1>(p, ctas, s)
                          : run_bwd<T, 16, 4, 1>(p, ctas, s);
}

// CTAs of the gradients, as far as there are rows.  The counts an SM are those
// of bfloat16 at 513 to 768 columns, which was measured; others hold fewer at
// once than they are given (bfloat16: 3 of 4 up to 512 and at 1025 to 2048
// columns, 1 of 2 at 769 to 1024 and 2049 to 4096; float32: half in every band
// up to 4096), so that theirs take more than one round.
int norm_ctas(int rows, int cols) {
  const int per = cols <= 256 ? 8 : cols <= 1024 ? 4 : 1;
  const int most = kSmCount * (cols <= 512 ? 4 : cols <= 1024 ? 2 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1);
  const long long want = ((long long)rows + per - 1) / per;
  return (int)(want < most ? want : most);
}

// part[p * stride + i] summed over p: R threads an element, each every R-th p.
template <int R>
__global__ void __launch_bounds__(32 * R) sum_parts_kernel(const float* part, int P, long long stride, long long n1,
                                                           float* out1, long long n2, float* out2, long long n3,
                                                           float* out3) {
  __shared__ float sh[R][33];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const long long n = n1 + n2 + n3, i = (long long)blockIdx.x * 32 + lane;
  float s = 0.f;
  wait_prior();
  if (i < n) {
#pragma unroll 4
    for (int q = r; q < P; q += R) s += part[q * stride + i];
  }
  sh[r][lane] = s;
  __syncthreads();
  if (r == 0 && i < n) {
    s = sh[0][lane];
#pragma unroll
    for (int k = 1; k < R; ++k) s += sh[k][lane];
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

cudaError_t launch_sum_parts(const float* part, int P, long long stride, long long n1, float* out1, long long n2,
                             float* out2, long long n3, float* out3, cudaStream_t s) {
  const long long n = n1 + n2 + n3;
  // its launch overlaps the end of the one before it.  Few parts and many
  // elements: smaller CTAs, of which more are under way (64 parts of 27648: 4.6
  // against 8.7 us)
  const dim3 grid((unsigned)((n + 31) / 32));
  return P <= 128 ? launch_dependent(sum_parts_kernel<8>, grid, dim3(256), 0, s, part, P, stride, n1, out1, n2, out2,
                                     n3, out3)
                  : launch_dependent(sum_parts_kernel<32>, grid, dim3(1024), 0, s, part, P, stride, n1, out1, n2, out2,
                                     n3, out3);
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
  return a.dtype == DT_BF16 ? run_fwd_any<__nv_bfloat16>(p, s) : run_fwd_any<float>(p, s);
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
  cudaError_t e = a.dtype == DT_BF16 ? run_bwd_any<__nv_bfloat16>(p, ctas, s) : run_bwd_any<float>(p, ctas, s);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(p.part, ctas, 2LL * a.cols, a.cols, a.dweight, a.cols, a.dbias, 0, nullptr, s);
}

}  // namespace lion
