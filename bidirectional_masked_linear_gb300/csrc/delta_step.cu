// delta_step.cu -- the gated delta rule for one token.
//
//   u = beta (v - e^g S^T k),  out = scale (e^g S^T q + (k . q) u),  S <- e^g S + k u^T
//
// S^T k and S^T q come from one pass over the state, which stays in registers
// until it is written back: the state is read once and written once.  A CTA
// takes 32 of a head's dv columns (256 x 16 x 128 x 128: 81 us, 6.6 TB/s; 64
// columns 103 us, 128 149 us), 16 rows at a time, a thread four columns of a row.
#include "lion_internal.h"
#include "ssm_common.cuh"

namespace lion {
namespace {

constexpr int kStepCols = 32;

template <typename T, int NV>   // NV: rows a thread holds, 16 apart
__global__ void __launch_bounds__(4 * kStepCols) delta_step_kernel(const lion_delta_step_args a, int slices) {
  constexpr int LPR = kStepCols / 4, WARPS = kStepCols / 8;   // LPR: lanes a row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c4 = lane % LPR;
  const unsigned bh = blockIdx.x / slices;
  const int slice = (int)(blockIdx.x - bh * slices);
  const int b = (int)(bh / a.Hv), hv = (int)(bh - (unsigned)b * a.Hv), hk = hv / (a.Hv / a.Hk);
  const int col = slice * kStepCols + 4 * c4, row0 = threadIdx.x / LPR;
  const bool in = col < a.dv;
  float* S = a.h + (size_t)bh * a.dk * a.dv + col;
  float4 x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int r = row0 + 16 * i;
    x[i] = in && r < a.dk ? *reinterpret_cast<const float4*>(S + (size_t)r * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const T* kp = static_cast<const T*>(a.k) + ((size_t)b * a.Hk + hk) * a.dk;
  const T* qp = static_cast<const T*>(a.q) + ((size_t)b * a.Hk + hk) * a.dk;
  float k[NV], q[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int r = row0 + 16 * i;
    k[i] = r < a.dk ? to_f32(kp[r]) : 0.f;
    q[i] = r < a.dk ? to_f32(qp[r]) : 0.f;
  }
  const float decay = expf(to_f32(static_cast<const T*>(a.g)[bh]));
  const float beta = to_f32(static_cast<const T*>(a.beta)[bh]);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = in ? to_f32(static_cast<const T*>(a.v)[(size_t)bh * a.dv + col + e]) : 0.f;
  float sum[9] = {};   // S^T k, S^T q, k . q
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float s[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum[e] = fmaf(s[e], k[i], sum[e]);
      sum[4 + e] = fmaf(s[e], q[i], sum[4 + e]);
    }
    sum[8] = fmaf(k[i], q[i], sum[8]);
  }
  __shared__ float sh[WARPS][LPR][9];
#pragma unroll
  for (int e = 0; e < 9; ++e) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
    if (lane < LPR) sh[warp][lane][e] = sum[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 9; ++e) {
    sum[e] = sh[0][c4][e];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) sum[e] += sh[w][c4][e];
  }
  float u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = beta * (v[e] - decay * sum[e]);
  if (!in) return;
  if (row0 == 0) {
    T* out = static_cast<T*>(a.out) + (size_t)bh * a.dv + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = from_f32<T>(a.scale * fmaf(sum[8], u[e], decay * sum[4 + e]));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int r = row0 + 16 * i;
    if (r < a.dk)
      *reinterpret_cast<float4*>(S + (size_t)r * a.dv) =
          make_float4(fmaf(k[i], u[0], decay * x[i].x), fmaf(k[i], u[1], decay * x[i].y),
                      fmaf(k[i], u[2], decay * x[i].z), fmaf(k[i], u[3], decay * x[i].w));
  }
}

template <typename T>
cudaError_t run_step(const lion_delta_step_args& a, cudaStream_t s) {
  const int slices = (a.dv + kStepCols - 1) / kStepCols;
  const unsigned grid = (unsigned)((long long)a.B * a.Hv * slices);
  if (a.dk <= 64)
    delta_step_kernel<T, 4><<<grid, 4 * kStepCols, 0, s>>>(a, slices);
  else
    delta_step_kernel<T, 8><<<grid, 4 * kStepCols, 0, s>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_step(const lion_delta_step_args& a, cudaStream_t s) {
  return a.dtype == DT_BF16 ? run_step<__nv_bfloat16>(a, s) : run_step<float>(a, s);
}

}  // namespace lion
