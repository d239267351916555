// ssm_common.cuh -- what the state space block's kernels share: eight
// elements at a time from and to rows of either type and any alignment, fp32
// nonlinearities, packed fp32 pairs, and the fixed-order sum of partials.
#pragma once

#include "lion_common.cuh"
#include "scan_plan.h"

namespace lion {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- eight elements

// n (<= 8) consecutive values as fp32, the rest 0; wide: p is 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, int n, bool wide, float (&v)[8]) {
  if (wide && n >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.f;
  }
}
__device__ __forceinline__ float2 unpack_bf16(unsigned w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_bf16(w[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, bool wide, float (&v)[8]) {
  if (wide && n >= 8) {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? __bfloat162float(p[e]) : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int n, bool wide, const float (&v)[8]) {
  if (wide && n >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, bool wide, const float (&v)[8]) {
  if (wide && n >= 8) {
    uint4 r;
    unsigned* w = reinterpret_cast<unsigned*>(&r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const unsigned*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = r;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = __float2bfloat16_rn(v[e]);
  }
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// ---------------------------------------------------------------- nonlinearities

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// ---------------------------------------------------------------- fp32 pairs

// Two fp32 values in one 64-bit register: an instruction issues for both, at
// the same rate of values, which leaves issue slots for everything else.
typedef float2 f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ float2 unpack2(f2 x) { return x; }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ f2 ex2_2(f2 x) {
  const float2 v = unpack2(x);
  return pack2(ex2(v.x), ex2(v.y));
}
__device__ __forceinline__ float sum2(f2 x) {
  const float2 v = unpack2(x);
  return v.x + v.y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// softplus(x) = max(x, 0) + log(1 + e), e = exp(-|x|).  With s = e / (2 + e)
// <= 1/3 the logarithm is 2 artanh(s) = s P(s^2), P fitted to the series in
// the Chebyshev sense on [0, 1/9] to 8e-9 of the result, so that a small e
// keeps its relative accuracy.
__device__ __forceinline__ f2 softplus2(float x0, float x1) {
  const f2 e = pack2(ex2(fabsf(x0) * -kLog2e), ex2(fabsf(x1) * -kLog2e));
  const float2 den = unpack2(add2(e, pack2(2.f, 2.f)));
  const f2 s = mul2(e, pack2(rcp(den.x), rcp(den.y))), q = mul2(s, s);
  f2 r = fma2(q, pack2(0.2817465663f, 0.2817465663f), pack2(0.2796141803f, 0.2796141803f));
  r = fma2(r, q, pack2(0.4002485275f, 0.4002485275f));
  r = fma2(r, q, pack2(0.6666631699f, 0.6666631699f));
  r = fma2(r, q, pack2(2.f, 2.f));
  return fma2(s, r, pack2(fmaxf(x0, 0.f), fmaxf(x1, 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return unpack2(softplus2(x, 0.f)).x; }

__device__ __forceinline__ f2 sigmoid2(float x0, float x1) {
  const f2 d = add2(pack2(ex2(x0 * -kLog2e), ex2(x1 * -kLog2e)), pack2(1.f, 1.f));
  return pack2(rcp(d.x), rcp(d.y));
}

// z sigmoid(z) of a pair, times o.
__device__ __forceinline__ f2 gate2(f2 o, float z0, float z1) {
  return mul2(mul2(o, pack2(z0, z1)), sigmoid2(z0, z1));
}

// For a kernel launched as a dependent (launch_dependent): the launch before it
// has ended and its writes are there.
__device__ __forceinline__ void wait_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether rows of es-byte elements, `stride` elements apart, all start on 16 bytes.
inline bool rows_wide(const void* p, long long stride, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
}

}  // namespace

// out[i] = sum over p < P of part[p * stride + i] for i < n1 + n2 + n3, the
// three ranges of i going to out1, out2 and out3 (a NULL one is dropped), in
// an order that P alone decides.
cudaError_t launch_sum_parts(const float* part, int P, long long stride, long long n1, float* out1, long long n2,
                             float* out2, long long n3, float* out3, cudaStream_t s);

}  // namespace lion
