// ssm_common.cuh -- what the state space block's kernels share: eight
// elements at a time from and to rows of either type and any alignment, fp32
// nonlinearities, packed fp32 pairs, and the fixed-order sum of partials.
#pragma once

#include "lion_common.cuh"

namespace lion {
namespace {

constexpr int kSmCount = 152;
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

// log(1 + e) for e in [0, 1] as 2 artanh(s), s = e / (2 + e) <= 1/3, by
// artanh's power series: the first term left out is below 2e-8 of the sum, and
// a small e keeps its relative accuracy.
__device__ __forceinline__ float log1p_unit(float e) {
  const float s = __fdividef(e, 2.f + e), q = s * s;
  float r = 1.f / 13.f;
  r = fmaf(r, q, 1.f / 11.f);
  r = fmaf(r, q, 1.f / 9.f);
  r = fmaf(r, q, 1.f / 7.f);
  r = fmaf(r, q, 1.f / 5.f);
  r = fmaf(r, q, 1.f / 3.f);
  r = fmaf(r, q, 1.f);
  return 2.f * s * r;
}
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1p_unit(__expf(-fabsf(x))); }

// ---------------------------------------------------------------- fp32 pairs

// Two fp32 values in one 64-bit register: an instruction issues for both, at
// the same rate of values, which leaves issue slots for everything else.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 ex2_2(f2 x) {
  const float2 v = unpack2(x);
  return pack2(ex2(v.x), ex2(v.y));
}
__device__ __forceinline__ float sum2(f2 x) {
  const float2 v = unpack2(x);
  return v.x + v.y;
}

// Whether rows of es-byte elements, `stride` elements apart, all start on 16 bytes.
inline bool rows_wide(const void* p, long long stride, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
}

}  // namespace

// out[i] = sum over p < P of part[p * stride + i] for i < n1 + n2 + n3, the
// three ranges of i going to out1, out2 and out3 (a NULL one is dropped), in
// an order that P alone decides.
cudaError_t launch_sum_parts(const float* part, int P, long long stride, long long n1, float* out1, long long n2, float* out2,
                             long long n3, float* out3, cudaStream_t s);

}  // namespace lion
