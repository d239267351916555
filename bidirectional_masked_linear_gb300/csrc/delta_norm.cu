// delta_norm.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and their gradients.
//
//   y = rot(x r w),  r = (sum x^2 / n + eps)^(-1/2),  n = 1 or d
//   dx = r g - x r^3 (sum g x) / n,  g = w rot^-1(dy);  dw = sum rot^-1(dy) x r
//
// A lane holds eight values of a head as two runs of four: adjacent ones, or
// those that the rotation pairs in the two halves, so that a pair never leaves
// its lane.  d / 8 lanes make a head (of a power of two, the rest idle), a
// warp takes a token, its groups of lanes the token's heads.  The four
// angles of a lane belong to all heads of the token: the groups work them out
// between them, one each at d = 64.
#include "lion_internal.h"
#include "ssm_common.cuh"

namespace lion {
namespace {

constexpr int kWarps = 4;
constexpr int kSmCount = 152, kPerSm = 4;   // CTAs an SM

struct QkP {
  const void* x[2];        // q, k
  const void* dy[2];
  void* y[2];              // outputs, or dx
  const float* w[2];
  const float* freqs;
  const int* positions;
  float* part;             // [CTA][2][d]
  long long x_ld[2];
  long long tokens;
  int per, at_once;        // a token's parts, and of each the heads a lane has
  int L, H[2], d, rp;      // rp: lanes of a head whose values turn (rot / 8)
  int interleaved;
  float inv_n, eps;
};

// A lane's eight values of a head as they lie in memory: runs of four at a and
// b.  WIDE: a run lies on its size.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
};
template <>
struct Raw<float> {
  float4 a, b;
};
template <bool WIDE>
__device__ __forceinline__ uint2 run_of(const __nv_bfloat16* p) {
  if (WIDE) return *reinterpret_cast<const uint2*>(p);
  const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
template <bool WIDE>
__device__ __forceinline__ float4 run_of(const float* p) {
  return WIDE ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ void values(uint2 r, f2* v) {
  v[0] = unpack_bf16(r.x);
  v[1] = unpack_bf16(r.y);
}
__device__ __forceinline__ void values(float4 r, f2* v) {
  v[0] = pack2(r.x, r.y);
  v[1] = pack2(r.z, r.w);
}
template <bool WIDE>
__device__ __forceinline__ void store4(float* p, const f2* v) {
  if (WIDE) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  } else {
    p[0] = v[0].x; p[1] = v[0].y; p[2] = v[1].x; p[3] = v[1].y;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store4(__nv_bfloat16* p, const f2* v) {
  if (WIDE) {
    const __nv_bfloat162 a = __float22bfloat162_rn(v[0]), b = __float22bfloat162_rn(v[1]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = __float2bfloat16_rn(e & 1 ? v[e >> 1].y : v[e >> 1].x);
  }
}

// f / (2 pi) as a fraction of a turn in units of 2^-64: the product with an
// integer position wraps at whole turns, and 32 bits of position leave 32 of
// the fraction exact.  1 / (2 pi) in two doubles, as the product's own error
// and the constant's would show from positions of about 2^28 on, and of f's
// magnitude, as a fraction above 0 has more bits than what it lacks to 1.
__device__ __forceinline__ unsigned long long turn_of(float f) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  const double x = fabsf(f), t = x * hi;
  const double rest = fma(x, hi, -t) + x * lo;
  const double frac = t - floor(t);   // exact
  const unsigned long long u = (unsigned long long)(frac * 18446744073709551616.0) +
                               (unsigned long long)(long long)(rest * 18446744073709551616.0);
  return f < 0.f ? 0 - u : u;
}

template <int LPH>
struct Turn {
  static constexpr int NG = 32 / LPH;                    // heads at a time
  static constexpr int OWN = NG >= 4 ? 1 : 4 / NG;       // angles of a lane's own
  unsigned long long u[OWN];

  // lane: this thread's, p: its place in the head
  __device__ __forceinline__ void init(const QkP& q, int lane, int p) {
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const int e = lane / LPH + o * NG;
      u[o] = p < q.rp && e < 4 ? turn_of(q.freqs[4 * p + e]) : 0;
    }
  }
  // cosines and sines (back: of the angles' negatives)
  template <bool BWD>
  __device__ __forceinline__ void at(int pos, int p, f2 (&c)[2], f2 (&s)[2], f2 (&minus)[2]) const {
    float co[OWN], so[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const unsigned long long t = u[o] * (unsigned long long)(long long)pos;
      sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &so[o], &co[o]);   // 2^-31: half turns
    }
    float ca[4], sa[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ca[e] = __shfl_sync(0xffffffffu, co[e / NG], (e % NG) * LPH + p);
      sa[e] = __shfl_sync(0xffffffffu, so[e / NG], (e % NG) * LPH + p);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      c[e] = pack2(ca[2 * e], ca[2 * e + 1]);
      const f2 x = pack2(sa[2 * e], sa[2 * e + 1]), y = pack2(-sa[2 * e], -sa[2 * e + 1]);
      s[e] = BWD ? y : x;
      minus[e] = BWD ? x : y;
    }
  }
};

// v[0], v[1] and v[2], v[3] are the lane's two runs; minus: the sines' negatives.
__device__ __forceinline__ void turn8(f2 (&v)[4], const f2 (&c)[2], const f2 (&s)[2], const f2 (&minus)[2],
                                      int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = v[e].x, b = v[e].y, ce = e & 1 ? c[e >> 1].y : c[e >> 1].x, se = e & 1 ? s[e >> 1].y : s[e >> 1].x;
      v[e] = pack2(a * ce - b * se, a * se + b * ce);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const f2 a = v[e], b = v[e + 2];
      v[e] = fma2(a, c[e], mul2(b, minus[e]));
      v[e + 2] = fma2(a, s[e], mul2(b, c[e]));
    }
  }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Heads a lane has under way: some 48 registers of raw values, this item's and
// the next one's.
template <typename T, bool BWD>
constexpr int heads_at_once() {
  return sizeof(T) == 2 ? (BWD ? 3 : 6) : (BWD ? 2 : 3);
}

// A warp goes through its tokens' heads in parts, as many at a time as a lane
// holds (evenly: 8 of them in two parts are 4 and 4); a part's values are read
// while the part before it is worked on.  2 x 24337 x 12 + 12 heads of 64 in
// bfloat16 50 us, 5.9 TB/s, 88% of a copy's rate (five CTAs an SM 51); 32 x 512 x 16 +
// 16 x 64 with rotation 31 us forward (4.3 TB/s), 47 back (4.2), with 56 and 59% of
// the issue slots at 24% of the warps: neither is full, a warp has one part ahead.
// Products of two values an instruction took 33 and 51 to that.
// Back in float32, which then spills up to 36 bytes a thread, four CTAs an SM are
// ahead of three (5 x 1021 x 6 + 2 x 72: 14 us against 19).
template <typename T, int LPH, bool WIDE, bool BWD>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) qknorm_kernel(const QkP q) {
  constexpr int NG = 32 / LPH, U = heads_at_once<T, BWD>();
  __shared__ __align__(16) float sw[2][8 * LPH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p = lane & (LPH - 1), g = lane / LPH;
  const bool there = 8 * p < q.d, turns = p < q.rp;
  const int a = q.interleaved || !turns ? 8 * p : 4 * p, b = q.interleaved || !turns ? 8 * p + 4 : 4 * (p + q.rp);
  for (int i = threadIdx.x; i < 2 * 8 * LPH; i += 32 * kWarps) {
    const int m = i / (8 * LPH), e = i % (8 * LPH);
    sw[m][e] = q.w[m] && e < q.d ? q.w[m][e] : 1.f;
  }
  Turn<LPH> turn;
  turn.init(q, lane, p);
  f2 dw[BWD ? 2 : 1][4] = {};
  const int heads = q.H[0] + q.H[1];
  __syncthreads();

  Raw<T> x[U], dy[BWD ? U : 1];
  const auto fetch = [&](long long t, int part) {
    const int h0 = part * NG * q.at_once + g;
    const T* xq = static_cast<const T*>(q.x[0]) + t * q.x_ld[0];
    const T* xk = static_cast<const T*>(q.x[1]) + t * q.x_ld[1] - (long long)q.H[0] * q.d;
    const T* dq = static_cast<const T*>(q.dy[0]) + t * q.H[0] * q.d;
    const T* dk = static_cast<const T*>(q.dy[1]) + (t * q.H[1] - q.H[0]) * q.d;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * NG;
      if (there && i < q.at_once && h < heads) {
        const T* s = (h < q.H[0] ? xq : xk) + (long long)h * q.d;
        x[i].a = run_of<WIDE>(s + a);
        x[i].b = run_of<WIDE>(s + b);
        if (BWD) {
          const T* d = (h < q.H[0] ? dq : dk) + (long long)h * q.d;
          dy[i].a = run_of<WIDE>(d + a);
          dy[i].b = run_of<WIDE>(d + b);
        }
      } else {
        x[i] = Raw<T>();
        if (BWD) dy[i] = Raw<T>();
      }
    }
  };
  const long long hop = (long long)gridDim.x * kWarps;
  long long tn = (long long)blockIdx.x * kWarps + warp;
  int pn = 0;
  f2 c[2] = {}, s[2] = {}, minus[2] = {};
  if (tn < q.tokens) fetch(tn, 0);
  while (tn < q.tokens) {
    const long long t = tn;
    const int part = pn, h0 = part * NG * q.at_once + g;
    Raw<T> xc[U], dc[BWD ? U : 1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      xc[i] = x[i];
      if (BWD) dc[i] = dy[i];
    }
    if (++pn == q.per) {
      pn = 0;
      tn += hop;
    }
    if (tn < q.tokens) fetch(tn, pn);
    if (q.rp && part == 0)
      turn.template at<BWD>(q.positions ? q.positions[t] : q.tokens >> 32 ? (int)(t % q.L) : (int)((unsigned)t % (unsigned)q.L), p, c, s,
              minus);
    T* yq = static_cast<T*>(q.y[0]) + t * q.H[0] * q.d;
    T* yk = static_cast<T*>(q.y[1]) + (t * q.H[1] - q.H[0]) * q.d;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * NG;
      if (i >= q.at_once || h - g >= heads) break;   // of all lanes
      const int m = h >= q.H[0];
      f2 v[4], w[4], o[4];
      values(xc[i].a, v);
      values(xc[i].b, v + 2);
      values(*reinterpret_cast<const float4*>(&sw[m][a]), w);
      values(*reinterpret_cast<const float4*>(&sw[m][b]), w + 2);
      f2 sum = mul2(v[0], v[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) sum = fma2(v[e], v[e], sum);
      const float r = rsqrtf(fmaf(head_sum<LPH>(sum.x + sum.y), q.inv_n, q.eps));   // to 2^-22
      const f2 r2 = pack2(r, r);
      if (!BWD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mul2(mul2(v[e], r2), w[e]);
        if (turns) turn8(o, c, s, minus, q.interleaved);
      } else {
        f2 z[4];
        values(dc[i].a, z);
        values(dc[i].b, z + 2);
        if (turns) turn8(z, c, s, minus, q.interleaved);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] = mul2(z[e], w[e]);
          sum = e ? fma2(o[e], v[e], sum) : mul2(o[e], v[e]);
        }
        if (q.part && h < heads) {
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = mul2(z[e], mul2(v[e], r2));
          if (m) {
#pragma unroll
            for (int e = 0; e < 4; ++e) dw[BWD ? 1 : 0][e] = add2(dw[BWD ? 1 : 0][e], z[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) dw[0][e] = add2(dw[0][e], z[e]);
          }
        }
        const float k = -(head_sum<LPH>(sum.x + sum.y) * q.inv_n * r * r);
        const f2 k2 = pack2(k, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mul2(r2, fma2(k2, v[e], o[e]));
      }
      if (there && h < heads) {
        T* dst = (m ? yk : yq) + (long long)h * q.d;
        store4<WIDE>(dst + a, o);
        store4<WIDE>(dst + b, o + 2);
      }
    }
  }
  if constexpr (BWD) {
    if (!q.part) return;
    __shared__ float sh[kWarps][2][8 * LPH];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = e & 1 ? dw[m][e >> 1].y : dw[m][e >> 1].x;
#pragma unroll
        for (int o = 16; o >= LPH; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (g == 0 && there) sh[warp][m][(e < 4 ? a : b - 4) + e] = x;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * q.d; i += 32 * kWarps) {
      const int m = i >= q.d, e = m ? i - q.d : i;
      float v = sh[0][m][e];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) v += sh[k][m][e];
      q.part[(size_t)blockIdx.x * 2 * q.d + i] = v;
    }
  }
}

int lanes_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }
// CTAs: a token a warp while that fills the SMs, else four CTAs an SM that go
// round, as registers have room for (the angles' frequencies are set up once a warp).
int qknorm_ctas(long long tokens) {
  const long long want = (tokens + kWarps - 1) / kWarps;
  return (int)(want < kPerSm * kSmCount ? want : kPerSm * kSmCount);
}

template <typename T, bool BWD>
cudaError_t run(QkP q, bool wide, cudaStream_t s) {
  const int by = 32 / lanes_of(q.d), turns = (q.H[0] + q.H[1] + by - 1) / by;
  q.per = (turns + heads_at_once<T, BWD>() - 1) / heads_at_once<T, BWD>();
  q.at_once = (turns + q.per - 1) / q.per;
  const dim3 grid(qknorm_ctas(q.tokens)), block(32 * kWarps);
  if (q.d <= 64)
    wide ? qknorm_kernel<T, 8, true, BWD><<<grid, block, 0, s>>>(q) : qknorm_kernel<T, 8, false, BWD><<<grid, block, 0, s>>>(q);
  else if (q.d <= 128)
    wide ? qknorm_kernel<T, 16, true, BWD><<<grid, block, 0, s>>>(q) : qknorm_kernel<T, 16, false, BWD><<<grid, block, 0, s>>>(q);
  else
    wide ? qknorm_kernel<T, 32, true, BWD><<<grid, block, 0, s>>>(q) : qknorm_kernel<T, 32, false, BWD><<<grid, block, 0, s>>>(q);
  return cudaGetLastError();
}

template <typename Args>
QkP fill(const Args& a) {
  QkP q = {};
  q.x[0] = a.q;
  q.x[1] = a.k;
  q.w[0] = a.q_weight;
  q.w[1] = a.k_weight;
  q.freqs = a.freqs;
  q.positions = a.positions;
  q.x_ld[0] = a.q_token ? a.q_token : (long long)a.Hq * a.d;
  q.x_ld[1] = a.k_token ? a.k_token : (long long)a.Hk * a.d;
  q.tokens = (long long)a.B * a.L;
  q.L = a.L;
  q.H[0] = a.Hq;
  q.H[1] = a.Hk;
  q.d = a.d;
  q.rp = a.rot / 8;
  q.interleaved = a.interleaved;
  q.inv_n = a.norm == LION_QKNORM_L2 ? 1.f : 1.f / a.d;
  q.eps = a.eps;
  return q;
}

// Whether all runs of four values lie on their size (heads do, as d is a multiple of 8).
bool on4(const void* p, long long ld, int es) {
  return reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && ld % 4 == 0;
}

}  // namespace

cudaError_t launch_qknorm_fwd(const lion_qknorm_args& a, cudaStream_t s) {
  QkP q = fill(a);
  q.y[0] = a.q_out;
  q.y[1] = a.k_out;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  const bool wide = on4(a.q, q.x_ld[0], es) && on4(a.k, q.x_ld[1], es) && on4(a.q_out, 0, es) && on4(a.k_out, 0, es);
  return a.dtype == DT_BF16 ? run<__nv_bfloat16, false>(q, wide, s) : run<float, false>(q, wide, s);
}

size_t qknorm_bwd_workspace_bytes(int B, int L, int, int, int d) {
  return sizeof(float) * 2 * d * (size_t)qknorm_ctas((long long)B * L);
}

cudaError_t launch_qknorm_bwd(const lion_qknorm_bwd_args& a, void* ws, cudaStream_t s) {
  QkP q = fill(a);
  q.dy[0] = a.dq_out;
  q.dy[1] = a.dk_out;
  q.y[0] = a.dq;
  q.y[1] = a.dk;
  q.part = static_cast<float*>(ws);
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  const bool wide = on4(a.q, q.x_ld[0], es) && on4(a.k, q.x_ld[1], es) && on4(a.dq, 0, es) && on4(a.dk, 0, es) &&
                    on4(a.dq_out, 0, es) && on4(a.dk_out, 0, es);
  const cudaError_t e = a.dtype == DT_BF16 ? run<__nv_bfloat16, true>(q, wide, s) : run<float, true>(q, wide, s);
  if (e != cudaSuccess || !ws) return e;
  const int ctas = qknorm_ctas(q.tokens);
  return launch_sum_parts(q.part, ctas, 2LL * a.d, a.d, a.dq_weight, a.d, a.dk_weight, 0, nullptr, s);
}

}  // namespace lion
