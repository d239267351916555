// ssm_scan_fwd.cu -- the selective scan, forward, and its one-token step.
#include "ssm_scan.cuh"

namespace lion {
namespace {

template <typename T, int LN, int W>
struct FwdSmem {
  using S = ScanTile<LN, W>;
  float4 dt[S::TT * S::SLOT];       // {delta, delta, delta u, delta u}
  float y[S::TT * S::SLOT];
  float Bm[S::TT * S::N];
  float Cm[S::TT * S::N];
};

// The state that enters the CTA's segment from the ones before it (h0 before the first).
template <int LN, int W>
__device__ __forceinline__ void enter_segment(const ScanP& p, const ScanAt& w, const int (&d)[2], const bool (&live)[2],
                                              int n0, const f2 (&A)[2][2], f2 (&h)[2][2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    load_pair(p.h0 + ((size_t)w.b * p.D + d[k]) * p.N + n0, live[k] && p.h0, h[k]);
#pragma unroll 4
    for (int s = 0; s < w.seg; ++s) {
      const size_t at = ((size_t)w.b * p.nseg + s) * p.D + d[k];
      f2 own[2];
      load_pair(p.seg_state + at * p.N + n0, live[k], own);
      const float sum = live[k] ? p.seg_sum[at] : 0.f;
      const f2 s2 = pack2(sum, sum);
#pragma unroll
      for (int q = 0; q < 2; ++q) h[k][q] = fma2(ex2_2(mul2(s2, A[k][q])), h[k][q], own[q]);
    }
  }
}

// MAIN: outputs, states, final state.  Otherwise: a segment's own
// contribution to the state that leaves it, from a zero state, and its sum of
// delta.
template <typename T, int LN, int W, bool MAIN>
__global__ void __launch_bounds__(32 * W) scan_fwd_kernel(ScanP p) {
  using S = ScanTile<LN, W>;
  constexpr int N = S::N, LC = S::LC, TT = S::TT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  FwdSmem<T, LN, W>& sm = *reinterpret_cast<FwdSmem<T, LN, W>*>(smem_raw);
  const ScanAt w = scan_at(p, S::CB);
  if (!MAIN && w.seg == p.nseg - 1) return;   // nothing comes after it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // element role
  const int vt = tid / S::VPT, vc = 8 * (tid % S::VPT), vd = w.d0 + vc, vn = min(8, w.nch - vc);
  // recurrence role
  const int ln = lane % LN, cl = warp * S::CW + lane / LN;
  const int d[2] = {w.d0 + cl, w.d0 + cl + LC};
  const bool live[2] = {cl < w.nch, cl + LC < w.nch};
  f2 A[2][2], h[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    load_pair(p.A + (size_t)d[k] * N + 4 * ln, live[k], A[k], kLog2e);
    h[k][0] = h[k][1] = pack2(0.f, 0.f);
  }
  if (MAIN) enter_segment<LN, W>(p, w, d, live, 4 * ln, A, h);
  float total[8], skip[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    total[e] = 0.f;
    skip[e] = MAIN && p.Dskip && e < vn ? p.Dskip[vd + e] : 0.f;
  }

  for (int i0 = w.i0; i0 < w.i1; i0 += TT) {
    const int i = i0 + vt;
    if (MAIN && p.states) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (live[k]) store_pair(p.states + (((size_t)w.b * p.nst + i0 / TT) * p.D + d[k]) * N + 4 * ln, h[k]);
    }
    const bool real = i >= w.v0 && i < w.v1 && i < w.i1;
    const long long row = (long long)w.b * p.L + token_of(p, i);
    const bool some = i0 + TT > w.v0 && i0 < w.v1;   // the tile has a token
    float u[8], z[8];
    if (some) {
      float dt[8], raw[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = dt[e] = z[e] = 0.f;
      if (real && vn > 0) {
        load8(static_cast<const T*>(p.u) + row * p.u_ld + vd, vn, p.u_wide, u);
        load8(static_cast<const T*>(p.dt) + row * p.dt_ld + vd, vn, p.dt_wide, dt);
        if (MAIN && p.z) load8(static_cast<const T*>(p.z) + row * p.z_ld + vd, vn, p.z_wide, z);
        deltas(p, vd, vn, dt, raw);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float du = dt[e] * u[e];
        sm.dt[vt * S::SLOT + slot_of(vc + e)] = make_float4(dt[e], dt[e], du, du);
        total[e] += dt[e];
      }
      load_bc<T, N, TT, S::NT>(p, w, p.Bm, p.b_ld, i0, sm.Bm);
      if (MAIN) load_bc<T, N, TT, S::NT>(p, w, p.Cm, p.c_ld, i0, sm.Cm);
      __syncthreads();
      constexpr int TG = LN / 2;   // tokens whose sums over the states are taken together
#pragma unroll 2
      for (int t0 = 0; t0 < TT; t0 += TG) {
        float v[LN];
#pragma unroll
        for (int t = 0; t < TG; ++t) {
          const float4 b4 = *reinterpret_cast<const float4*>(sm.Bm + (t0 + t) * N + 4 * ln);
          const f2 Bt[2] = {pack2(b4.x, b4.y), pack2(b4.z, b4.w)};
          f2 Ct[2];
          if (MAIN) {
            const float4 c4 = *reinterpret_cast<const float4*>(sm.Cm + (t0 + t) * N + 4 * ln);
            Ct[0] = pack2(c4.x, c4.y);
            Ct[1] = pack2(c4.z, c4.w);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 q4 = sm.dt[(t0 + t) * S::SLOT + slot_of(cl + k * LC)];
            const f2 dt2 = pack2(q4.x, q4.y), du2 = pack2(q4.z, q4.w);
            f2 y;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              h[k][q] = fma2(ex2_2(mul2(dt2, A[k][q])), h[k][q], mul2(du2, Bt[q]));
              if (MAIN) y = q == 0 ? mul2(Ct[0], h[k][0]) : fma2(Ct[q], h[k][q], y);
            }
            if (MAIN) v[2 * t + k] = sum2(y);
          }
        }
        if (MAIN) {
          const float y = sum_states<LN>(v, ln);
          sm.y[(t0 + (ln >> 1)) * S::SLOT + slot_of(cl + (ln & 1) * LC)] = y;
        }
      }
      __syncthreads();
    }
    if (MAIN && p.out && i < w.i1 && vn > 0) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = 0.f;
        if (real) {
          o[e] = fmaf(skip[e], u[e], sm.y[vt * S::SLOT + slot_of(vc + e)]);
          if (p.z) o[e] *= z[e] * sigmoid(z[e]);
        }
      }
      store8(static_cast<T*>(p.out) + row * p.D + vd, vn, p.o_wide, o);
    }
  }

  if (MAIN) {
    if (p.h_out && w.seg == p.nseg - 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (live[k]) store_pair(p.h_out + ((size_t)w.b * p.D + d[k]) * N + 4 * ln, h[k]);
    }
  } else {
    const size_t at = ((size_t)w.b * p.nseg + w.seg) * p.D;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (live[k]) store_pair(p.seg_state + (at + d[k]) * N + 4 * ln, h[k]);
    // the threads of a channel vector add up their tokens' delta
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sm.y[vt * S::SLOT + slot_of(vc + e)] = total[e];
    __syncthreads();
    for (int c = tid; c < w.nch; c += S::NT) {
      float s = 0.f;
#pragma unroll 8
      for (int t = 0; t < TT; ++t) s += sm.y[t * S::SLOT + slot_of(c)];
      p.seg_sum[at + w.d0 + c] = s;
    }
  }
}

constexpr int kFwdWarps = 4;

template <typename T, int LN, bool MAIN>
cudaError_t run_kernel(const ScanP& p, cudaStream_t s) {
  using S = ScanTile<LN, kFwdWarps>;
  auto kern = scan_fwd_kernel<T, LN, kFwdWarps, MAIN>;
  const size_t smem = sizeof(FwdSmem<T, LN, kFwdWarps>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.nblk * p.G * p.nseg * p.B, S::NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int LN>
cudaError_t run_fwd(const ScanP& p, cudaStream_t s) {
  if (p.nseg > 1) {
    cudaError_t e = run_kernel<T, LN, false>(p, s);
    if (e != cudaSuccess) return e;
  }
  return run_kernel<T, LN, true>(p, s);
}

// One token: a thread holds four states of a channel; bound by the states'
// traffic, read and written once, 16 bytes a thread.
template <typename T, int LN>
__global__ void __launch_bounds__(128) scan_step_kernel(lion_scan_step_args a) {
  constexpr int N = 4 * LN;
  const long long item = (long long)blockIdx.x * 128 + threadIdx.x;
  const int ln = (int)(item % LN);
  const long long ch = item / LN;   // b * D + d
  const bool live = ch < (long long)a.B * a.D;
  float y = 0.f, u = 0.f;
  int b = 0, d = 0;
  if (live) {
    b = (int)(ch / a.D);
    d = (int)(ch - (long long)b * a.D);
    const float4 A = *reinterpret_cast<const float4*>(a.A + (size_t)d * N + 4 * ln);
    float4* hp = reinterpret_cast<float4*>(a.h + (size_t)ch * N + 4 * ln);
    float4 h = *hp;
    u = to_f32(static_cast<const T*>(a.u)[ch]);
    float dt = to_f32(static_cast<const T*>(a.dt)[ch]);
    if (a.dt_bias) dt += a.dt_bias[d];
    if (a.dt_softplus) dt = softplus(dt);
    const size_t bc = ((size_t)b * a.G + d / (a.D / a.G)) * N + 4 * ln;
    const T* Bp = static_cast<const T*>(a.Bm) + bc;
    const T* Cp = static_cast<const T*>(a.Cm) + bc;
    const float du = dt * u, s = dt * kLog2e;
    h.x = fmaf(ex2(s * A.x), h.x, du * to_f32(Bp[0]));
    h.y = fmaf(ex2(s * A.y), h.y, du * to_f32(Bp[1]));
    h.z = fmaf(ex2(s * A.z), h.z, du * to_f32(Bp[2]));
    h.w = fmaf(ex2(s * A.w), h.w, du * to_f32(Bp[3]));
    *hp = h;
    y = fmaf(to_f32(Cp[0]), h.x, fmaf(to_f32(Cp[1]), h.y, fmaf(to_f32(Cp[2]), h.z, to_f32(Cp[3]) * h.w)));
  }
#pragma unroll
  for (int o = LN / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (live && ln == 0) {
    if (a.Dskip) y = fmaf(a.Dskip[d], u, y);
    if (a.z) {
      const float z = to_f32(static_cast<const T*>(a.z)[ch]);
      y *= z * sigmoid(z);
    }
    static_cast<T*>(a.out)[ch] = from_f32<T>(y);
  }
}

template <typename T, int LN>
cudaError_t run_step(const lion_scan_step_args& a, cudaStream_t s) {
  const long long n = (long long)a.B * a.D * LN;
  scan_step_kernel<T, LN><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// A sequence is cut into segments only while its channels alone leave the SMs
// short of CTAs: each cut costs a second pass over the exponentials.
ScanPlan scan_plan(int B, int L, int D, int N, int G, int W) {
  ScanPlan r;
  const int cb = scan_channels(N, W);
  r.nblk = (D / G + cb - 1) / cb;
  const long long ctas = (long long)B * G * r.nblk;
  const long long want = kSmCount * (16 / W);
  long long nseg = ctas >= want / 2 ? 1 : (want + ctas - 1) / ctas;
  const long long most = L / 128 > 1 ? L / 128 : 1;
  if (nseg > most) nseg = most;
  long long len = (L + nseg - 1) / nseg;
  len = (len + 63) / 64 * 64;   // whole tiles
  r.seglen = (int)len;
  r.nseg = (int)((L + len - 1) / len);
  return r;
}

size_t scan_workspace_bytes(int B, int L, int D, int N, int G) {
  const ScanPlan r = scan_plan(B, L, D, N, G, kFwdWarps);
  if (r.nseg == 1) return 0;
  return up256(sizeof(float) * (size_t)B * r.nseg * D * N) + up256(sizeof(float) * (size_t)B * r.nseg * D);
}

void fill_scan(ScanP& p, const lion_scan_args& a) {
  p.u = a.u;
  p.dt = a.dt;
  p.z = a.z;
  p.Bm = a.Bm;
  p.Cm = a.Cm;
  p.A = a.A;
  p.Dskip = a.Dskip;
  p.dt_bias = a.dt_bias;
  p.h0 = a.h0;
  p.lengths = a.lengths;
  p.out = a.out;
  p.h_out = a.h_out;
  p.states = a.states;
  p.B = a.B;
  p.L = a.L;
  p.D = a.D;
  p.N = a.N;
  p.G = a.G;
  p.Dg = a.D / a.G;
  p.u_ld = a.u_token ? a.u_token : a.D;
  p.dt_ld = a.dt_token ? a.dt_token : a.D;
  p.z_ld = a.z_token ? a.z_token : a.D;
  p.b_ld = a.b_token ? a.b_token : (long long)a.G * a.N;
  p.c_ld = a.c_token ? a.c_token : (long long)a.G * a.N;
  p.softplus = a.dt_softplus;
  p.reverse = a.reverse;
  p.nst = (a.L + a.N - 1) / a.N;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  const bool whole = a.G == 1 || p.Dg * es % 16 == 0;   // a group's first channel keeps the alignment
  p.u_wide = whole && rows_wide(a.u, p.u_ld, es);
  p.dt_wide = whole && rows_wide(a.dt, p.dt_ld, es);
  p.z_wide = whole && rows_wide(a.z, p.z_ld, es);
  p.o_wide = whole && rows_wide(a.out, a.D, es);
}

cudaError_t launch_scan_fwd(const lion_scan_args& a, void* ws, cudaStream_t s) {
  ScanP p = {};
  fill_scan(p, a);
  const ScanPlan r = scan_plan(a.B, a.L, a.D, a.N, a.G, kFwdWarps);
  p.nblk = r.nblk;
  p.nseg = r.nseg;
  p.seglen = r.seglen;
  p.seg_state = static_cast<float*>(ws);
  p.seg_sum = reinterpret_cast<float*>(static_cast<char*>(ws) + up256(sizeof(float) * (size_t)a.B * r.nseg * a.D * a.N));
  return LION_SCAN_DISPATCH(run_fwd, a.dtype, a.N, p, s);
}

cudaError_t launch_scan_step(const lion_scan_step_args& a, cudaStream_t s) {
  return LION_SCAN_DISPATCH(run_step, a.dtype, a.N, a, s);
}

}  // namespace lion
