// ssm_scan_bwd.cu -- gradients of the selective scan.
//
// With G_i the gradient of h_i and g_i = a_i G_i what it passes on,
//   G_i = C_i dy_i + g_{i+1},   q = g_i h_{i-1}
//   dA = sum q delta,  ddelta = sum_n q A + u sum_n G B,  du = Dskip dy + delta sum_n G B
//   dB = sum_c G delta u,  dC = sum_c dy h,  dh0 = g_0.
// The walk runs against the forward's order.  A tile starts from the state
// before its first token; its states are computed forwards eight tokens at a
// time and stay in registers, with the decays, for the way back.
#include "ssm_scan.cuh"

namespace lion {
namespace {

// A row of partial sums, dA then dDskip then ddt_bias, its start on 16 bytes.
__host__ __device__ inline size_t par_stride(int D, int N) { return ((size_t)D * (N + 2) + 3) / 4 * 4; }

constexpr int kSub = 8;   // tokens whose states and decays are held in registers

template <int LN, int W>
struct BwdSmem {
  using S = ScanTile<LN, W>;
  float4 dt[S::TT * S::SLOT];        // {delta, delta, delta u, delta u}
  float2 dy[S::TT * S::SLOT];        // {dy, dy}
  float gb[S::TT * S::SLOT];         // sum_n G B
  float qa[S::TT * S::SLOT];         // sum_n q A (A scaled by log2 e)
  float y[S::TT * S::SLOT];          // sum_n C h
  float Bm[S::TT * S::N];
  float Cm[S::TT * S::N];
  float hs[(S::TT / kSub) * 8 * S::NT];       // states at the sub-blocks' starts, a thread's own
  float red[W * kSub * 2 * S::N];             // dB, dC of a sub-block, one part a warp
};

// A segment's own contribution to what it passes back, and its sum of delta.
template <typename T, int LN, int W>
__global__ void __launch_bounds__(32 * W) scan_bwd_segment_kernel(ScanP p) {
  using S = ScanTile<LN, W>;
  constexpr int N = S::N, LC = S::LC, TT = S::TT;
  __shared__ float2 sdt[TT * S::SLOT];   // {delta, dy}
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float* sC = reinterpret_cast<float*>(smem_raw);
  const ScanAt w = scan_at(p, S::CB);
  if (w.seg == 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int vt = tid / S::VPT, vc = 8 * (tid % S::VPT), vd = w.d0 + vc, vn = min(8, w.nch - vc);
  const int ln = lane % LN, cl = warp * S::CW + lane / LN;
  const int d[2] = {w.d0 + cl, w.d0 + cl + LC};
  const bool live[2] = {cl < w.nch, cl + LC < w.nch};
  f2 A[2][2], g[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    load_pair(p.A + (size_t)d[k] * N + 4 * ln, live[k], A[k], kLog2e);
    g[k][0] = g[k][1] = pack2(0.f, 0.f);
  }
  float total[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) total[e] = 0.f;
  for (int i0 = w.i0 + (w.i1 - w.i0 - 1) / TT * TT; i0 >= w.i0; i0 -= TT) {
    if (i0 + TT <= w.v0 || i0 >= w.v1) continue;
    const int i = i0 + vt;
    const bool real = i >= w.v0 && i < w.v1 && i < w.i1 && vn > 0;
    const long long row = (long long)w.b * p.L + token_of(p, i);
    float dt[8], raw[8], dy[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dt[e] = dy[e] = 0.f;
    if (real) {
      load8(static_cast<const T*>(p.dt) + row * p.dt_ld + vd, vn, p.dt_wide, dt);
      load8(static_cast<const T*>(p.dout) + row * p.D + vd, vn, p.d_wide, dy);
      if (p.z) {
        float z[8];
        load8(static_cast<const T*>(p.z) + row * p.z_ld + vd, vn, p.z_wide, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) dy[e] *= z[e] * sigmoid(z[e]);
      }
      deltas(p, vd, vn, dt, raw);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sdt[vt * S::SLOT + slot_of(vc + e)] = make_float2(dt[e], dy[e]);
      total[e] += dt[e];
    }
    load_bc<T, N, TT, S::NT>(p, w, p.Cm, p.c_ld, i0, sC);
    __syncthreads();
#pragma unroll 4
    for (int t = TT - 1; t >= 0; --t) {
      const float4 c4 = *reinterpret_cast<const float4*>(sC + t * N + 4 * ln);
      const f2 Ct[2] = {pack2(c4.x, c4.y), pack2(c4.z, c4.w)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x = sdt[t * S::SLOT + slot_of(cl + k * LC)];
        const f2 dt2 = pack2(x.x, x.x), dy2 = pack2(x.y, x.y);
#pragma unroll
        for (int q = 0; q < 2; ++q) g[k][q] = mul2(ex2_2(mul2(dt2, A[k][q])), fma2(Ct[q], dy2, g[k][q]));
      }
    }
    __syncthreads();
  }
  const size_t at = ((size_t)w.b * p.nseg + w.seg) * p.D;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (live[k]) store_pair(p.seg_state + (at + d[k]) * N + 4 * ln, g[k]);
#pragma unroll
  for (int e = 0; e < 8; ++e) sdt[vt * S::SLOT + slot_of(vc + e)].x = total[e];
  __syncthreads();
  for (int c = tid; c < w.nch; c += S::NT) {
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < TT; ++t) s += sdt[t * S::SLOT + slot_of(c)].x;
    p.seg_sum[at + w.d0 + c] = s;
  }
}

template <typename T, int LN, int W>
__global__ void __launch_bounds__(32 * W) scan_bwd_kernel(ScanP p) {
  using S = ScanTile<LN, W>;
  constexpr int N = S::N, LC = S::LC, TT = S::TT, NT = S::NT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<LN, W>& sm = *reinterpret_cast<BwdSmem<LN, W>*>(smem_raw);
  const ScanAt w = scan_at(p, S::CB);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int vt = tid / S::VPT, vc = 8 * (tid % S::VPT), vd = w.d0 + vc, vn = min(8, w.nch - vc);
  const int ln = lane % LN, lc = lane / LN, cl = warp * S::CW + lc;
  const int d[2] = {w.d0 + cl, w.d0 + cl + LC};
  const bool live[2] = {cl < w.nch, cl + LC < w.nch};
  f2 A[2][2], g[2][2], dA[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    load_pair(p.A + (size_t)d[k] * N + 4 * ln, live[k], A[k], kLog2e);
    dA[k][0] = dA[k][1] = pack2(0.f, 0.f);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)   // what the segments after this one pass back into it
    load_pair(p.seg_state + (((size_t)w.b * p.nseg + w.seg) * p.D + d[k]) * N + 4 * ln, live[k] && p.nseg > 1, g[k]);
  float skip[8], dskip[8], dbias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    skip[e] = p.Dskip && e < vn ? p.Dskip[vd + e] : 0.f;
    dskip[e] = dbias[e] = 0.f;
  }

  for (int i0 = w.i0 + (w.i1 - w.i0 - 1) / TT * TT; i0 >= w.i0; i0 -= TT) {
    const int i = i0 + vt;
    const bool real = i >= w.v0 && i < w.v1 && i < w.i1 && vn > 0;
    const bool some = i0 + TT > w.v0 && i0 < w.v1;
    const long long row = (long long)w.b * p.L + token_of(p, i);
    float u[8], dt[8], raw[8], z[8], dout[8], dy[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = dt[e] = raw[e] = z[e] = dout[e] = dy[e] = 0.f;
    if (some) {
      if (real) {
        load8(static_cast<const T*>(p.u) + row * p.u_ld + vd, vn, p.u_wide, u);
        load8(static_cast<const T*>(p.dt) + row * p.dt_ld + vd, vn, p.dt_wide, dt);
        load8(static_cast<const T*>(p.dout) + row * p.D + vd, vn, p.d_wide, dout);
        if (p.z) load8(static_cast<const T*>(p.z) + row * p.z_ld + vd, vn, p.z_wide, z);
        deltas(p, vd, vn, dt, raw);
#pragma unroll
        for (int e = 0; e < 8; ++e) dy[e] = p.z ? dout[e] * z[e] * sigmoid(z[e]) : dout[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float du = dt[e] * u[e];
        sm.dt[vt * S::SLOT + slot_of(vc + e)] = make_float4(dt[e], dt[e], du, du);
        sm.dy[vt * S::SLOT + slot_of(vc + e)] = make_float2(dy[e], dy[e]);
      }
      load_bc<T, N, TT, NT>(p, w, p.Bm, p.b_ld, i0, sm.Bm);
      load_bc<T, N, TT, NT>(p, w, p.Cm, p.c_ld, i0, sm.Cm);
      f2 h0[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        load_pair(p.states + (((size_t)w.b * p.nst + i0 / TT) * p.D + d[k]) * N + 4 * ln, live[k], h0[k]);
      __syncthreads();
      // the states at the sub-blocks' starts
      for (int sb = 0; sb < TT / kSub; ++sb) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 x = unpack2(h0[k][q]);
            sm.hs[((sb * 2 + k) * 2 + q) * 2 * NT + tid] = x.x;
            sm.hs[(((sb * 2 + k) * 2 + q) * 2 + 1) * NT + tid] = x.y;
          }
        if (sb == TT / kSub - 1) break;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
          const int at = sb * kSub + t;
          const float4 b4 = *reinterpret_cast<const float4*>(sm.Bm + at * N + 4 * ln);
          const f2 Bt[2] = {pack2(b4.x, b4.y), pack2(b4.z, b4.w)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 q4 = sm.dt[at * S::SLOT + slot_of(cl + k * LC)];
            const f2 dt2 = pack2(q4.x, q4.y), du2 = pack2(q4.z, q4.w);
#pragma unroll
            for (int q = 0; q < 2; ++q)
              h0[k][q] = fma2(ex2_2(mul2(dt2, A[k][q])), h0[k][q], mul2(du2, Bt[q]));
          }
        }
      }
      for (int sb = TT / kSub - 1; sb >= 0; --sb) {
        f2 a[kSub][2][2], h[kSub + 1][2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            h[0][k][q] = pack2(sm.hs[((sb * 2 + k) * 2 + q) * 2 * NT + tid],
                               sm.hs[(((sb * 2 + k) * 2 + q) * 2 + 1) * NT + tid]);
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
          const int at = sb * kSub + t;
          const float4 b4 = *reinterpret_cast<const float4*>(sm.Bm + at * N + 4 * ln);
          const f2 Bt[2] = {pack2(b4.x, b4.y), pack2(b4.z, b4.w)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 q4 = sm.dt[at * S::SLOT + slot_of(cl + k * LC)];
            const f2 dt2 = pack2(q4.x, q4.y), du2 = pack2(q4.z, q4.w);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              a[t][k][q] = ex2_2(mul2(dt2, A[k][q]));
              h[t + 1][k][q] = fma2(a[t][k][q], h[t][k][q], mul2(du2, Bt[q]));
            }
          }
        }
#pragma unroll
        for (int t = kSub - 1; t >= 0; --t) {
          const int at = sb * kSub + t;
          const float4 b4 = *reinterpret_cast<const float4*>(sm.Bm + at * N + 4 * ln);
          const float4 c4 = *reinterpret_cast<const float4*>(sm.Cm + at * N + 4 * ln);
          const f2 Bt[2] = {pack2(b4.x, b4.y), pack2(b4.z, b4.w)};
          const f2 Ct[2] = {pack2(c4.x, c4.y), pack2(c4.z, c4.w)};
          f2 dB[2], dC[2];
          float gb[2], qa[2], y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 q4 = sm.dt[at * S::SLOT + slot_of(cl + k * LC)];
            const f2 dt2 = pack2(q4.x, q4.y), du2 = pack2(q4.z, q4.w);
            const float2 y2 = sm.dy[at * S::SLOT + slot_of(cl + k * LC)];
            const f2 dy2 = pack2(y2.x, y2.y);
            f2 sgb, sqa, sy;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const f2 G = fma2(Ct[q], dy2, g[k][q]);
              dC[q] = k == 0 ? mul2(dy2, h[t + 1][k][q]) : fma2(dy2, h[t + 1][k][q], dC[q]);
              dB[q] = k == 0 ? mul2(du2, G) : fma2(du2, G, dB[q]);
              sgb = q == 0 ? mul2(G, Bt[q]) : fma2(G, Bt[q], sgb);
              sy = q == 0 ? mul2(Ct[q], h[t + 1][k][q]) : fma2(Ct[q], h[t + 1][k][q], sy);
              g[k][q] = mul2(G, a[t][k][q]);
              const f2 e = mul2(g[k][q], h[t][k][q]);
              dA[k][q] = fma2(e, dt2, dA[k][q]);
              sqa = q == 0 ? mul2(e, A[k][q]) : fma2(e, A[k][q], sqa);
            }
            gb[k] = sum2(sgb);
            qa[k] = sum2(sqa);
            y[k] = sum2(sy);
          }
          // over the states: every lane of a channel gets the sums
#pragma unroll
          for (int o = 1; o < LN; o <<= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              gb[k] += __shfl_xor_sync(0xffffffffu, gb[k], o);
              qa[k] += __shfl_xor_sync(0xffffffffu, qa[k], o);
              y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
            }
          if (ln < 2) {
            const int at_c = at * S::SLOT + slot_of(cl + ln * LC);
            sm.gb[at_c] = ln ? gb[1] : gb[0];
            sm.qa[at_c] = ln ? qa[1] : qa[0];
            sm.y[at_c] = ln ? y[1] : y[0];
          }
          // over the channels: lanes LN apart
          float r[8];
          const float2 b0 = unpack2(dB[0]), b1 = unpack2(dB[1]), c0 = unpack2(dC[0]), c1 = unpack2(dC[1]);
          r[0] = b0.x; r[1] = b0.y; r[2] = b1.x; r[3] = b1.y;
          r[4] = c0.x; r[5] = c0.y; r[6] = c1.x; r[7] = c1.y;
          int first = 0;   // which of the eight sums this lane ends with
          int count = 8;
#pragma unroll
          for (int o = LN; o < 32; o <<= 1) {
            if (count > 1) {
              const bool up = lane & o;
              count /= 2;
              if (up) first += count;
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (v < count) {
                  const float keep = up ? r[v + count] : r[v], send = up ? r[v] : r[v + count];
                  r[v] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            } else {
              r[0] += __shfl_xor_sync(0xffffffffu, r[0], o);
            }
          }
          float* red = sm.red + (warp * kSub + t) * 2 * N;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            if (v < count && (count > 1 || LC <= 8 || lane < 8 * LN)) {
              const int which = first + v;   // 0..3 dB, 4..7 dC of this lane's states
              red[(which >> 2) * N + 4 * ln + (which & 3)] = r[v];
            }
        }
        __syncthreads();
        // one part a CTA: the warps' sums in their order
        for (int k = tid; k < kSub * 2 * N; k += NT) {
          const int t = k / (2 * N), i_t = i0 + sb * kSub + t;
          if (i_t >= w.i1) continue;
          float s = 0.f;
#pragma unroll
          for (int v = 0; v < W; ++v) s += sm.red[(v * kSub + t) * 2 * N + k % (2 * N)];
          p.part_bc[((((size_t)w.blk * p.B + w.b) * p.L + token_of(p, i_t)) * p.G + w.g) * 2 * N + k % (2 * N)] = s;
        }
        __syncthreads();
      }
    }
    if (i < w.i1 && vn > 0) {
      float du[8], ddt[8], dz[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        du[e] = ddt[e] = dz[e] = 0.f;
        if (real) {
          const int at = vt * S::SLOT + slot_of(vc + e);
          const float gb = sm.gb[at];
          du[e] = fmaf(dt[e], gb, skip[e] * dy[e]);
          ddt[e] = fmaf(u[e], gb, kLn2 * sm.qa[at]);
          if (p.softplus) ddt[e] *= sigmoid(raw[e]);
          dskip[e] = fmaf(dy[e], u[e], dskip[e]);
          dbias[e] += ddt[e];
          if (p.z) {
            const float s = sigmoid(z[e]);
            dz[e] = dout[e] * fmaf(skip[e], u[e], sm.y[at]) * s * fmaf(z[e], 1.f - s, 1.f);
          }
        }
      }
      store8(static_cast<T*>(p.du) + row * p.D + vd, vn, p.o_wide, du);
      store8(static_cast<T*>(p.ddt) + row * p.D + vd, vn, p.o_wide, ddt);
      if (p.z) store8(static_cast<T*>(p.dz) + row * p.D + vd, vn, p.o_wide, dz);
    }
    if (some) __syncthreads();   // the sums are read before the next tile's are written
  }

  float* part = p.part_par + ((size_t)w.b * p.nseg + w.seg) * par_stride(p.D, N);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!live[k]) continue;
    store_pair(part + (size_t)d[k] * N + 4 * ln, dA[k]);
    if (p.dh0 && w.seg == 0) store_pair(p.dh0 + ((size_t)w.b * p.D + d[k]) * N + 4 * ln, g[k]);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sm.gb[vt * S::SLOT + slot_of(vc + e)] = dskip[e];
    sm.qa[vt * S::SLOT + slot_of(vc + e)] = dbias[e];
  }
  __syncthreads();
  for (int c = tid; c < w.nch; c += NT) {
    float s = 0.f, b = 0.f;
#pragma unroll 8
    for (int t = 0; t < TT; ++t) {
      s += sm.gb[t * S::SLOT + slot_of(c)];
      b += sm.qa[t * S::SLOT + slot_of(c)];
    }
    part[(size_t)p.D * N + w.d0 + c] = s;
    part[(size_t)p.D * (N + 1) + w.d0 + c] = b;
  }
}

// dB and dC: the channel blocks' parts in their order.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(ScanP p, T* dB, T* dC) {
  const long long n = (long long)p.B * p.L * p.G * 2 * p.N, k = (long long)blockIdx.x * 256 + threadIdx.x;
  if (k >= n) return;
  const int N2 = 2 * p.N, v = (int)(k % N2);
  const long long tok = k / N2 / p.G;   // b * L + t
  const int b = (int)(tok / p.L), t = (int)(tok - (long long)b * p.L);
  float s = 0.f;
  if (!p.lengths || t < p.lengths[b])
    for (int q = 0; q < p.nblk; ++q) s += p.part_bc[(size_t)q * n + k];
  (v < p.N ? dB : dC)[k / N2 * p.N + v % p.N] = from_f32<T>(s);
}

constexpr int kBwdWarps = 8;
template <int LN>
struct BwdW {
  static constexpr int W = kBwdWarps;
};

template <typename T, int N>
cudaError_t run_bwd(const ScanP& p, cudaStream_t s) {
  constexpr int LN = N / 4;
  constexpr int W = BwdW<LN>::W;
  using S = ScanTile<LN, W>;
  const unsigned ctas = (unsigned)p.nblk * p.G * p.nseg * p.B;
  if (p.nseg > 1) {
    auto seg = scan_bwd_segment_kernel<T, LN, W>;
    seg<<<ctas, S::NT, sizeof(float) * S::TT * S::N, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_scan_chain(p, true, nullptr, s);
    if (e != cudaSuccess) return e;
  }
  auto kern = scan_bwd_kernel<T, LN, W>;
  const size_t smem = sizeof(BwdSmem<LN, W>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<ctas, S::NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_bc(const ScanP& p, void* dB, void* dC, cudaStream_t s) {
  const long long n = (long long)p.B * p.L * p.G * 2 * p.N;
  scan_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, static_cast<T*>(dB), static_cast<T*>(dC));
  return cudaGetLastError();
}

// The workspace's parts: the forward's own, the states, the segments, the
// partial sums.
struct BwdPlan {
  ScanPlan r;
  size_t fwd, states, seg_state, seg_sum, bc, par, total;
};
BwdPlan bwd_plan(int B, int L, int D, int N, int G, bool have_states) {
  BwdPlan q;
  q.r = scan_plan(B, L, D, G, scan_channels(N, kBwdWarps), kBwdWarps, 8 * kSmCount, 32 * kSmCount);
  size_t at = 0;
  auto take = [&](size_t floats) {
    const size_t here = at;
    at += up256(sizeof(float) * floats);
    return here;
  };
  q.fwd = at;
  if (!have_states) at += up256(scan_workspace_bytes(B, L, D, N, G));
  q.states = take(have_states ? 0 : (size_t)B * ((L + N - 1) / N) * D * N);
  q.seg_state = take(q.r.nseg > 1 ? (size_t)B * q.r.nseg * D * N : 0);
  q.seg_sum = take(q.r.nseg > 1 ? (size_t)B * q.r.nseg * D : 0);
  q.bc = take((size_t)q.r.nblk * B * L * G * 2 * N);
  q.par = take((size_t)B * q.r.nseg * par_stride(D, N));
  q.total = at;
  return q;
}

}  // namespace

size_t scan_bwd_workspace_bytes(int B, int L, int D, int N, int G, bool have_states) {
  return bwd_plan(B, L, D, N, G, have_states).total;
}

cudaError_t launch_scan_bwd(const lion_scan_bwd_args& a, void* ws, cudaStream_t s) {
  const BwdPlan q = bwd_plan(a.B, a.L, a.D, a.N, a.G, a.states != nullptr);
  char* base = static_cast<char*>(ws);
  lion_scan_args f = {};
  f.u = a.u;
  f.dt = a.dt;
  f.A = a.A;
  f.Bm = a.Bm;
  f.Cm = a.Cm;
  f.Dskip = a.Dskip;
  f.dt_bias = a.dt_bias;
  f.h0 = a.h0;
  f.lengths = a.lengths;
  f.states = const_cast<float*>(a.states);
  f.u_token = a.u_token;
  f.dt_token = a.dt_token;
  f.z_token = a.z_token;
  f.b_token = a.b_token;
  f.c_token = a.c_token;
  f.B = a.B;
  f.L = a.L;
  f.D = a.D;
  f.N = a.N;
  f.G = a.G;
  f.dt_softplus = a.dt_softplus;
  f.reverse = a.reverse;
  f.dtype = a.dtype;
  if (!a.states) {
    f.states = reinterpret_cast<float*>(base + q.states);
    const cudaError_t e = launch_scan_fwd(f, base + q.fwd, s);
    if (e != cudaSuccess) return e;
  }
  f.z = a.z;
  ScanP p = {};
  fill_scan(p, f);
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  const bool whole = a.G == 1 || p.Dg * es % 16 == 0;
  p.dout = a.dout;
  p.d_wide = whole && rows_wide(a.dout, a.D, es);
  p.o_wide = whole && rows_wide(a.du, a.D, es) && rows_wide(a.ddt, a.D, es) && rows_wide(a.dz, a.D, es);
  p.du = a.du;
  p.ddt = a.ddt;
  p.dz = a.dz;
  p.dh0 = a.dh0;
  p.nblk = q.r.nblk;
  p.nseg = q.r.nseg;
  p.seglen = q.r.seglen;
  p.seg_state = reinterpret_cast<float*>(base + q.seg_state);
  p.seg_sum = reinterpret_cast<float*>(base + q.seg_sum);
  p.part_bc = reinterpret_cast<float*>(base + q.bc);
  p.part_par = reinterpret_cast<float*>(base + q.par);
  cudaError_t e = LION_SCAN_DISPATCH(run_bwd, a.dtype, a.N, p, s);
  if (e != cudaSuccess) return e;
  e = a.dtype == DT_BF16 ? run_bc<__nv_bfloat16>(p, a.dB, a.dC, s) : run_bc<float>(p, a.dB, a.dC, s);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(p.part_par, a.B * q.r.nseg, (long long)par_stride(a.D, a.N), (long long)a.D * a.N, a.dA, a.D, a.dDskip, a.D, a.ddt_bias, s);
}

}  // namespace lion
