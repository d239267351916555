// ssm_scan_fwd.cu -- the selective scan, forward, and its one-token step.
//
// A warp walks a segment of one sequence for its CW channels in tiles of TT
// tokens, alone: no barrier wider than the warp.  Raw inputs arrive in shared
// memory a tile ahead (asynchronous copies); the element lanes turn them into
// delta and delta u once; the recurrence lanes, 32 states each (all of a
// channel's up to 16, of as many channels as that allows), read those and B,
// C, and leave sum_n C h in delta's place for the element lanes, which gate and
// store.
//
// What bounds it: a token, channel and state costs one exponential (32 a clock
// and SM) and four fp32 operations (128 a clock and SM), which at N = 16 is more
// than the 8 bytes a token and channel of HBM traffic (2 x 24337 x 1536 x 16:
// 126 us of exponentials, 90 us of bytes).  With packed pairs a scheduler
// reaches about 45 clocks for the exponentials and products of 16 channels'
// token against 32 at the pipes' rates; loads, softplus, gate and stores add
// about 40.  Measured: 86 clocks, 330 us (14.5e12 operations a second with the
// segments' pass, 552 us; 1576 in the first form).  32 states a lane are what
// keeps shared memory from being the bound: a token costs a lane one read of
// delta and one of delta u for them, and B and C are broadcasts (four states of
// four channels a lane: 689 us, bound by shared-memory reads; of two: 865).
// More warps an SM than the 12 that 168 registers leave do not help, fewer
// hurt (8: 615 us).  float32's shared memory leaves 11 at N = 16 and 9 at N = 32.
//
// Few channels: the sequences are cut into segments.  A first launch takes each
// segment's own contribution to the state that leaves it (the same walk without
// C, gate and outputs), a small one chains them, and the main launch starts
// every segment from its state.  (A warp that only has the recurrence, four
// lanes a channel, with another one preparing its tiles and no segments, took
// 130 clocks a token, its latencies one after the other: 1711 us.)
#include <algorithm>

#include "ssm_scan.cuh"

namespace lion {
namespace {

constexpr int kFwdWarps = kScanFwdWarps;

template <typename T, int N_>
struct FwdTile {
  static constexpr int N = N_;
  static constexpr int RN = N < 16 ? N : 16;          // states of a channel in a lane
  static constexpr int LN = N / RN;                   // lanes of a channel
  static constexpr int RC = 32 / RN;                  // adjacent channels of a lane
  static constexpr int CW = 32 / LN * RC;             // channels of a warp
  static constexpr int TT = N == 64 ? 16 : 512 / CW;  // tokens of a tile
  static_assert(kFwdWarps * CW == scan_fwd_channels(N), "the plan cuts the channels alike");
  static constexpr int VT = CW / 4;                   // vectors of four channels: of a token,
  static constexpr int VL = TT * VT / 32;             // and of a lane, 32 / VT tokens apart
  static constexpr bool kConvert = sizeof(T) == 2;    // B and C: fp32 copies of raw bf16
};
template <typename T, int N_>
struct FwdWarp {
  using S = FwdTile<T, N_>;
  alignas(16) float dt[S::TT * S::CW];   // delta, then sum_n C h
  alignas(16) float du[S::TT * S::CW];   // delta u
  alignas(16) float Bf[S::kConvert ? S::TT * S::N : 4];
  alignas(16) float Cf[S::kConvert ? S::TT * S::N : 4];
  struct Raw {
    alignas(16) T u[S::TT * S::CW];
    alignas(16) T dt[S::TT * S::CW];
    alignas(16) T z[S::TT * S::CW];
    alignas(16) T Bm[S::TT * S::N];
    alignas(16) T Cm[S::TT * S::N];
  } raw[2];
};

// R adjacent floats.
template <int R>
__device__ __forceinline__ void get_some(const float* p, float (&v)[R]) {
  static_assert(R == 2 || R == 4, "");
  if (R == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[R - 2] = x.z; v[R - 1] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x; v[1] = x.y;
  }
}

// RN states of a channel (fp32, 16-byte aligned) as pairs.
template <int RN>
__device__ __forceinline__ void load_states(const float* src, bool there, f2 (&v)[RN / 2]) {
#pragma unroll
  for (int k = 0; k < RN / 4; ++k) {
    f2 x[2];
    load_pair(src + 4 * k, there, x);
    v[2 * k] = x[0];
    v[2 * k + 1] = x[1];
  }
}
template <int RN>
__device__ __forceinline__ void store_states(float* dst, const f2 (&v)[RN / 2]) {
#pragma unroll
  for (int k = 0; k < RN / 4; ++k) {
    const f2 x[2] = {v[2 * k], v[2 * k + 1]};
    store_pair(dst + 4 * k, x);
  }
}

// MAIN: outputs, states, final state.  Otherwise: a segment's own
// contribution to the state that leaves it, from a zero state, and its sum of
// delta.
template <typename T, int N, bool MAIN>
__global__ void __launch_bounds__(32 * kFwdWarps, (N == 64 ? 8 : 12) / kFwdWarps) scan_fwd_kernel(ScanP p) {
  using S = FwdTile<T, N>;
  typedef typename FwdWarp<T, N>::Raw Raw;
  constexpr int RN = S::RN, LN = S::LN, RC = S::RC, TT = S::TT, CW = S::CW, VT = S::VT, VL = S::VL;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  FwdWarp<T, N>& sm = reinterpret_cast<FwdWarp<T, N>*>(smem_raw)[warp];
  ScanAt w = scan_at(p, kFwdWarps * CW);
  w.d0 += warp * CW;
  w.nch = min(CW, w.nch - warp * CW);
  if (w.nch <= 0) return;
  if (!MAIN && w.seg == p.nseg - 1) return;   // nothing comes after it
  // element role: VL vectors of four channels, 32 / VT tokens apart
  const int vt = lane / VT, vc = lane % VT * 4, vd = w.d0 + vc, vn = min(4, w.nch - vc);
  // recurrence role: states n0 .. n0 + RN - 1 of RC adjacent channels; with two
  // lanes a channel the odd one holds them in the other order, so that the
  // first step of a sum over the states sends the same register from both
  const int ln = lane % LN, n0 = ln * RN, odd = RC == 2 ? ln & 1 : 0, c0 = lane / LN * RC;
  f2 A[RC][RN / 2], h[RC][RN / 2];
  const size_t state_at = (size_t)(w.d0 + c0) * N + n0;
  bool live[RC];
#pragma unroll
  for (int k = 0; k < RC; ++k) {
    live[k] = c0 + (k ^ odd) < w.nch;
    load_states<RN>(p.A + state_at + (k ^ odd) * N, live[k], A[k]);
#pragma unroll
    for (int q = 0; q < RN / 2; ++q) {
      A[k][q] = pack2(decay(A[k][q].x), decay(A[k][q].y));
      h[k][q] = pack2(0.f, 0.f);
    }
  }
  float total[4], bias[4], skip[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    total[e] = 0.f;
    bias[e] = p.dt_bias && e < vn ? p.dt_bias[vd + e] : 0.f;
    skip[e] = MAIN && p.Dskip && e < vn ? p.Dskip[vd + e] : 0.f;
  }
  const bool plain = w.nch == CW && p.o_wide &&
                     (p.u_align & p.dt_align & p.b_align & p.c_align & (p.z ? p.z_align : 16)) == 16;
  // the tiles that have tokens; MAIN visits the others to write zeros and states
  const int a0 = max(w.i0, w.v0 - w.v0 % TT), a1 = min(w.i1, w.v1), r0 = max(w.i0, w.v0);
  Feed<T, TT, CW> fu, fdt, fz;
  Feed<T, TT, N> fb, fc;
  fu.start(p.u, p.u_ld, w.d0, p, w, a0, lane, w.nch);
  fdt.start(p.dt, p.dt_ld, w.d0, p, w, a0, lane, w.nch);
  fz.start(p.z, p.z_ld, w.d0, p, w, a0, lane, w.nch);
  fb.start(p.Bm, p.b_ld, w.g * N, p, w, a0, lane, N);
  fc.start(p.Cm, p.c_ld, w.g * N, p, w, a0, lane, N);
  const int dir = p.reverse ? -TT : TT;
  auto fetch_tile = [&](Raw& to, int i0) {
    const int lo = r0 - i0, hi = a1 - i0;
    const bool whole = plain && lo <= 0 && hi >= TT;
    fu.next(to.u, lo, hi, lane, p.u_align, whole, dir * p.u_ld);
    fdt.next(to.dt, lo, hi, lane, p.dt_align, whole, dir * p.dt_ld);
    if (MAIN && p.z) fz.next(to.z, lo, hi, lane, p.z_align, whole, dir * p.z_ld);
    fb.next(to.Bm, lo, hi, lane, p.b_align, whole, dir * p.b_ld);
    if (MAIN) fc.next(to.Cm, lo, hi, lane, p.c_align, whole, dir * p.c_ld);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (a0 < a1) fetch_tile(sm.raw[0], a0);
  if (MAIN) {
    if (p.nseg > 1) wait_prior();
    const float* from = p.nseg > 1 ? p.seg_state + ((size_t)w.b * p.nseg + w.seg) * p.D * N
                        : p.h0     ? p.h0 + (size_t)w.b * p.D * N
                                   : nullptr;
#pragma unroll
    for (int k = 0; k < RC; ++k) load_states<RN>(from + state_at + (k ^ odd) * N, live[k] && from, h[k]);
  }
  T* out = nullptr;
  long long out_hop = 0;   // from a lane's vector to its next
  if (MAIN && p.out) {
    out = static_cast<T*>(p.out) + ((long long)w.b * p.L + token_of(p, w.i0 + vt)) * p.D + vd;
    out_hop = (long long)(p.reverse ? -(32 / VT) : 32 / VT) * p.D;
  }

  int stage = 0;
  for (int i0 = MAIN ? w.i0 : a0; i0 < (MAIN ? w.i1 : a1); i0 += TT) {
    if (MAIN && p.states && i0 % kStateEvery == 0) {
      float* to = p.states + ((size_t)w.b * p.nst + i0 / kStateEvery) * p.D * N + state_at;
#pragma unroll
      for (int k = 0; k < RC; ++k)
        if (live[k]) store_states<RN>(to + (k ^ odd) * N, h[k]);
    }
    const bool some = i0 >= a0 && i0 < a1;
    const bool whole = plain && i0 >= r0 && i0 + TT <= a1;   // every lane has full vectors of tokens
    Raw& raw = sm.raw[stage];
    if (some) {
      if (i0 + TT < a1) {
        fetch_tile(sm.raw[stage ^ 1], i0 + TT);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int at = (lane + 32 * j) * 4, i = i0 + vt + j * (32 / VT);
        float u[4], dt[4];
        get(raw.u + at, u);
        get(raw.dt + at, dt);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          f2 x = add2(pack2(dt[e], dt[e + 1]), pack2(bias[e], bias[e + 1]));
          if (p.softplus) {
            const float2 r = unpack2(x);
            x = softplus2(r.x, r.y);
          }
          if (!whole) {
            const bool real = i >= r0 && i < a1;
            x = pack2(real && e < vn ? unpack2(x).x : 0.f, real && e + 1 < vn ? unpack2(x).y : 0.f);
          }
          const float2 dl = unpack2(x), d2 = unpack2(mul2(x, pack2(u[e], u[e + 1])));
          dt[e] = dl.x; dt[e + 1] = dl.y;
          u[e] = d2.x; u[e + 1] = d2.y;
          if (!MAIN) {
            total[e] += dl.x;
            total[e + 1] += dl.y;
          }
        }
        *reinterpret_cast<float4*>(sm.dt + at) = make_float4(dt[0], dt[1], dt[2], dt[3]);
        *reinterpret_cast<float4*>(sm.du + at) = make_float4(u[0], u[1], u[2], u[3]);
      }
      const float* Bt = as_fp32<TT * N>(raw.Bm, sm.Bf, lane) + n0;
      const float* Ct = MAIN ? as_fp32<TT * N>(raw.Cm, sm.Cf, lane) + n0 : nullptr;
      __syncwarp();
#pragma unroll(TT < 8 ? TT : 8)
      for (int t = 0; t < TT; ++t) {
        float dt[RC], du[RC];
        get_some<RC>(sm.dt + t * CW + c0, dt);
        get_some<RC>(sm.du + t * CW + c0, du);
        if (RC == 2 && LN > 1) {   // the odd lane's order
          const float a = dt[0], b = du[0];
          dt[0] = odd ? dt[1] : a; dt[1] = odd ? a : dt[1];
          du[0] = odd ? du[1] : b; du[1] = odd ? b : du[1];
        }
        f2 y[RC];
#pragma unroll
        for (int n = 0; n < RN / 4; ++n) {
          const float4 b4 = *reinterpret_cast<const float4*>(Bt + t * N + 4 * n);
          const f2 b2[2] = {pack2(b4.x, b4.y), pack2(b4.z, b4.w)};
          f2 c2[2];
          if (MAIN) {
            const float4 c4 = *reinterpret_cast<const float4*>(Ct + t * N + 4 * n);
            c2[0] = pack2(c4.x, c4.y);
            c2[1] = pack2(c4.z, c4.w);
          }
#pragma unroll
          for (int k = 0; k < RC; ++k) {
            const f2 dt2 = pack2(dt[k], dt[k]), du2 = pack2(du[k], du[k]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              f2& s = h[k][2 * n + q];
              s = fma2(ex2_2(mul2(dt2, A[k][2 * n + q])), s, mul2(du2, b2[q]));
              if (MAIN) y[k] = n + q == 0 ? mul2(c2[q], s) : fma2(c2[q], s, y[k]);
            }
          }
        }
        if (MAIN) {
          float v[RC];
#pragma unroll
          for (int k = 0; k < RC; ++k) v[k] = sum2(y[k]);
          float* yo = sm.dt + t * CW + c0;
          if (LN > 1) {
            float r = v[0] + __shfl_xor_sync(0xffffffffu, v[1], 1);
#pragma unroll
            for (int o = 2; o < LN; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
            __syncwarp();   // the channel's lanes have read this delta; a shuffle orders no memory
            yo[odd] = r;    // lanes of one parity hold the same sum
          } else if (RC == 4) {
            *reinterpret_cast<float4*>(yo) = make_float4(v[0], v[1], v[RC - 2], v[RC - 1]);
          } else {
            *reinterpret_cast<float2*>(yo) = make_float2(v[0], v[1]);
          }
        }
      }
      __syncwarp();
    }
    if (MAIN && out) {
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int at = (lane + 32 * j) * 4, i = i0 + vt + j * (32 / VT);
        if (whole || (i < w.i1 && vn > 0)) {
          float o[4] = {0.f, 0.f, 0.f, 0.f};
          if (whole || (i >= r0 && i < a1)) {
            float u[4];
            get(raw.u + at, u);
            get(sm.dt + at, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(skip[e], u[e], o[e]);
            if (p.z) {
              float z[4];
              get(raw.z + at, z);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float2 g = unpack2(gate2(pack2(o[e], o[e + 1]), z[e], z[e + 1]));
                o[e] = g.x;
                o[e + 1] = g.y;
              }
            }
          }
          put(out, whole ? 4 : vn, whole || p.o_wide, o);
        }
        out += out_hop;
      }
    }
    if (some) {
      stage ^= 1;
      __syncwarp();   // this tile's raw inputs are read before the copies after next overwrite them
    }
  }

  if (MAIN) {
    if (p.h_out && w.seg == p.nseg - 1) {
      float* to = p.h_out + (size_t)w.b * p.D * N + state_at;
#pragma unroll
      for (int k = 0; k < RC; ++k)
        if (live[k]) store_states<RN>(to + (k ^ odd) * N, h[k]);
    }
  } else {
    const size_t at = ((size_t)w.b * p.nseg + w.seg) * p.D;
#pragma unroll
    for (int k = 0; k < RC; ++k)
      if (live[k]) store_states<RN>(p.seg_state + at * N + state_at + (k ^ odd) * N, h[k]);
    // a channel's delta: over the lanes that hold its tokens
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = VT; o < 32; o <<= 1) total[e] += __shfl_xor_sync(0xffffffffu, total[e], o);
      if (vt == 0 && e < vn) p.seg_sum[at + vd + e] = total[e];
    }
  }
}

template <typename T, int N, bool MAIN>
cudaError_t run_kernel(const ScanP& p, cudaStream_t s) {
  auto kern = scan_fwd_kernel<T, N, MAIN>;
  const size_t smem = sizeof(FwdWarp<T, N>) * kFwdWarps;
  static_assert(sizeof(FwdWarp<T, N>) * kFwdWarps <= 48 * 1024, "more shared memory has to be asked for");
  const dim3 grid((unsigned)p.nblk * p.G * p.nseg * p.B);
  if (MAIN && p.nseg > 1) return launch_dependent(kern, grid, dim3(32 * kFwdWarps), smem, s, p);   // of the chain
  kern<<<grid, 32 * kFwdWarps, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int N>
cudaError_t run_fwd(const ScanP& p, cudaStream_t s) {
  if (p.nseg > 1) {
    cudaError_t e = run_kernel<T, N, false>(p, s);
    if (e == cudaSuccess) e = launch_scan_chain(p, false, p.h0, s);
    if (e != cudaSuccess) return e;
  }
  return run_kernel<T, N, true>(p, s);
}

// One token: a thread holds four states of a channel for kStepRows sequences;
// bound by the states' traffic, read and written once, 16 bytes a thread and
// sequence with the rows' reads in flight together.  Of a channel's lanes the
// r-th takes what there is one of for row r: the step size and the gate.  256 x
// 2048 x 16, 67 MB of states: 10.3 us with them in L2, 18.7 from HBM (every lane
// taking both: 12.3 and 22; B and C value by value: 19.2; four rows, larger
// CTAs, or rows read ahead in a loop: no faster).
constexpr int kStepRows = 2;   // at most the lanes of a channel at N = 8

// Four values of B or C, in one read where they lie aligned.
__device__ __forceinline__ float4 four(const float* p, bool wide) {
  return wide ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ float4 four(const __nv_bfloat16* p, bool wide) {
  if (wide) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack_bf16(r.x), b = unpack_bf16(r.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
}

template <typename T, int N>
__global__ void __launch_bounds__(128) scan_step_kernel(lion_scan_step_args a, bool bc_wide) {
  constexpr int LN = N / 4;
  // a CTA has 128 / LN channels (their lanes' number, D N / 4, can pass 32 bits)
  const int lane = threadIdx.x & 31, ln = threadIdx.x % LN, d = (int)(blockIdx.x * (128 / LN) + threadIdx.x / LN);
  const bool live = d < a.D;
  const int b0 = blockIdx.y * kStepRows;
  float4* hp = reinterpret_cast<float4*>(a.h + ((size_t)b0 * a.D + d) * N) + ln;
  const size_t h_hop = (size_t)a.D * N / 4, bc_hop = (size_t)a.G * N;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f), h[kStepRows], Bv[kStepRows], Cv[kStepRows];
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) h[r] = Bv[r] = Cv[r] = A;
  float u = 0.f, dt = 0.f, z = 0.f, skip = 0.f;
  const bool mine = live && ln < kStepRows && b0 + ln < a.B;
  const size_t ch = (size_t)(b0 + ln) * a.D + d;
  if (live) {
    const size_t bc = ((size_t)b0 * a.G + d / (a.D / a.G)) * N + 4 * ln;
#pragma unroll
    for (int r = 0; r < kStepRows; ++r)
      if (b0 + r < a.B) h[r] = hp[r * h_hop];
    if (mine) {
      u = to_f32(static_cast<const T*>(a.u)[ch]);
      dt = to_f32(static_cast<const T*>(a.dt)[ch]);
      if (a.z) z = to_f32(static_cast<const T*>(a.z)[ch]);
      if (a.dt_bias) dt += a.dt_bias[d];
      if (a.Dskip) skip = a.Dskip[d];
    }
    A = *reinterpret_cast<const float4*>(a.A + (size_t)d * N + 4 * ln);
#pragma unroll
    for (int r = 0; r < kStepRows; ++r)
      if (b0 + r < a.B) {
        Bv[r] = four(static_cast<const T*>(a.Bm) + bc + r * bc_hop, bc_wide);
        Cv[r] = four(static_cast<const T*>(a.Cm) + bc + r * bc_hop, bc_wide);
      }
  }
  if (a.dt_softplus) dt = softplus(dt);
  const float du = dt * u;
  float out = 0.f;
#pragma unroll
  for (int r = 0; r < kStepRows; ++r) {
    const int from = lane - ln + r;   // the lane that has row r's step size
    const float s = __shfl_sync(0xffffffffu, dt, from) * kLog2e, x = __shfl_sync(0xffffffffu, du, from);
    h[r].x = fmaf(ex2(s * A.x), h[r].x, x * Bv[r].x);
    h[r].y = fmaf(ex2(s * A.y), h[r].y, x * Bv[r].y);
    h[r].z = fmaf(ex2(s * A.z), h[r].z, x * Bv[r].z);
    h[r].w = fmaf(ex2(s * A.w), h[r].w, x * Bv[r].w);
    float y = fmaf(Cv[r].x, h[r].x, fmaf(Cv[r].y, h[r].y, fmaf(Cv[r].z, h[r].z, Cv[r].w * h[r].w)));
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (ln == r) out = y;
    if (live && b0 + r < a.B) hp[r * h_hop] = h[r];
  }
  if (mine) {
    out = fmaf(skip, u, out);
    if (a.z) out *= z * sigmoid(z);
    static_cast<T*>(a.out)[ch] = from_f32<T>(out);
  }
}

template <typename T, int N>
cudaError_t run_step(const lion_scan_step_args& a, cudaStream_t s) {
  const long long n = (long long)a.D * (N / 4);
  const int rows = (a.B + kStepRows - 1) / kStepRows;
  const int bc_align = std::min(rows_align(a.Bm, 0, 0, sizeof(T)), rows_align(a.Cm, 0, 0, sizeof(T)));
  const bool bc_wide = bc_align >= 4 * (int)sizeof(T);
  scan_step_kernel<T, N><<<dim3((unsigned)((n + 127) / 128), rows), 128, 0, s>>>(a, bc_wide);
  return cudaGetLastError();
}

}  // namespace

// Turns the segments' own contributions into the states that enter them, in
// place: X_{s+1} = exp(A sum_s) X_s + own_s from the walk's start, or, back,
// X_{s-1} = exp(A sum_s) X_s + own_s from its end.  A thread has four states
// of a channel and reads kAhead segments ahead.  A growing state's factor can
// pass fp32 where the state, 0 or tiny, does not: it is the cube of a finite
// one, multiplied in one by one, so that a product overflows only if the whole
// does (2^378 takes the least positive state there).
namespace {
constexpr int kAhead = 16;

__global__ void __launch_bounds__(64) scan_chain_kernel(ScanP p, bool back, const float* first) {
  const int per = p.N / 4;
  const long long k = (long long)blockIdx.x * 64 + threadIdx.x;
  if (k >= (long long)p.B * p.D * per) return;
  const int n0 = 4 * (int)(k % per);
  const long long bd = k / per;
  const int b = (int)(bd / p.D), d = (int)(bd - (long long)b * p.D);
  f2 A[2], x[2];
  load_decays(p.A + (size_t)d * p.N + n0, true, A);
#pragma unroll
  for (int e = 0; e < 2; ++e) A[e] = mul2(A[e], pack2(1.f / 3.f, 1.f / 3.f));
  load_pair(first + bd * p.N + n0, first != nullptr, x);
  wait_prior();
  for (int s0 = 0; s0 < p.nseg; s0 += kAhead) {
    f2 own[kAhead][2];
    float sum[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      // the last of the walk has no contribution: nothing follows it
      const bool there = s0 + q < p.nseg - 1;
      const int s = back ? p.nseg - 1 - s0 - q : s0 + q;
      const size_t at = ((size_t)b * p.nseg + s) * p.D + d;
      load_pair(p.seg_state + at * p.N + n0, there, own[q]);
      sum[q] = there ? p.seg_sum[at] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (s0 + q >= p.nseg) break;
      const int s = back ? p.nseg - 1 - s0 - q : s0 + q;
      store_pair(p.seg_state + (((size_t)b * p.nseg + s) * p.D + d) * p.N + n0, x);
      const f2 s2 = pack2(sum[q], sum[q]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const f2 t = mul2(s2, A[e]);
        const f2 f = ex2_2(pack2(t.x > 126.f ? 126.f : t.x, t.y > 126.f ? 126.f : t.y));   // a NaN stays one
        x[e] = fma2(f, mul2(f, mul2(f, x[e])), own[q][e]);
      }
    }
  }
}
}  // namespace

cudaError_t launch_scan_chain(const ScanP& p, bool back, const float* first, cudaStream_t s) {
  const long long n = (long long)p.B * p.D * (p.N / 4);
  return launch_dependent(scan_chain_kernel, dim3((unsigned)((n + 63) / 64)), dim3(64), 0, s, p, back, first);
}

size_t scan_workspace_bytes(int B, int L, int D, int N, int G) {
  size_t most = 0;
  for (int ragged = 0; ragged < 2; ++ragged) {
    const size_t nseg = scan_fwd_plan(B, L, D, N, G, ragged).nseg;
    if (nseg > 1) most = std::max(most, up256(sizeof(float) * B * nseg * D * N) + up256(sizeof(float) * B * nseg * D));
  }
  return most;
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
  p.nst = (a.L + kStateEvery - 1) / kStateEvery;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  const long long group = a.G > 1 ? p.Dg : 0;
  p.u_align = rows_align(a.u, p.u_ld, group, es);
  p.dt_align = rows_align(a.dt, p.dt_ld, group, es);
  p.z_align = rows_align(a.z, p.z_ld, group, es);
  p.b_align = rows_align(a.Bm, p.b_ld, 0, es);
  p.c_align = rows_align(a.Cm, p.c_ld, 0, es);
  p.o_wide = rows_align(a.out, a.D, group, es) == 16;
}

cudaError_t launch_scan_fwd(const lion_scan_args& a, void* ws, cudaStream_t s) {
  ScanP p = {};
  fill_scan(p, a);
  const ScanPlan r = scan_fwd_plan(a.B, a.L, a.D, a.N, a.G, a.lengths != nullptr);
  p.nblk = r.nblk;
  p.nseg = r.nseg;
  p.seglen = r.seglen;
  p.seg_state = static_cast<float*>(ws);
  p.seg_sum =
      reinterpret_cast<float*>(static_cast<char*>(ws) + up256(sizeof(float) * (size_t)a.B * r.nseg * a.D * a.N));
  return LION_SCAN_DISPATCH(run_fwd, a.dtype, a.N, p, s);
}

cudaError_t launch_scan_step(const lion_scan_step_args& a, cudaStream_t s) {
  return LION_SCAN_DISPATCH(run_step, a.dtype, a.N, a, s);
}

}  // namespace lion
