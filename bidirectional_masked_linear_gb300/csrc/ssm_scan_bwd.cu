// ssm_scan_bwd.cu -- gradients of the selective scan.
//
// With G_i the gradient of h_i and g_i = a_i G_i what it passes on,
//   G_i = C_i dy_i + g_{i+1},   q = g_i h_{i-1}
//   dA = sum q delta,  ddelta = sum_n q A + u sum_n G B,  du = Dskip dy + delta sum_n G B
//   dB = sum_c G delta u,  dC = sum_c dy h,  dh0 = g_0.
// The walk runs against the forward's order, a tile of kStateEvery tokens at a
// time, each from the forward's state before it.  A lane first walks the tile
// forwards to the states at every fourth token, then takes the four-token
// blocks from the last one: forwards once more, the four states and decays
// staying in registers, and back through them.
//
// What bounds it: twelve fp32 operations a token, channel and state at the
// least, 14 with the first walk, against 22 bytes a token and channel (64 x 197
// x 1536 x 16: 98 us of operations, 68 us of bytes), and the sums over states
// and over channels, which go through shuffles and shared memory.  The states
// and decays of a block take the registers, so that two warps share a scheduler
// and cover half of their latencies: measured 380 us, 47% of the issue slots,
// 39% of the fp32 pipe.  (float32 at N = 16 and 64 has one: its 129,024 and
// 116,736 bytes of shared memory leave an SM one CTA.)  Eight products a lane instead of sixteen doubles the
// warps and, with them, the shared-memory traffic of the sums, which then is
// the bound (570 us); inputs read a tile ahead cost more instructions than they
// hide (443 us).
#include <algorithm>

#include "ssm_scan.cuh"

namespace lion {
namespace {

// A row of partial sums, dA then dDskip then ddt_bias, its start on 16 bytes.
__host__ __device__ inline size_t par_stride(int D, int N) { return ((size_t)D * (N + 2) + 3) / 4 * 4; }

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
    load_decays(p.A + (size_t)d[k] * N + 4 * ln, live[k], A[k]);
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
      load8(static_cast<const T*>(p.dt) + row * p.dt_ld + vd, vn, p.dt_align == 16, dt);
      load8(static_cast<const T*>(p.dout) + row * p.D + vd, vn, p.d_align == 16, dy);
      if (p.z) {
        float z[8];
        load8(static_cast<const T*>(p.z) + row * p.z_ld + vd, vn, p.z_align == 16, z);
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

constexpr int kBwdWarps = kScanBwdWarps;
constexpr int kBlock = 4;   // tokens whose states and decays are held in registers

// A lane holds eight states of RC channels: sixteen products a token, as many
// as leave room for a block's states and decays in 255 registers.  A sum over
// the states is then one exchange at N = 16 and a sum over the channels 15.
template <typename T, int N_>
struct BwdTile {
  static constexpr int N = N_, RN = 8, LN = N / RN;
  static constexpr int RC = N == 8 ? 1 : 2;
  static constexpr int LC = 32 / LN;                  // channel lanes
  static constexpr int CW = LC * RC;                  // channels of a warp
  static constexpr int CB = kBwdWarps * CW;           // and of a CTA
  static_assert(CB == scan_bwd_channels(N), "the plan cuts the channels alike");
  static constexpr int TT = kStateEvery;
  static constexpr int VT = CW / 4, VL = TT * VT / 32;
  static constexpr int NB = TT / kBlock;
  static constexpr int GR = LC / 2;                   // lanes that share four states after a sum's first step
  static constexpr int GS = GR * N + 16;              // a token's row of their parts, padded off its neighbour's banks
};
template <typename T, int N>
struct BwdSmem {
  using S = BwdTile<T, N>;
  struct Warp {
    alignas(16) float dt[S::TT * S::CW];   // delta
    alignas(16) float du[S::TT * S::CW];   // delta u, then sum_n q A (A scaled by log2 e)
    alignas(16) float dy[S::TT * S::CW];   // dy, then sum_n G B
    alignas(16) float y[S::TT * S::CW];    // sum_n C h
    alignas(16) float hs[S::NB][S::RN * S::RC / 4][32][4];   // states at the blocks' starts, a lane's own
    alignas(16) float part[2][kBlock][S::GS];   // dB, dC of a block: [lane group][N]
    alignas(16) float red[S::TT * 2 * N];       // dB, dC of the warp's channels
    alignas(16) T ru[S::TT * S::CW];       // raw inputs
    alignas(16) T rdt[S::TT * S::CW];
    alignas(16) T rz[S::TT * S::CW];
    alignas(16) T rdo[S::TT * S::CW];
  } warp[kBwdWarps];
  alignas(16) T rB[S::TT * N];
  alignas(16) T rC[S::TT * N];
  alignas(16) float Bm[S::TT * N];
  alignas(16) float Cm[S::TT * N];
};

template <typename T, int N, bool GATE>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) scan_bwd_kernel(ScanP p) {
  using S = BwdTile<T, N>;
  constexpr int RN = S::RN, LN = S::LN, RC = S::RC, LC = S::LC, CW = S::CW, TT = S::TT, VT = S::VT, VL = S::VL;
  constexpr int NT = 32 * kBwdWarps;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<T, N>& sh = *reinterpret_cast<BwdSmem<T, N>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  typename BwdSmem<T, N>::Warp& sm = sh.warp[warp];
  ScanAt w = scan_at(p, S::CB);
  w.d0 += warp * CW;
  w.nch = max(0, min(CW, w.nch - warp * CW));   // a warp without channels goes along: the CTA has barriers
  // element role: VL vectors of four channels, 32 / VT tokens apart
  const int vt = lane / VT, vc = lane % VT * 4, vd = w.d0 + vc, vn = min(4, w.nch - vc);
  // recurrence role.  Lanes of odd ln hold their two channels, and lanes of odd
  // channel place their two blocks of four states, in the other order: the
  // first step of either sum then sends the same registers from every lane.
  const int ln = lane % LN, lc = lane / LN, odd = RC == 2 && LN > 1 ? ln & 1 : 0, flip = lc & 1;
  int c[RC];
  bool live[RC];
#pragma unroll
  for (int k = 0; k < RC; ++k) {
    c[k] = lc + (k ^ odd) * LC;
    live[k] = c[k] < w.nch;
  }
  const int n0 = ln * RN + 4 * flip, n1 = ln * RN + 4 * (flip ^ 1);   // the first and the second block's states
  auto load_h = [&](const float* from, bool have, f2 (&v)[RC][4]) {
#pragma unroll
    for (int k = 0; k < RC; ++k) {
      f2 a[2], b[2];
      const float* row = from + (size_t)(w.d0 + c[k]) * N;
      load_pair(row + n0, have && live[k], a);
      load_pair(row + n1, have && live[k], b);
      v[k][0] = a[0]; v[k][1] = a[1]; v[k][2] = b[0]; v[k][3] = b[1];
    }
  };
  auto store_h = [&](float* to, const f2 (&v)[RC][4]) {
#pragma unroll
    for (int k = 0; k < RC; ++k) {
      if (!live[k]) continue;
      float* row = to + (size_t)(w.d0 + c[k]) * N;
      const f2 a[2] = {v[k][0], v[k][1]}, b[2] = {v[k][2], v[k][3]};
      store_pair(row + n0, a);
      store_pair(row + n1, b);
    }
  };
  f2 A[RC][4], g[RC][4], dA[RC][4];
  load_h(p.A, true, A);
  // what the segments after this one pass back into it
  load_h(p.nseg > 1 ? p.seg_state + ((size_t)w.b * p.nseg + w.seg) * p.D * N : p.A, p.nseg > 1, g);
#pragma unroll
  for (int k = 0; k < RC; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      A[k][q] = pack2(decay(A[k][q].x), decay(A[k][q].y));
      dA[k][q] = pack2(0.f, 0.f);
    }
  float bias[4], skip[4], dskip[4], dbias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bias[e] = p.dt_bias && e < vn ? p.dt_bias[vd + e] : 0.f;
    skip[e] = p.Dskip && e < vn ? p.Dskip[vd + e] : 0.f;
    dskip[e] = dbias[e] = 0.f;
  }
  const int r0 = max(w.i0, w.v0), r1 = min(w.i1, w.v1);   // the tokens that there are
  const bool plain = w.nch == CW && p.o_wide && (p.u_align & p.dt_align & p.d_align & (GATE ? p.z_align : 16)) == 16;

  for (int i0 = w.i0 + (w.i1 - w.i0 - 1) / TT * TT; i0 >= w.i0; i0 -= TT) {
    const bool some = i0 + TT > r0 && i0 < r1;
    const bool whole = plain && i0 >= r0 && i0 + TT <= r1;
    if (some) {
      // raw inputs of this tile
      const int lo = r0 - i0, hi = r1 - i0;
      {
        Feed<T, TT, CW> f;
        f.start(p.u, p.u_ld, w.d0, p, w, i0, lane, w.nch);
        f.next(sm.ru, lo, hi, lane, p.u_align, whole, 0);
        f.start(p.dt, p.dt_ld, w.d0, p, w, i0, lane, w.nch);
        f.next(sm.rdt, lo, hi, lane, p.dt_align, whole, 0);
        f.start(p.dout, p.D, w.d0, p, w, i0, lane, w.nch);
        f.next(sm.rdo, lo, hi, lane, p.d_align, whole, 0);
        if (GATE) {
          f.start(p.z, p.z_ld, w.d0, p, w, i0, lane, w.nch);
          f.next(sm.rz, lo, hi, lane, p.z_align, whole, 0);
        }
        // B by the first warp, C by the second
        Feed<T, TT, N> fb;
        if (warp < 2) {
          fb.start(warp ? p.Cm : p.Bm, warp ? p.c_ld : p.b_ld, w.g * N, p, w, i0, lane, N);
          fb.next(warp ? sh.rC : sh.rB, lo, hi, lane, warp ? p.c_align : p.b_align, false, 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      f2 h[RC][4];
      load_h(p.states + ((size_t)w.b * p.nst + i0 / TT) * p.D * N, true, h);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      for (int k = tid; k < TT * N; k += NT) {
        sh.Bm[k] = to_f32(sh.rB[k]);
        sh.Cm[k] = to_f32(sh.rC[k]);
      }
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int at = (lane + 32 * j) * 4, i = i0 + vt + j * (32 / VT);
        float u[4], dt[4], dy[4];
        get(sm.ru + at, u);
        get(sm.rdt + at, dt);
        get(sm.rdo + at, dy);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          f2 x = add2(pack2(dt[e], dt[e + 1]), pack2(bias[e], bias[e + 1]));
          if (p.softplus) x = softplus2(x.x, x.y);
          if (!whole) {
            const bool real = i >= r0 && i < r1;
            x = pack2(real && e < vn ? x.x : 0.f, real && e + 1 < vn ? x.y : 0.f);
          }
          const f2 d2 = mul2(x, pack2(u[e], u[e + 1]));
          dt[e] = x.x; dt[e + 1] = x.y;
          u[e] = d2.x; u[e + 1] = d2.y;
        }
        if (GATE) {
          float z[4];
          get(sm.rz + at, z);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const f2 x = gate2(pack2(dy[e], dy[e + 1]), z[e], z[e + 1]);
            dy[e] = x.x; dy[e + 1] = x.y;
          }
        }
        *reinterpret_cast<float4*>(sm.dt + at) = make_float4(dt[0], dt[1], dt[2], dt[3]);
        *reinterpret_cast<float4*>(sm.du + at) = make_float4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<float4*>(sm.dy + at) = make_float4(dy[0], dy[1], dy[2], dy[3]);
      }
      __syncthreads();

      // forwards to the states at the blocks' starts
      auto keep = [&](int blk) {
#pragma unroll
        for (int k = 0; k < RC; ++k)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<float4*>(sm.hs[blk][2 * k + q][lane]) =
                make_float4(h[k][2 * q].x, h[k][2 * q].y, h[k][2 * q + 1].x, h[k][2 * q + 1].y);
      };
      auto row4 = [&](const float* m, int t, f2 (&v)[4]) {
        const float4 a = *reinterpret_cast<const float4*>(m + t * N + n0);
        const float4 b = *reinterpret_cast<const float4*>(m + t * N + n1);
        v[0] = pack2(a.x, a.y); v[1] = pack2(a.z, a.w);
        v[2] = pack2(b.x, b.y); v[3] = pack2(b.z, b.w);
      };
      keep(0);
      for (int blk = 1; blk < S::NB; ++blk) {
#pragma unroll
        for (int s = 0; s < kBlock; ++s) {
          const int t = (blk - 1) * kBlock + s;
          f2 b2[4];
          row4(sh.Bm, t, b2);
#pragma unroll
          for (int k = 0; k < RC; ++k) {
            const float dt = sm.dt[t * CW + c[k]], du = sm.du[t * CW + c[k]];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              h[k][q] = fma2(ex2_2(mul2(pack2(dt, dt), A[k][q])), h[k][q], mul2(pack2(du, du), b2[q]));
          }
        }
        keep(blk);
      }

#pragma unroll 1
      for (int blk = S::NB - 1; blk >= 0; --blk) {
        f2 a[kBlock][RC][4], hh[kBlock + 1][RC][4];
#pragma unroll
        for (int k = 0; k < RC; ++k)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(sm.hs[blk][2 * k + q][lane]);
            hh[0][k][2 * q] = pack2(x.x, x.y);
            hh[0][k][2 * q + 1] = pack2(x.z, x.w);
          }
#pragma unroll
        for (int s = 0; s < kBlock; ++s) {
          const int t = blk * kBlock + s;
          f2 b2[4];
          row4(sh.Bm, t, b2);
#pragma unroll
          for (int k = 0; k < RC; ++k) {
            const float dt = sm.dt[t * CW + c[k]], du = sm.du[t * CW + c[k]];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              a[s][k][q] = ex2_2(mul2(pack2(dt, dt), A[k][q]));
              hh[s + 1][k][q] = fma2(a[s][k][q], hh[s][k][q], mul2(pack2(du, du), b2[q]));
            }
          }
        }
        // A token's reads stand before the stores of the token walked before it: a read does not pass a store ahead
        // of it that could go to its place, and the tokens would wait for one another's sums.
        f2 b2[4], c2[4];
        float vt_[RC], vu_[RC], vy_[RC];
        auto read_token = [&](int t) {
          row4(sh.Bm, t, b2);
          row4(sh.Cm, t, c2);
#pragma unroll
          for (int k = 0; k < RC; ++k) {
            vt_[k] = sm.dt[t * CW + c[k]];
            vu_[k] = sm.du[t * CW + c[k]];
            vy_[k] = sm.dy[t * CW + c[k]];
          }
        };
        read_token(blk * kBlock + kBlock - 1);
#pragma unroll
        for (int s = kBlock - 1; s >= 0; --s) {
          const int t = blk * kBlock + s;
          f2 dB[4], dC[4];
          float gb[RC], qa[RC], y[RC];
#pragma unroll
          for (int k = 0; k < RC; ++k) {
            const f2 dt2 = pack2(vt_[k], vt_[k]), du2 = pack2(vu_[k], vu_[k]), dy2 = pack2(vy_[k], vy_[k]);
            f2 sgb, sqa, sy;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f2 G = fma2(c2[q], dy2, g[k][q]);
              dC[q] = k == 0 ? mul2(dy2, hh[s + 1][k][q]) : fma2(dy2, hh[s + 1][k][q], dC[q]);
              dB[q] = k == 0 ? mul2(du2, G) : fma2(du2, G, dB[q]);
              sgb = q == 0 ? mul2(G, b2[q]) : fma2(G, b2[q], sgb);
              if (GATE) sy = q == 0 ? mul2(c2[q], hh[s + 1][k][q]) : fma2(c2[q], hh[s + 1][k][q], sy);
              g[k][q] = mul2(G, a[s][k][q]);
              const f2 e = mul2(g[k][q], hh[s][k][q]);
              dA[k][q] = fma2(e, dt2, dA[k][q]);
              sqa = q == 0 ? mul2(e, A[k][q]) : fma2(e, A[k][q], sqa);
            }
            gb[k] = sum2(sgb);
            qa[k] = sum2(sqa);
            if (GATE) y[k] = sum2(sy);
          }
          if (s > 0) read_token(t - 1);
          // over the states
          if (LN > 1) {
            gb[0] += __shfl_xor_sync(0xffffffffu, gb[RC - 1], 1);
            qa[0] += __shfl_xor_sync(0xffffffffu, qa[RC - 1], 1);
            if (GATE) y[0] += __shfl_xor_sync(0xffffffffu, y[RC - 1], 1);
#pragma unroll
            for (int o = 2; o < LN; o <<= 1) {
              gb[0] += __shfl_xor_sync(0xffffffffu, gb[0], o);
              qa[0] += __shfl_xor_sync(0xffffffffu, qa[0], o);
              if (GATE) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
            }
          }
          if (LN > 1) __syncwarp();   // the channel's lanes have read dy and delta u; a shuffle orders no memory
          sm.dy[t * CW + c[0]] = gb[0];   // lanes of one parity hold the same sums
          sm.du[t * CW + c[0]] = qa[0];
          if (GATE) sm.y[t * CW + c[0]] = y[0];
          // over the channels, LN lanes apart: first between lanes that hold the blocks of states in opposite
          // order, the rest in shared memory
          float r[8];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            r[2 * q] = dB[q].x + __shfl_xor_sync(0xffffffffu, dB[q + 2].x, LN);
            r[2 * q + 1] = dB[q].y + __shfl_xor_sync(0xffffffffu, dB[q + 2].y, LN);
            r[4 + 2 * q] = dC[q].x + __shfl_xor_sync(0xffffffffu, dC[q + 2].x, LN);
            r[4 + 2 * q + 1] = dC[q].y + __shfl_xor_sync(0xffffffffu, dC[q + 2].y, LN);
          }
          const int at_r = (lc >> 1) * N + n0;
          *reinterpret_cast<float4*>(sm.part[0][s] + at_r) = make_float4(r[0], r[1], r[2], r[3]);
          *reinterpret_cast<float4*>(sm.part[1][s] + at_r) = make_float4(r[4], r[5], r[6], r[7]);
        }
        __syncwarp();
#pragma unroll
        for (int o = lane; o < 2 * kBlock * N / 4; o += 32) {
          const int n = o % (N / 4) * 4, s = o / (N / 4) % kBlock, kind = o / (N / 4) / kBlock;
          const float* from = sm.part[kind][s] + n;
          f2 a = pack2(0.f, 0.f), b = a;
#pragma unroll
          for (int v = 0; v < S::GR; ++v) {
            const float4 x = *reinterpret_cast<const float4*>(from + v * N);
            a = add2(a, pack2(x.x, x.y));
            b = add2(b, pack2(x.z, x.w));
          }
          *reinterpret_cast<float4*>(sm.red + (blk * kBlock + s) * 2 * N + kind * N + n) =
              make_float4(a.x, a.y, b.x, b.y);
        }
        __syncwarp();
      }
      __syncthreads();
      // one part a CTA: the warps' sums in their order
      for (int k = tid; k < TT * 2 * N; k += NT) {
        const int t = k / (2 * N), i = i0 + t;
        if (i >= w.i1) break;
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < kBwdWarps; ++v) s += sh.warp[v].red[k];
        p.part_bc[((((size_t)w.blk * p.B + w.b) * p.L + token_of(p, i)) * p.G + w.g) * 2 * N + k % (2 * N)] = s;
      }
    }
#pragma unroll
    for (int j = 0; j < VL; ++j) {
      const int at = (lane + 32 * j) * 4, i = i0 + vt + j * (32 / VT);
      if (i >= w.i1 || vn <= 0) continue;
      float du[4] = {0.f, 0.f, 0.f, 0.f}, ddt[4] = {0.f, 0.f, 0.f, 0.f}, dz[4] = {0.f, 0.f, 0.f, 0.f};
      if (i >= r0 && i < r1) {
        float u[4], raw[4], dl[4], dout[4], gb[4], qa[4];
        get(sm.ru + at, u);
        get(sm.rdt + at, raw);
        get(sm.rdo + at, dout);
        get(sm.dt + at, dl);
        get(sm.dy + at, gb);
        get(sm.du + at, qa);
        float z[4], y[4];
        if (GATE) {
          get(sm.rz + at, z);
          get(sm.y + at, y);
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const f2 u2 = pack2(u[e], u[e + 1]), sk2 = pack2(skip[e], skip[e + 1]), gb2 = pack2(gb[e], gb[e + 1]);
          f2 dy2 = pack2(dout[e], dout[e + 1]);
          if (GATE) {
            const f2 s2 = sigmoid2(z[e], z[e + 1]), z2 = pack2(z[e], z[e + 1]), zs = mul2(z2, s2);
            // silu'(z) = s + z s (1 - s) = s + zs - zs s
            const f2 ds = add2(s2, fma2(zs, pack2(-s2.x, -s2.y), zs));
            const f2 x = mul2(mul2(dy2, fma2(sk2, u2, pack2(y[e], y[e + 1]))), ds);
            dz[e] = x.x; dz[e + 1] = x.y;
            dy2 = mul2(dy2, zs);
          }
          const f2 x = fma2(pack2(dl[e], dl[e + 1]), gb2, mul2(sk2, dy2));
          du[e] = x.x; du[e + 1] = x.y;
          f2 d = fma2(u2, gb2, mul2(pack2(qa[e], qa[e + 1]), pack2(kLn2, kLn2)));
          if (p.softplus) d = mul2(d, sigmoid2(raw[e] + bias[e], raw[e + 1] + bias[e + 1]));
          ddt[e] = d.x; ddt[e + 1] = d.y;
          const f2 ws = fma2(dy2, u2, pack2(dskip[e], dskip[e + 1]));
          dskip[e] = ws.x; dskip[e + 1] = ws.y;
          dbias[e] += d.x;
          dbias[e + 1] += d.y;
        }
      }
      const long long row = ((long long)w.b * p.L + token_of(p, i)) * p.D + vd;
      put(static_cast<T*>(p.du) + row, vn, p.o_wide, du);
      put(static_cast<T*>(p.ddt) + row, vn, p.o_wide, ddt);
      if (GATE) put(static_cast<T*>(p.dz) + row, vn, p.o_wide, dz);
    }
    if (some) __syncthreads();   // red, B and C are read before the next tile's are written
  }

  float* part = p.part_par + ((size_t)w.b * p.nseg + w.seg) * par_stride(p.D, N);
  store_h(part, dA);
  if (p.dh0 && w.seg == 0) store_h(p.dh0 + (size_t)w.b * p.D * N, g);
  // the element lanes of a channel vector
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int o = VT; o < 32; o <<= 1) {
      dskip[e] += __shfl_xor_sync(0xffffffffu, dskip[e], o);
      dbias[e] += __shfl_xor_sync(0xffffffffu, dbias[e], o);
    }
    if (vt == 0 && e < vn) {
      part[(size_t)p.D * N + vd + e] = dskip[e];
      part[(size_t)p.D * (N + 1) + vd + e] = dbias[e];
    }
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
  wait_prior();
  if (!p.lengths || t < p.lengths[b])
    for (int q = 0; q < p.nblk; ++q) s += p.part_bc[(size_t)q * n + k];
  (v < p.N ? dB : dC)[k / N2 * p.N + v % p.N] = from_f32<T>(s);
}

template <typename T, int N, bool GATE>
cudaError_t run_main(const ScanP& p, cudaStream_t s) {
  auto kern = scan_bwd_kernel<T, N, GATE>;
  const size_t smem = sizeof(BwdSmem<T, N>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.nblk * p.G * p.nseg * p.B, 32 * kBwdWarps, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int N>
cudaError_t run_bwd(const ScanP& p, cudaStream_t s) {
  if (p.nseg > 1) {
    constexpr int LN = N / 4, W = N == 8 ? 4 : 8;
    using S = ScanTile<LN, W>;
    static_assert(S::CB == BwdTile<T, N>::CB, "both kernels cut the channels alike");
    scan_bwd_segment_kernel<T, LN, W>
        <<<(unsigned)p.nblk * p.G * p.nseg * p.B, S::NT, sizeof(float) * S::TT * S::N, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_scan_chain(p, true, nullptr, s);
    if (e != cudaSuccess) return e;
  }
  return p.z ? run_main<T, N, true>(p, s) : run_main<T, N, false>(p, s);
}

template <typename T>
cudaError_t run_bc(const ScanP& p, void* dB, void* dC, cudaStream_t s) {
  const long long n = (long long)p.B * p.L * p.G * 2 * p.N;
  return launch_dependent(scan_bc_kernel<T>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p, static_cast<T*>(dB),
                          static_cast<T*>(dC));
}

// The workspace's parts: the forward's own, the states, the segments, the
// partial sums.
struct BwdPlan {
  ScanPlan r;
  size_t fwd, states, seg_state, seg_sum, bc, par, total;
};
BwdPlan bwd_plan(int B, int L, int D, int N, int G, bool have_states, bool ragged) {
  BwdPlan q;
  q.r = scan_bwd_plan(B, L, D, N, G, ragged);
  size_t at = 0;
  auto take = [&](size_t floats) {
    const size_t here = at;
    at += up256(sizeof(float) * floats);
    return here;
  };
  q.fwd = at;
  if (!have_states) at += up256(scan_workspace_bytes(B, L, D, N, G));
  q.states = take(have_states ? 0 : (size_t)B * ((L + kStateEvery - 1) / kStateEvery) * D * N);
  q.seg_state = take(q.r.nseg > 1 ? (size_t)B * q.r.nseg * D * N : 0);
  q.seg_sum = take(q.r.nseg > 1 ? (size_t)B * q.r.nseg * D : 0);
  q.bc = take((size_t)q.r.nblk * B * L * G * 2 * N);
  q.par = take((size_t)B * q.r.nseg * par_stride(D, N));
  q.total = at;
  return q;
}

}  // namespace

size_t scan_bwd_workspace_bytes(int B, int L, int D, int N, int G, bool have_states) {
  return std::max(bwd_plan(B, L, D, N, G, have_states, false).total, bwd_plan(B, L, D, N, G, have_states, true).total);
}

cudaError_t launch_scan_bwd(const lion_scan_bwd_args& a, void* ws, cudaStream_t s) {
  const BwdPlan q = bwd_plan(a.B, a.L, a.D, a.N, a.G, a.states != nullptr, a.lengths != nullptr);
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
  const long long group = a.G > 1 ? p.Dg : 0;
  p.dout = a.dout;
  p.d_align = rows_align(a.dout, a.D, group, es);
  p.o_wide = (rows_align(a.du, a.D, group, es) & rows_align(a.ddt, a.D, group, es) &
              rows_align(a.dz, a.D, group, es)) == 16;
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
  return launch_sum_parts(p.part_par, a.B * q.r.nseg, (long long)par_stride(a.D, a.N), (long long)a.D * a.N, a.dA, a.D,
                          a.dDskip, a.D, a.ddt_bias, s);
}

}  // namespace lion
