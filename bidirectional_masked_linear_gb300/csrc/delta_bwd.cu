// delta_bwd.cu -- gradients of the gated delta rule over chunks: a walk back
// over the chunks carries dS and leaves dV = dR and every 64th token's dS'; the
// rest needs no order and runs on blocks of 64 tokens side by side.
#include "delta_chain.cuh"
#include "delta_internal.h"

namespace lion {
namespace {

// ------------------------------------------------------- what dO gives a chunk
//
// A warp a chunk: P^T dO, transposed as the chain's accumulators are, and
// (scale e^G o dO)^T as its A operands.  Bytes bound it: 16 x 4096 x 8 x 64 in
// bfloat16 59 us at 5.7 TB/s.

template <typename T, int DK>
__global__ void __launch_bounds__(32) delta_back_prep_kernel(const DeltaP p) {
  typedef ChunkData<T, DK, true, sizeof(T) == 4> D;
  constexpr int NI = D::NI, NS = D::NS, NPP = D::NPP, val = kChunk * kSlice * 2;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned base = shared_at(smem), tiles = base + NPP * kTile;
  const int lane = threadIdx.x, q4 = lane & 3;
  const long long bh = blockIdx.x / p.nc;
  const int c = (int)(blockIdx.x - bh * p.nc), b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv);
  const int n = delta_length(p, b), i0 = c * kChunk;
  if (i0 >= n) return;
  const char* chunk = p.chunks + (long long)blockIdx.x * D::bytes;
  copy_block<NPP * kTile, 32>(base, chunk + D::P, lane);
  for (int s = 0; s < p.slices; ++s)
    load_tile<kSlice, kChunk, 32>(tiles + s * NI * val, val,
                                  rows_of<T>(p, p.dout, (long long)p.Hv * p.dv, (long long)hv * p.dv + s * kSlice, b, n),
                                  i0, n, p.dv - s * kSlice, p.do_wide, lane);
  copy_commit();
  float2 g[2][2];
  const float* coef = reinterpret_cast<const float*>(chunk + D::coef);
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int h = 0; h < 2; ++h) g[ks][h] = *reinterpret_cast<const float2*>(coef + 16 * ks + 8 * h + 2 * q4);
  copy_wait<0>();
  __syncwarp();
  float4* Z = reinterpret_cast<float4*>(p.U) + (long long)blockIdx.x * p.dvp * (kChunk / 4) + lane;
  uint4* out = p.dO + (long long)blockIdx.x * (p.dvp / 16) * 2 * NS * 32 + lane;
  for (int mt = 0; 16 * mt < p.dvp; ++mt) {
    float z[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      unsigned a[NI][4];
      float f[2][4] = {};
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        ldsm_t(a[j], tiles + (mt >> 2) * NI * val + j * val + at_a_rows_k<kSlice>(16 * ks, 16 * (mt & 3), lane));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = unpack_bf16(a[j][e]);
          f[e >> 1][2 * (e & 1)] += v.x;
          f[e >> 1][2 * (e & 1) + 1] += v.y;
        }
      }
#pragma unroll
      for (int np = 0; np <= ks; ++np)
        mma_tile<NI, NPP, true>(z[2 * np], z[2 * np + 1], a, base + at_b_rows_k<kChunk, true>(16 * ks, 16 * np, lane), kTile);
      unsigned s[NS][4];
      to_a<NS>(f[0], f[1], g[ks][0], g[ks][1], s);
#pragma unroll
      for (int y = 0; y < NS; ++y) out[((mt * 2 + ks) * NS + y) * 32] = make_uint4(s[y][0], s[y][1], s[y][2], s[y][3]);
    }
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) Z[(mt * 4 + nb) * 32] = make_float4(z[nb][0], z[nb][1], z[nb][2], z[nb][3]);
  }
}

// ------------------------------------------------------------- the chain back
//
// As delta_chain_kernel with dS^T in the registers:
//   X^T = dO^T P + beta e^(G_C - G) o (dS'^T K^T);  dR^T = X^T T
//   dS^T = e^G_C dS'^T + (scale e^G o dO)^T Q - X^T W
// Bound as that one is: 64 x 197 x 12 x 64 in bfloat16 54 us.

template <typename T, int DK>
struct Back {
  typedef ChunkData<T, DK, true, sizeof(T) == 4> D;
  typedef Stage<T, DK, D::coef, D::bytes> L;
  static constexpr int stages = sizeof(T) == 4 ? 2 : 3;
  static constexpr int smem = stages * L::bytes + 4 * out_bytes<T>();
};

template <typename T, int DK>
__global__ void __launch_bounds__(128) delta_back_kernel(const DeltaP p) {
  typedef Back<T, DK> C;
  typedef typename C::D D;
  typedef typename C::L L;
  constexpr int NST = C::stages, NI = D::NI, NS = D::NS, PER = kStateChunk / kChunk;
  constexpr bool KQ = L::KQ;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, q4 = lane & 3;
  unsigned char* buf = smem + NST * L::bytes + w * out_bytes<T>();
  const long long at = blockIdx.x / p.slices;
  const int slice = (int)(blockIdx.x - at * p.slices), rank = (int)(at / p.Hv), hv = (int)(at - (long long)rank * p.Hv);
  const int b = by_length(p, rank);
  const long long bh = (long long)b * p.Hv + hv;
  const int hk = hv / (p.Hv / p.Hk);
  const int n = delta_length(p, b), nc = (n + kChunk - 1) / kChunk;
  const int m0 = slice * kSlice + 16 * w, cols = p.dv - m0 < 16 ? p.dv - m0 : 16;
  const Rows<T> xq = rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n);
  const Rows<T> xk = rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n);
  const Rows<T> xv = rows_of<T>(p, p.dv_out, (long long)p.Hv * p.dv, (long long)hv * p.dv + m0, b, n);
  const char* chunk = p.chunks + bh * p.nc * D::bytes;
  const long long at_last = bh * p.nc + nc - 1;
  const float4* Z = reinterpret_cast<const float4*>(p.U) + (at_last * p.dvp + m0) * (kChunk / 4) + lane;
  const uint4* dO = p.dO + (at_last * (p.dvp / 16) + m0 / 16) * 2 * NS * 32 + lane;

  float s[DK / 8][4] = {};   // dS^T
  wait_prior();
#pragma unroll
  for (int st = 0; st < NST - 1; ++st) {
    const int c = nc - 1 - st;
    if (c >= 0) L::template load<128>(p, base + st * L::bytes, chunk + (long long)c * D::bytes, xq, xk, c * kChunk, n, tid);
    copy_commit();
  }
  float4 znext[4];
  uint4 onext[2][NS];
  if (cols > 0 && nc > 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) znext[e] = Z[32 * e];
#pragma unroll
    for (int e = 0; e < 2 * NS; ++e) onext[e / NS][e % NS] = dO[32 * e];
  }
  for (int step = 0; step < nc; ++step) {
    const int c = nc - 1 - step, ahead = c - (NST - 1);
    copy_wait<NST - 2>();
    __syncthreads();
    if (ahead >= 0)
      L::template load<128>(p, base + (step + NST - 1) % NST * L::bytes, chunk + (long long)ahead * D::bytes, xq, xk,
                            ahead * kChunk, n, tid);
    copy_commit();
    if (cols <= 0) continue;
    const unsigned st = base + step % NST * L::bytes;
    const float* coef = reinterpret_cast<const float*>(smem + step % NST * L::bytes + L::at(D::coef));
    if (step == 0 || c % PER == PER - 1)
      store_blocks<DK / 8>(static_cast<T*>(p.dstates) + ((bh * p.nc64 + c / PER) * p.dvp + m0) * DK, s, lane);

    float4 z[4];
    unsigned g[2][NS][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = znext[e];
#pragma unroll
    for (int e = 0; e < 2 * NS; ++e) {
      const uint4 v = onext[e / NS][e % NS];
      unsigned(&d)[4] = g[e / NS][e % NS];
      d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
    }
    if (c > 0) {
      Z -= p.dvp * (kChunk / 4);
      dO -= (p.dvp / 16) * 2 * NS * 32;
#pragma unroll
      for (int e = 0; e < 4; ++e) znext[e] = Z[32 * e];
#pragma unroll
      for (int e = 0; e < 2 * NS; ++e) onext[e / NS][e % NS] = dO[32 * e];
    }
    // X^T
    float x[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
      for (int np = 0; np < 2; ++np)
        mma_tile<NS, NI, false>(x[2 * np], x[2 * np + 1], a, st + L::k + at_b_rows_n<DK, KQ>(16 * np, 16 * ks, lane), L::row);
    }
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float2 l = *reinterpret_cast<const float2*>(coef + kChunk + 8 * nb + 2 * q4);
      x[nb][0] = fmaf(l.x, x[nb][0], z[nb].x);
      x[nb][1] = fmaf(l.y, x[nb][1], z[nb].y);
      x[nb][2] = fmaf(l.x, x[nb][2], z[nb].z);
      x[nb][3] = fmaf(l.y, x[nb][3], z[nb].w);
    }
    // dS^T and dR^T
    scale_by(s, coef[2 * kChunk]);
    float y[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(x[2 * ks], x[2 * ks + 1], a);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn) {
        mma_tile<NS, NI, true>(s[2 * nn], s[2 * nn + 1], g[ks], st + L::q + at_b_rows_k<DK, KQ>(16 * ks, 16 * nn, lane), L::row);
        mma_tile<NS, NS, true>(s[2 * nn], s[2 * nn + 1], a,
                               st + L::at(D::W) + at_b_rows_k<DK, true>(16 * ks, 16 * nn, lane), L::row);
      }
#pragma unroll
      for (int np = 0; np <= ks; ++np)
        mma_tile<NS, NS, true>(y[2 * np], y[2 * np + 1], a,
                               st + L::at(D::Tm) + at_b_rows_k<kChunk, true>(16 * ks, 16 * np, lane), kTile);
    }
    const int i = c * kChunk + lane;
    store_rows(buf, y, lane, cols, p.dv_wide, i < n ? const_cast<T*>(xv.at(i)) : nullptr);
  }
  copy_wait<0>();
  if (cols <= 0) return;
  if (p.dh0) keep_state<DK>(p, p.dh0, bh, m0, cols, lane, s);
  zero_rows<T>(p, p.dv_out, n, b, hv, m0, cols, p.dv_wide, lane);
}

// The same with a helper to each warp, which has the loads, dR, what the other
// gradients take, and dO's part of the next dS, ready when the warp has X: 1330 ns
// a chunk of 64 columns where an SM has one CTA (16 x 4096 x 8 x 64: 174 us, 33%
// of the tensor cores', 31% of the issue slots).

template <typename T, int DK, int PAIRS>
struct BackTeam {
  static constexpr int width = 16 * PAIRS, half = 32 * PAIRS;
  static constexpr bool KQ = sizeof(T) == 4;
  typedef ChunkData<T, DK, true, KQ> D;
  static constexpr int row = kChunk * DK * 2;
  // a stage: q, k, coefficients, -W and T, the slice of P^T dO
  static constexpr int q = 0, k = D::NI * row, coef = 2 * D::NI * row, W = coef + (D::W - D::coef), Tm = W + (D::Tm - D::W);
  static constexpr int Z = Tm + (D::bytes - D::Tm), bytes = Z + width * kChunk * 4;
  static constexpr int stages = 3;
  static constexpr int S = 0, X = KQ ? 0 : DK / 16 * 512, swap = X + 2 * D::NS * 512;   // a warp's buffer to its helper
  static constexpr int Y = DK / 8 * 512;                               // and back: dO's part of dS^T
  static constexpr int swaps = stages * bytes, ys = swaps + 2 * PAIRS * swap, out = ys + PAIRS * Y;
  static constexpr int smem = out + PAIRS * out_bytes<T>();
  static_assert(smem <= 227 * 1024 - 1024);
};

template <typename T, int DK, int PAIRS>
__global__ void __launch_bounds__(64 * PAIRS) delta_back_team_kernel(const DeltaP p, int slices) {
  typedef BackTeam<T, DK, PAIRS> C;
  typedef typename C::D D;
  constexpr int NST = C::stages, NI = D::NI, NS = D::NS, PER = kStateChunk / kChunk;
  constexpr int HALF = C::half;
  constexpr bool KQ = C::KQ;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x & (HALF - 1), lane = tid & 31, w = tid >> 5, q4 = lane & 3;
  const bool helper = threadIdx.x >= HALF;
  const long long part = blockIdx.x / slices, at = part / p.nseg;
  const int slice = (int)(blockIdx.x - part * slices), seg = (int)(part - at * p.nseg);
  const int rank = (int)(at / p.Hv), hv = (int)(at - (long long)rank * p.Hv), b = by_length(p, rank);
  const long long bh = (long long)b * p.Hv + hv;
  const int hk = hv / (p.Hv / p.Hk);
  const int n = delta_length(p, b), all = (n + kChunk - 1) / kChunk, c0 = seg * p.seglen;
  const int nc = all - c0 < 0 ? 0 : all - c0 < p.seglen ? all - c0 : p.seglen, last = c0 + nc - 1;   // the segment's
  const int m0 = slice * C::width + 16 * w, cols = p.dv - m0 < 16 ? p.dv - m0 : 16;
  const unsigned swap = base + C::swaps + w * C::swap;   // the second buffer PAIRS swaps behind
  const unsigned ys = base + C::ys + w * C::Y;
  wait_prior();
  if (helper) {
    const Rows<T> xq = rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n);
    const Rows<T> xk = rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n);
    const Rows<T> xv = rows_of<T>(p, p.dv_out, (long long)p.Hv * p.dv, (long long)hv * p.dv + m0, b, n);
    const char* chunks = p.chunks + bh * p.nc * D::bytes;
    const float* Zs = p.U + (bh * p.nc * p.dvp + slice * C::width) * kChunk;
    const uint4* dO = p.dO + (bh * p.nc * (p.dvp / 16) + m0 / 16) * 2 * NS * 32 + lane;
    const int rows = p.dvp - slice * C::width < C::width ? p.dvp - slice * C::width : C::width;
    unsigned char* buf = smem + C::out + w * out_bytes<T>();
    const auto load = [&](int i) {   // the segment's i-th chunk from the end
      const int c = last - i;
      const unsigned st = base + i % NST * C::bytes;
      if (KQ) {
        copy_block<2 * NI * C::row, HALF>(st, chunks + (long long)c * D::bytes, tid);
      } else {
        load_tile<DK, kChunk, HALF>(st + C::k, 0, xk, c * kChunk, n, p.dk, p.k_wide, tid);
        load_tile<DK, kChunk, HALF>(st + C::q, 0, xq, c * kChunk, n, p.dk, p.q_wide, tid);
      }
      copy_block<D::bytes - D::coef, HALF>(st + C::coef, chunks + (long long)c * D::bytes + D::coef, tid);
      copy_slice<C::width, HALF>(st + C::Z, Zs + (long long)c * p.dvp * kChunk, rows, tid);
    };
    uint4 g[2][NS];
    const auto fetch = [&](int i) {
      const uint4* s = dO + (long long)(last - i) * (p.dvp / 16) * 2 * NS * 32;
#pragma unroll
      for (int e = 0; e < 2 * NS; ++e) g[e / NS][e % NS] = s[32 * e];
    };
    if (nc > 0) {
      load(0);
      if (cols > 0) fetch(0);
    }
    copy_commit();
    for (int i = 0; i <= nc; ++i) {
      copy_wait<0>();
      __syncthreads();
      if (i + 1 < nc) load(i + 1);
      copy_commit();
      if (i + 2 < nc) {   // as in the forward walk
        const long long c = last - 2 - i;
        to_l2<D::bytes - D::coef, HALF>(chunks + c * D::bytes + D::coef, D::bytes - D::coef, tid);
        to_l2<C::width * kChunk * 4, HALF>(Zs + c * p.dvp * kChunk, rows * kChunk * 4, tid);
        if constexpr (KQ) {
          to_l2<2 * NI * C::row, HALF>(chunks + c * D::bytes, 2 * NI * C::row, tid);
        } else {
          rows_to_l2(xk, (int)c * kChunk, n, tid - (HALF - 64));
          rows_to_l2(xq, (int)c * kChunk, n, tid - (HALF - 32));
        }
        if (cols > 0) to_l2<2 * NS * 512, 32>(dO - lane + c * (p.dvp / 16) * 2 * NS * 32, 2 * NS * 512, lane);
      }
      if (i < nc && cols > 0) {   // (scale e^G o dO)^T Q
        const unsigned st = base + i % NST * C::bytes;
        float y[DK / 8][4] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          unsigned a[NS][4];
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            a[j][0] = g[ks][j].x; a[j][1] = g[ks][j].y; a[j][2] = g[ks][j].z; a[j][3] = g[ks][j].w;
          }
#pragma unroll
          for (int nn = 0; nn < DK / 16; ++nn)
            mma_tile<NS, NI, true>(y[2 * nn], y[2 * nn + 1], a, st + C::q + at_b_rows_k<DK, KQ>(16 * ks, 16 * nn, lane), C::row);
        }
        put_sums(ys, y, lane);
        asm volatile("barrier.cta.arrive %0, 64;" ::"r"(1 + w) : "memory");
        if (i + 1 < nc) fetch(i + 1);
      }
      if (i == 0 || cols <= 0) continue;
      const int j = i - 1, c = last - j;
      const unsigned st = base + j % NST * C::bytes, x = swap + (j & 1) * PAIRS * C::swap;
      if constexpr (!KQ) {
        if (c == all - 1 || c % PER == PER - 1)
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks) {
            unsigned a[4];
            get_a(x + C::S + ks * 512, a, lane);
            store_a<DK / 8>(static_cast<T*>(p.dstates) + ((bh * p.nc64 + c / PER) * p.dvp + m0) * DK + ks * 128, a, lane);
          }
      }
      float y[4][4] = {};   // dR^T
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        unsigned a[NS][4];
#pragma unroll
        for (int e = 0; e < NS; ++e) get_a(x + C::X + (ks * NS + e) * 512, a[e], lane);
#pragma unroll
        for (int np = 0; np <= ks; ++np)
          mma_tile<NS, NS, true>(y[2 * np], y[2 * np + 1], a,
                                 st + C::Tm + at_b_rows_k<kChunk, true>(16 * ks, 16 * np, lane), kTile);
      }
      const int t = c * kChunk + lane;
      store_rows(buf, y, lane, cols, p.dv_wide, t < n ? const_cast<T*>(xv.at(t)) : nullptr);
    }
    if (cols > 0 && seg == 0) zero_rows<T>(p, p.dv_out, n, b, hv, m0, cols, p.dv_wide, lane);
    return;
  }
  float s[DK / 8][4];   // dS^T
  load_state<DK>(p, seg < p.nseg - 1 ? p.starts : nullptr, bh * p.nseg + seg, m0, cols, lane, s);
  for (int i = 0; i <= nc; ++i) {
    __syncthreads();
    if (i == nc || cols <= 0) continue;
    const unsigned st = base + i % NST * C::bytes, x = swap + (i & 1) * PAIRS * C::swap;
    const float* coef = reinterpret_cast<const float*>(smem + i % NST * C::bytes + C::coef);
    if constexpr (KQ) {
      const int c = last - i;
      if (c == all - 1 || c % PER == PER - 1)
        store_blocks<DK / 8>(static_cast<T*>(p.dstates) + ((bh * p.nc64 + c / PER) * p.dvp + m0) * DK, s, lane);
    }
    // X^T
    float r[4][4] = {};
    unsigned plain[DK / 16][4], a[2][NS][4];   // to the helper at the end, as in the forward walk
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned d[NS][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], d);
#pragma unroll
      for (int e = 0; e < 4; ++e) plain[ks][e] = d[0][e];
#pragma unroll
      for (int np = 0; np < 2; ++np)
        mma_tile<NS, NI, false>(r[2 * np], r[2 * np + 1], d, st + C::k + at_b_rows_n<DK, KQ>(16 * np, 16 * ks, lane), C::row);
    }
    scale_by(s, coef[2 * kChunk]);
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float2 l = *reinterpret_cast<const float2*>(coef + kChunk + 8 * nb + 2 * q4);
      const float4 z = get_f4(st + C::Z + (w * 4 + nb) * 512, lane);
      r[nb][0] = fmaf(l.x, r[nb][0], z.x);
      r[nb][1] = fmaf(l.y, r[nb][1], z.y);
      r[nb][2] = fmaf(l.x, r[nb][2], z.z);
      r[nb][3] = fmaf(l.y, r[nb][3], z.w);
    }
    // dS^T
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      to_a<NS>(r[2 * ks], r[2 * ks + 1], a[ks]);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn)
        mma_tile<NS, NS, true>(s[2 * nn], s[2 * nn + 1], a[ks], st + C::W + at_b_rows_k<DK, true>(16 * ks, 16 * nn, lane), C::row);
    }
    asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + w) : "memory");
#pragma unroll
    for (int nb = 0; nb < DK / 8; ++nb) {
      const float4 y = get_f4(ys + nb * 512, lane);
      s[nb][0] += y.x;
      s[nb][1] += y.y;
      s[nb][2] += y.z;
      s[nb][3] += y.w;
    }
    if (!KQ)
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) put_a(x + C::S + ks * 512, plain[ks], lane);
#pragma unroll
    for (int e = 0; e < 2 * NS; ++e) put_a(x + C::X + e * 512, a[e / NS][e % NS], lane);
  }
  if (p.dh0 && cols > 0 && seg == 0) keep_state<DK>(p, p.dh0, bh, m0, cols, lane, s);
}

// Segments as in the forward walk, from their ends: dS = M dS' + N with the
// transpose of that one's M, N the walk back from zeros: 2 x 24337 x 12 x 64, in
// one piece 992 us, in segments 375: N and M 171, the chain 25, the walks 179.
// CTAs for 8 x 16 columns of [N | M] of a segment; past dk = 64 one an SM, as the
// columns of dS take half of 128 registers.
template <int DK>
struct BackMove {
  static constexpr int row = kChunk * DK * 2;
  static constexpr int q = 0, k = row, coef = 2 * row, W = coef + kCoefs * 4, bytes = W + 2 * row, stages = 3;
  static constexpr int smem = stages * bytes;
};

template <int DK>
__global__ void __launch_bounds__(kMoveThreads, DK == 64 ? 2 : 1) delta_back_move_kernel(const DeltaP p, int groups) {
  typedef __nv_bfloat16 T;
  typedef BackMove<DK> C;
  typedef ChunkData<T, DK, true, false> D;
  constexpr int NST = C::stages, NS = 2;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x, lane = tid & 31, q4 = lane & 3;
  const long long part = blockIdx.x / groups, bh = part / (p.nseg - 1);
  const int group = (int)(blockIdx.x - part * groups), seg = 1 + (int)(part - bh * (p.nseg - 1));
  const int b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv), hk = hv / (p.Hv / p.Hk);
  const int n = delta_length(p, b), all = (n + kChunk - 1) / kChunk, c0 = seg * p.seglen;
  const int nc = all - c0 < 0 ? 0 : all - c0 < p.seglen ? all - c0 : p.seglen, last = c0 + nc - 1;
  const int m0 = 16 * (group * 8 + (tid >> 5));        // the warp's first column of [N | M]
  const bool move = m0 >= p.dvp;                       // of M
  const bool mine = move ? seg < p.nseg - 1 && m0 - p.dvp < p.dk : true;
  const Rows<T> xq = rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n);
  const Rows<T> xk = rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n);
  const char* chunks = p.chunks + bh * p.nc * D::bytes;
  const float4* Z = reinterpret_cast<const float4*>(p.U) + ((bh * p.nc + last) * p.dvp + m0) * (kChunk / 4) + lane;
  const uint4* dO = p.dO + ((bh * p.nc + last) * (p.dvp / 16) + m0 / 16) * 2 * NS * 32 + lane;
  float s[DK / 8][4];
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[j][e] = move && 8 * j + 2 * q4 + (e & 1) == m0 - p.dvp + (lane >> 2) + 8 * (e >> 1) ? 1.f : 0.f;
  const auto load = [&](int i) {   // the i-th from the end
    const int c = last - i;
    const unsigned st = base + i % NST * C::bytes;
    load_tile<DK, kChunk, kMoveThreads>(st + C::q, 0, xq, c * kChunk, n, p.dk, p.q_wide, tid);
    load_tile<DK, kChunk, kMoveThreads>(st + C::k, 0, xk, c * kChunk, n, p.dk, p.k_wide, tid);
    copy_block<D::Tm - D::coef, kMoveThreads>(st + C::coef, chunks + (long long)c * D::bytes + D::coef, tid);
  };
  Raised raised;
  wait_prior();
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    if (i < nc) load(i);
    copy_commit();
  }
  const bool given = mine && !move;
  float4 next[4] = {};
  if (given && nc > 0)
#pragma unroll
    for (int e = 0; e < 4; ++e) next[e] = Z[32 * e];
  for (int i = 0; i < nc; ++i) {
    copy_wait<NST - 2>();
    __syncthreads();
    if (i + NST - 1 < nc) load(i + NST - 1);
    copy_commit();
    if (!mine) continue;
    const unsigned st = base + i % NST * C::bytes;
    const float* coef = reinterpret_cast<const float*>(smem + i % NST * C::bytes + C::coef);
    uint4 g[2][NS] = {};
    if (given)
#pragma unroll
      for (int e = 0; e < 2 * NS; ++e) g[e / NS][e % NS] = dO[32 * e];
    dO -= (p.dvp / 16) * 2 * NS * 32;
    // X^T
    float x[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
      for (int np = 0; np < 2; ++np)
        mma_tile<NS, 1, false>(x[2 * np], x[2 * np + 1], a, st + C::k + at_b_rows_n<DK>(16 * np, 16 * ks, lane), 0);
    }
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float2 l = *reinterpret_cast<const float2*>(coef + kChunk + 8 * nb + 2 * q4);
      x[nb][0] = fmaf(l.x, x[nb][0], next[nb].x);
      x[nb][1] = fmaf(l.y, x[nb][1], next[nb].y);
      x[nb][2] = fmaf(l.x, x[nb][2], next[nb].z);
      x[nb][3] = fmaf(l.y, x[nb][3], next[nb].w);
    }
    if (given && i + 1 < nc) {
      Z -= p.dvp * (kChunk / 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) next[e] = Z[32 * e];
    }
    // dS^T
    scale_by(s, coef[2 * kChunk]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(x[2 * ks], x[2 * ks + 1], a);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn)
        mma_tile<NS, NS, true>(s[2 * nn], s[2 * nn + 1], a, st + C::W + at_b_rows_k<DK, true>(16 * ks, 16 * nn, lane), C::row);
    }
    if (given) {   // dO's part added as a whole, as above: the same bits
      unsigned a[2][NS][4];
#pragma unroll
      for (int e = 0; e < 2 * NS; ++e) {
        const uint4 v = g[e / NS][e % NS];
        unsigned(&d)[4] = a[e / NS][e % NS];
        d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
      }
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn) {
        float y[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          mma_tile<NS, 1, true>(y[0], y[1], a[ks], st + C::q + at_b_rows_k<DK>(16 * ks, 16 * nn, lane), 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[2 * nn + (e >> 2)][e & 3] += y[e >> 2][e & 3];
      }
    }
    if (move) raised.after(s, coef[2 * kChunk]);
  }
  copy_wait<0>();
  if (!mine) return;
  if (m0 == p.dvp && lane == 0) p.raised[bh * p.nseg + seg] = raised.by;
  const int width = p.dvp + p.dk, cols = width - m0 < 16 ? width - m0 : 16;
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kx = 8 * j + 2 * q4 + (e & 1), col = (lane >> 2) + 8 * (e >> 1);
      if (kx < p.dk && col < cols) p.moves[((bh * p.nseg + seg) * p.dk + kx) * width + m0 + col] = s[j][e];
    }
}

// ------------------------------------------------------------- all other gradients
//
// A block of 64 tokens with the state S before it and dS' after it, D as above:
//   A = scale D o (dO R^T) (i >= j),  E = -D o (dR R^T) (i > j)
//   dQ = scale e^G o (dO S^T) + (A beta) K
//   F  = -e^G o (dR S^T) + (E beta) K                    (keys as they erase)
//   W  = e^(G_C - G) o (R dS'^T) + A^T Q + E^T K         (keys as they write)
//   dK = beta o W + F,  dbeta_i = k_i . W_i
// A decay g_t is in every factor that reaches over it: of tokens i >= t with
// the state, of tokens i < t with dS', of S with dS', and of pairs i >= t > j,
//   dg_t = sum_{i >= t} (q_i . dQ1_i + k_i . F1_i) + sum_{i < t} beta_i k_i . W1_i + e^G_C <S, dS'>
//          + sum_{i >= t > j} beta_j p_ij,   p_ij = A_ij q_i . k_j + E_ij k_i . k_j
// (dQ1, F1, W1: the first terms), each sum of its own terms alone: sums over all
// of q . dq - k . dk from t on would be shorter, but pairs on one side of t would
// have to cancel in them, and beside a strong decay nothing else is left.  With
// the pairs at hand, dbeta_j = k_j . W1_j + sum_{i >= j} p_ij.
//
// A warp has 16 rows and half or a quarter of the dk columns, and of A and E
// two blocks or one of 16 columns: eight warps and two CTAs an SM in bfloat16 up
// to dk = 64 (16 x 4096 x 8 x 64: 261 us, sixteen warps 310), else sixteen.  R,
// dR, S and dS' come in the inputs' type: in bfloat16 each is one rounding of
// 2^-9, as A beta and E beta are.  Instructions bound it, 18,100 of a warp a block
// at 49% of the issue slots, of which one in seventeen is a product: the rest
// makes tiles, D, p and the sums of it; 24% of the tensor cores', 29% of DRAM.  A
// third CTA an SM would leave a thread 80 registers, as many as its sums take.

constexpr int kPairRow = 65;   // floats of a row of p, of 64

template <typename T, int DK, int DV>
struct Grad {
  static constexpr int NI = Planes<T>::in;
  static constexpr int groups = DK == 64 && sizeof(T) == 2 ? 2 : 4, blocks = 4 / groups, threads = 128 * groups;
  static constexpr int N = DK / 8 / groups;   // a warp's blocks of eight columns
  static constexpr int row = 64 * DK * 2, val = 64 * DV * 2, sta = DV * DK * 2, pair = 64 * 64 * 2;
  static constexpr int k = 0, q = NI * row, dO = 2 * NI * row, dR = dO + NI * val, R = dR + NI * val;
  static constexpr int S = R + NI * val, dS = S + NI * sta, end = dS + NI * sta;
  static constexpr int A = dO, E = A + NI * pair, pairs = E + NI * pair;   // over the values' tiles, when they are done with
  static constexpr int last = pairs + 64 * kPairRow * 4;
  static constexpr int smem = end > last ? end : last;
};

// Blocks of 8 x 8 as the chains left them: `units` rows of eight values to
// UNITS in shared memory, zeros behind them.
template <int UNITS, int THREADS>
__device__ __forceinline__ void load_blocks(unsigned dst, int, const __nv_bfloat16* src, int units, int tid) {
#pragma unroll
  for (int i = tid; i < UNITS; i += THREADS) copy16(dst + 16 * i, src + 8 * (i < units ? i : 0), i < units);
}
template <int UNITS, int THREADS>
__device__ __forceinline__ void load_blocks(unsigned dst, int plane, const float* src, int units, int tid) {
  constexpr int N = (UNITS + THREADS - 1) / THREADS, AHEAD = N < 4 ? N : 4;
#pragma unroll 1
  for (int i = tid; i < UNITS; i += AHEAD * THREADS) {
    float v[AHEAD][8];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = i + j * THREADS;
      load8(src + 8 * (long long)k, k < units ? 8 : 0, true, v[j]);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j * THREADS < UNITS) store_planes(dst + 16 * (i + j * THREADS), plane, v[j]);
  }
}

__device__ __forceinline__ float2 pair_of(unsigned addr) {
  unsigned v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return unpack_bf16(v);
}
__device__ __forceinline__ void put_pair(unsigned addr, unsigned v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Two adjacent values, all planes.
template <int NP>
__device__ __forceinline__ float2 plane_sum(unsigned addr, int plane) {
  float2 s = pair_of(addr);
#pragma unroll
  for (int j = 1; j < NP; ++j) {
    const float2 t = pair_of(addr + j * plane);
    s.x += t.x;
    s.y += t.y;
  }
  return s;
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(Grad<T, DK, DV>::threads, Grad<T, DK, DV>::groups == 2 ? 2 : 1) delta_grad_kernel(const DeltaP p) {
  typedef Grad<T, DK, DV> G;
  constexpr int NI = G::NI, THREADS = G::threads, NQ = G::groups, N = G::N, PARTS = THREADS / 64;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 sG[64];
  __shared__ float sGrown[64], sLeft[64], sBeta[64], sI[NQ][64], sW[NQ][64], sB[64], sCol[4][64], sDot[4 * NQ];
  __shared__ float sPart[PARTS][64];
  __shared__ double sCarry;
  __shared__ bool sRoots;
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, grp = w >> 2;
  // lower rows have more blocks left of the diagonal: a scheduler's warps take a low and a high one (float32, 3 x 1021 x
  // 6 x 40 x 72: 46 us against 48; 8192 x 16 x 128 in bfloat16 172 against 177; dk = 64 in bfloat16 the same)
  const int rw = grp & 1 ? 3 - (w & 3) : w & 3;
  const int r = lane >> 2, q4 = lane & 3;
  const long long bh = blockIdx.x / p.nc64;
  const int c = (int)(blockIdx.x - bh * p.nc64);
  const int b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv), group = p.Hv / p.Hk, hk = hv / group;
  const int n = delta_length(p, b), i0 = c * kStateChunk;
  const auto token = [&](int row) -> long long {   // also of rows that the sequence does not have, -1 past L
    const int i = i0 + row;
    return i >= p.L ? -1 : (long long)b * p.L + (i < n && p.reverse ? n - 1 - i : i);
  };
  // eight values of q's or k's gradient: to their place, or per value head in fp32
  const auto put = [&](void* out, float* part, int row, int col, const float (&v)[8]) {
    const long long t = token(row);
    if (t < 0 || col >= p.dk) return;
    if (part) {
      store8(part + (t * p.Hv + hv) * p.dk + col, 8, true, v);
    } else {
      T* d = static_cast<T*>(out) + (t * p.Hk + hk) * p.dk + col;
      store8(d, 8, reinterpret_cast<uintptr_t>(d) % 16 == 0, v);
    }
  };
  if (i0 >= n) {
    const float zero[8] = {};
    for (int i = tid; i < 64 * DK / 8; i += THREADS) {
      put(p.dq, p.dq_part, i / (DK / 8), i % (DK / 8) * 8, zero);
      put(p.dk_out, p.dk_part, i / (DK / 8), i % (DK / 8) * 8, zero);
    }
    if (tid < 64 && token(tid) >= 0) {
      static_cast<T*>(p.dg)[token(tid) * p.Hv + hv] = from_f32<T>(0.f);
      static_cast<T*>(p.dbeta)[token(tid) * p.Hv + hv] = from_f32<T>(0.f);
    }
    return;
  }
  load_tile<DK, 64, THREADS>(base + G::k, G::row, rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n), i0, n, p.dk,
                             p.k_wide, tid);
  load_tile<DK, 64, THREADS>(base + G::q, G::row, rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n), i0, n, p.dk,
                             p.q_wide, tid);
  // decays; beside one above 1 each power of them is its root twice, as over 64 tokens it may be past fp32 where over 32 it
  // is not, and what it multiplies small or 0 (for blocks with none, 16 x 4096 x 8 x 64: 258 us before this, 261 with it)
  double Gs = 0.0;
  bool grows = false;
  if (tid < 64) {
    float beta = 0.f;
    if (i0 + tid < n) {
      const float g = to_f32(static_cast<const T*>(p.g)[token(tid) * p.g_ld + hv]);
      beta = to_f32(static_cast<const T*>(p.beta)[token(tid) * p.beta_ld + hv]);
      Gs = (g < -1000.f ? -1000.0 : (double)g) * 1.4426950408889634;
      grows = g > 0.f;
    }
    sBeta[tid] = beta;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, Gs, o);
      if (lane >= o) Gs += x;
    }
    if (tid == 31) sCarry = Gs;
  }
  const bool roots = __syncthreads_or(grows);
  if (tid >= 32 && tid < 64) Gs += sCarry;
  __syncthreads();
  if (tid < 64) {
    if (roots) Gs *= 0.5;
    const float hi = (float)Gs;
    sG[tid] = make_float2(hi, (float)(Gs - hi));
    sGrown[tid] = ex2(hi);
    if (tid == 63) sCarry = Gs;
    if (tid == 0) sRoots = roots;
  }
  __syncthreads();
  if (tid < 64) sLeft[tid] = ex2((float)(sCarry - Gs));

  float dP[G::blocks][2][4] = {}, dN[G::blocks][2][4] = {}, dq[N][4] = {}, f[N][4] = {}, W[N][4] = {};
  float dot = 0.f;
  wait_prior();
  for (int d0 = 0; d0 < p.dv; d0 += DV) {
    if (d0) __syncthreads();
    const int cols = p.dv - d0, some = p.dvp - d0 < DV ? p.dvp - d0 : DV;
    const long long ld = (long long)p.Hv * p.dv, head = (long long)hv * p.dv + d0;
    load_tile<DV, 64, THREADS>(base + G::dO, G::val, rows_of<T>(p, p.dout, ld, head, b, n), i0, n, cols, p.do_wide, tid);
    load_tile<DV, 64, THREADS>(base + G::dR, G::val, rows_of<T>(p, p.dv_out, ld, head, b, n), i0, n, cols, p.dv_wide, tid);
#pragma unroll
    for (int h = 0; h < 2; ++h)   // R^T of 32 tokens each
      load_blocks<DV * 4, THREADS>(base + G::R + h * G::val / 2, G::val,
                                   static_cast<const T*>(p.R) + ((bh * p.nc + 2 * c + h) * p.dvp + d0) * kChunk,
                                   i0 + h * kChunk < n ? some * 4 : 0, tid);
    const long long state = ((bh * p.nc64 + c) * p.dvp + d0) * DK;
    load_blocks<DV * DK / 8, THREADS>(base + G::S, G::sta, static_cast<const T*>(p.states) + state, some * (DK / 8), tid);
    load_blocks<DV * DK / 8, THREADS>(base + G::dS, G::sta, static_cast<const T*>(p.dstates) + state, some * (DK / 8), tid);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < DV * DK / 2; i += THREADS) {
      const float2 x = plane_sum<NI>(base + G::S + 4 * i, G::sta), y = plane_sum<NI>(base + G::dS + 4 * i, G::sta);
      dot = fmaf(x.x, y.x, fmaf(x.y, y.y, dot));
    }
#pragma unroll
    for (int ks = 0; ks < DV / 16; ++ks) {
      unsigned ao[NI][4], ad[NI][4], ar[NI][4];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const unsigned at = base + j * G::val + at_a_rows_m<DV>(16 * rw, 16 * ks, lane);
        ldsm(ao[j], at + G::dO);
        ldsm(ad[j], at + G::dR);
        ldsm_t(ar[j], base + G::R + j * G::val + (rw >> 1) * (G::val / 2) +
                          at_a_rows_k<kChunk, true>(16 * ks, 16 * (rw & 1), lane));
      }
#pragma unroll
      for (int i = 0; i < G::blocks; ++i) {
        const int np = grp + NQ * i;
        if (np <= rw)
          mma_tile2<NI, NI, true>(
              dP[i][0], dP[i][1], ao, dN[i][0], dN[i][1], ad,
              base + G::R + (np >> 1) * (G::val / 2) + at_b_rows_k<kChunk, true>(16 * ks, 16 * (np & 1), lane), G::val);
      }
#pragma unroll
      for (int nn = 0; nn < N / 2; ++nn) {
        const unsigned at = base + at_b_rows_k<DK, true>(16 * ks, 8 * N * grp + 16 * nn, lane);
        mma_tile2<NI, NI, true>(dq[2 * nn], dq[2 * nn + 1], ao, f[2 * nn], f[2 * nn + 1], ad, at + G::S, G::sta);
        mma_tile<NI, NI, true>(W[2 * nn], W[2 * nn + 1], ar, at + G::dS, G::sta);
      }
    }
  }
  dot = warp_sum(dot);
  if (sRoots) {   // a root once, the other below
    dot *= sGrown[63];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 16 * rw + r + 8 * h;
      const float grown = sGrown[row], left = sLeft[row];
#pragma unroll
      for (int nb = 0; nb < N; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          dq[nb][2 * h + e] *= grown;
          f[nb][2 * h + e] *= grown;
          W[nb][2 * h + e] *= left;
        }
    }
  }
  if (lane == 0) sDot[w] = dot;

  // the first terms, their products with q and k, and f as dK's beginning
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 16 * rw + r + 8 * h;
    const float grown = sGrown[i], left = sLeft[i], beta = sBeta[i], gq = p.scale * grown;
    float si = 0.f, sw = 0.f;
#pragma unroll
    for (int nb = 0; nb < N; ++nb) {
      const unsigned at = base + unit_at<DK>(i, N * grp + nb) + 4 * q4;
      const float2 qv = plane_sum<NI>(at + G::q, G::row), kv = plane_sum<NI>(at + G::k, G::row);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float &x = dq[nb][2 * h + e], &y = f[nb][2 * h + e];
        const float z = left * W[nb][2 * h + e], qe = e ? qv.y : qv.x, ke = e ? kv.y : kv.x;
        x *= gq;
        y *= -grown;
        si = fmaf(qe, x, fmaf(ke, y, si));
        sw = fmaf(ke, z, sw);
        y = fmaf(beta, z, y);
      }
    }
    si = quad_sum(si);
    sw = quad_sum(sw);
    if (q4 == 0) {
      sI[grp][i] = si;
      sW[grp][i] = sw;
    }
  }
  __syncthreads();   // the values' tiles are done with
  if (tid < 64) {
    float si = sI[0][tid], sw = sW[0][tid];
#pragma unroll
    for (int h = 1; h < NQ; ++h) {
      si += sI[h][tid];
      sw += sW[h][tid];
    }
    sI[0][tid] = si;
    sB[tid] = sw;
    sW[0][tid] = sw * sBeta[tid];
  }
  float* pairs = reinterpret_cast<float*>(smem + G::pairs);
#pragma unroll
  for (int i = 0; i < G::blocks; ++i) {
    const int np = grp + NQ * i;
    float col[4] = {0.f, 0.f, 0.f, 0.f};
    if (np <= rw) {
      if (sRoots) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ii = 16 * rw + r + 8 * (e >> 1 & 1), j = 16 * np + 8 * (e >> 2) + 2 * q4 + (e & 1);
          const float2 gi = sG[ii], gj = sG[j];
          const float d = ii >= j ? ex2((gi.x - gj.x) + (gi.y - gj.y)) : 0.f;
          dP[i][e >> 2][e & 3] *= d;
          dN[i][e >> 2][e & 3] *= d;
        }
      }
      float qk[2][4] = {}, kk[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        unsigned aq[NI][4], ak[NI][4];
        const unsigned aa = base + at_a_rows_m<DK>(16 * rw, 16 * ks, lane);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          ldsm(aq[j], aa + G::q + j * G::row);
          ldsm(ak[j], aa + G::k + j * G::row);
        }
        mma_tile2<NI, NI, false>(qk[0], qk[1], aq, kk[0], kk[1], ak, base + G::k + at_b_rows_n<DK>(16 * np, 16 * ks, lane),
                                 G::row);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 16 * np + 8 * h + 2 * q4;
        const float4 gj = *reinterpret_cast<const float4*>(&sG[j]);
        const float2 bj = *reinterpret_cast<const float2*>(&sBeta[j]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int ii = 16 * rw + r + 8 * half;
          const float2 gi = sG[ii];
          float av[2], ev[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = ex2(e ? (gi.x - gj.z) + (gi.y - gj.w) : (gi.x - gj.x) + (gi.y - gj.y));
            const float x = ii >= j + e ? p.scale * d * dP[i][h][2 * half + e] : 0.f;
            const float y = ii > j + e ? -d * dN[i][h][2 * half + e] : 0.f;
            const float v = fmaf(x, qk[h][2 * half + e], y * kk[h][2 * half + e]);
            pairs[ii * kPairRow + j + e] = v;
            col[2 * h + e] += v;
            av[e] = x * (e ? bj.y : bj.x);
            ev[e] = y * (e ? bj.y : bj.x);
          }
          const unsigned at = base + unit_at<64>(ii, 2 * np + h) + 4 * q4;
          unsigned t[NI];
          split<NI>(av[0], av[1], t);
#pragma unroll
          for (int y = 0; y < NI; ++y) put_pair(at + G::A + y * G::pair, t[y]);
          split<NI>(ev[0], ev[1], t);
#pragma unroll
          for (int y = 0; y < NI; ++y) put_pair(at + G::E + y * G::pair, t[y]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) col[e] += __shfl_xor_sync(0xffffffffu, col[e], o);
      if (r == 0) sCol[rw][16 * np + 8 * (e >> 1) + 2 * q4 + (e & 1)] = col[e];
    }
  }
  __syncthreads();   // A, E and p are there
  if (NQ == 2 || rw >= 2) {   // a row's sums of beta p up to each token, four threads a row
    const int i = (NQ == 2 ? tid : (rw - 2) * 32 + grp * 64 + lane) >> 2, j0 = 16 * (lane & 3);
    float* row = pairs + i * kPairRow + j0;
    float v[16], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = sum;
      sum += j0 + j < i ? sBeta[j0 + j] * row[j] : 0.f;
    }
    float before = __shfl_up_sync(0xffffffffu, sum, 1, 4), x = q4 >= 1 ? before : 0.f;
    before = __shfl_up_sync(0xffffffffu, sum, 2, 4);
    x += q4 >= 2 ? before : 0.f;
    before = __shfl_up_sync(0xffffffffu, sum, 3, 4);
    x += q4 >= 3 ? before : 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) row[j] = v[j] + x;
  }
  // dQ += (A beta) K, dK += (E beta) K + (A beta)^T Q + (E beta)^T K
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    if (ks <= rw) {
      unsigned aa[NI][4], ae[NI][4];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const unsigned at = base + j * G::pair + at_a_rows_m<64>(16 * rw, 16 * ks, lane);
        ldsm(aa[j], at + G::A);
        ldsm(ae[j], at + G::E);
      }
#pragma unroll
      for (int nn = 0; nn < N / 2; ++nn)
        mma_tile2<NI, NI, true>(dq[2 * nn], dq[2 * nn + 1], aa, f[2 * nn], f[2 * nn + 1], ae,
                                base + G::k + at_b_rows_k<DK>(16 * ks, 8 * N * grp + 16 * nn, lane), G::row);
    }
    if (ks >= rw) {
      unsigned aa[NI][4], ae[NI][4];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const unsigned at = base + j * G::pair + at_a_rows_k<64>(16 * ks, 16 * rw, lane);
        ldsm_t(aa[j], at + G::A);
        ldsm_t(ae[j], at + G::E);
      }
#pragma unroll
      for (int nn = 0; nn < N / 2; ++nn) {
        const unsigned at = base + at_b_rows_k<DK>(16 * ks, 8 * N * grp + 16 * nn, lane);
        mma_tile<NI, NI, true>(f[2 * nn], f[2 * nn + 1], aa, at + G::q, G::row);
        mma_tile<NI, NI, true>(f[2 * nn], f[2 * nn + 1], ae, at + G::k, G::row);
      }
    }
  }
  __syncthreads();   // the sums of rows are there, and q and k done with
  // dg's sums, some rows a thread
  {
    const int t = tid & 63, part = tid >> 6;
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 64 / PARTS; ++x) {
      const int i = 64 / PARTS * part + x;
      sum += i >= t ? sI[0][i] + pairs[i * kPairRow + t] : sW[0][i];
    }
    sPart[part][t] = sum;
  }
  // dQ and dK through q's and k's place, for whole rows
  if (sizeof(T) == 2 && !p.dq_part) {
#pragma unroll
    for (int nb = 0; nb < N; ++nb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned at = base + unit_at<DK>(16 * rw + r + 8 * h, N * grp + nb) + 4 * q4;
        put_pair(at + G::q, pack_bf16(dq[nb][2 * h], dq[nb][2 * h + 1]));
        put_pair(at + G::k, pack_bf16(f[nb][2 * h], f[nb][2 * h + 1]));
      }
  } else {
#pragma unroll
    for (int nb = 0; nb < N; ++nb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const long long t = token(16 * rw + r + 8 * h);
        const int col = 8 * N * grp + 8 * nb + 2 * q4;
        if (t < 0 || col >= p.dk) continue;
        const float2 x = make_float2(dq[nb][2 * h], dq[nb][2 * h + 1]), y = make_float2(f[nb][2 * h], f[nb][2 * h + 1]);
        if (p.dq_part) {
          const long long at = (t * p.Hv + hv) * p.dk + col;
          *reinterpret_cast<float2*>(p.dq_part + at) = x;
          *reinterpret_cast<float2*>(p.dk_part + at) = y;
        } else {
          const long long at = (t * p.Hk + hk) * p.dk + col;
          float* d[2] = {reinterpret_cast<float*>(p.dq) + at, reinterpret_cast<float*>(p.dk_out) + at};
          d[0][0] = x.x;
          d[0][1] = x.y;
          d[1][0] = y.x;
          d[1][1] = y.y;
        }
      }
  }
  __syncthreads();
  if (sizeof(T) == 2 && !p.dq_part) {
#pragma unroll 2
    for (int i = tid; i < 2 * 64 * (DK / 8); i += THREADS) {
      const int second = i >= 64 * (DK / 8), x = i - second * 64 * (DK / 8), row = x / (DK / 8), u = x % (DK / 8);
      const long long t = token(row);
      if (t < 0 || 8 * u >= p.dk) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(smem + (second ? G::k : G::q) + unit_at<DK>(row, u));
      T* d = static_cast<T*>(second ? p.dk_out : p.dq) + (t * p.Hk + hk) * p.dk + 8 * u;
      if (reinterpret_cast<uintptr_t>(d) % 16 == 0) {
        *reinterpret_cast<uint4*>(d) = v;
      } else {
        const unsigned s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) reinterpret_cast<unsigned short*>(d)[e] = (unsigned short)(s[e >> 1] >> 16 * (e & 1));
      }
    }
  }
  if (tid < 64 && token(tid) >= 0) {
    float dg = 0.f, db = 0.f;
    if (i0 + tid < n) {
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < 4 * NQ; ++k) d += sDot[k];
#pragma unroll
      for (int k = 0; k < PARTS; ++k) dg += sPart[k][tid];
      dg += sGrown[63] * d;
      db = sB[tid] + ((sCol[0][tid] + sCol[1][tid]) + (sCol[2][tid] + sCol[3][tid]));
    }
    static_cast<T*>(p.dg)[token(tid) * p.Hv + hv] = from_f32<T>(dg);
    static_cast<T*>(p.dbeta)[token(tid) * p.Hv + hv] = from_f32<T>(db);
  }
}

// dq and dk of a query and key head: the sum over its value heads, in order.
template <typename T>
__global__ void __launch_bounds__(256) delta_heads_kernel(const float* part_q, const float* part_k, T* dq, T* dk,
                                                          long long vectors, int units, int group) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;   // eight values of a head
  wait_prior();
  if (i >= 2 * vectors) return;
  const bool second = i >= vectors;
  const long long at = second ? i - vectors : i, head = at / units;
  const float* src = (second ? part_k : part_q) + (head * group * units + (at - head * units)) * 8;
  float s[8], v[8];
  load8(src, 8, true, s);
  for (int g = 1; g < group; ++g) {
    load8(src + (long long)g * units * 8, 8, true, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += v[e];
  }
  T* dst = (second ? dk : dq) + at * 8;
  store8(dst, 8, reinterpret_cast<uintptr_t>(dst) % 16 == 0, s);
}

template <typename T, int DK, int DV>
cudaError_t run_grad(const DeltaP& p, cudaStream_t s) {
  const auto grad = delta_grad_kernel<T, DK, DV>;
  const cudaError_t e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, Grad<T, DK, DV>::smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(grad, dim3((unsigned)((long long)p.B * p.Hv * p.nc64)), dim3(Grad<T, DK, DV>::threads),
                          (size_t)Grad<T, DK, DV>::smem, s, p);
}
// Columns of dv at a time: all of them in bfloat16, what shared memory holds in three planes.
template <int DK>
cudaError_t run_grad_any(const DeltaP& p, __nv_bfloat16*, cudaStream_t s) {
  return p.dv <= 64 ? run_grad<__nv_bfloat16, DK, 64>(p, s) : run_grad<__nv_bfloat16, DK, 128>(p, s);
}
template <int DK>
cudaError_t run_grad_any(const DeltaP& p, float*, cudaStream_t s) {
  return run_grad<float, DK, 32>(p, s);
}

template <typename T, int DK>
cudaError_t run_alone(const DeltaP& p, cudaStream_t s) {
  const auto kern = delta_back_kernel<T, DK>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Back<T, DK>::smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)((long long)p.B * p.Hv * p.slices)), dim3(128), (size_t)Back<T, DK>::smem, s, p);
}
template <typename T, int DK, int PAIRS>
cudaError_t run_team(const DeltaP& p, cudaStream_t s) {
  typedef BackTeam<T, DK, PAIRS> C;
  const auto kern = delta_back_team_kernel<T, DK, PAIRS>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  const int slices = (p.dv + C::width - 1) / C::width;
  return launch_dependent(kern, dim3((unsigned)((long long)p.B * p.Hv * p.nseg * slices)), dim3(2 * C::half),
                          (size_t)C::smem, s, p, slices);
}
// Helpers where the forward walk has them.
template <int DK>
cudaError_t run_walk(const DeltaP& p, __nv_bfloat16*, cudaStream_t s) {
  if (crowded(p)) return run_alone<__nv_bfloat16, DK>(p, s);
  if (p.nseg > 1) {
    const auto move = delta_back_move_kernel<DK>;
    cudaError_t e = cudaFuncSetAttribute(move, cudaFuncAttributeMaxDynamicSharedMemorySize, BackMove<DK>::smem);
    if (e != cudaSuccess) return e;
    const int groups = (p.dvp + p.dk + 127) / 128;
    e = launch_dependent(move, dim3((unsigned)((long long)p.B * p.Hv * (p.nseg - 1) * groups)), dim3(kMoveThreads),
                         (size_t)BackMove<DK>::smem, s, p, groups);
    if (e != cudaSuccess) return e;
    e = run_starts<true>(p, s);
    if (e != cudaSuccess) return e;
  }
  return few(p) ? run_team<__nv_bfloat16, DK, 2>(p, s) : run_team<__nv_bfloat16, DK, 4>(p, s);
}
template <int DK>
cudaError_t run_walk(const DeltaP& p, float*, cudaStream_t s) {
  if constexpr (DK == 64)
    if (few(p)) return run_team<float, DK, 2>(p, s);
  return run_alone<float, DK>(p, s);
}

template <typename T, int DK>
cudaError_t run_back(const DeltaP& p, cudaStream_t s) {
  typedef ChunkData<T, DK, true, sizeof(T) == 4> D;
  const auto prep = delta_back_prep_kernel<T, DK>;
  const int smem = D::NPP * kTile + p.slices * D::NI * kChunk * kSlice * 2;
  prep<<<(unsigned)((long long)p.B * p.Hv * p.nc), 32, smem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = run_walk<DK>(p, (T*)nullptr, s);
  if (e != cudaSuccess) return e;
  e = run_grad_any<DK>(p, (T*)nullptr, s);
  if (e != cudaSuccess || !p.dq_part) return e;
  const long long vectors = (long long)p.B * p.L * p.Hk * (p.dk / 8);
  return launch_dependent(delta_heads_kernel<T>, dim3((unsigned)((2 * vectors + 255) / 256)), dim3(256), (size_t)0, s,
                          (const float*)p.dq_part, (const float*)p.dk_part, static_cast<T*>(p.dq),
                          static_cast<T*>(p.dk_out), vectors, p.dk / 8, p.Hv / p.Hk);
}

// The workspace going back: U's place, dO's fragments, dS', the parts of dq and
// dk, and without the forward's `saved` what that would hold.
struct BackLayout {
  size_t dO, dstates, parts, part, saved, bytes;
};
BackLayout back_layout(int B, int L, int Hk, int Hv, int dk, int dv, int dtype, bool have_saved) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const DeltaLayout f = delta_layout(B, L, Hv, dk, dv, dtype, true);
  const size_t planes = dtype == DT_BF16 ? Planes<__nv_bfloat16>::mid : Planes<float>::mid;
  BackLayout l;
  l.dO = f.beside;
  l.dstates = l.dO + up((size_t)B * Hv * f.nc * kChunk * f.dvp * 2 * planes);
  l.parts = l.dstates + (f.bytes - f.states);   // as large as the states
  l.part = Hv > Hk ? up(sizeof(float) * (size_t)B * L * Hv * dk) : 0;
  l.saved = l.parts + 2 * l.part;
  l.bytes = l.saved + (have_saved ? 0 : f.bytes);
  return l;
}

}  // namespace

size_t delta_bwd_workspace_bytes(int B, int L, int Hk, int Hv, int dk, int dv, int dtype, bool have_saved) {
  return back_layout(B, L, Hk, Hv, dk, dv, dtype, have_saved).bytes;
}

cudaError_t launch_delta_bwd(const lion_delta_bwd_args& a, void* ws, cudaStream_t s) {
  const BackLayout l = back_layout(a.B, a.L, a.Hk, a.Hv, a.dk, a.dv, a.dtype, a.saved != nullptr);
  char* base = static_cast<char*>(ws);
  DeltaP p = delta_params(a, a.saved ? static_cast<char*>(const_cast<void*>(a.saved)) : base + l.saved, base, true);
  if (!a.saved) {
    const cudaError_t e = launch_delta_chain(p, a.dtype, true, s);
    if (e != cudaSuccess) return e;
  }
  p.dout = a.dout;
  p.dv_out = a.dv_out;
  p.dO = reinterpret_cast<uint4*>(base + l.dO);
  p.dstates = base + l.dstates;
  p.dh0 = a.dh0;
  p.dq = a.dq;
  p.dk_out = a.dk_out;
  p.dg = a.dg;
  p.dbeta = a.dbeta;
  if (l.part) {
    p.dq_part = reinterpret_cast<float*>(base + l.parts);
    p.dk_part = reinterpret_cast<float*>(base + l.parts + l.part);
  }
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.do_wide = rows_wide(a.dout, 0, es);
  p.dv_wide = rows_wide(a.dv_out, 0, es);
  return a.dtype == DT_BF16 ? (a.dk <= 64 ? run_back<__nv_bfloat16, 64>(p, s) : run_back<__nv_bfloat16, 128>(p, s))
                            : (a.dk <= 64 ? run_back<float, 64>(p, s) : run_back<float, 128>(p, s));
}

}  // namespace lion
