// delta_fwd.cu -- the gated delta rule over chunks: a first launch works out
// what a chunk's tokens are to one another (delta_common.cuh), all chunks at
// once; a second one walks the chunks with the state in registers.
#include "delta_chain.cuh"
#include "delta_internal.h"

namespace lion {
namespace {

// ---------------------------------------------------------- P, T, U, W of a chunk
//
// A warp a chunk.  T comes by substitution, a column a lane: t_i = I_i -
// sum_{m < i} M_im t_m, 496 products a chunk with M's rows read from shared
// memory by all lanes at once.  Its pairs of adjacent columns are the B operand
// of U^T = V^T T^T and, times -e^G of their column, the A operand of -W = -T (e^G
// o K), so that K and V stay exact.  G is summed in 64 bits and kept as two
// floats: differences within a chunk are exact to 2^-46 of its largest sum, also
// next to a decay of 0 (g = -inf, held at -1000, of which e^g is 0 in fp32 as
// well).
//
// What it writes bounds it: 16 x 4096 x 8 x 64 in bfloat16 for a training step 91
// us at 5.6 TB/s, 71% of DRAM's cycles and 45% of the issue slots.  A warp's CTA
// needs no barrier, and up to fourteen of them an SM read and write at once.

template <typename T, int DK>
struct Prep {
  static constexpr int NI = Planes<T>::in;
  static constexpr int row = kChunk * DK * 2, val = kChunk * kSlice * 2;
  static constexpr int k = 0, q = NI * row, M = 2 * NI * row, MR = kChunk + 4;   // MR: floats of a row of M
  static constexpr int v = M + kChunk * MR * 4;                                  // slices of 64 columns
  static int smem(int slices) { return v + slices * NI * val; }
};

template <typename T, int DK, bool SAVE>
__global__ void __launch_bounds__(32) delta_prep_kernel(const DeltaP p) {
  typedef Prep<T, DK> X;
  constexpr bool KQ = sizeof(T) == 4;
  typedef ChunkData<T, DK, SAVE, KQ> D;
  constexpr int NI = D::NI, NS = D::NS, NPP = D::NPP;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned base = shared_at(smem);
  const int lane = threadIdx.x, r = lane >> 2, q4 = lane & 3;
  const long long bh = blockIdx.x / p.nc;
  const int c = (int)(blockIdx.x - bh * p.nc), b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv);
  const int hk = hv / (p.Hv / p.Hk), n = delta_length(p, b), i0 = c * kChunk;
  if (i0 >= n) return;
  load_tile<DK, kChunk, 32>(base + X::k, X::row, rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n), i0, n, p.dk,
                            p.k_wide, lane);
  load_tile<DK, kChunk, 32>(base + X::q, X::row, rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n), i0, n, p.dk,
                            p.q_wide, lane);
  for (int s = 0; s < p.slices; ++s)
    load_tile<kSlice, kChunk, 32>(base + X::v + s * NI * X::val, X::val,
                                  rows_of<T>(p, p.v, p.v_ld, (long long)hv * p.dv + s * kSlice, b, n), i0, n,
                                  p.dv - s * kSlice, p.v_wide, lane);
  copy_commit();

  // decays: lane i has token i's
  const long long tok = (long long)b * p.L + (p.reverse ? n - 1 - i0 - lane : i0 + lane);
  double G = 0.0;
  float beta = 0.f;
  if (i0 + lane < n) {
    const float g = to_f32(static_cast<const T*>(p.g)[tok * p.g_ld + hv]);
    beta = to_f32(static_cast<const T*>(p.beta)[tok * p.beta_ld + hv]);
    G = (g < -1000.f ? -1000.0 : (double)g) * 1.4426950408889634;   // powers of 2
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, G, o);
    if (lane >= o) G += x;
  }
  const double last = __shfl_sync(0xffffffffu, G, 31);
  char* out = p.chunks + (long long)blockIdx.x * D::bytes;
  const float grown = ex2((float)G), hi = (float)G, lo = (float)(G - hi);
  {
    float* coef = reinterpret_cast<float*>(out + D::coef);
    coef[lane] = p.scale * grown;
    coef[kChunk + lane] = beta * ex2((float)(last - G));
    if (lane == 31) coef[2 * kChunk] = grown;
  }
  copy_wait<0>();
  __syncwarp();

  // k k^T and q k^T below the diagonal: rows 0-15 two column blocks, rows 16-31 four
  float kk[6][4] = {}, qk[6][4] = {};
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    unsigned ka[2][NI][4], qa[2][NI][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const unsigned at = base + j * X::row + at_a_rows_m<DK>(16 * m, 16 * ks, lane);
        ldsm(ka[m][j], at + X::k);
        ldsm(qa[m][j], at + X::q);
        if (KQ) {   // blocks of 8 x 8: rows 0-7 and 8-15, then the next eight columns
          unsigned* d = reinterpret_cast<unsigned*>(out + D::q + j * D::row) + lane;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int blk = ((2 * m + (e & 1)) * (DK / 8) + 2 * ks + (e >> 1)) * 32;
            d[blk] = qa[m][j][e];
            d[(D::k - D::q) / 4 + blk] = ka[m][j][e];
          }
        }
      }
#pragma unroll
    for (int np = 0; np < 2; ++np)
#pragma unroll
      for (int m = np; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const unsigned kb[4] = {ka[np][j][0], ka[np][j][2], ka[np][j][1], ka[np][j][3]};   // as B operands
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (i + j < NI) {
              mma(kk[2 * m + 2 * np], ka[m][i], kb[0], kb[1]);
              mma(kk[2 * m + 2 * np + 1], ka[m][i], kb[2], kb[3]);
              mma(qk[2 * m + 2 * np], qa[m][i], kb[0], kb[1]);
              mma(qk[2 * m + 2 * np + 1], qa[m][i], kb[2], kb[3]);
            }
        }
  }
  float* Ms = reinterpret_cast<float*>(smem + X::M);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nb = 0; nb < 2 * (m + 1); ++nb) {
      const int j = 8 * nb + 2 * q4;
      const float h0 = __shfl_sync(0xffffffffu, hi, j), h1 = __shfl_sync(0xffffffffu, hi, j + 1);
      const float l0 = __shfl_sync(0xffffffffu, lo, j), l1 = __shfl_sync(0xffffffffu, lo, j + 1);
      const float b0 = __shfl_sync(0xffffffffu, beta, j), b1 = __shfl_sync(0xffffffffu, beta, j + 1);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = 16 * m + r + 8 * half;
        const float hx = __shfl_sync(0xffffffffu, hi, i), lx = __shfl_sync(0xffffffffu, lo, i);
        const float d0 = b0 * ex2((hx - h0) + (lx - l0)), d1 = b1 * ex2((hx - h1) + (lx - l1));
        const float* a = kk[2 * m + nb] + 2 * half;
        const float* x = qk[2 * m + nb] + 2 * half;
        *reinterpret_cast<float2*>(Ms + i * X::MR + j) =
            make_float2(i > j ? d0 * a[0] : 0.f, i > j + 1 ? d1 * a[1] : 0.f);
        unsigned pp[NPP];
        split<NPP>(i >= j ? p.scale * (d0 * x[0]) : 0.f, i >= j + 1 ? p.scale * (d1 * x[1]) : 0.f, pp);
#pragma unroll
        for (int e = 0; e < NPP; ++e)
          reinterpret_cast<unsigned*>(out + D::P + e * kTile)[((2 * m + half) * 4 + nb) * 32 + lane] = pp[e];
      }
    }
  __syncwarp();
  {
    float t[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 a = *reinterpret_cast<const float4*>(Ms + i * X::MR + m);   // zeros from the diagonal on
        s0 = fmaf(-a.x, t[m], s0);
        if (m + 1 < i) s1 = fmaf(-a.y, t[m + 1], s1);
        if (m + 2 < i) s0 = fmaf(-a.z, t[m + 2], s0);
        if (m + 3 < i) s1 = fmaf(-a.w, t[m + 3], s1);
      }
      t[i] = s0 + s1;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunk; ++i) Ms[i * X::MR + lane] = t[i];
    __syncwarp();
  }
  // the 16 x 16 blocks (0, 0), (1, 0) and (1, 1) of T: pairs of rows r, columns 2 q4 of their four 8 x 8 blocks
  float2 t[3][4];
  unsigned tb[3][NS][4];   // as B operands: blocks (0, 0), (0, 1), (1, 0), (1, 1)
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int i = x ? 16 : 0, j = x == 2 ? 16 : 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[x][e] = *reinterpret_cast<const float2*>(Ms + (i + 8 * (e >> 1) + r) * X::MR + j + 8 * (e & 1) + 2 * q4);
      unsigned s[NS];
      split<NS>(t[x][e].x, t[x][e].y, s);
#pragma unroll
      for (int y = 0; y < NS; ++y) {
        tb[x][y][e] = s[y];
        if (SAVE)
          reinterpret_cast<unsigned*>(out + D::Tm + y * kTile)[((i / 8 + (e >> 1)) * 4 + j / 8 + (e & 1)) * 32 + lane] = s[y];
      }
    }
  }
  // U^T = V^T T^T, the accumulators as they are
  float4* U = reinterpret_cast<float4*>(p.U) + (long long)blockIdx.x * p.dvp * (kChunk / 4) + lane;
  for (int mt = 0; 16 * mt < p.dvp; ++mt) {
    float u[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      unsigned va[NI][4];
#pragma unroll
      for (int j = 0; j < NI; ++j)
        ldsm_t(va[j], base + X::v + (mt >> 2) * NI * X::val + j * X::val + at_a_rows_k<kSlice>(16 * ks, 16 * (mt & 3), lane));
#pragma unroll
      for (int np = ks; np < 2; ++np) {
        const int x = np + ks;
        mma_planes<NI, NS, 0>(u[2 * np], u[2 * np + 1], va, tb[x][0]);
        mma_planes<NI, NS, 1>(u[2 * np], u[2 * np + 1], va, tb[x][1]);
        if (NS > 2) mma_planes<NI, NS, 2>(u[2 * np], u[2 * np + 1], va, tb[x][NS - 1]);
      }
    }
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) U[(mt * 4 + nb) * 32] = make_float4(u[nb][0], u[nb][1], u[nb][2], u[nb][3]);
  }
  // -W = (-T e^G) K
  unsigned ta[3][NS][4];
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int j = x == 2 ? 16 : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float g0 = -__shfl_sync(0xffffffffu, grown, j + 8 * h + 2 * q4);
      const float g1 = -__shfl_sync(0xffffffffu, grown, j + 8 * h + 2 * q4 + 1);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        unsigned s[NS];
        split<NS>(g0 * t[x][2 * half + h].x, g1 * t[x][2 * half + h].y, s);
#pragma unroll
        for (int y = 0; y < NS; ++y) ta[x][y][2 * h + half] = s[y];
      }
    }
  }
#pragma unroll 2
  for (int nn = 0; nn < DK / 16; ++nn) {
    float w[2][2][4] = {};   // [row block][column block]
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int m = ks; m < 2; ++m)
        mma_tile<NS, NI, true>(w[m][0], w[m][1], ta[m + ks], base + X::k + at_b_rows_k<DK>(16 * ks, 16 * nn, lane), X::row);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          unsigned s[NS];
          split<NS>(w[m][h][2 * half], w[m][h][2 * half + 1], s);
#pragma unroll
          for (int y = 0; y < NS; ++y)
            reinterpret_cast<unsigned*>(out + D::W + y * D::row)[((2 * m + half) * (DK / 8) + 2 * nn + h) * 32 + lane] = s[y];
        }
  }
}

// ------------------------------------------------------------------ the chain
//
// A CTA holds 64 columns of a head's state, a warp 16 of them as rows of S^T;
// all a chunk does to them stays in the warp's registers, and the tiles that
// all columns share come through shared memory a few chunks ahead.  Two products
// that wait for one another bound it, and what stands beside them in one warp's
// order: 64 x 197 x 12 x 64 in bfloat16, five CTAs one after the other on an SM,
// 47 us.

template <typename T, int DK, bool SAVE>
struct Chain {
  typedef ChunkData<T, DK, SAVE, sizeof(T) == 4> D;
  typedef Stage<T, DK, D::P, D::Tm> L;
  static constexpr int stages = sizeof(T) == 4 ? 2 : 3;
  static constexpr int smem = stages * L::bytes + 4 * out_bytes<T>();
};

template <typename T, int DK, bool SAVE>
__global__ void __launch_bounds__(128) delta_chain_kernel(const DeltaP p) {
  typedef Chain<T, DK, SAVE> C;
  typedef typename C::D D;
  typedef typename C::L L;
  constexpr int NST = C::stages, NI = D::NI, NS = D::NS;
  constexpr int NO = NI == 1 ? 1 : NS;   // planes of S and R that a bfloat16 output takes: one rounding of 2^-9 each
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
  const int m0 = slice * kSlice + 16 * w;              // the warp's first column of the state
  const int cols = p.dv - m0 < 16 ? p.dv - m0 : 16;    // 0 or less: none
  const Rows<T> xq = rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n);
  const Rows<T> xk = rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n);
  const Rows<T> xo = rows_of<T>(p, p.out, (long long)p.Hv * p.dv, (long long)hv * p.dv + m0, b, n);
  const char* chunk = p.chunks + bh * p.nc * D::bytes;
  const float4* U = reinterpret_cast<const float4*>(p.U) + (bh * p.nc * p.dvp + m0) * (kChunk / 4) + lane;

  float s[DK / 8][4];   // S^T
  load_state<DK>(p, p.h0, bh, m0, cols, lane, s);
  wait_prior();
#pragma unroll
  for (int st = 0; st < NST - 1; ++st) {
    if (st < nc)
      L::template load<128>(p, base + st * L::bytes, chunk + (long long)st * D::bytes, xq, xk, st * kChunk, n, tid);
    copy_commit();
  }
  float4 next[4];
  if (cols > 0 && nc > 0)
#pragma unroll
    for (int e = 0; e < 4; ++e) next[e] = U[32 * e];
  for (int c = 0; c < nc; ++c) {
    copy_wait<NST - 2>();
    __syncthreads();
    if (c + NST - 1 < nc)
      L::template load<128>(p, base + (c + NST - 1) % NST * L::bytes, chunk + (long long)(c + NST - 1) * D::bytes, xq, xk,
                            (c + NST - 1) * kChunk, n, tid);
    copy_commit();
    if (cols <= 0) continue;
    const unsigned st = base + c % NST * L::bytes;
    const float* coef = reinterpret_cast<const float*>(smem + c % NST * L::bytes + L::at(D::coef));
    if (SAVE && c % (kStateChunk / kChunk) == 0)
      store_blocks<DK / 8>(static_cast<T*>(p.states) + ((bh * p.nc64 + c / (kStateChunk / kChunk)) * p.dvp + m0) * DK, s, lane);

    // R^T = U^T - S^T W^T; S^T Q^T
    float x[4][4], o[4][4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i][0] = next[i].x; x[i][1] = next[i].y; x[i][2] = next[i].z; x[i][3] = next[i].w;
    }
    if (c + 1 < nc) {
      U += p.dvp * (kChunk / 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) next[e] = U[32 * e];
    }
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned a[NS][4], ao[NO][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
      for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ao[i][e] = a[i][e];
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        mma_tile<NS, NS, false>(x[2 * np], x[2 * np + 1], a, st + L::at(D::W) + at_b_rows_n<DK, true>(16 * np, 16 * ks, lane),
                                L::row);
        mma_tile<NO, NI, false>(o[2 * np], o[2 * np + 1], ao, st + L::q + at_b_rows_n<DK, KQ>(16 * np, 16 * ks, lane), L::row);
      }
    }
    if (SAVE) store_blocks<4>(static_cast<T*>(p.R) + ((bh * p.nc + c) * p.dvp + m0) * kChunk, x, lane);
    // S^T = e^G_C S^T + (beta left R)^T K; O^T = scale e^G (S^T Q^T) + R^T P^T
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float2 g = *reinterpret_cast<const float2*>(coef + 8 * nb + 2 * q4);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nb][e] *= e & 1 ? g.y : g.x;
    }
    scale_by(s, coef[2 * kChunk]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const float* l = coef + kChunk + 16 * ks + 2 * q4;
      unsigned a[NS][4], ao[NO][4];
      to_a<NS>(x[2 * ks], x[2 * ks + 1], *reinterpret_cast<const float2*>(l), *reinterpret_cast<const float2*>(l + 8), a);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn)
        mma_tile<NS, NI, true>(s[2 * nn], s[2 * nn + 1], a, st + L::k + at_b_rows_k<DK, KQ>(16 * ks, 16 * nn, lane), L::row);
      to_a<NO>(x[2 * ks], x[2 * ks + 1], ao);
#pragma unroll
      for (int np = ks; np < 2; ++np)
        mma_tile<NO, NO, false>(o[2 * np], o[2 * np + 1], ao,
                                st + L::at(D::P) + at_b_rows_n<kChunk, true>(16 * np, 16 * ks, lane), kTile);
    }
    if (p.out) {
      const int i = c * kChunk + lane;
      store_rows(buf, o, lane, cols, p.o_wide, i < n ? const_cast<T*>(xo.at(i)) : nullptr);
    }
  }
  copy_wait<0>();
  if (cols <= 0) return;
  if (p.h_out) keep_state<DK>(p, p.h_out, bh, m0, cols, lane, s);
  if (p.out) zero_rows<T>(p, p.out, n, b, hv, m0, cols, p.o_wide, lane);
}

// The same with a helper to each warp: the warp has the two products between one
// state and the next, the helper the loads, the output and what the gradients
// keep.  One warp for all of it is 1206 ns a chunk at 2 x
// 24337 x 12 x 64, of which the loads are 256, the output 227, U's read 146;
// two warps with half of the tokens and of dk each took longer (1430), as every
// half has to pass between them within a chunk.  With helpers, and the tiles two
// chunks ahead on their way to L2, a chunk of 64 columns takes 1130 ns where an
// SM has one CTA (16 x 4096 x 8 x 64: 145 us): 32% of the tensor cores' and 32% of
// the issue slots, the rest what one product waits for another, shared memory
// and the chunk's barrier.  Copies by the bulk engine into rings two chunks
// ahead were no faster (1066 to 1108 against 1066).
//
// Four pairs put a warp and its helper on each of an SM's four schedulers, two
// pairs (32 columns) every warp on one of its own: for walks of no more such CTAs
// than SMs, 3 heads of 197 x 64 in bfloat16 7.7 us against 9.4, and in float32,
// where six products for one keep a scheduler's tensor core busy, 3 x 1021 x 6 x
// 40 x 72 52 us, back 49, against 77 and 83 with four pairs and 84 and 76 without
// helpers.  Float32's longer walks than that have none.  At the border and twice
// past it, in bfloat16 with two and with four pairs, forward and back: 152 CTAs (1 x
// 480 x 76 x 64) 16 and 20 us, 20 and 23; (1 x 480 x 38 x 128) 24 and 27, 29 and 35;
// 304 CTAs (2 x 480 x 76 x 64) 22 and 21, 27 and 25; (1 x 480 x 76 x 128) 45 and 29, 56 and 36.

// PAIRS: of a warp and its helper in a CTA.
template <typename T, int DK, bool SAVE, int PAIRS>
struct Team {
  static constexpr int width = 16 * PAIRS, half = 32 * PAIRS;   // columns; threads of the warps, and of the helpers
  static constexpr bool KQ = sizeof(T) == 4;
  typedef ChunkData<T, DK, SAVE, KQ> D;
  static constexpr int NO = D::NI == 1 ? 1 : D::NS;   // planes of S, R and P that the output takes, as above
  static constexpr int row = kChunk * DK * 2;
  // a stage: q, k, P, coefficients and -W, the slice of U
  static constexpr int q = 0, k = D::NI * row, P = 2 * D::NI * row, coef = P + NO * kTile, W = coef + (D::W - D::coef);
  static constexpr int U = W + (D::Tm - D::W), bytes = U + width * kChunk * 4, stages = 3;
  // a warp's buffer to its helper: operands in bfloat16, float32's sums as they are
  static constexpr int S = 0, R = DK / 16 * (KQ ? 1024 : 512), swap = R + 2 * (KQ ? 1024 : 512);
  static constexpr int swaps = stages * bytes, out = swaps + 2 * PAIRS * swap, smem = out + PAIRS * out_bytes<T>();
  static_assert(smem <= 227 * 1024 - 1024);
};

template <typename T, int DK, bool SAVE, int PAIRS>
__global__ void __launch_bounds__(64 * PAIRS, DK == 64 && sizeof(T) == 2 ? 2 : 1)
    delta_team_kernel(const DeltaP p, int slices) {
  typedef Team<T, DK, SAVE, PAIRS> C;
  typedef typename C::D D;
  constexpr int NST = C::stages, NI = D::NI, NS = D::NS, NO = C::NO, PER = kStateChunk / kChunk;
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
  const bool ends = seg == p.nseg - 1;
  const int nc = all - c0 < 0 ? 0 : ends || all - c0 < p.seglen ? all - c0 : p.seglen;   // chunks of the segment, from c0 on
  const int m0 = slice * C::width + 16 * w, cols = p.dv - m0 < 16 ? p.dv - m0 : 16;
  const unsigned swap = base + C::swaps + w * C::swap;   // the second buffer PAIRS swaps behind
  wait_prior();
  if (helper) {
    const Rows<T> xq = rows_of<T>(p, p.q, p.q_ld, (long long)hk * p.dk, b, n);
    const Rows<T> xk = rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n);
    const Rows<T> xo = rows_of<T>(p, p.out, (long long)p.Hv * p.dv, (long long)hv * p.dv + m0, b, n);
    const char* chunks = p.chunks + (bh * p.nc + c0) * D::bytes;
    const float* Us = p.U + ((bh * p.nc + c0) * p.dvp + slice * C::width) * kChunk;
    const int rows = p.dvp - slice * C::width < C::width ? p.dvp - slice * C::width : C::width;
    unsigned char* buf = smem + C::out + w * out_bytes<T>();
    const auto load = [&](int c) {
      const unsigned st = base + c % NST * C::bytes;
      const char* chunk = chunks + (long long)c * D::bytes;
      if (KQ) {
        copy_block<2 * NI * C::row, HALF>(st, chunk, tid);
      } else {
        load_tile<DK, kChunk, HALF>(st + C::k, 0, xk, (c0 + c) * kChunk, n, p.dk, p.k_wide, tid);
        load_tile<DK, kChunk, HALF>(st + C::q, 0, xq, (c0 + c) * kChunk, n, p.dk, p.q_wide, tid);
      }
      copy_block<NO * kTile, HALF>(st + C::P, chunk + D::P, tid);
      copy_block<D::Tm - D::coef, HALF>(st + C::coef, chunk + D::coef, tid);
      copy_slice<C::width, HALF>(st + C::U, Us + (long long)c * p.dvp * kChunk, rows, tid);
    };
    if (nc > 0) load(0);
    copy_commit();
    for (int i = 0; i <= nc; ++i) {
      copy_wait<0>();
      __syncthreads();
      if (i + 1 < nc) load(i + 1);
      copy_commit();
      if (i + 2 < nc) {   // a load has a chunk's time, which covers L2's latency and not HBM's
        to_l2<D::Tm - D::P, HALF>(chunks + (long long)(i + 2) * D::bytes + D::P, D::Tm - D::P, tid);
        to_l2<C::width * kChunk * 4, HALF>(Us + (long long)(i + 2) * p.dvp * kChunk, rows * kChunk * 4, tid);
        if constexpr (KQ) {
          to_l2<2 * NI * C::row, HALF>(chunks + (long long)(i + 2) * D::bytes, 2 * NI * C::row, tid);
        } else {
          rows_to_l2(xk, (c0 + i + 2) * kChunk, n, tid - (HALF - 64));
          rows_to_l2(xq, (c0 + i + 2) * kChunk, n, tid - (HALF - 32));
        }
      }
      if (i == 0 || cols <= 0) continue;
      const unsigned st = base + (i - 1) % NST * C::bytes, x = swap + (i - 1 & 1) * PAIRS * C::swap;
      const float* coef = reinterpret_cast<const float*>(smem + (i - 1) % NST * C::bytes + C::coef);
      const int c = c0 + i - 1;
      // O^T = scale e^G (S^T Q^T) + R^T P^T
      float o[4][4] = {};
      unsigned a[DK / 16][NO][4], r[2][NO][4];
      if constexpr (KQ) {
        float s[DK / 8][4], rs[4][4];
        get_sums(x + C::S, s, lane);
        get_sums(x + C::R, rs, lane);
        if (SAVE) {
          if (c % PER == 0)
            store_blocks<DK / 8>(static_cast<T*>(p.states) + ((bh * p.nc64 + c / PER) * p.dvp + m0) * DK, s, lane);
          store_blocks<4>(static_cast<T*>(p.R) + ((bh * p.nc + c) * p.dvp + m0) * kChunk, rs, lane);
        }
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) to_a<NO>(s[2 * ks], s[2 * ks + 1], a[ks]);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) to_a<NO>(rs[2 * ks], rs[2 * ks + 1], r[ks]);
      } else {
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) get_a(x + C::S + ks * 512, a[ks][0], lane);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) get_a(x + C::R + ks * 512, r[ks][0], lane);
      }
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks)
#pragma unroll
        for (int np = 0; np < 2; ++np)
          mma_tile<NO, NI, false>(o[2 * np], o[2 * np + 1], a[ks], st + C::q + at_b_rows_n<DK, KQ>(16 * np, 16 * ks, lane), C::row);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const float2 g = *reinterpret_cast<const float2*>(coef + 8 * nb + 2 * q4);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nb][e] *= e & 1 ? g.y : g.x;
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int np = ks; np < 2; ++np)
          mma_tile<NO, NO, false>(o[2 * np], o[2 * np + 1], r[ks],
                                  st + C::P + at_b_rows_n<kChunk, true>(16 * np, 16 * ks, lane), kTile);
      if constexpr (SAVE && !KQ) {
        if (c % PER == 0)
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            store_a<DK / 8>(static_cast<T*>(p.states) + ((bh * p.nc64 + c / PER) * p.dvp + m0) * DK + ks * 128, a[ks][0], lane);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          store_a<4>(static_cast<T*>(p.R) + ((bh * p.nc + c) * p.dvp + m0) * kChunk + ks * 128, r[ks][0], lane);
      }
      if (p.out) {
        const int t = c * kChunk + lane;
        store_rows(buf, o, lane, cols, p.o_wide, t < n ? const_cast<T*>(xo.at(t)) : nullptr);
      }
    }
    if (p.out && cols > 0 && ends) zero_rows<T>(p, p.out, n, b, hv, m0, cols, p.o_wide, lane);
    return;
  }
  float s[DK / 8][4];   // S^T
  seg > 0 ? load_state<DK>(p, p.starts, bh * p.nseg + seg, m0, cols, lane, s) : load_state<DK>(p, p.h0, bh, m0, cols, lane, s);
  for (int i = 0; i <= nc; ++i) {
    __syncthreads();
    if (i == nc || cols <= 0) continue;
    const unsigned st = base + i % NST * C::bytes, x = swap + (i & 1) * PAIRS * C::swap;
    const float* coef = reinterpret_cast<const float*>(smem + i % NST * C::bytes + C::coef);
    if (KQ) put_sums(x + C::S, s, lane);
    float r[4][4];
    unsigned plain[DK / 16][4], rplain[2][1][4];   // to the helper at the end: a store would hold back the reads behind it
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float4 u = get_f4(st + C::U + (w * 4 + nb) * 512, lane);
      r[nb][0] = u.x; r[nb][1] = u.y; r[nb][2] = u.z; r[nb][3] = u.w;
    }
    // R^T = U^T - S^T W^T
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
      for (int e = 0; e < 4; ++e) plain[ks][e] = a[0][e];
#pragma unroll
      for (int np = 0; np < 2; ++np)
        mma_tile<NS, NS, false>(r[2 * np], r[2 * np + 1], a, st + C::W + at_b_rows_n<DK, true>(16 * np, 16 * ks, lane), C::row);
    }
    if (KQ) put_sums(x + C::R, r, lane);
    // S^T = e^G_C S^T + (beta left R)^T K
    scale_by(s, coef[2 * kChunk]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const float* l = coef + kChunk + 16 * ks + 2 * q4;
      unsigned a[NS][4];
      to_a<NS>(r[2 * ks], r[2 * ks + 1], *reinterpret_cast<const float2*>(l), *reinterpret_cast<const float2*>(l + 8), a);
      to_a<1>(r[2 * ks], r[2 * ks + 1], rplain[ks]);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn)
        mma_tile<NS, NI, true>(s[2 * nn], s[2 * nn + 1], a, st + C::k + at_b_rows_k<DK, KQ>(16 * ks, 16 * nn, lane), C::row);
    }
    if constexpr (!KQ) {
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) put_a(x + C::S + ks * 512, plain[ks], lane);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) put_a(x + C::R + ks * 512, rplain[ks][0], lane);
    }
  }
  if (p.h_out && cols > 0 && ends) keep_state<DK>(p, p.h_out, bh, m0, cols, lane, s);
}

// ------------------------------------------------------------------- segments
//
// Few heads leave most SMs idle, and a head's chunks follow one another.  Then
// a sequence is cut into segments.  A segment makes S' = M S + N of the state
// before it; N is its walk from zeros (the first one's from the state that is
// given), M the walk of the identity with U = 0, both without outputs and all
// segments' at once.  A second launch chains them, and the walks with outputs
// start from there.  Three walks' work for one, so only where it finds idle SMs:
// 2 x 24337 x 12 x 64, 24 heads, in one piece 896 us, in 12 segments 363: prep 93,
// M and N 130, the chain 26, the walks 115.

template <int DK>
struct Move {
  static constexpr int row = kChunk * DK * 2;
  static constexpr int k = 0, coef = row, W = coef + kCoefs * 4, bytes = W + 2 * row, stages = 3, smem = stages * bytes;
};

// CTAs for 8 x 16 columns of [N | M] of a segment, two an SM: past dk = 64 that
// spills 92 bytes a thread and is as fast as one that does not (1 x 8192 x 8/16 x
// 128: 117 us against 118).
template <int DK, bool SAVE>
__global__ void __launch_bounds__(kMoveThreads, 2) delta_move_kernel(const DeltaP p, int groups) {
  typedef __nv_bfloat16 T;
  typedef Move<DK> C;
  typedef ChunkData<T, DK, SAVE, false> D;
  constexpr int NST = C::stages, NS = 2;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x, lane = tid & 31, q4 = lane & 3;
  const long long part = blockIdx.x / groups, bh = part / (p.nseg - 1);
  const int group = (int)(blockIdx.x - part * groups), seg = (int)(part - bh * (p.nseg - 1));
  const int b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv), hk = hv / (p.Hv / p.Hk);
  const int n = delta_length(p, b), all = (n + kChunk - 1) / kChunk, c0 = seg * p.seglen;
  const int nc = all - c0 < 0 ? 0 : all - c0 < p.seglen ? all - c0 : p.seglen;
  const int m0 = 16 * (group * 8 + (tid >> 5));        // the warp's first column of [N | M]
  const bool move = m0 >= p.dvp;                       // of M
  const bool mine = move ? seg > 0 && m0 - p.dvp < p.dk : true;
  const Rows<T> xk = rows_of<T>(p, p.k, p.k_ld, (long long)hk * p.dk, b, n);
  const char* chunks = p.chunks + (bh * p.nc + c0) * D::bytes;
  const float4* U = reinterpret_cast<const float4*>(p.U) + ((bh * p.nc + c0) * p.dvp + m0) * (kChunk / 4) + lane;
  float s[DK / 8][4];
  if (move) {
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 8 * j + 2 * q4 + (e & 1) == m0 - p.dvp + (lane >> 2) + 8 * (e >> 1) ? 1.f : 0.f;
  } else {
    load_state<DK>(p, seg == 0 ? p.h0 : nullptr, bh, m0, p.dv - m0 < 16 ? p.dv - m0 : 16, lane, s);
  }
  const auto load = [&](int c) {
    const unsigned st = base + c % NST * C::bytes;
    load_tile<DK, kChunk, kMoveThreads>(st + C::k, 0, xk, (c0 + c) * kChunk, n, p.dk, p.k_wide, tid);
    copy_block<D::Tm - D::coef, kMoveThreads>(st + C::coef, chunks + (long long)c * D::bytes + D::coef, tid);
  };
  Raised raised;
  wait_prior();
#pragma unroll
  for (int c = 0; c < NST - 1; ++c) {
    if (c < nc) load(c);
    copy_commit();
  }
  float4 next[4] = {};
  if (mine && !move && nc > 0)
#pragma unroll
    for (int e = 0; e < 4; ++e) next[e] = U[32 * e];
  for (int c = 0; c < nc; ++c) {
    copy_wait<NST - 2>();
    __syncthreads();
    if (c + NST - 1 < nc) load(c + NST - 1);
    copy_commit();
    if (!mine) continue;
    const unsigned st = base + c % NST * C::bytes;
    const float* coef = reinterpret_cast<const float*>(smem + c % NST * C::bytes + C::coef);
    float r[4][4];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      r[nb][0] = next[nb].x; r[nb][1] = next[nb].y; r[nb][2] = next[nb].z; r[nb][3] = next[nb].w;
    }
    if (!move && c + 1 < nc) {
      U += p.dvp * (kChunk / 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) next[e] = U[32 * e];
    }
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
      for (int np = 0; np < 2; ++np)
        mma_tile<NS, NS, false>(r[2 * np], r[2 * np + 1], a, st + C::W + at_b_rows_n<DK, true>(16 * np, 16 * ks, lane), C::row);
    }
    scale_by(s, coef[2 * kChunk]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const float* l = coef + kChunk + 16 * ks + 2 * q4;
      unsigned a[NS][4];
      to_a<NS>(r[2 * ks], r[2 * ks + 1], *reinterpret_cast<const float2*>(l), *reinterpret_cast<const float2*>(l + 8), a);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn)
        mma_tile<NS, 1, true>(s[2 * nn], s[2 * nn + 1], a, st + C::k + at_b_rows_k<DK>(16 * ks, 16 * nn, lane), 0);
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

template <typename T, int DK, bool SAVE>
cudaError_t run_alone(const DeltaP& p, cudaStream_t s) {
  typedef Chain<T, DK, SAVE> C;
  const auto kern = delta_chain_kernel<T, DK, SAVE>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)((long long)p.B * p.Hv * p.slices)), dim3(128), (size_t)C::smem, s, p);
}
template <typename T, int DK, bool SAVE, int PAIRS>
cudaError_t run_team(const DeltaP& p, cudaStream_t s) {
  typedef Team<T, DK, SAVE, PAIRS> C;
  const auto kern = delta_team_kernel<T, DK, SAVE, PAIRS>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  const int slices = (p.dv + C::width - 1) / C::width;
  return launch_dependent(kern, dim3((unsigned)((long long)p.B * p.Hv * p.nseg * slices)), dim3(2 * C::half),
                          (size_t)C::smem, s, p, slices);
}
// Helpers make a chunk's walk shorter, and fewer CTAs fit an SM: with them two at
// dk = 64, one back and at dk = 128; without three, at dk = 128 two, one with
// `saved` and back.  One rule for all, helpers for up to two walks an SM; us with
// them and alone, forward with `saved`, then back:
//   4 x 4096 x 38 x 64, 152 walks  152 180  178 220    4 x 4096 x 19 x 128, 152  211 233  272 288
//   4 x 4096 x 64 x 64, 256 walks  242 248  345 276    4 x 4096 x 32 x 128, 256  411 452  535 562
//   4 x 4096 x 77 x 64, 308 walks  380 349  515 401    4 x 4096 x 39 x 128, 312  617 675  801 844
// and at dk = 128 without `saved` 193 249, 378 359 and 568 563.  In float32 at dk
// > 64 three stages do not fit.
template <int DK, bool SAVE>
cudaError_t run_walk(const DeltaP& p, float*, cudaStream_t s) {
  if constexpr (DK == 64)
    if (few(p)) return run_team<float, DK, SAVE, 2>(p, s);
  return run_alone<float, DK, SAVE>(p, s);
}
template <int DK, bool SAVE>
cudaError_t run_walk(const DeltaP& p, __nv_bfloat16*, cudaStream_t s) {
  const unsigned heads = (unsigned)((long long)p.B * p.Hv);
  cudaError_t e;
  if (crowded(p)) return run_alone<__nv_bfloat16, DK, SAVE>(p, s);
  if (p.nseg > 1) {
    const auto move = delta_move_kernel<DK, SAVE>;
    e = cudaFuncSetAttribute(move, cudaFuncAttributeMaxDynamicSharedMemorySize, Move<DK>::smem);
    if (e != cudaSuccess) return e;
    const int groups = (p.dvp + p.dk + 127) / 128;
    e = launch_dependent(move, dim3(heads * (p.nseg - 1) * groups), dim3(kMoveThreads), (size_t)Move<DK>::smem, s, p, groups);
    if (e != cudaSuccess) return e;
    e = run_starts<false>(p, s);
    if (e != cudaSuccess) return e;
  }
  return few(p) ? run_team<__nv_bfloat16, DK, SAVE, 2>(p, s) : run_team<__nv_bfloat16, DK, SAVE, 4>(p, s);
}

template <typename T, int DK, bool SAVE>
cudaError_t run_chain(const DeltaP& p, cudaStream_t s) {
  const auto prep = delta_prep_kernel<T, DK, SAVE>;
  cudaError_t e = cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, Prep<T, DK>::smem(2));
  if (e != cudaSuccess) return e;
  prep<<<(unsigned)((long long)p.B * p.Hv * p.nc), 32, Prep<T, DK>::smem(p.slices), s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return run_walk<DK, SAVE>(p, (T*)nullptr, s);
}
template <typename T>
cudaError_t run_chain_any(const DeltaP& p, bool save, cudaStream_t s) {
  return p.dk <= 64 ? (save ? run_chain<T, 64, true>(p, s) : run_chain<T, 64, false>(p, s))
                    : (save ? run_chain<T, 128, true>(p, s) : run_chain<T, 128, false>(p, s));
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaP& p, int dtype, bool save, cudaStream_t s) {
  return dtype == DT_BF16 ? run_chain_any<__nv_bfloat16>(p, save, s) : run_chain_any<float>(p, save, s);
}

size_t delta_saved_bytes(int B, int L, int Hv, int dk, int dv, int dtype) {
  return delta_layout(B, L, Hv, dk, dv, dtype, true).bytes;
}
size_t delta_workspace_bytes(int B, int L, int Hv, int dk, int dv, int dtype, bool save) {
  const DeltaLayout l = delta_layout(B, L, Hv, dk, dv, dtype, save);
  return l.beside + (save ? 0 : l.bytes);
}

cudaError_t launch_delta_fwd(const lion_delta_args& a, void* ws, cudaStream_t s) {
  const bool save = a.saved != nullptr;
  const DeltaLayout l = delta_layout(a.B, a.L, a.Hv, a.dk, a.dv, a.dtype, save);
  char* beside = static_cast<char*>(ws);
  DeltaP p = delta_params(a, save ? static_cast<char*>(a.saved) : beside + l.beside, beside, save);
  p.out = a.out;
  p.h_out = a.h_out;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.o_wide = rows_wide(a.out, 0, es);
  return launch_delta_chain(p, a.dtype, save, s);
}

}  // namespace lion
