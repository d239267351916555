// delta_fwd.cu -- the gated delta rule over chunks: a first launch works out
// what a chunk's tokens are to one another (T and P of delta_common.cuh, and
// the decays), all chunks at once; a second one walks the chunks with the state
// in registers.
#include "delta_chain.cuh"
#include "delta_internal.h"

namespace lion {
namespace {

// ------------------------------------------------------------ T, P and decays
//
// A warp a chunk.  A lane reads 16 bytes of a row where the products take two
// blocks of eight: which columns meet in a product is free as long as both
// factors agree, so eight adjacent values of q and k serve as columns 2c, 2c + 1
// and 2c + 8, 2c + 9 of two products.  The same registers are A operand and B
// operand.  T comes by substitution, a column a lane: t_i = I_i - sum_{m < i}
// M_im t_m, 496 products a chunk with M's rows read from shared memory by all
// lanes at once.  G is summed in 64 bits and kept as two floats: differences
// within a chunk are exact to 2^-46 of its largest sum, also next to a decay of
// 0 (g = -inf, held at -1000, of which e^g is 0 in fp32 as well).

constexpr int kPrepWarps = 4;

// Eight values of a row (zeros if it is not there) as packed pairs in NP planes.
template <typename T, int NP>
__device__ __forceinline__ void row8(const T* s, bool there, bool wide, unsigned (&w)[4][NP]) {
  if (NP == 1 && wide) {
    const uint4 r = there ? *reinterpret_cast<const uint4*>(s) : make_uint4(0, 0, 0, 0);
    w[0][0] = r.x; w[1][0] = r.y; w[2][0] = r.z; w[3][0] = r.w;
  } else {
    float v[8];
    load8(s, there ? 8 : 0, wide, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) split<NP>(v[2 * e], v[2 * e + 1], w[e]);
  }
}

template <typename T, int DK, int NPP>   // NPP: planes of P
__global__ void __launch_bounds__(32 * kPrepWarps) delta_prep_kernel(const DeltaP p, long long chunks) {
  constexpr int NI = Planes<T>::in, NS = Planes<T>::mid;
  __shared__ __align__(16) float sh[kPrepWarps][kChunk][kChunk + 4];
  __shared__ float2 shG[kPrepWarps][kChunk];
  __shared__ float shB[kPrepWarps][kChunk];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long at = (long long)blockIdx.x * kPrepWarps + w;
  if (at >= chunks) return;
  const long long bh = at / p.nc;
  const int c = (int)(at - bh * p.nc), b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv);
  const int hk = hv / (p.Hv / p.Hk), n = delta_length(p, b), i0 = c * kChunk;
  if (i0 >= n) return;
  char* tp = static_cast<char*>(p.tp) + at * p.tp_chunk;

  // decays: lane i has token i's
  const int mine = i0 + lane;
  const long long tok = (long long)b * p.L + (p.reverse ? n - 1 - mine : mine);
  double G = 0.0;
  float beta = 0.f;
  if (mine < n) {
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
  {
    float* coef = reinterpret_cast<float*>(tp + (NS + NPP) * kTile);
    const float grown = ex2((float)G);
    coef[lane] = grown;
    coef[kChunk + lane] = p.scale * grown;
    coef[2 * kChunk + lane] = ex2((float)(last - G));
    coef[3 * kChunk + lane] = beta;
    const float hi = (float)G;
    shG[w][lane] = make_float2(hi, (float)(G - hi));
    shB[w][lane] = beta;
  }

  // k k^T and q k^T below the diagonal: rows 0-15 two column blocks, rows 16-31 four
  const int r = lane >> 2, q4 = lane & 3;
  float kk[6][4], qk[6][4];
#pragma unroll
  for (int i = 0; i < 6; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[i][e] = qk[i][e] = 0.f;
  const T* kb = static_cast<const T*>(p.k) + (long long)hk * p.dk;
  const T* qb = static_cast<const T*>(p.q) + (long long)hk * p.dk;
  long long kr[4], qr[4];
  bool in[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = i0 + r + 8 * e;
    in[e] = i < n;
    const long long t = (long long)b * p.L + (in[e] ? (p.reverse ? n - 1 - i : i) : 0);
    kr[e] = t * p.k_ld;
    qr[e] = t * p.q_ld;
  }
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    const int col = 32 * s + 8 * q4;
    unsigned kw[4][4][NI], qw[4][4][NI];   // [row block][pair][plane]
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool there = in[e] && col < p.dk;
      row8<T, NI>(kb + kr[e] + col, there, p.k_wide, kw[e]);
      row8<T, NI>(qb + qr[e] + col, there, p.q_wide, qw[e]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)   // pairs 0, 1, then 2, 3
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if (i + j < NI)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const unsigned ka[4] = {kw[2 * m][2 * h][i], kw[2 * m + 1][2 * h][i], kw[2 * m][2 * h + 1][i],
                                      kw[2 * m + 1][2 * h + 1][i]};
              const unsigned qa[4] = {qw[2 * m][2 * h][i], qw[2 * m + 1][2 * h][i], qw[2 * m][2 * h + 1][i],
                                      qw[2 * m + 1][2 * h + 1][i]};
#pragma unroll
              for (int nb = 0; nb < 2 * (m + 1); ++nb) {
                mma(kk[2 * m + nb], ka, kw[nb][2 * h][j], kw[nb][2 * h + 1][j]);
                mma(qk[2 * m + nb], qa, kw[nb][2 * h][j], kw[nb][2 * h + 1][j]);
              }
            }
  }
  __syncwarp();
  unsigned char* tT = reinterpret_cast<unsigned char*>(tp);
  unsigned char* tPp = reinterpret_cast<unsigned char*>(tp) + NS * kTile;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nb = 0; nb < 2 * (m + 1); ++nb)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = 16 * m + r + 8 * half, j = 8 * nb + 2 * q4;
        const float2 gi = shG[w][i], g0 = shG[w][j], g1 = shG[w][j + 1];
        const float d0 = ex2((gi.x - g0.x) + (gi.y - g0.y)), d1 = ex2((gi.x - g1.x) + (gi.y - g1.y));
        const float* a = kk[2 * m + nb] + 2 * half;
        const float* x = qk[2 * m + nb] + 2 * half;
        *reinterpret_cast<float2*>(&sh[w][i][j]) =
            make_float2(i > j ? d0 * a[0] * shB[w][j] : 0.f, i > j + 1 ? d1 * a[1] * shB[w][j + 1] : 0.f);
        unsigned pp[NPP];
        split<NPP>(i >= j ? p.scale * (d0 * x[0]) : 0.f, i >= j + 1 ? p.scale * (d1 * x[1]) : 0.f, pp);
#pragma unroll
        for (int e = 0; e < NPP; ++e)
          *reinterpret_cast<unsigned*>(tPp + e * kTile + unit_at<kChunk>(i, j >> 3) + 2 * (j & 7)) = pp[e];
      }
  __syncwarp();
  float t[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
    for (int m = 0; m < i; m += 4) {
      const float4 a = *reinterpret_cast<const float4*>(&sh[w][i][m]);   // zeros from the diagonal on
      s0 = fmaf(-a.x, t[m], s0);
      if (m + 1 < i) s1 = fmaf(-a.y, t[m + 1], s1);
      if (m + 2 < i) s0 = fmaf(-a.z, t[m + 2], s0);
      if (m + 3 < i) s1 = fmaf(-a.w, t[m + 3], s1);
    }
    t[i] = s0 + s1;
  }
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    unsigned pl[NS];
    split<NS>(t[i], 0.f, pl);
#pragma unroll
    for (int e = 0; e < NS; ++e)
      *reinterpret_cast<unsigned short*>(tT + e * kTile + unit_at<kChunk>(i, lane >> 3) + 2 * (lane & 7)) =
          (unsigned short)pl[e];
  }
}

// ------------------------------------------------------------------ the chain
//
// A CTA holds 64 columns of a head's state, a warp 16 of them as rows of S^T;
// all a chunk does to them stays in the warp's registers, and the tiles that
// all columns share (K, Q, T, P) come through shared memory a few chunks ahead.

template <typename T, int DK, bool SAVE>
struct Chain {
  static constexpr int NPP = SAVE || sizeof(T) == 4 ? Planes<T>::mid : 1;
  static constexpr int stages = sizeof(T) == 4 ? 2 : 3;
  static constexpr int smem = stages * ChainTiles<T, DK, NPP>::bytes + 4 * kOutBytes;
};

template <typename T, int DK, bool SAVE>
__global__ void __launch_bounds__(128) delta_chain_kernel(const DeltaP p) {
  constexpr int NPP = Chain<T, DK, SAVE>::NPP, NST = Chain<T, DK, SAVE>::stages;
  constexpr int NI = Planes<T>::in, NS = Planes<T>::mid;
  constexpr int NO = NI == 1 ? 1 : NS;   // planes of S and U that a bfloat16 output takes: one rounding of 2^-9 each
  typedef ChainTiles<T, DK, NPP> L;
  extern __shared__ __align__(1024) unsigned char smem[];
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int r = lane >> 2, q4 = lane & 3;
  float* buf = reinterpret_cast<float*>(smem + NST * L::bytes + w * kOutBytes);
  const long long bh = blockIdx.x / p.slices;
  const int slice = (int)(blockIdx.x - bh * p.slices);
  const int b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv), hk = hv / (p.Hv / p.Hk);
  const int n = delta_length(p, b), nc = (n + kChunk - 1) / kChunk;
  const int m0 = slice * kSlice + 16 * w;              // the warp's first column of the state
  const int cols = p.dv - m0 < 16 ? p.dv - m0 : 16;    // 0 or less: none

  float s[DK / 8][4];   // S^T
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kx = 8 * j + 2 * q4 + (e & 1), col = r + 8 * (e >> 1);
      s[j][e] = p.h0 && kx < p.dk && col < cols ? p.h0[(bh * p.dk + kx) * p.dv + m0 + col] : 0.f;
    }
  wait_prior();
#pragma unroll
  for (int st = 0; st < NST - 1; ++st) {
    if (st < nc) load_chunk<T, DK, NPP>(p, base + st * L::bytes, st, b, hv, hk, slice, n, p.v, p.v_ld, p.v_wide, tid);
    copy_commit();
  }
  for (int c = 0; c < nc; ++c) {
    copy_wait<NST - 2>();
    __syncthreads();
    if (c + NST - 1 < nc)
      load_chunk<T, DK, NPP>(p, base + (c + NST - 1) % NST * L::bytes, c + NST - 1, b, hv, hk, slice, n, p.v, p.v_ld,
                             p.v_wide, tid);
    copy_commit();
    if (cols <= 0) continue;
    const unsigned st = base + c % NST * L::bytes;
    const float* coef = reinterpret_cast<const float*>(smem + c % NST * L::bytes + L::coef);

    if (SAVE && c % (kStateChunk / kChunk) == 0)
      save_state<T, DK>(p, p.states, bh, c / (kStateChunk / kChunk), s, m0, cols, lane);

    // S^T K^T and S^T Q^T
    float x[4][4], o[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = o[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        const unsigned at = at_b_rows_n<DK>(16 * np, 16 * ks, lane);
        unsigned bk[4];
#define LION_PLANE(J)                                                          \
  if (J < NI) {                                                                \
    ldsm(bk, st + L::k + J * L::row + at);                                     \
    mma_planes<NS, NI, J>(x[2 * np], x[2 * np + 1], a, bk);                    \
    ldsm(bk, st + L::q + J * L::row + at);                                     \
    if (NO == 1) {                                                             \
      mma(o[2 * np], a[0], bk[0], bk[1]);                                      \
      mma(o[2 * np + 1], a[0], bk[2], bk[3]);                                  \
    } else {                                                                   \
      mma_planes<NS, NI, J>(o[2 * np], o[2 * np + 1], a, bk);                  \
    }                                                                          \
  }
        LION_PLANE(0) LION_PLANE(1) LION_PLANE(2)
#undef LION_PLANE
      }
    }
    // X^T = V^T - e^G (S^T K^T)
#pragma unroll
    for (int np = 0; np < 2; ++np) {
      float v[2][4] = {};
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        unsigned t[4];
        ldsm_t(t, st + L::v + j * L::val + at_a_rows_k<kSlice>(16 * np, 16 * w, lane));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16(t[e]);
          v[e >> 1][2 * (e & 1)] += f.x;
          v[e >> 1][2 * (e & 1) + 1] += f.y;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 g = *reinterpret_cast<const float2*>(coef + 16 * np + 8 * h + 2 * q4);
        const float2 gq = *reinterpret_cast<const float2*>(coef + kChunk + 16 * np + 8 * h + 2 * q4);
        float(&xx)[4] = x[2 * np + h];
        float(&oo)[4] = o[2 * np + h];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xx[e] = fmaf(-(e & 1 ? g.y : g.x), xx[e], v[h][e]);
          oo[e] *= e & 1 ? gq.y : gq.x;
        }
      }
    }
    // R^T = X^T T^T, below the diagonal
    float u[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      unsigned a[NS][4];
      to_a<NS>(x[2 * ks], x[2 * ks + 1], a);
#pragma unroll
      for (int np = ks; np < 2; ++np) {
        const unsigned at = st + L::tp + at_b_rows_n<kChunk>(16 * np, 16 * ks, lane);
        unsigned bt[4];
        ldsm(bt, at);
        mma_planes<NS, NS, 0>(u[2 * np], u[2 * np + 1], a, bt);
        ldsm(bt, at + kTile);
        mma_planes<NS, NS, 1>(u[2 * np], u[2 * np + 1], a, bt);
        if (NS > 2) {
          ldsm(bt, at + 2 * kTile);
          mma_planes<NS, NS, 2>(u[2 * np], u[2 * np + 1], a, bt);
        }
      }
    }
    if (SAVE) {
      T* to = static_cast<T*>(p.R) + ((bh * p.nc + c) * kChunk) * p.dv + m0;
      store_rows<T>(buf, u, lane, cols, true, [&](int t) { return to + (long long)t * p.dv; });
    }
    // U = beta R; O^T += U^T P^T; S^T = e^G_C S^T + (left U)^T K
    const float last = coef[kChunk - 1];
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] *= last;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int j0 = 16 * ks + 2 * q4;
      const float2 b0 = *reinterpret_cast<const float2*>(coef + 3 * kChunk + j0);
      const float2 b1 = *reinterpret_cast<const float2*>(coef + 3 * kChunk + j0 + 8);
      const float2 l0 = *reinterpret_cast<const float2*>(coef + 2 * kChunk + j0);
      const float2 l1 = *reinterpret_cast<const float2*>(coef + 2 * kChunk + j0 + 8);
      {
        unsigned a[NO][4];
        to_a<NO>(u[2 * ks], u[2 * ks + 1], b0, b1, a);
#pragma unroll
        for (int np = ks; np < 2; ++np) {
          const unsigned at = st + L::tp + NS * kTile + at_b_rows_n<kChunk>(16 * np, 16 * ks, lane);
          unsigned bt[4];
          ldsm(bt, at);
          mma_planes<NO, NO, 0>(o[2 * np], o[2 * np + 1], a, bt);
          if (NO > 1) {
            ldsm(bt, at + kTile);
            mma_planes<NO, NO, 1>(o[2 * np], o[2 * np + 1], a, bt);
            ldsm(bt, at + 2 * kTile);
            mma_planes<NO, NO, 2>(o[2 * np], o[2 * np + 1], a, bt);
          }
        }
      }
      unsigned a[NS][4];
      to_a<NS>(u[2 * ks], u[2 * ks + 1], make_float2(b0.x * l0.x, b0.y * l0.y), make_float2(b1.x * l1.x, b1.y * l1.y),
               a);
#pragma unroll
      for (int nn = 0; nn < DK / 16; ++nn) {
        const unsigned at = st + L::k + at_b_rows_k<DK>(16 * ks, 16 * nn, lane);
        unsigned bk[4];
        ldsm_t(bk, at);
        mma_planes<NS, NI, 0>(s[2 * nn], s[2 * nn + 1], a, bk);
        if (NI > 1) {
          ldsm_t(bk, at + L::row);
          mma_planes<NS, NI, 1>(s[2 * nn], s[2 * nn + 1], a, bk);
          ldsm_t(bk, at + 2 * L::row);
          mma_planes<NS, NI, 2>(s[2 * nn], s[2 * nn + 1], a, bk);
        }
      }
    }
    if (p.out)
      store_rows<T>(buf, o, lane, cols, p.o_wide, [&](int t) -> T* {
        const int i = c * kChunk + t;
        if (i >= n) return nullptr;
        return static_cast<T*>(p.out) + (((long long)b * p.L + (p.reverse ? n - 1 - i : i)) * p.Hv + hv) * p.dv + m0;
      });
  }
  copy_wait<0>();
  if (cols <= 0) return;
  if (p.h_out) {
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kx = 8 * j + 2 * q4 + (e & 1), col = r + 8 * (e >> 1);
        if (kx < p.dk && col < cols) p.h_out[(bh * p.dk + kx) * p.dv + m0 + col] = s[j][e];
      }
  }
  if (p.out) zero_rows<T>(p, p.out, n, b, hv, m0, cols, p.o_wide, lane);
}

template <typename T, int DK, bool SAVE>
cudaError_t run_chain(const DeltaP& p, cudaStream_t s) {
  typedef Chain<T, DK, SAVE> C;
  const long long chunks = (long long)p.B * p.Hv * p.nc;
  delta_prep_kernel<T, DK, C::NPP><<<(unsigned)((chunks + kPrepWarps - 1) / kPrepWarps), 32 * kPrepWarps, 0, s>>>(p, chunks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const auto kern = delta_chain_kernel<T, DK, SAVE>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)((long long)p.B * p.Hv * p.slices)), dim3(128), C::smem, s, p);
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
size_t delta_workspace_bytes(int B, int L, int Hv, int dk, int dv, int dtype) {
  return delta_layout(B, L, Hv, dk, dv, dtype, false).bytes;
}

cudaError_t launch_delta_fwd(const lion_delta_args& a, void* ws, cudaStream_t s) {
  DeltaP p = delta_params(a, a.saved ? a.saved : ws, a.saved != nullptr);
  p.out = a.out;
  p.h_out = a.h_out;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.o_wide = rows_wide(a.out, 0, es);
  return launch_delta_chain(p, a.dtype, a.saved != nullptr, s);
}

}  // namespace lion
