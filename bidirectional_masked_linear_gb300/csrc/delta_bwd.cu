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
// (scale e^G o dO)^T as its A operands.

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
  const long long bh = blockIdx.x / p.slices;
  const int slice = (int)(blockIdx.x - bh * p.slices);
  const int b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv), hk = hv / (p.Hv / p.Hk);
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
//          + sum_{i >= t > j} beta_j (A_ij q_i . k_j + E_ij k_i . k_j)
// (dQ1, F1, W1: the first terms), each sum of its own terms alone: sums over all
// of q . dq - k . dk from t on would be shorter, but pairs on one side of t would
// have to cancel in them, and beside a strong decay nothing else is left.
//
// A warp has 16 rows and 64 of the dk columns.  R, dR, S and dS' come in the
// inputs' type: in bfloat16 each is one rounding of 2^-9, as A and E are.

constexpr int kPairRow = 65;

template <typename T, int DK>
struct Grad {
  static constexpr int NI = Planes<T>::in;
  static constexpr int halves = DK / 64, warps = 4 * halves;
  static constexpr int dvs = sizeof(T) == 4 ? 32 : 64;   // columns of dv at a time: what shared memory holds
  static constexpr int row = 64 * DK * 2, val = 64 * dvs * 2, sta = dvs * DK * 2, pair = 64 * 64 * 2;
  static constexpr int k = 0, q = NI * row, dO = 2 * NI * row, dR = dO + NI * val, R = dR + NI * val;
  static constexpr int S = R + NI * val, dS = S + NI * sta, end = dS + NI * sta;
  static constexpr int A = dO, E = A + NI * pair;        // over the values' tiles, when they are done with
  static constexpr int pairs = E + NI * pair, last = pairs + 64 * kPairRow * 4;   // the pairs' terms, fp32
  static constexpr int smem = end > last ? end : last;
};

// Blocks of 8 x 8 as the chains left them: `units` rows of eight values to
// UNITS in shared memory, zeros behind them.
template <int UNITS, int THREADS>
__device__ __forceinline__ void load_blocks(unsigned dst, int, const __nv_bfloat16* src, int units, int tid) {
#pragma unroll
  for (int k = 0; k < UNITS / THREADS; ++k) {
    const int i = tid + k * THREADS;
    copy16(dst + 16 * i, src + 8 * (i < units ? i : 0), i < units);
  }
  static_assert(UNITS % THREADS == 0, "");
}
template <int UNITS, int THREADS>
__device__ __forceinline__ void load_blocks(unsigned dst, int plane, const float* src, int units, int tid) {
#pragma unroll 2
  for (int i = tid; i < UNITS; i += THREADS) {
    float v[8];
    load8(src + 8 * (long long)i, i < units ? 8 : 0, true, v);
    store_planes(dst + 16 * i, plane, v);
  }
}

__device__ __forceinline__ float2 pair_of(unsigned addr) {
  unsigned v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return unpack_bf16(v);
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
template <int W, int NP>
__device__ __forceinline__ float2 tile_pair(unsigned tile, int plane, int row, int col) {
  return plane_sum<NP>(tile + unit_at<W>(row, col >> 3) + 2 * (col & 7), plane);
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <typename T, int DK>
__global__ void __launch_bounds__(32 * Grad<T, DK>::warps, DK == 64 ? 2 : 1) delta_grad_kernel(const DeltaP p) {
  typedef Grad<T, DK> G;
  constexpr int NI = G::NI, THREADS = 32 * G::warps;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 sG[64];
  __shared__ float sGrown[64], sLeft[64], sBeta[64], sI[2][64], sW[2][64], sB[2][64], sDot[G::warps];
  __shared__ double sCarry;
  const unsigned base = shared_at(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, rw = w & 3, half = w >> 2;
  const int r = lane >> 2, q4 = lane & 3;
  const long long bh = blockIdx.x / p.nc64;
  const int c = (int)(blockIdx.x - bh * p.nc64);
  const int b = (int)(bh / p.Hv), hv = (int)(bh - (long long)b * p.Hv), group = p.Hv / p.Hk, hk = hv / group;
  const int n = delta_length(p, b), i0 = c * kStateChunk;
  const auto token = [&](int row) -> long long {   // also of rows that the sequence does not have, -1 past L
    const int i = i0 + row;
    return i >= p.L ? -1 : (long long)b * p.L + (i < n && p.reverse ? n - 1 - i : i);
  };
  // the gradients of q and k: to their places, or per value head in fp32
  const auto put = [&](void* out, float* part, int row, int col, float x, float y) {
    const long long t = token(row);
    if (t < 0 || col >= p.dk) return;
    if (part) {
      *reinterpret_cast<float2*>(part + (t * p.Hv + hv) * p.dk + col) = make_float2(x, y);
    } else {
      T* d = static_cast<T*>(out) + (t * p.Hk + hk) * p.dk + col;
      d[0] = from_f32<T>(x);
      d[1] = from_f32<T>(y);
    }
  };
  if (i0 >= n) {
    for (int i = tid; i < 64 * DK / 2; i += THREADS) {
      put(p.dq, p.dq_part, i / (DK / 2), i % (DK / 2) * 2, 0.f, 0.f);
      put(p.dk_out, p.dk_part, i / (DK / 2), i % (DK / 2) * 2, 0.f, 0.f);
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
  // decays
  double Gs = 0.0;
  if (tid < 64) {
    float beta = 0.f;
    if (i0 + tid < n) {
      const float g = to_f32(static_cast<const T*>(p.g)[token(tid) * p.g_ld + hv]);
      beta = to_f32(static_cast<const T*>(p.beta)[token(tid) * p.beta_ld + hv]);
      Gs = (g < -1000.f ? -1000.0 : (double)g) * 1.4426950408889634;
    }
    sBeta[tid] = beta;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, Gs, o);
      if (lane >= o) Gs += x;
    }
    if (tid == 31) sCarry = Gs;
  }
  __syncthreads();
  if (tid >= 32 && tid < 64) Gs += sCarry;
  __syncthreads();
  if (tid < 64) {
    const float hi = (float)Gs;
    sG[tid] = make_float2(hi, (float)(Gs - hi));
    sGrown[tid] = ex2(hi);
    if (tid == 63) sCarry = Gs;
  }
  __syncthreads();
  if (tid < 64) sLeft[tid] = ex2((float)(sCarry - Gs));

  float dP[8][4] = {}, N[8][4] = {}, dq[8][4] = {}, f[8][4] = {}, W[8][4] = {};
  float dot = 0.f;
  wait_prior();
  for (int d0 = 0; d0 < p.dv; d0 += G::dvs) {
    if (d0) __syncthreads();
    const int cols = p.dv - d0, some = p.dvp - d0 < G::dvs ? p.dvp - d0 : G::dvs;
    const long long ld = (long long)p.Hv * p.dv, head = (long long)hv * p.dv + d0;
    load_tile<G::dvs, 64, THREADS>(base + G::dO, G::val, rows_of<T>(p, p.dout, ld, head, b, n), i0, n, cols, p.do_wide, tid);
    load_tile<G::dvs, 64, THREADS>(base + G::dR, G::val, rows_of<T>(p, p.dv_out, ld, head, b, n), i0, n, cols, p.dv_wide, tid);
#pragma unroll
    for (int h = 0; h < 2; ++h)   // R^T of 32 tokens each
      load_blocks<G::dvs * 4, THREADS>(base + G::R + h * G::val / 2, G::val,
                                       static_cast<const T*>(p.R) + ((bh * p.nc + 2 * c + h) * p.dvp + d0) * kChunk,
                                       i0 + h * kChunk < n ? some * 4 : 0, tid);
    const long long state = ((bh * p.nc64 + c) * p.dvp + d0) * DK;
    load_blocks<G::dvs * DK / 8, THREADS>(base + G::S, G::sta, static_cast<const T*>(p.states) + state, some * (DK / 8), tid);
    load_blocks<G::dvs * DK / 8, THREADS>(base + G::dS, G::sta, static_cast<const T*>(p.dstates) + state, some * (DK / 8), tid);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < G::dvs * DK / 2; i += THREADS) {
      const float2 x = plane_sum<NI>(base + G::S + 4 * i, G::sta), y = plane_sum<NI>(base + G::dS + 4 * i, G::sta);
      dot = fmaf(x.x, y.x, fmaf(x.y, y.y, dot));
    }
#pragma unroll
    for (int ks = 0; ks < G::dvs / 16; ++ks) {
      unsigned ao[NI][4], ad[NI][4], ar[NI][4];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const unsigned at = base + j * G::val + at_a_rows_m<G::dvs>(16 * rw, 16 * ks, lane);
        ldsm(ao[j], at + G::dO);
        ldsm(ad[j], at + G::dR);
        ldsm_t(ar[j], base + G::R + j * G::val + (rw >> 1) * (G::val / 2) +
                          at_a_rows_k<kChunk, true>(16 * ks, 16 * (rw & 1), lane));
      }
#pragma unroll
      for (int np = 0; np < 4; ++np)
        if (np <= rw) {
          const unsigned at =
              base + G::R + (np >> 1) * (G::val / 2) + at_b_rows_k<kChunk, true>(16 * ks, 16 * (np & 1), lane);
          unsigned x[4];
#define LION_PLANE(J)                                               \
  if (J < NI) {                                                     \
    ldsm_t(x, at + J * G::val);                                     \
    mma_planes<NI, NI, J>(dP[2 * np], dP[2 * np + 1], ao, x);       \
    mma_planes<NI, NI, J>(N[2 * np], N[2 * np + 1], ad, x);         \
  }
          LION_PLANE(0) LION_PLANE(1) LION_PLANE(2)
#undef LION_PLANE
        }
#pragma unroll
      for (int nn = 0; nn < 4; ++nn) {
        const unsigned at = base + at_b_rows_k<DK, true>(16 * ks, 64 * half + 16 * nn, lane);
        unsigned x[4];
#define LION_PLANE(J)                                               \
  if (J < NI) {                                                     \
    ldsm_t(x, at + G::S + J * G::sta);                              \
    mma_planes<NI, NI, J>(dq[2 * nn], dq[2 * nn + 1], ao, x);       \
    mma_planes<NI, NI, J>(f[2 * nn], f[2 * nn + 1], ad, x);         \
    ldsm_t(x, at + G::dS + J * G::sta);                             \
    mma_planes<NI, NI, J>(W[2 * nn], W[2 * nn + 1], ar, x);         \
  }
        LION_PLANE(0) LION_PLANE(1) LION_PLANE(2)
#undef LION_PLANE
      }
    }
  }
  dot = warp_sum(dot);
  if (lane == 0) sDot[w] = dot;

  // the first terms, and their products with q and k
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 16 * rw + r + 8 * h;
    const float grown = sGrown[i], left = sLeft[i];
    float si = 0.f, sw = 0.f;
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      const float2 qv = tile_pair<DK, NI>(base + G::q, G::row, i, 64 * half + 8 * nb + 2 * q4);
      const float2 kv = tile_pair<DK, NI>(base + G::k, G::row, i, 64 * half + 8 * nb + 2 * q4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dq[nb][2 * h + e] *= p.scale * grown;
        f[nb][2 * h + e] *= -grown;
        W[nb][2 * h + e] *= left;
        const float qe = e ? qv.y : qv.x, ke = e ? kv.y : kv.x;
        si = fmaf(qe, dq[nb][2 * h + e], fmaf(ke, f[nb][2 * h + e], si));
        sw = fmaf(ke, W[nb][2 * h + e], sw);
      }
    }
    si = quad_sum(si);
    sw = quad_sum(sw);
    if (q4 == 0) {
      sI[half][i] = si;
      sW[half][i] = sw * sBeta[i];
    }
  }
  // A and E, in the registers of dP and N
#pragma unroll
  for (int nb = 0; nb < 8; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * rw + r + 8 * (e >> 1), j = 8 * nb + 2 * q4 + (e & 1);
      const float2 gi = sG[i], gj = sG[j];
      const float d = i >= j ? ex2((gi.x - gj.x) + (gi.y - gj.y)) : 0.f;
      dP[nb][e] = i >= j ? p.scale * d * dP[nb][e] : 0.f;
      N[nb][e] = i > j ? -d * N[nb][e] : 0.f;
    }
  __syncthreads();   // the values' tiles are done with
#pragma unroll
  for (int nb = 0; nb < 8; ++nb)
    if (nb < 2 * rw + 2)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned at = base + unit_at<64>(16 * rw + r + 8 * h, nb) + 4 * q4;
        unsigned t[NI];
        if (half == 0) {
          split<NI>(dP[nb][2 * h], dP[nb][2 * h + 1], t);
#pragma unroll
          for (int j = 0; j < NI; ++j) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + G::A + j * G::pair), "r"(t[j]) : "memory");
        }
        if (half == G::halves - 1) {
          split<NI>(N[nb][2 * h], N[nb][2 * h + 1], t);
#pragma unroll
          for (int j = 0; j < NI; ++j) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + G::E + j * G::pair), "r"(t[j]) : "memory");
        }
      }
  // the pairs' terms; with two halves each has every other block
  float* pairs = reinterpret_cast<float*>(smem + G::pairs);
#pragma unroll
  for (int np = 0; np < 4; ++np)
    if (np <= rw && np % G::halves == half) {
      float qk[2][4] = {}, kk[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        unsigned aq[NI][4], ak[NI][4], x[4];
        const unsigned aa = base + at_a_rows_m<DK>(16 * rw, 16 * ks, lane);
        const unsigned bb = base + G::k + at_b_rows_n<DK>(16 * np, 16 * ks, lane);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          ldsm(aq[j], aa + G::q + j * G::row);
          ldsm(ak[j], aa + G::k + j * G::row);
        }
#define LION_PLANE(J)                                    \
  if (J < NI) {                                          \
    ldsm(x, bb + J * G::row);                            \
    mma_planes<NI, NI, J>(qk[0], qk[1], aq, x);          \
    mma_planes<NI, NI, J>(kk[0], kk[1], ak, x);          \
  }
        LION_PLANE(0) LION_PLANE(1) LION_PLANE(2)
#undef LION_PLANE
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int nb = 2 * np + h, i = 16 * rw + r + 8 * (e >> 1), j = 8 * nb + 2 * q4 + (e & 1);
          pairs[i * kPairRow + j] = sBeta[j] * fmaf(dP[nb][e], qk[h][e], N[nb][e] * kk[h][e]);
        }
    }
  // dQ += (A beta) K, F += (E beta) K
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    if (ks <= rw) {
      const int j0 = 16 * ks + 2 * q4;
      const float2 b0 = make_float2(sBeta[j0], sBeta[j0 + 1]), b1 = make_float2(sBeta[j0 + 8], sBeta[j0 + 9]);
      unsigned aa[NI][4], ae[NI][4];
      to_a<NI>(dP[2 * ks], dP[2 * ks + 1], b0, b1, aa);
      to_a<NI>(N[2 * ks], N[2 * ks + 1], b0, b1, ae);
#pragma unroll
      for (int nn = 0; nn < 4; ++nn) {
        const unsigned at = base + G::k + at_b_rows_k<DK>(16 * ks, 64 * half + 16 * nn, lane);
        unsigned x[4];
#define LION_PLANE(J)                                               \
  if (J < NI) {                                                     \
    ldsm_t(x, at + J * G::row);                                     \
    mma_planes<NI, NI, J>(dq[2 * nn], dq[2 * nn + 1], aa, x);       \
    mma_planes<NI, NI, J>(f[2 * nn], f[2 * nn + 1], ae, x);         \
  }
        LION_PLANE(0) LION_PLANE(1) LION_PLANE(2)
#undef LION_PLANE
      }
    }
#pragma unroll
  for (int nb = 0; nb < 8; ++nb)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      put(p.dq, p.dq_part, 16 * rw + r + 8 * h, 64 * half + 8 * nb + 2 * q4, dq[nb][2 * h], dq[nb][2 * h + 1]);
  __syncthreads();   // A and E are there
  if (rw >= 2 && half == 0) {   // a pair row's sums up to each token; the warps with the fewest products below
    float* row = pairs + (tid - 64) * kPairRow;
    float sum = 0.f;
#pragma unroll 8
    for (int j = 0; j < 64; ++j) {
      const float x = j < tid - 64 ? row[j] : 0.f;
      row[j] = sum;
      sum += x;
    }
  }
  // W += A^T Q + E^T K
#pragma unroll
  for (int ib = 0; ib < 4; ++ib)
    if (ib >= rw) {
      unsigned aa[NI][4], ae[NI][4];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const unsigned at = base + j * G::pair + at_a_rows_k<64>(16 * ib, 16 * rw, lane);
        ldsm_t(aa[j], at + G::A);
        ldsm_t(ae[j], at + G::E);
      }
#pragma unroll
      for (int nn = 0; nn < 4; ++nn) {
        const unsigned at = base + at_b_rows_k<DK>(16 * ib, 64 * half + 16 * nn, lane);
        unsigned x[4];
#define LION_PLANE(J)                                               \
  if (J < NI) {                                                     \
    ldsm_t(x, at + G::q + J * G::row);                              \
    mma_planes<NI, NI, J>(W[2 * nn], W[2 * nn + 1], aa, x);         \
    ldsm_t(x, at + G::k + J * G::row);                              \
    mma_planes<NI, NI, J>(W[2 * nn], W[2 * nn + 1], ae, x);         \
  }
        LION_PLANE(0) LION_PLANE(1) LION_PLANE(2)
#undef LION_PLANE
      }
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 16 * rw + r + 8 * h;
    const float beta = sBeta[i];
    float sb = 0.f;
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      const int col = 64 * half + 8 * nb + 2 * q4;
      const float2 kv = tile_pair<DK, NI>(base + G::k, G::row, i, col);
      sb = fmaf(kv.x, W[nb][2 * h], fmaf(kv.y, W[nb][2 * h + 1], sb));
      put(p.dk_out, p.dk_part, i, col, fmaf(beta, W[nb][2 * h], f[nb][2 * h]),
          fmaf(beta, W[nb][2 * h + 1], f[nb][2 * h + 1]));
    }
    sb = quad_sum(sb);
    if (q4 == 0) sB[half][i] = sb;
  }
  __syncthreads();
  if (tid < 64 && token(tid) >= 0) {
    float dg = 0.f, db = 0.f;
    if (i0 + tid < n) {
      float inner = 0.f, before = 0.f, across = 0.f;
#pragma unroll 8
      for (int i = 0; i < 64; ++i) {
        float a = 0.f, bw = 0.f;
#pragma unroll
        for (int h = 0; h < G::halves; ++h) {
          a += sI[h][i];
          bw += sW[h][i];
        }
        if (i >= tid) {
          inner += a;
          across += pairs[i * kPairRow + tid];
        } else {
          before += bw;
        }
      }
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < G::warps; ++k) d += sDot[k];
      dg = inner + before + across + sGrown[63] * d;
#pragma unroll
      for (int h = 0; h < G::halves; ++h) db += sB[h][tid];
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

template <typename T, int DK>
cudaError_t run_back(const DeltaP& p, cudaStream_t s) {
  typedef ChunkData<T, DK, true, sizeof(T) == 4> D;
  const auto prep = delta_back_prep_kernel<T, DK>;
  const int smem = D::NPP * kTile + p.slices * D::NI * kChunk * kSlice * 2;
  prep<<<(unsigned)((long long)p.B * p.Hv * p.nc), 32, smem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const auto back = delta_back_kernel<T, DK>;
  e = cudaFuncSetAttribute(back, cudaFuncAttributeMaxDynamicSharedMemorySize, Back<T, DK>::smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(back, dim3((unsigned)((long long)p.B * p.Hv * p.slices)), dim3(128), (size_t)Back<T, DK>::smem, s, p);
  if (e != cudaSuccess) return e;
  const auto grad = delta_grad_kernel<T, DK>;
  e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, Grad<T, DK>::smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(grad, dim3((unsigned)((long long)p.B * p.Hv * p.nc64)), dim3(32 * Grad<T, DK>::warps),
                       (size_t)Grad<T, DK>::smem, s, p);
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
  l.dO = f.U;
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
