// delta_common.cuh -- what the gated delta rule's chunk kernels share: the
// formulas' names, split operands, fragments and tiles.
//
// A chunk of C tokens with the state S before it, G the inclusive sums of the
// logarithms g of its decays and D_ij = e^(G_i - G_j) for i >= j:
//   M_ij = D_ij (k_i . k_j) beta_j  (i > j),   T = (I + M)^-1
//   R = T (V - e^G o (K S)) = U - W S,  U = T V,  W = T (e^G o K)
//   O = scale e^G o (Q S) + P R,  P_ij = scale D_ij (q_i . k_j) beta_j  (i >= j)
//   S' = e^G_C S + (beta e^(G_C - G) o K)^T R
// T, U, W and P need no state: all chunks have theirs worked out at once, and
// the walk over the chunks has two products between one state and the next.  R
// does not depend on where the chunks are cut; it is what the gradients start
// from.  Given dO and dS' the gradients run back with
//   X = P^T dO + beta e^(G_C - G) o (K dS'),  dR = T^T X = dV
//   dS = e^G_C dS' + (scale e^G o Q)^T dO - W^T X
//
// Products run on the tensor cores in bfloat16 with fp32 sums.  A factor is a
// sum of planes, x = bf16(x) + bf16(x - bf16(x)) + ...: bfloat16 inputs are one
// plane and exact; what is computed (states, T, W, R, P) has two planes beside
// them, 2^-18 of a value, which keeps the float32 state that a call hands back
// to about 1e-6; float32 inputs and everything beside them have three, 2^-26.
// Products of planes i and j with i + j past the finer factor's last plane are
// below its rounding and are left out.
//
// A step's products are 16 columns of the state by 32 tokens by 64: too small
// to fill a tcgen05 tile, and each waits for the one before.  mma.sync takes
// them from registers to registers in 20 clocks, where a tile in tensor memory
// would go out and back between any two.
#pragma once

#include "lion_internal.h"
#include "ssm_common.cuh"

namespace lion {

struct DeltaP {
  const void *q, *k, *v, *g, *beta, *dout;
  const int* lengths;
  const float* h0;
  void* out;
  float* h_out;
  char* chunks;            // per head and chunk: a ChunkData
  float* U;                // per head and chunk: U^T in fragments; going back P^T dO
  uint4* dO;               // per head and chunk: (scale e^G o dO)^T in fragments
  void *R, *states;        // per head: R^T in blocks of 32 tokens, S^T before every 64th token; NULL: not wanted
  void *dv_out, *dstates;  // gradients: dV [B][L][Hv][dv]; dS' as states
  float* dh0;
  void *dq, *dk_out, *dg, *dbeta;
  float *dq_part, *dk_part;   // per value head, [B][L][Hv][dk], where a query head has several
  long long q_ld, k_ld, v_ld, g_ld, beta_ld;
  int B, L, Hk, Hv, dk, dv, dvp, nc, nc64, slices;   // dvp: dv up to whole warps' 16
  int nseg, seglen;        // the forward walk's segments, of seglen chunks
  float *moves, *starts;   // per head and segment: what it makes of a state, [dk][dvp + dk]; the state before it, [dk][dv]
  int* raised;             // per head and segment: M is 2^raised times what moves holds of it
  float scale;
  int reverse;
  int q_wide, k_wide, v_wide, o_wide, do_wide, dv_wide;
};

namespace {

constexpr int kChunk = 32;          // tokens of a step of the chains
constexpr int kSlice = 64;          // columns of the state a chain's CTA holds, 16 a warp
constexpr int kStateChunk = 64;     // tokens between saved states, and of a block of the gradients
constexpr int kTile = kChunk * kChunk * 2;   // bytes of a plane of T or P
// a chunk's coefficients: scale e^G, beta e^(G_C - G), then e^G_C
constexpr int kCoefs = 2 * kChunk + 16;

// Planes of an input and of what is computed from it.
template <typename T>
struct Planes {
  static constexpr int in = 1, mid = 2;
};
template <>
struct Planes<float> {
  static constexpr int in = 3, mid = 3;
};

// What the chains need of a chunk, in bytes from its start: copies of q and k
// where the chains do not read the tensors themselves (KQ), P, coefficients,
// -W, and for the gradients (SAVE) T.
template <typename T, int DK, bool SAVE, bool KQ>
struct ChunkData {
  static constexpr int NI = Planes<T>::in, NS = Planes<T>::mid;
  static constexpr int NPP = SAVE || NI > 1 ? NS : 1;   // planes of P: one for a bfloat16 output alone
  static constexpr int row = kChunk * DK * 2;
  static constexpr int q = 0, k = NI * row, P = KQ ? 2 * NI * row : 0, coef = P + NPP * kTile, W = coef + kCoefs * 4;
  static constexpr int Tm = W + NS * row, bytes = Tm + (SAVE ? NS * kTile : 0);
};

__device__ __forceinline__ int delta_length(const DeltaP& p, int b) {
  if (!p.lengths) return p.L;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// ------------------------------------------------------------------ fragments
//
// mma.m16n8k16, lane l, c = l % 4, r = l / 4: an accumulator holds rows r and
// r + 8, columns 2c and 2c + 1; an A operand the same of two 8-column blocks,
// so that accumulators become A operands in place; a B operand holds column r
// and rows 2c, 2c + 1 (and 8 more).  The chains keep everything transposed --
// S^T, R^T, O^T have the state's columns as rows -- so that a warp's 16 columns
// never leave its registers.

__device__ __forceinline__ void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm_t(unsigned addr, unsigned a, unsigned b, unsigned c, unsigned d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&b);
}
// A pair in NP planes.
template <int NP>
__device__ __forceinline__ void split(float x, float y, unsigned (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    p[i] = pack_bf16(x, y);
    if (i + 1 < NP) {
      const float2 f = unpack_bf16(p[i]);
      x -= f.x;
      y -= f.y;
    }
  }
}
// Two accumulators (8-column blocks of 16 columns) as an A operand in NP planes.
template <int NP>
__device__ __forceinline__ void to_a(const float (&c0)[4], const float (&c1)[4], unsigned (&a)[NP][4]) {
  unsigned t[NP];
  split<NP>(c0[0], c0[1], t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][0] = t[i];
  split<NP>(c0[2], c0[3], t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][1] = t[i];
  split<NP>(c1[0], c1[1], t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][2] = t[i];
  split<NP>(c1[2], c1[3], t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][3] = t[i];
}
// Each value times f of its column first.
template <int NP>
__device__ __forceinline__ void to_a(const float (&c0)[4], const float (&c1)[4], float2 f0, float2 f1,
                                     unsigned (&a)[NP][4]) {
  const float x[4] = {c0[0] * f0.x, c0[1] * f0.y, c0[2] * f0.x, c0[3] * f0.y};
  const float y[4] = {c1[0] * f1.x, c1[1] * f1.y, c1[2] * f1.x, c1[3] * f1.y};
  to_a<NP>(x, y, a);
}
// c0, c1 += A (NA planes) times the two B operands of b, plane J of NB.
template <int NA, int NB, int J>
__device__ __forceinline__ void mma_planes(float (&c0)[4], float (&c1)[4], const unsigned (&a)[NA][4],
                                           const unsigned (&b)[4]) {
  constexpr int MOST = NA > NB ? NA : NB;
#pragma unroll
  for (int i = 0; i < NA; ++i)
    if (i + J < MOST) {
      mma(c0, a[i], b[0], b[1]);
      mma(c1, a[i], b[2], b[3]);
    }
}
// The same over all planes of B: of a tile at `at`, `plane` bytes apart.
template <int NA, int NB, bool TRANS>
__device__ __forceinline__ void mma_tile(float (&c0)[4], float (&c1)[4], const unsigned (&a)[NA][4], unsigned at,
                                         int plane) {
  unsigned b[4];
  TRANS ? ldsm_t(b, at) : ldsm(b, at);
  mma_planes<NA, NB, 0>(c0, c1, a, b);
  if (NB > 1) {
    TRANS ? ldsm_t(b, at + plane) : ldsm(b, at + plane);
    mma_planes<NA, NB, 1>(c0, c1, a, b);
  }
  if (NB > 2) {
    TRANS ? ldsm_t(b, at + 2 * plane) : ldsm(b, at + 2 * plane);
    mma_planes<NA, NB, 2>(c0, c1, a, b);
  }
}

// Two A operands on the same B.
template <int NA, int NB, bool TRANS>
__device__ __forceinline__ void mma_tile2(float (&c0)[4], float (&c1)[4], const unsigned (&a)[NA][4], float (&d0)[4],
                                          float (&d1)[4], const unsigned (&e)[NA][4], unsigned at, int plane) {
  unsigned b[4];
  TRANS ? ldsm_t(b, at) : ldsm(b, at);
  mma_planes<NA, NB, 0>(c0, c1, a, b);
  mma_planes<NA, NB, 0>(d0, d1, e, b);
  if (NB > 1) {
    TRANS ? ldsm_t(b, at + plane) : ldsm(b, at + plane);
    mma_planes<NA, NB, 1>(c0, c1, a, b);
    mma_planes<NA, NB, 1>(d0, d1, e, b);
  }
  if (NB > 2) {
    TRANS ? ldsm_t(b, at + 2 * plane) : ldsm(b, at + 2 * plane);
    mma_planes<NA, NB, 2>(c0, c1, a, b);
    mma_planes<NA, NB, 2>(d0, d1, e, b);
  }
}

// ---------------------------------------------------------------------- tiles
//
// A plane of a tile: rows of W bfloat16 values.  What comes from a tensor has
// the 16-byte units of a row in an order that its number decides, so that the
// eight rows an ldmatrix reads lie in different banks; what a kernel computed
// is kept in blocks of 8 x 8 (BLK), 128 bytes each, which is what a register of
// a warp's fragments holds.

__device__ __forceinline__ unsigned shared_at(const void* p) {
  return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
template <int W, bool BLK = false>
__device__ __forceinline__ unsigned unit_at(int row, int unit) {
  return BLK ? (unsigned)((((row >> 3) * (W / 8) + unit) << 7) + ((row & 7) << 4))
             : (unsigned)(row * (W * 2) + ((unit ^ (W >= 64 ? row & 7 : (row >> 1) & 3)) << 4));
}
// Per-lane addresses of the four ways an operand is read.  m0, n0, k0: its
// first row, column or depth; `rows` says which of them the tile's rows are.
template <int W, bool BLK = false>
__device__ __forceinline__ unsigned at_b_rows_n(int n0, int k0, int lane) {   // ldsm: B, rows are columns n
  return unit_at<W, BLK>(n0 + ((lane >> 4) << 3) + (lane & 7), (k0 >> 3) + ((lane >> 3) & 1));
}
template <int W, bool BLK = false>
__device__ __forceinline__ unsigned at_b_rows_k(int k0, int n0, int lane) {   // ldsm_t: B, rows are the depth k
  return unit_at<W, BLK>(k0 + (lane & 15), (n0 >> 3) + (lane >> 4));
}
template <int W, bool BLK = false>
__device__ __forceinline__ unsigned at_a_rows_m(int m0, int k0, int lane) {   // ldsm: A, rows are rows m
  return unit_at<W, BLK>(m0 + (lane & 15), (k0 >> 3) + (lane >> 4));
}
template <int W, bool BLK = false>
__device__ __forceinline__ unsigned at_a_rows_k(int k0, int m0, int lane) {   // ldsm_t: A, rows are the depth k
  return unit_at<W, BLK>(k0 + ((lane >> 4) << 3) + (lane & 7), (m0 >> 3) + ((lane >> 3) & 1));
}

__device__ __forceinline__ void copy16(unsigned dst, const void* src, bool there) {
  const int n = there ? 16 : 0;   // 0: zeros are written, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store16(unsigned dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// BYTES (of a multiple of 16) from a place on 16 bytes.
template <int BYTES, int THREADS>
__device__ __forceinline__ void copy_block(unsigned dst, const char* src, int tid) {
#pragma unroll
  for (int i = 0; i < BYTES / 16 / THREADS; ++i) copy16(dst + 16 * (tid + i * THREADS), src + 16 * (tid + i * THREADS), true);
  constexpr int REST = BYTES / 16 % THREADS, AT = BYTES / 16 / THREADS * THREADS;
  if (REST && tid < REST) copy16(dst + 16 * (tid + AT), src + 16 * (tid + AT), true);
}

// A head's rows of a token-major tensor in the order they are walked.
template <typename T>
struct Rows {
  const T* first;
  long long step;
  __device__ __forceinline__ const T* at(int i) const { return first + (long long)i * step; }
};
template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const DeltaP& p, const void* x, long long ld, long long column, int b, int n) {
  return {static_cast<const T*>(x) + ((long long)b * p.L + (p.reverse ? n - 1 : 0)) * ld + column, p.reverse ? -ld : ld};
}

// Rows i0 ... i0 + ROWS - 1 of a sequence of n, of up to W values, into the
// planes at `dst` (`plane` bytes apart), zeros where there is no row or column.
// wide: every row lies on 16 bytes.  bfloat16's wide rows arrive asynchronously,
// all others before the call returns.
template <int W, int ROWS, int THREADS>
__device__ __forceinline__ void load_tile(unsigned dst, int, Rows<__nv_bfloat16> x, int i0, int n, int cols, bool wide,
                                          int tid) {
  constexpr int RS = THREADS / (W / 8);   // rows at a time, of the same unit
  static_assert(THREADS % (W / 8) == 0 && ROWS % RS == 0, "");
  const int u = tid % (W / 8), r0 = tid / (W / 8);
  const __nv_bfloat16* s = x.at(i0 + r0) + 8 * u;
  const long long hop = RS * x.step;
#pragma unroll
  for (int k = 0; k < ROWS / RS; ++k) {
    const bool there = i0 + r0 + k * RS < n && 8 * u < cols;
    const unsigned at = dst + unit_at<W>(r0 + k * RS, u);
    if (wide) {
      copy16(at, there ? s : x.first, there);
    } else {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (there) {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(s);
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
      store16(at, v);
    }
    s += hop;
  }
}
__device__ __forceinline__ void store_planes(unsigned dst, int plane, const float (&v)[8]) {
  unsigned w[4][3];
#pragma unroll
  for (int e = 0; e < 4; ++e) split<3>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
  for (int j = 0; j < 3; ++j) store16(dst + j * plane, make_uint4(w[0][j], w[1][j], w[2][j], w[3][j]));
}
template <int W, int ROWS, int THREADS>
__device__ __forceinline__ void load_tile(unsigned dst, int plane, Rows<float> x, int i0, int n, int cols, bool wide,
                                          int tid) {
  constexpr int UNITS = ROWS * (W / 8), N = (UNITS + THREADS - 1) / THREADS, AHEAD = N < 4 ? N : 4;   // reads under way
#pragma unroll 1
  for (int i = tid; i < UNITS; i += AHEAD * THREADS) {
    float v[AHEAD][8];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = i + j * THREADS, row = k / (W / 8), u = k % (W / 8);
      load8(x.at(i0 + row) + 8 * u, k < UNITS && i0 + row < n && 8 * u < cols ? 8 : 0, wide, v[j]);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = i + j * THREADS;
      if (k < UNITS) store_planes(dst + unit_at<W>(k / (W / 8), k % (W / 8)), plane, v[j]);
    }
  }
}

}  // namespace
}  // namespace lion
