// delta_common.cuh -- what the gated delta rule's chunk kernels share: the
// formulas' names, split operands, fragments and tiles.
//
// A chunk of C tokens with the state S before it, G the inclusive sums of the
// logarithms g of its decays and D_ij = e^(G_i - G_j) for i >= j:
//   M_ij = D_ij (k_i . k_j) beta_j  (i > j),   T = (I + M)^-1
//   R = T (V - e^G o (K S)),  U = beta o R
//   O = scale (e^G o (Q S)) + P U,  P_ij = scale D_ij (q_i . k_j)  (i >= j)
//   S' = e^G_C S + (e^(G_C - G) o K)^T U
// R does not depend on where the chunks are cut; it is what the gradients
// start from.  Given dO and dS' the gradients run back with
//   dU = P^T dO + e^(G_C - G) o (K dS'),  dR = T^T (beta o dU) = dV
//   dS = e^G_C dS' + (scale e^G o Q)^T dO - (e^G o K)^T dR
//
// Products run on the tensor cores in bfloat16 with fp32 sums.  A factor is a
// sum of planes, x = bf16(x) + bf16(x - bf16(x)) + ...: bfloat16 inputs are one
// plane and exact; what is computed (states, T, R, P) has two planes beside
// them, 2^-18 of a value, which keeps the float32 state that a call hands back
// to about 1e-6; float32 inputs and everything beside them have three, 2^-26.
// Products of planes i and j with i + j past the finer factor's last plane are
// below its rounding and are left out.
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
  void* tp;                // per head and chunk: planes of T, planes of P, coefficients
  void *R, *states;        // per head: R [nc * 32][dv], states [nc64][dv][dk]; NULL: not wanted
  void *dv_out, *dstates;  // gradients: dV [B][L][Hv][dv]; dS' as states
  float* dh0;
  long long q_ld, k_ld, v_ld, g_ld, beta_ld;
  void *dq, *dk_out, *dg, *dbeta;
  float *dq_part, *dk_part;   // per value head, [B][L][Hv][dk], where a query head has several
  long long tp_chunk;      // bytes of a chunk in tp
  int B, L, Hk, Hv, dk, dv, nc, nc64, slices;
  float scale;
  int reverse;
  int q_wide, k_wide, v_wide, o_wide, do_wide, dv_wide;
};

namespace {

constexpr int kChunk = 32;          // tokens of a step of the chains
constexpr int kSlice = 64;          // columns of the state a chain's CTA holds, 16 a warp
constexpr int kStateChunk = 64;     // tokens between saved states, and of a block of the gradients
constexpr int kTile = kChunk * kChunk * 2;   // bytes of a plane of T or P
constexpr int kCoefs = 4 * kChunk;           // floats: e^G, scale e^G, e^(G_C - G), beta

// Planes of an input and of what is computed from it.
template <typename T>
struct Planes {
  static constexpr int in = 1, mid = 2;
};
template <>
struct Planes<float> {
  static constexpr int in = 3, mid = 3;
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
// Two accumulators (8-column blocks of 16 columns), each value times f[its
// column], as an A operand in NP planes.
template <int NP>
__device__ __forceinline__ void to_a(const float (&c0)[4], const float (&c1)[4], float2 f0, float2 f1,
                                     unsigned (&a)[NP][4]) {
  unsigned t[NP];
  split<NP>(c0[0] * f0.x, c0[1] * f0.y, t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][0] = t[i];
  split<NP>(c0[2] * f0.x, c0[3] * f0.y, t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][1] = t[i];
  split<NP>(c1[0] * f1.x, c1[1] * f1.y, t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][2] = t[i];
  split<NP>(c1[2] * f1.x, c1[3] * f1.y, t);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][3] = t[i];
}
template <int NP>
__device__ __forceinline__ void to_a(const float (&c0)[4], const float (&c1)[4], unsigned (&a)[NP][4]) {
  to_a<NP>(c0, c1, make_float2(1.f, 1.f), make_float2(1.f, 1.f), a);
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

// ---------------------------------------------------------------------- tiles
//
// A plane of a tile in shared memory: rows of W bfloat16 values, the 16-byte
// units of a row in an order that its number decides, so that the eight rows
// an ldmatrix reads lie in different banks.

__device__ __forceinline__ unsigned shared_at(const void* p) {
  return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
template <int W>
__device__ __forceinline__ unsigned unit_at(int row, int unit) {
  return W >= 64 ? (unsigned)(row * (W * 2) + ((unit ^ (row & 7)) << 4))
                 : (unsigned)(row * (W * 2) + ((unit ^ ((row >> 1) & 3)) << 4));
}
// Per-lane addresses of the four ways an operand is read.  m0, n0, k0: its
// first row, column or depth; `rows` says which of them the tile's rows are.
template <int W>
__device__ __forceinline__ unsigned at_b_rows_n(int n0, int k0, int lane) {   // ldsm: B, rows are columns n
  return unit_at<W>(n0 + ((lane >> 4) << 3) + (lane & 7), (k0 >> 3) + ((lane >> 3) & 1));
}
template <int W>
__device__ __forceinline__ unsigned at_b_rows_k(int k0, int n0, int lane) {   // ldsm_t: B, rows are the depth k
  return unit_at<W>(k0 + (lane & 15), (n0 >> 3) + (lane >> 4));
}
template <int W>
__device__ __forceinline__ unsigned at_a_rows_m(int m0, int k0, int lane) {   // ldsm: A, rows are rows m
  return unit_at<W>(m0 + (lane & 15), (k0 >> 3) + (lane >> 4));
}
template <int W>
__device__ __forceinline__ unsigned at_a_rows_k(int k0, int m0, int lane) {   // ldsm_t: A, rows are the depth k
  return unit_at<W>(k0 + ((lane >> 4) << 3) + (lane & 7), (m0 >> 3) + ((lane >> 3) & 1));
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

// ROWS rows of up to W values into the planes at `dst` (PLANE bytes apart),
// zeros where there is no row or column.  src(row): the row's first value, or
// NULL; base: memory that may be read.  wide: every row lies on 16 bytes.  bfloat16's wide rows arrive
// asynchronously, all others before the call returns.
template <int W, int ROWS, int THREADS, typename F>
__device__ __forceinline__ void load_tile(unsigned dst, int, const __nv_bfloat16* base, F src, int cols, bool wide, int tid) {
#pragma unroll
  for (int i = tid; i < ROWS * (W / 8); i += THREADS) {
    const int row = i / (W / 8), u = i % (W / 8);
    const __nv_bfloat16* s = src(row);
    const bool there = s != nullptr && 8 * u < cols;
    const unsigned at = dst + unit_at<W>(row, u);
    if (wide) {
      copy16(at, there ? s + 8 * u : base, there);
    } else {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (there) {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(s + 8 * u);
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
      store16(at, v);
    }
  }
}
template <int W, int ROWS, int THREADS, typename F>
__device__ __forceinline__ void load_tile(unsigned dst, int plane, const float*, F src, int cols, bool wide, int tid) {
#pragma unroll 4
  for (int i = tid; i < ROWS * (W / 8); i += THREADS) {
    const int row = i / (W / 8), u = i % (W / 8);
    const float* s = src(row);
    float v[8];
    load8(s + 8 * u, s != nullptr && 8 * u < cols ? 8 : 0, wide, v);
    unsigned w[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split<3>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
    for (int j = 0; j < 3; ++j)
      store16(dst + j * plane + unit_at<W>(row, u), make_uint4(w[0][j], w[1][j], w[2][j], w[3][j]));
  }
}

}  // namespace
}  // namespace lion
