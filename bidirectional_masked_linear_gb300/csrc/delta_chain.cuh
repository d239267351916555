// delta_chain.cuh -- what the chains over chunks share, forward and back: the
// tiles all of a head's columns read, and the ways out for results.
#pragma once

#include "delta_common.cuh"

namespace lion {
namespace {

// A chunk's tiles in shared memory: q and k, then ChunkData's bytes FROM to TO.
template <typename T, int DK, int FROM, int TO>
struct Stage {
  static constexpr bool KQ = sizeof(T) == 4;
  static constexpr int NI = Planes<T>::in, row = kChunk * DK * 2;
  static constexpr int q = 0, k = NI * row, rest = 2 * NI * row, bytes = rest + TO - FROM;
  static constexpr int at(int offset) { return rest + offset - FROM; }

  template <int THREADS>
  static __device__ __forceinline__ void load(const DeltaP& p, unsigned dst, const char* chunk, const Rows<T>& xq,
                                              const Rows<T>& xk, int i0, int n, int tid) {
    if (KQ) {
      copy_block<2 * NI * row, THREADS>(dst, chunk, tid);
    } else {
      load_tile<DK, kChunk, THREADS>(dst + q, row, xq, i0, n, p.dk, p.q_wide, tid);
      load_tile<DK, kChunk, THREADS>(dst + k, row, xk, i0, n, p.dk, p.k_wide, tid);
    }
    copy_block<TO - FROM, THREADS>(dst + rest, chunk + FROM, tid);
  }
};

// Two warps share 16 columns of a head's state: a warp's `side` says which half
// of a chunk's tokens and which half of the dk values are its own.  What the
// other one needs of it passes through shared memory as A operands, a register
// quad a lane.
template <typename T, int DK, int EXTRA>
struct Swap {
  static constexpr int NS = Planes<T>::mid;
  static constexpr int state = DK / 16 * NS * 512;       // bytes a pair: S^T, all dk
  static constexpr int row = (2 * NS + EXTRA) * 512;     // and R^T or X^T of 32 tokens
  static constexpr int bytes = state + row;
};
__device__ __forceinline__ void pair_sync(int pair) {
  asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + pair) : "memory");
}
__device__ __forceinline__ void put_a(unsigned at, const unsigned (&a)[4], int lane) {
  store16(at + 16 * lane, make_uint4(a[0], a[1], a[2], a[3]));
}
__device__ __forceinline__ void get_a(unsigned at, unsigned (&a)[4], int lane) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(at + 16 * lane)
               : "memory");
}
// A warp's half of S^T, in planes, to where both read it.
template <int DK, int NS>
__device__ __forceinline__ void put_state(unsigned at, const float (&s)[DK / 16][4], int side, int lane) {
#pragma unroll
  for (int ks = 0; ks < DK / 32; ++ks) {
    unsigned a[NS][4];
    to_a<NS>(s[2 * ks], s[2 * ks + 1], a);
#pragma unroll
    for (int j = 0; j < NS; ++j) put_a(at + ((side * (DK / 32) + ks) * NS + j) * 512, a[j], lane);
  }
}

// Bytes of a warp's buffer for results on their way out, tokens in rows.
template <typename T>
constexpr int out_bytes() {
  return sizeof(T) == 2 ? 16 * 48 : 0;
}
// A warp's accumulators [16 columns][16 tokens] to a token-major tensor: tokens
// i0 ... of n from `x` on, as far as there are columns.
__device__ __forceinline__ void store_rows(unsigned char* buf, const float (&o)[2][4], int lane, int cols, bool wide,
                                           const Rows<__nv_bfloat16>& x, int i0, int n) {
  stsm_t(shared_at(buf) + ((lane >> 4) * 8 + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16, pack_bf16(o[0][0], o[0][1]),
         pack_bf16(o[0][2], o[0][3]), pack_bf16(o[1][0], o[1][1]), pack_bf16(o[1][2], o[1][3]));
  __syncwarp();
  const int t = lane >> 1, u = lane & 1;
  const uint4 v = *reinterpret_cast<const uint4*>(buf + t * 48 + u * 16);
  if (i0 + t < n && 8 * u < cols) {
    __nv_bfloat16* d = const_cast<__nv_bfloat16*>(x.at(i0 + t)) + 8 * u;
    if (wide) {
      *reinterpret_cast<uint4*>(d) = v;
    } else {
      const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) reinterpret_cast<unsigned short*>(d)[e] = (unsigned short)(w[e >> 1] >> 16 * (e & 1));
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void store_rows(unsigned char*, const float (&o)[2][4], int lane, int cols, bool,
                                           const Rows<float>& x, int i0, int n) {
  const int r = lane >> 2, q4 = lane & 3;   // eight lanes write 32 bytes of a token
#pragma unroll
  for (int nb = 0; nb < 2; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 8 * nb + 2 * q4 + (e & 1), col = r + 8 * (e >> 1);
      if (i < n && col < cols) const_cast<float*>(x.at(i))[col] = o[nb][e];
    }
}

// Accumulators [16 columns][8 N values] as blocks of 8 x 8 in the inputs' type,
// in rows of ROW blocks: what the gradients' tiles are loaded from.
template <int N, int ROW>
__device__ __forceinline__ void store_blocks(__nv_bfloat16* to, const float (&s)[N][4], int lane) {
  unsigned* d = reinterpret_cast<unsigned*>(to) + lane;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    d[j * 32] = pack_bf16(s[j][0], s[j][1]);
    d[(ROW + j) * 32] = pack_bf16(s[j][2], s[j][3]);
  }
}
template <int N, int ROW>
__device__ __forceinline__ void store_blocks(float* to, const float (&s)[N][4], int lane) {
  float2* d = reinterpret_cast<float2*>(to) + lane;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    d[j * 32] = make_float2(s[j][0], s[j][1]);
    d[(ROW + j) * 32] = make_float2(s[j][2], s[j][3]);
  }
}

// Tokens that a sequence does not have, in a warp's columns.
template <typename T>
__device__ __forceinline__ void zero_rows(const DeltaP& p, void* out, int n, int b, int hv, int m0, int cols, bool wide,
                                          int side, int lane) {
  const float zero[8] = {};
  for (long long t = n + 16 * side + (lane >> 1); t < p.L; t += 32) {
    const int u = lane & 1;
    if (8 * u < cols)
      store8(static_cast<T*>(out) + (((long long)b * p.L + t) * p.Hv + hv) * p.dv + m0 + 8 * u, 8, wide, zero);
  }
}

// A warp's part of the [dk][dv] state of a head, from column m0 and value k0 on, as accumulators.
template <int N>
__device__ __forceinline__ void load_state(const DeltaP& p, const float* h, long long bh, int m0, int cols, int k0, int lane,
                                           float (&s)[N][4]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kx = k0 + 8 * j + 2 * (lane & 3) + (e & 1), col = (lane >> 2) + 8 * (e >> 1);
      s[j][e] = h && kx < p.dk && col < cols ? h[(bh * p.dk + kx) * p.dv + m0 + col] : 0.f;
    }
}
template <int N>
__device__ __forceinline__ void keep_state(const DeltaP& p, float* h, long long bh, int m0, int cols, int k0, int lane,
                                           const float (&s)[N][4]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kx = k0 + 8 * j + 2 * (lane & 3) + (e & 1), col = (lane >> 2) + 8 * (e >> 1);
      if (kx < p.dk && col < cols) h[(bh * p.dk + kx) * p.dv + m0 + col] = s[j][e];
    }
}

// x *= f, all of it
template <int N>
__device__ __forceinline__ void scale_by(float (&x)[N][4], float f) {
  const f2 g = pack2(f, f);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const f2 a = mul2(pack2(x[j][0], x[j][1]), g), b = mul2(pack2(x[j][2], x[j][3]), g);
    x[j][0] = a.x; x[j][1] = a.y; x[j][2] = b.x; x[j][3] = b.y;
  }
}

}  // namespace
}  // namespace lion
