// delta_chain.cuh -- what the chains over chunks share, forward and back: a
// chunk's tiles in shared memory, their loads, and the way out for results.
#pragma once

#include "delta_common.cuh"

namespace lion {
namespace {

template <typename T, int DK, int NPP>
struct ChainTiles {
  static constexpr int NI = Planes<T>::in, NS = Planes<T>::mid;
  static constexpr int row = kChunk * DK * 2, val = kChunk * kSlice * 2;   // bytes of a plane
  static constexpr int k = 0, q = NI * row, v = 2 * NI * row, tp = v + NI * val;
  static constexpr int coef = tp + (NS + NPP) * kTile;
  static constexpr int bytes = coef + kCoefs * 4;
};
// rows of 16 of a warp's outputs on their way out, 80 bytes apart
constexpr int kOutRow = 20;
constexpr int kOutBytes = kChunk * kOutRow * 4;

template <typename T, int DK, int NPP>
__device__ __forceinline__ void load_chunk(const DeltaP& p, unsigned dst, int c, int b, int hv, int hk, int slice, int n,
                                           const void* val, long long val_ld, int val_wide, int tid) {
  typedef ChainTiles<T, DK, NPP> L;
  const auto token = [&](int row) {
    const int i = c * kChunk + row;
    return i < n ? (long long)b * p.L + (p.reverse ? n - 1 - i : i) : -1LL;
  };
  const auto rows = [&](const void* x, long long ld, long long first) {
    return [=](int row) -> const T* {
      const long long t = token(row);
      return t < 0 ? nullptr : static_cast<const T*>(x) + t * ld + first;
    };
  };
  load_tile<DK, kChunk, 128>(dst + L::k, L::row, static_cast<const T*>(p.k), rows(p.k, p.k_ld, (long long)hk * p.dk),
                             p.dk, p.k_wide, tid);
  load_tile<DK, kChunk, 128>(dst + L::q, L::row, static_cast<const T*>(p.q), rows(p.q, p.q_ld, (long long)hk * p.dk),
                             p.dk, p.q_wide, tid);
  load_tile<kSlice, kChunk, 128>(dst + L::v, L::val, static_cast<const T*>(val),
                                 rows(val, val_ld, (long long)hv * p.dv + slice * kSlice), p.dv - slice * kSlice,
                                 val_wide, tid);
  const char* tp = static_cast<const char*>(p.tp) + (((long long)b * p.Hv + hv) * p.nc + c) * p.tp_chunk;
  for (int i = tid; i < (L::bytes - L::tp) / 16; i += 128) copy16(dst + L::tp + 16 * i, tp + 16 * i, true);
}

// A warp's [16 columns][32 tokens] accumulators to rows of a [tokens][columns] tensor: 16 values of a token a lane.
template <typename T, typename F>
__device__ __forceinline__ void store_rows(float* buf, const float (&o)[4][4], int lane, int cols, bool wide, F row) {
  const int r = lane >> 2, q4 = lane & 3;
#pragma unroll
  for (int nb = 0; nb < 4; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) buf[(8 * nb + 2 * q4 + (e & 1)) * kOutRow + r + 8 * (e >> 1)] = o[nb][e];
  __syncwarp();
  T* dst = row(lane);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float v[8];
    const float4 x = *reinterpret_cast<const float4*>(buf + lane * kOutRow + 8 * u);
    const float4 y = *reinterpret_cast<const float4*>(buf + lane * kOutRow + 8 * u + 4);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    if (dst && 8 * u < cols) store8(dst + 8 * u, 8, wide, v);
  }
  __syncwarp();
}

// Tokens that a sequence does not have, in a warp's columns.
template <typename T>
__device__ __forceinline__ void zero_rows(const DeltaP& p, void* out, int n, int b, int hv, int m0, int cols, bool wide,
                                          int lane) {
  const float zero[8] = {};
  for (long long t = n + (lane >> 1); t < p.L; t += 16) {
    const int u = lane & 1;
    if (8 * u < cols) store8(static_cast<T*>(out) + (((long long)b * p.L + t) * p.Hv + hv) * p.dv + m0 + 8 * u, 8, wide, zero);
  }
}

// A warp's columns of S^T, two rows of 16 adjacent values a lane pair, as a saved state [dv][dk].
template <typename T, int DK>
__device__ __forceinline__ void save_state(const DeltaP& p, void* states, long long bh, int at, const float (&s)[DK / 8][4],
                                           int m0, int cols, int lane) {
  const int r = lane >> 2, q4 = lane & 3;
  T* to = static_cast<T*>(states) + (bh * p.nc64 + at) * p.dv * p.dk;
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kx = 8 * j + 2 * q4, col = r + 8 * h;
      if (kx < p.dk && col < cols) {
        T* d = to + (long long)(m0 + col) * p.dk + kx;
        if (sizeof(T) == 2)
          *reinterpret_cast<unsigned*>(d) = pack_bf16(s[j][2 * h], s[j][2 * h + 1]);
        else
          *reinterpret_cast<float2*>(d) = make_float2(s[j][2 * h], s[j][2 * h + 1]);
      }
    }
}

}  // namespace
}  // namespace lion
