// ssm_scan.cuh -- what the selective scan's kernels share.
//
//   h_i[n] = a_i[n] h_{i-1}[n] + b_i[n],  a = exp(delta A[n]),  b = delta u B[n]
//
// Channels are cut into blocks within their group and sequences, where that
// leaves too few CTAs, into segments; a walk goes tile by tile.  For the
// element-wise parts (loads, softplus, gate, stores) a lane holds adjacent
// channels of one token of the tile; for the recurrence it holds some states of
// some channels over all of its tokens.  The two meet in shared memory.
#pragma once

#include "lion_internal.h"
#include "scan_plan.h"
#include "ssm_common.cuh"

namespace lion {

constexpr int kStateEvery = LION_SCAN_STATE_EVERY;

struct ScanP {
  const void* u;
  const void* dt;
  const void* z;
  const void* Bm;
  const void* Cm;
  const void* dout;
  const float* A;
  const float* Dskip;
  const float* dt_bias;
  const float* h0;
  const int* lengths;
  void* out;
  float* h_out;
  float* states;        // [B][nst][D][N]
  // gradients
  void* du;
  void* ddt;
  void* dz;
  float* dh0;
  float* part_bc;       // [channel block of a group][B][L][G][2][N]
  float* part_par;      // [B * nseg][D*N | D | D], rows padded to four
  // segments
  float* seg_state;     // [B][nseg][D][N]: a segment's own contribution to the state that leaves it, then
                        // (chained) the state that enters it
  float* seg_sum;       // [B][nseg][D]: its sum of delta
  long long u_ld, dt_ld, z_ld, b_ld, c_ld;
  int B, L, D, N, G, Dg;
  int nblk, nseg, seglen, nst;
  int softplus, reverse;
  // the alignment in bytes, 16 at most, of every row of a tensor (d: dout)
  int u_align, dt_align, z_align, b_align, c_align, d_align;
  bool o_wide;   // the outputs' rows lie on 16 bytes
};

namespace {

// The tile of the gradients' segment pass: a lane holds four states of two
// channels, LN lanes a channel's N = 4 LN.
template <int LN_, int W_>
struct ScanTile {
  static constexpr int LN = LN_, W = W_;
  static constexpr int N = 4 * LN;
  static constexpr int LC = 32 / LN;        // channel lanes of a warp
  static constexpr int CW = 2 * LC;         // channels of a warp
  static constexpr int CB = W * CW;         // channels of a CTA
  static constexpr int TT = N;              // tokens of a tile: eight elements a thread
  static constexpr int NT = 32 * W;
  static constexpr int VPT = CB / 8;        // vectors of a token
  static constexpr int SLOT = CB + CB / 8;  // a token's row of per-channel slots, one slot of padding after eight:
                                            // the element threads' 16-byte accesses then start on different banks
  static_assert(TT * CB == 8 * NT, "eight elements a thread");
};
__device__ __forceinline__ int slot_of(int c) { return c + (c >> 3); }


// A CTA's place: channel block, segment and sequence.
struct ScanAt {
  int g, blk, seg, b;
  int d0;       // first channel within D
  int nch;      // channels of the block
  int i0, i1;   // processing indices of the segment
  int v0, v1;   // processing indices with a token
};
__device__ __forceinline__ ScanAt scan_at(const ScanP& p, int CB) {
  ScanAt w;
  unsigned x = blockIdx.x;
  w.blk = x % p.nblk;
  x /= p.nblk;
  w.g = x % p.G;
  x /= p.G;
  w.seg = x % p.nseg;
  w.b = x / p.nseg;
  w.d0 = w.g * p.Dg + w.blk * CB;
  w.nch = min(CB, p.Dg - w.blk * CB);
  w.i0 = w.seg * p.seglen;
  w.i1 = min(p.L, w.i0 + p.seglen);
  const int len = p.lengths ? min(max(p.lengths[w.b], 0), p.L) : p.L;
  w.v0 = p.reverse ? p.L - len : 0;
  w.v1 = p.reverse ? p.L : len;
  return w;
}
__device__ __forceinline__ int token_of(const ScanP& p, int i) { return p.reverse ? p.L - 1 - i : i; }

// B or C of a tile's tokens as fp32 rows of N (tokens outside [v0, v1): 0).
template <typename T, int N, int TT, int NT>
__device__ __forceinline__ void load_bc(const ScanP& p, const ScanAt& w, const void* src, long long ld, int i0,
                                        float* dst) {
#pragma unroll 4
  for (int k = threadIdx.x; k < TT * N; k += NT) {
    const int i = i0 + k / N;
    float v = 0.f;
    if (i >= w.v0 && i < w.v1 && i < w.i1)
      v = to_f32(static_cast<const T*>(src)[((long long)w.b * p.L + token_of(p, i)) * ld + w.g * N + k % N]);
    dst[k] = v;
  }
}

// The state's four values of a channel.
__device__ __forceinline__ void load_pair(const float* src, bool there, f2 (&v)[2]) {
  const float4 x = there ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
  v[0] = pack2(x.x, x.y);
  v[1] = pack2(x.z, x.w);
}
// A as the kernels use it: times log2 e.  -inf (a state that keeps nothing) becomes a finite value that keeps as
// little: the step of a place without a token is 0, and 0 times it has to be 0.
__device__ __forceinline__ float decay(float a) {
  const float x = a * kLog2e;
  return x < -3e38f ? -3e38f : x;   // a NaN stays one
}
__device__ __forceinline__ void load_decays(const float* src, bool there, f2 (&v)[2]) {
  load_pair(src, there, v);
#pragma unroll
  for (int k = 0; k < 2; ++k) v[k] = pack2(decay(v[k].x), decay(v[k].y));
}
__device__ __forceinline__ void store_pair(float* dst, const f2 (&v)[2]) {
  const float2 a = unpack2(v[0]), b = unpack2(v[1]);
  *reinterpret_cast<float4*>(dst) = make_float4(a.x, a.y, b.x, b.y);
}

// Four adjacent elements of shared or global memory.
__device__ __forceinline__ void get(const float* p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void get(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  const float2 a = unpack_bf16(r.x), b = unpack_bf16(r.y);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void put(float* p, int n, bool wide, const float (&v)[4]) {
  if (wide && n >= 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void put(__nv_bfloat16* p, int n, bool wide, const float (&v)[4]) {
  if (wide && n >= 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = __float2bfloat16_rn(v[e]);
  }
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}
// n <= V = 16 bytes' worth of elements to shared memory, zeros behind them,
// asynchronously as far as the source's alignment (in bytes) allows.
template <typename T>
__device__ __forceinline__ void fetch(T* dst, const T* src, int n, int align) {
  constexpr int V = 16 / (int)sizeof(T);
  if (n >= V && align >= 4) {
    if (align == 16) {
      copy_async<16>(dst, src);
    } else if (align == 8) {
      copy_async<8>(dst, src);
      copy_async<8>(dst + V / 2, src + V / 2);
    } else {
#pragma unroll
      for (int e = 0; e < V; e += V / 4) copy_async<4>(dst + e, src + e);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (sizeof(T) == 4 && e < n) copy_async<4>(dst + e, src + e);
      else dst[e] = e < n ? src[e] : from_f32<T>(0.f);
    }
  }
}

// A warp's copies of [TT][W] rows in pieces of 16 bytes: piece q = lane + 32 k
// is PV elements of token q / PPR.  The source moves on a tile at a time.
template <typename T, int TT, int W>
struct Feed {
  static constexpr int PV = 16 / (int)sizeof(T), PPR = W / PV, PIECES = TT * PPR, PK = (PIECES + 31) / 32;
  static_assert(PPR <= 32 && 32 % PPR == 0, "a lane's pieces have one place in their tokens");
  const T* src;
  long long hop;   // elements from a lane's piece to its next, 32 / PPR tokens on
  int n;           // elements there are of a piece
  __device__ __forceinline__ void start(const void* base, long long ld, long long off, const ScanP& p, const ScanAt& w,
                                        int i0, int lane, int width) {
    const int c = lane % PPR * PV;
    src = static_cast<const T*>(base) + ((long long)w.b * p.L + token_of(p, i0 + lane / PPR)) * ld + off + c;
    hop = (p.reverse ? -(32 / PPR) : 32 / PPR) * ld;
    n = min(PV, width - c);
  }
  __device__ __forceinline__ void next(T* dst, int lo, int hi, int lane, int align, bool whole, long long tile) {
    if (whole) {
#pragma unroll
      for (int k = 0; k < PK; ++k) {
        const int q = lane + 32 * k;
        if (PIECES % 32 == 0 || q < PIECES) copy_async<16>(dst + q * PV, src + k * hop);
      }
    } else {
#pragma unroll 2
      for (int k = 0; k < PK; ++k) {
        const int q = lane + 32 * k, t = q / PPR;
        if (PIECES % 32 == 0 || q < PIECES)
          fetch<T>(dst + q * PV, src + k * hop, t >= lo && t < hi ? n : 0, align);
      }
    }
    src += tile;
  }
};

template <int COUNT>
__device__ __forceinline__ const float* as_fp32(const float* raw, float*, int) { return raw; }
template <int COUNT>
__device__ __forceinline__ const float* as_fp32(const __nv_bfloat16* raw, float* dst, int lane) {
#pragma unroll
  for (int k = 0; k < (COUNT / 4 + 31) / 32; ++k) {
    const int q = lane + 32 * k;
    if (COUNT / 4 % 32 == 0 || q < COUNT / 4) {
      float v[4];
      get(raw + 4 * q, v);
      *reinterpret_cast<float4*>(dst + 4 * q) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  return dst;
}

// delta of eight channels from the step sizes read.
__device__ __forceinline__ void deltas(const ScanP& p, int d, int n, float (&dt)[8], float (&raw)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    raw[e] = p.dt_bias && e < n ? dt[e] + p.dt_bias[d + e] : dt[e];
    dt[e] = e < n ? (p.softplus ? softplus(raw[e]) : raw[e]) : 0.f;
  }
}

// ---------------------------------------------------------------- host side

#define LION_SCAN_DISPATCH(RUN, dtype, N, ...)                                        \
  (dtype == DT_BF16 ? (N == 8    ? RUN<__nv_bfloat16, 8>(__VA_ARGS__)                 \
                       : N == 16 ? RUN<__nv_bfloat16, 16>(__VA_ARGS__)                \
                       : N == 32 ? RUN<__nv_bfloat16, 32>(__VA_ARGS__)                \
                                 : RUN<__nv_bfloat16, 64>(__VA_ARGS__))               \
                    : (N == 8    ? RUN<float, 8>(__VA_ARGS__)                         \
                       : N == 16 ? RUN<float, 16>(__VA_ARGS__)                        \
                       : N == 32 ? RUN<float, 32>(__VA_ARGS__)                        \
                                 : RUN<float, 64>(__VA_ARGS__)))

// 16, 8, 4 or 2: what divides the address, the distance between rows and that between groups.
inline int rows_align(const void* p, long long stride, long long group, int es) {
  const unsigned long long x =
      reinterpret_cast<uintptr_t>(p) | (unsigned long long)stride * es | (unsigned long long)group * es;
  return x % 16 == 0 ? 16 : x % 8 == 0 ? 8 : x % 4 == 0 ? 4 : 2;
}
inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

void fill_scan(ScanP& p, const lion_scan_args& a);   // everything but the plan and the workspace
cudaError_t launch_scan_chain(const ScanP& p, bool back, const float* first, cudaStream_t s);

}  // namespace lion
