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

// Bytes of a warp's buffer for results on their way out: tokens in rows, 48
// bytes apart for bfloat16 and 80 for float32.
template <typename T>
constexpr int out_bytes() {
  return kChunk * (sizeof(T) == 2 ? 48 : 80);
}
// A warp's accumulators [16 columns][32 tokens] to rows of a token-major
// tensor: a token a lane, to `row` (NULL: nowhere).
__device__ __forceinline__ void store_rows(unsigned char* buf, const float (&o)[4][4], int lane, int cols, bool wide,
                                           __nv_bfloat16* row) {
  const unsigned at = shared_at(buf) + ((lane >> 4) * 8 + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16;
#pragma unroll
  for (int np = 0; np < 2; ++np)
    stsm_t(at + np * 16 * 48, pack_bf16(o[2 * np][0], o[2 * np][1]), pack_bf16(o[2 * np][2], o[2 * np][3]),
           pack_bf16(o[2 * np + 1][0], o[2 * np + 1][1]), pack_bf16(o[2 * np + 1][2], o[2 * np + 1][3]));
  __syncwarp();
  const uint4* s = reinterpret_cast<const uint4*>(buf + lane * 48);
  const uint4 x = s[0], y = s[1];
  if (row) {
    if (wide) {
      *reinterpret_cast<uint4*>(row) = x;
      if (cols > 8) *reinterpret_cast<uint4*>(row + 8) = y;
    } else {
      const unsigned w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (2 * e < cols) {
          reinterpret_cast<unsigned short*>(row)[2 * e] = (unsigned short)w[e];
          reinterpret_cast<unsigned short*>(row)[2 * e + 1] = (unsigned short)(w[e] >> 16);
        }
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void store_rows(unsigned char* raw, const float (&o)[4][4], int lane, int cols, bool wide,
                                           float* row) {
  float* buf = reinterpret_cast<float*>(raw);
  const int r = lane >> 2, q4 = lane & 3;
#pragma unroll
  for (int nb = 0; nb < 4; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) buf[(8 * nb + 2 * q4 + (e & 1)) * 20 + r + 8 * (e >> 1)] = o[nb][e];
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float v[8];
    load8(buf + lane * 20 + 8 * u, 8, true, v);
    if (row && 8 * u < cols) store8(row + 8 * u, 8, wide, v);
  }
  __syncwarp();
}

// Accumulators [16 columns][8 N values] as blocks of 8 x 8 in the inputs' type,
// rows of N blocks: what the gradients' tiles are loaded from.
template <int N>
__device__ __forceinline__ void store_blocks(__nv_bfloat16* to, const float (&s)[N][4], int lane) {
  unsigned* d = reinterpret_cast<unsigned*>(to) + lane;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    d[j * 32] = pack_bf16(s[j][0], s[j][1]);
    d[(N + j) * 32] = pack_bf16(s[j][2], s[j][3]);
  }
}
template <int N>
__device__ __forceinline__ void store_blocks(float* to, const float (&s)[N][4], int lane) {
  float2* d = reinterpret_cast<float2*>(to) + lane;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    d[j * 32] = make_float2(s[j][0], s[j][1]);
    d[(N + j) * 32] = make_float2(s[j][2], s[j][3]);
  }
}

// ------------------------------------------------- two warps for 16 columns
//
// A warp that carries the state has a second one beside it, its helper, for all
// that the next chunk does not wait for: outputs, what the gradients keep, the
// loads.  Between them lie A operands, or float32's sums, in shared memory, a
// register quad a lane, in two buffers: the helper works on the chunk before.

__device__ __forceinline__ void put_a(unsigned at, const unsigned (&a)[4], int lane) {
  store16(at + 16 * lane, make_uint4(a[0], a[1], a[2], a[3]));
}
__device__ __forceinline__ void get_a(unsigned at, unsigned (&a)[4], int lane) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(at + 16 * lane)
               : "memory");
}
__device__ __forceinline__ float4 get_f4(unsigned at, int lane) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at + 16 * lane)
               : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void put_sums(unsigned at, const float (&s)[N][4], int lane) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at + j * 512 + 16 * lane), "f"(s[j][0]), "f"(s[j][1]),
                 "f"(s[j][2]), "f"(s[j][3])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void get_sums(unsigned at, float (&s)[N][4], int lane) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float4 v = get_f4(at + j * 512, lane);
    s[j][0] = v.x; s[j][1] = v.y; s[j][2] = v.z; s[j][3] = v.w;
  }
}
// An A operand [16 columns][16 values] as four of the blocks of 8 x 8 that
// store_blocks writes, in rows of ROW blocks.
template <int ROW>
__device__ __forceinline__ void store_a(__nv_bfloat16* to, const unsigned (&a)[4], int lane) {
  unsigned* d = reinterpret_cast<unsigned*>(to) + lane;
  d[0] = a[0];
  d[ROW * 32] = a[1];
  d[32] = a[2];
  d[(ROW + 1) * 32] = a[3];
}
// `bytes`, at most MOST, on their way to L2, a line of 128 a thread.
template <int MOST, int THREADS>
__device__ __forceinline__ void to_l2(const void* p, int bytes, int tid) {
#pragma unroll
  for (int i = 0; i < (MOST / 128 + THREADS) / THREADS; ++i)
    if (128 * (tid + i * THREADS) < bytes)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + 128 * (tid + i * THREADS)));
}
// A chunk's rows, a line a thread (of longer rows their beginnings).
__device__ __forceinline__ void rows_to_l2(const Rows<__nv_bfloat16>& x, int i0, int n, int row) {
  if (row >= 0 && row < kChunk && i0 + row < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(x.at(i0 + row)));
}
// A slice's fragments of a chunk: `rows` columns of 32 floats to shared memory.
template <int COLS, int THREADS>
__device__ __forceinline__ void copy_slice(unsigned dst, const float* src, int rows, int tid) {
#pragma unroll
  for (int i = 0; i < COLS * kChunk / 4 / THREADS; ++i) {
    const int u = tid + i * THREADS;
    copy16(dst + 16 * u, src + (u < rows * (kChunk / 4) ? 4 * u : 0), u < rows * (kChunk / 4));
  }
}

// The i-th longest sequence of a ragged batch: CTAs start in their order, and a
// long walk that starts last is waited for alone (16 ragged prompts of up to
// 4096 tokens, 8 x 128 x 128: 245 us in the batch's order, 191 in this).  Of all threads;
// batches of up to 128, more are spread well enough.
__device__ __forceinline__ int by_length(const DeltaP& p, int i) {
  __shared__ int found;
  if (!p.lengths || p.B == 1 || p.B > 128) return i;
  const int t = threadIdx.x;
  if (t < p.B) {
    const int n = delta_length(p, t);
    int rank = 0;
    for (int j = 0; j < p.B; ++j) {
      const int m = delta_length(p, j);
      rank += m > n || (m == n && j < t);
    }
    if (rank == i) found = t;
  }
  __syncthreads();
  return found;
}

// Tokens that a sequence does not have, in a warp's columns.
template <typename T>
__device__ __forceinline__ void zero_rows(const DeltaP& p, void* out, int n, int b, int hv, int m0, int cols, bool wide,
                                          int lane) {
  const float zero[8] = {};
  for (long long t = n + (lane >> 1); t < p.L; t += 16) {
    const int u = lane & 1;
    if (8 * u < cols)
      store8(static_cast<T*>(out) + (((long long)b * p.L + t) * p.Hv + hv) * p.dv + m0 + 8 * u, 8, wide, zero);
  }
}

// A warp's columns of the [dk][dv] state of a head, as accumulators.
template <int DK>
__device__ __forceinline__ void load_state(const DeltaP& p, const float* h, long long bh, int m0, int cols, int lane,
                                           float (&s)[DK / 8][4]) {
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kx = 8 * j + 2 * (lane & 3) + (e & 1), col = (lane >> 2) + 8 * (e >> 1);
      s[j][e] = h && kx < p.dk && col < cols ? h[(bh * p.dk + kx) * p.dv + m0 + col] : 0.f;
    }
}
template <int DK>
__device__ __forceinline__ void keep_state(const DeltaP& p, float* h, long long bh, int m0, int cols, int lane,
                                           const float (&s)[DK / 8][4]) {
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kx = 8 * j + 2 * (lane & 3) + (e & 1), col = (lane >> 2) + 8 * (e >> 1);
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

// ------------------------------------------------------------------- segments

// A segment's M is a product over hundreds of tokens, which decays above 1 may take past fp32 although the state that it
// multiplies is small there, or 0.  So a walk of M takes powers of two out of it that hold it to the 1 it starts from
// (no more than one chunk's decays may then take it past fp32), and puts them back as decays below 1 follow.  Where
// decays' products stay below 1 there are none.
struct Raised {
  float log2 = 0.f;   // of the decays' product
  int by = 0;
  template <int N>
  __device__ __forceinline__ void after(float (&s)[N][4], float decay) {
    log2 += __log2f(decay);
    if (log2 > (float)by || (by > 0 && log2 < (float)(by - 32))) {
      const int want = log2 > 0.f ? (int)log2 + 1 : 0, to = want < by - 64 ? by - 64 : want;
      scale_by(s, ldexpf(1.f, by - to));
      by = to;
    }
  }
};

// The states before the segments (BACK: dS after them), given what each makes of
// one: a CTA for 16 columns of a head, a thread for four of them and every 64th
// row, S' = M S + N in fp32.  The next segment's M is copied to shared memory
// meanwhile (24 us at 2 x 24337 x 12 x 64, with M's powers of two 26; read from L2
// as it was used 43).
constexpr int starts_row(int dk) { return dk + 4; }   // floats of a row of M there: rows 64 apart in different banks
inline int starts_smem(int dk) { return 2 * dk * starts_row(dk) * 4; }

template <bool BACK>
__global__ void __launch_bounds__(256) delta_starts_kernel(const DeltaP p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float4 sh[LION_DELTA_MAX_D][4];
  const int tiles = p.dvp / 16, width = p.dvp + p.dk, ld = starts_row(p.dk);
  const long long bh = blockIdx.x / tiles;
  const int c4 = threadIdx.x & 3, col = 16 * (int)(blockIdx.x - bh * tiles) + 4 * c4, row = threadIdx.x >> 2;
  const float* moves = p.moves + bh * p.nseg * p.dk * width;
  float* Ms = reinterpret_cast<float*>(smem);
  const auto load = [&](int i) {   // the i-th in order
    const float* m = moves + (long long)(BACK ? p.nseg - 1 - i : i) * p.dk * width + p.dvp;
    for (int j = threadIdx.x; j < p.dk * (p.dk / 4); j += 256) {
      const int r = j / (p.dk / 4), u = j - r * (p.dk / 4);
      copy16(shared_at(Ms + ((i & 1) * p.dk + r) * ld + 4 * u), m + (long long)r * width + 4 * u, true);
    }
  };
  wait_prior();
  int raised = 0;   // of this segment's M; the first one's is not needed
  for (int at = 0; at < p.nseg - 1; ++at) {
    const int seg = BACK ? p.nseg - 1 - at : at, next = BACK ? seg - 1 : seg + 1;
    if (at + 1 < p.nseg - 1) load(at + 1);
    copy_commit();
    const float* n = moves + (long long)seg * p.dk * width + col;
    float4 x[LION_DELTA_MAX_D / 64];
#pragma unroll
    for (int i = 0; i < LION_DELTA_MAX_D / 64; ++i)
      if (row + 64 * i < p.dk) x[i] = *reinterpret_cast<const float4*>(n + (long long)(row + 64 * i) * width);
    const int raised_next = at + 1 < p.nseg - 1 ? p.raised[bh * p.nseg + next] : 0;
    copy_wait<1>();
    __syncthreads();   // M is there, and S of the threads' before
    if (at > 0) {
#pragma unroll
      for (int i = 0; i < LION_DELTA_MAX_D / 64; ++i) {
        if (row + 64 * i >= p.dk) continue;
        const float4 given = x[i];
        if (raised) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* m = Ms + ((at & 1) * p.dk + row + 64 * i) * ld;
#pragma unroll 2
        for (int k = 0; k < p.dk; k += 4) {
          const float4 a4 = *reinterpret_cast<const float4*>(m + k);
          const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 y = sh[k + e][c4];
            x[i].x = fmaf(a[e], y.x, x[i].x);
            x[i].y = fmaf(a[e], y.y, x[i].y);
            x[i].z = fmaf(a[e], y.z, x[i].z);
            x[i].w = fmaf(a[e], y.w, x[i].w);
          }
        }
        if (raised)
          x[i] = make_float4(given.x + ldexpf(x[i].x, raised), given.y + ldexpf(x[i].y, raised),
                             given.z + ldexpf(x[i].z, raised), given.w + ldexpf(x[i].w, raised));
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LION_DELTA_MAX_D / 64; ++i) {
      const int r = row + 64 * i;
      if (r >= p.dk) continue;
      sh[r][c4] = x[i];
      if (col < p.dv)
        *reinterpret_cast<float4*>(p.starts + ((bh * p.nseg + next) * p.dk + r) * p.dv + col) = x[i];
    }
    raised = raised_next;
  }
  copy_wait<0>();
}

template <bool BACK>
cudaError_t run_starts(const DeltaP& p, cudaStream_t s) {
  const auto kern = delta_starts_kernel<BACK>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, starts_smem(LION_DELTA_MAX_D));
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)((long long)p.B * p.Hv * (p.dvp / 16))), dim3(256),
                          (size_t)starts_smem(p.dk), s, p);
}

constexpr int kMoveThreads = 256;   // of the segments' walks: 8 x 16 columns of [N | M]

}  // namespace
}  // namespace lion
