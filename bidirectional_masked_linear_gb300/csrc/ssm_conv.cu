// ssm_conv.cu -- the short causal depthwise convolution along the tokens, its
// gradients and its one-token step.
//
//   p_i = bias + sum_{j<K} w[K-1-j] x_{i-j},  y_i = act(p_i)
//   dx_i = sum_{j<K} w[K-1-j] dp_{i+j},  dp = dy act'(p)
//   dw[K-1-j] = sum_{b,i} dp_i x_{i-j},  dbias = sum_{b,i} dp_i
// with i the order in which tokens are walked.  2 K operations a value: bound
// by HBM.  A thread walks a run of tokens for four channels with the window in
// registers; the next few tokens are read while it works on the last ones, so
// an input is read once plus K-1 tokens before each run (and behind it, for
// the gradients), which the neighbouring runs leave in the caches.  Measured at
// 64 x 197 x 1536, K = 4, bf16: 22 us forward and 34 us for the gradients (79
// and 116 MB: 3.6 and 3.4 TB/s; 63 and 199 with eight channels a thread and
// reads as they are needed); 16 prompts of up to 4096 x 1024: 44 us, 4.6 TB/s.
#include <algorithm>
#include <cmath>

#include "lion_internal.h"
#include "ssm_common.cuh"

namespace lion {
namespace {

struct ConvP {
  const void* x;
  const void* dy;
  const float* weight;
  const float* bias;
  const void* state;
  const int* lengths;
  void* out;          // y, or dx
  void* state_out;    // or dstate
  float* part;        // [parts][D*K | D]
  long long x_ld;
  int B, L, D;
  int act, reverse;
  int nvec;           // vectors of four channels
  int run, runs;      // tokens of a run; runs of a sequence
  bool x_wide, o_wide, s_wide, w_wide, items32;
};

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int L) {
  return lengths ? min(max(lengths[b], 0), L) : L;
}

// Tokens read ahead: 8 bytes of bfloat16 or 16 of fp32 a token and thread.
template <typename T>
struct Ahead {
  static constexpr int N = sizeof(T) == 2 ? 8 : 4;
};

// Four channels as two pairs.
struct Quad {
  f2 p[2];
  __device__ __forceinline__ Quad() {}
  __device__ __forceinline__ explicit Quad(const float (&v)[4]) { p[0] = pack2(v[0], v[1]); p[1] = pack2(v[2], v[3]); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = p[0].x; v[1] = p[0].y; v[2] = p[1].x; v[3] = p[1].y;
  }
};
__device__ __forceinline__ Quad zero4() {
  Quad q;
  q.p[0] = q.p[1] = pack2(0.f, 0.f);
  return q;
}

// Four raw elements.
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 r;
  __device__ __forceinline__ void zero() { r = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool wide) {
    if (wide) {
      r = *reinterpret_cast<const uint2*>(p);
    } else {
      unsigned short h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = e < n ? reinterpret_cast<const unsigned short*>(p)[e] : 0;
      r = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    }
  }
  __device__ __forceinline__ Quad get() const {
    Quad q;
    q.p[0] = unpack_bf16(r.x);
    q.p[1] = unpack_bf16(r.y);
    return q;
  }
};
template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p, int n, bool wide) {
    if (wide) r = *reinterpret_cast<const float4*>(p);
    else r = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
  }
  __device__ __forceinline__ Quad get() const {
    Quad q;
    q.p[0] = pack2(r.x, r.y);
    q.p[1] = pack2(r.z, r.w);
    return q;
  }
};
__device__ __forceinline__ void store4(float* p, int n, bool wide, const Quad& q) {
  float v[4];
  q.get(v);
  if (wide) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, int n, bool wide, const Quad& q) {
  float v[4];
  q.get(v);
  if (wide) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = __float2bfloat16_rn(v[e]);
  }
}

// The taps of channels c0 .. c0 + 3 (adjacent in memory) and their bias.
template <int K>
__device__ __forceinline__ void load_taps(const ConvP& p, int c0, Quad (&w)[K], Quad& bias) {
  float f[4 * K], b[4];
  const int n = p.D - c0;
  if (p.w_wide && n >= 4) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(p.weight + (size_t)c0 * K + 4 * k);
      f[4 * k] = x.x; f[4 * k + 1] = x.y; f[4 * k + 2] = x.z; f[4 * k + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4 * K; ++k) f[k] = k < n * K ? p.weight[(size_t)c0 * K + k] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = p.bias && e < n ? p.bias[c0 + e] : 0.f;
  bias = Quad(b);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float v[4] = {f[k], f[K + k], f[2 * K + k], f[3 * K + k]};
    w[k] = Quad(v);
  }
}

// A thread's line: four channels of one sequence.
template <typename T, int K>
struct Line {
  int b, c0, n, len;
  bool xw, ow, sw;   // whole aligned vectors: x, the tight activations, the states
  __device__ __forceinline__ Line(const ConvP& p, int b_, int c0_) : b(b_), c0(c0_) {
    n = p.D - c0;
    len = clamp_len(p.lengths, b, p.L);
    xw = p.x_wide && n >= 4;
    ow = p.o_wide && n >= 4;
    sw = p.s_wide && n >= 4;
  }
  __device__ __forceinline__ int token(const ConvP& p, int i) const { return p.reverse ? len - 1 - i : i; }
  // The input processed i-th (i < 0: from the state; zeros where there is none).
  __device__ __forceinline__ Raw4<T> at(const ConvP& p, int i) const {
    Raw4<T> r;
    r.zero();
    if (i >= 0 && i < len)
      r.load(static_cast<const T*>(p.x) + ((long long)b * p.L + token(p, i)) * p.x_ld + c0, n, xw);
    else if (i < 0 && i >= -(K - 1) && p.state)
      r.load(static_cast<const T*>(p.state) + ((long long)b * (K - 1) + K - 1 + i) * p.D + c0, n, sw);
    return r;
  }
};

// bias + sum_k w_k win_k
template <int K>
__device__ __forceinline__ f2 taps(const Quad (&w)[K], const Quad (&win)[K], f2 bias, int h) {
#pragma unroll
  for (int k = 0; k < K; ++k) bias = fma2(w[k].p[h], win[k].p[h], bias);
  return bias;
}

template <typename T, int K>
__global__ void __launch_bounds__(128) conv_fwd_kernel(ConvP p) {
  constexpr int A = Ahead<T>::N;
  const unsigned long long item = (unsigned long long)blockIdx.x * 128 + threadIdx.x;
  // divisions in 32 bits wherever the problem allows
  const unsigned line = p.items32 ? (unsigned)item / (unsigned)p.nvec : (unsigned)(item / (unsigned)p.nvec);
  const int b = (int)(line / (unsigned)p.runs), i0 = (int)(line - (unsigned)b * p.runs) * p.run;
  if (b >= p.B) return;
  const Line<T, K> l(p, b, 4 * (int)(item - (unsigned long long)line * p.nvec));
  const int i1 = min(i0 + p.run, p.L);
  Quad w[K], bias, win[K];
  const long long x_hop = p.reverse ? -p.x_ld : p.x_ld, y_hop = p.reverse ? -p.D : p.D;
  const T* x = static_cast<const T*>(p.x) + ((long long)b * p.L + l.token(p, i0)) * p.x_ld + l.c0;
  T* y = static_cast<T*>(p.out) + ((long long)b * p.L + l.token(p, i0)) * p.D + l.c0;
  const int real = min(i1, l.len) - i0;   // tokens of the run that there are
  Raw4<T> next[A];
  auto read = [&](int j) {
#pragma unroll
    for (int a = 0; a < A; ++a) {
      next[a].zero();
      if (j + a < real) next[a].load(x + a * x_hop, l.n, l.xw);
    }
    x += A * x_hop;
  };
  read(0);
#pragma unroll
  for (int k = 1; k < K; ++k) win[k] = l.at(p, i0 - K + k).get();
  load_taps<K>(p, l.c0, w, bias);
  for (int j = 0; j < real; j += A) {
    Raw4<T> now[A];
#pragma unroll
    for (int a = 0; a < A; ++a) now[a] = next[a];
    if (j + A < real) read(j + A);
    const bool full = l.ow && j + A <= real;
#pragma unroll
    for (int a = 0; a < A; ++a) {
#pragma unroll
      for (int k = 0; k + 1 < K; ++k) win[k] = win[k + 1];
      win[K - 1] = now[a].get();
      Quad o;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f2 s = taps<K>(w, win, bias.p[h], h);
        o.p[h] = p.act ? mul2(s, sigmoid2(s.x, s.y)) : s;
      }
      if (full) store4(y + a * y_hop, 4, true, o);
      else if (j + a < real) store4(y + a * y_hop, l.n, l.ow, o);
    }
    y += A * y_hop;
  }
  // tokens past the length are not part of the walk: zeros where they lie
  for (int i = max(i0, l.len); i < i1; ++i)
    store4(static_cast<T*>(p.out) + ((long long)b * p.L + i) * p.D + l.c0, l.n, l.ow, zero4());
  if (p.state_out && i0 == 0) {
    T* st = static_cast<T*>(p.state_out) + (long long)b * (K - 1) * p.D + l.c0;
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      store4(st + (long long)k * p.D, l.n, l.sw, l.at(p, l.len - (K - 1) + k).get());
  }
}

constexpr int kBwdRows = 8;   // runs that a CTA walks at a time

// One CTA: 32 channel vectors (lanes) x kBwdRows runs.  Each thread keeps its
// channels' share of dweight and dbias over all the runs it walks.
template <typename T, int K>
__global__ void __launch_bounds__(32 * kBwdRows, 2) conv_bwd_kernel(ConvP p) {
  constexpr int A = sizeof(T) == 2 ? 4 : 2;   // tokens read ahead, of both inputs
  __shared__ float sh[kBwdRows][32][4];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int c0 = 4 * (blockIdx.x * 32 + lane);
  const bool live = c0 < p.D;
  Quad w[K], bias, dw[K], db = zero4();
  load_taps<K>(p, live ? c0 : p.D, w, bias);
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k] = zero4();
  const long long x_hop = p.reverse ? -p.x_ld : p.x_ld, d_hop = p.reverse ? -p.D : p.D;
  const unsigned lines = p.B * p.runs;   // fewer than 2^31: a step past them stays in 32 bits
  for (unsigned next = blockIdx.y * kBwdRows + r; live && next < lines; next += gridDim.y * kBwdRows) {
    const int line = (int)next;   // (an unsigned division costs 0.5 us of 55 at 64 x 197 x 1536)
    const int b = line / p.runs, i0 = (line - b * p.runs) * p.run;
    const Line<T, K> l(p, b, c0);
    const int i1 = min(i0 + p.run, p.L), mine = min(i1, l.len) - i0;
    // the sums that end in the run need dp up to K-1 tokens behind it
    const int real = mine > 0 || (i0 == 0 && p.state_out) ? min(i1 + K - 1, l.len) - i0 : 0;
    const T* x = static_cast<const T*>(p.x) + ((long long)b * p.L + l.token(p, i0)) * p.x_ld + c0;
    const T* dy = static_cast<const T*>(p.dy) + ((long long)b * p.L + l.token(p, i0)) * p.D + c0;
    T* dx = static_cast<T*>(p.out) + ((long long)b * p.L + l.token(p, i0)) * p.D + c0;
    Raw4<T> nx[A], ny[A];
    auto read = [&](int j) {
#pragma unroll
      for (int a = 0; a < A; ++a) {
        nx[a].zero();
        ny[a].zero();
        if (j + a < real) {
          nx[a].load(x + a * x_hop, l.n, l.xw);
          ny[a].load(dy + a * d_hop, l.n, l.ow);
        }
      }
      x += A * x_hop;
      dy += A * d_hop;
    };
    read(0);
    // win[k] = x_{i-K+1+k}, dp[k] = dp_{i-K+1+k}
    Quad win[K], dp[K];
#pragma unroll
    for (int k = 0; k < K; ++k) dp[k] = zero4();
    // (the state before a sequence without tokens meets no gradient, whatever it holds)
#pragma unroll
    for (int k = 1; k < K; ++k) win[k] = l.at(p, l.len > 0 ? i0 - K + k : -K).get();
    const int last = mine + K - 1;   // steps until the run's last dx is complete
    for (int j = 0; j < last; j += A) {
      Raw4<T> vx[A], vy[A];
#pragma unroll
      for (int a = 0; a < A; ++a) {
        vx[a] = nx[a];
        vy[a] = ny[a];
      }
      if (j + A < last) read(j + A);
      // every token of the batch counts, and every sum that it completes is one of the run's
      const bool full = l.ow && j >= K - 1 && j + A <= mine;
#pragma unroll
      for (int a = 0; a < A; ++a) {
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) {
          win[k] = win[k + 1];
          dp[k] = dp[k + 1];
        }
        win[K - 1] = vx[a].get();
        const Quad g = vy[a].get();   // 0 where there is no token
        Quad o;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f2 d = g.p[h];
          if (p.act) {
            const f2 s = taps<K>(w, win, bias.p[h], h), sg = sigmoid2(s.x, s.y);
            // silu'(s) = sg + s sg (1 - sg)
            d = mul2(d, fma2(mul2(s, sg), fma2(sg, pack2(-1.f, -1.f), pack2(1.f, 1.f)), sg));
          }
          if (!full && j + a >= real) d = pack2(0.f, 0.f);
          dp[K - 1].p[h] = d;
          f2 dm = d;
          if (!full && j + a >= mine) dm = pack2(0.f, 0.f);
          db.p[h] = add2(db.p[h], dm);
#pragma unroll
          for (int k = 0; k < K; ++k) dw[k].p[h] = fma2(dm, win[k].p[h], dw[k].p[h]);
          // dx_m for m = i - K + 1 is complete
          o.p[h] = mul2(w[K - 1].p[h], dp[0].p[h]);
#pragma unroll
          for (int q = 1; q < K; ++q) o.p[h] = fma2(w[K - 1 - q].p[h], dp[q].p[h], o.p[h]);
        }
        const int m = j + a - K + 1;
        if (full)
          store4(dx + m * d_hop, 4, true, o);
        else if (m >= 0 && m < mine)
          store4(dx + m * d_hop, l.n, l.ow, o);
        else if (m < 0 && i0 == 0 && p.state_out)
          store4(static_cast<T*>(p.state_out) + ((long long)b * (K - 1) + K - 1 + m) * p.D + c0, l.n, l.sw, o);
      }
    }
    for (int i = max(i0, l.len); i < i1; ++i)
      store4(static_cast<T*>(p.out) + ((long long)b * p.L + i) * p.D + c0, l.n, l.ow, zero4());
  }
  float* part = p.part + (size_t)blockIdx.y * p.D * (K + 1);
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    float v[4];
    (k < K ? dw[k < K ? k : 0] : db).get(v);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) sh[r][lane][e] = v[e];
    __syncthreads();
    if (r < 4 && c0 + r < p.D) {   // thread (lane, r): channel c0 + r
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < kBwdRows; ++q) s += sh[q][lane][r];
      if (k < K) part[(size_t)(c0 + r) * K + k] = s;
      else part[(size_t)p.D * K + c0 + r] = s;
    }
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(128) conv_step_kernel(const T* x, T* state, const float* weight, const float* bias,
                                                        T* y, int B, int D, int act) {
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
  if (i >= (long long)B * D) return;
  const int b = (int)(i / D), c = (int)(i - (long long)b * D);
  T* st = state + (long long)b * (K - 1) * D + c;
  T win[K];
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) win[k] = st[(long long)k * D];
  win[K - 1] = x[i];
  float a = bias ? bias[c] : 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) a = fmaf(weight[(size_t)c * K + k], to_f32(win[k]), a);
  y[i] = from_f32<T>(act ? a * sigmoid(a) : a);
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) st[(long long)k * D] = win[k + 1];
}

#define LION_CONV_DISPATCH(RUN, dtype, K, ...)                                                     \
  (dtype == DT_BF16 ? (K == 2   ? RUN<__nv_bfloat16, 2>(__VA_ARGS__)                               \
                       : K == 3 ? RUN<__nv_bfloat16, 3>(__VA_ARGS__)                               \
                                : RUN<__nv_bfloat16, 4>(__VA_ARGS__))                              \
                    : (K == 2   ? RUN<float, 2>(__VA_ARGS__)                                       \
                       : K == 3 ? RUN<float, 3>(__VA_ARGS__)                                       \
                                : RUN<float, 4>(__VA_ARGS__)))

template <typename T, int K>
cudaError_t run_fwd(const ConvP& p, cudaStream_t s) {
  const long long items = (long long)p.B * p.runs * p.nvec;
  ConvP q = p;
  q.items32 = items + 128 < 0x100000000LL;
  conv_fwd_kernel<T, K><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(q);
  return cudaGetLastError();
}
template <typename T, int K>
cudaError_t run_bwd(const ConvP& p, int parts, cudaStream_t s) {
  conv_bwd_kernel<T, K><<<dim3((p.nvec + 31) / 32, parts), 32 * kBwdRows, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int K>
cudaError_t run_step(const void* x, void* state, const float* weight, const float* bias, void* y, int B, int D,
                     int act, cudaStream_t s) {
  const long long n = (long long)B * D;
  conv_step_kernel<T, K><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(
      static_cast<const T*>(x), static_cast<T*>(state), weight, bias, static_cast<T*>(y), B, D, act);
  return cudaGetLastError();
}

// Tokens of a run (a multiple of eight, less what the gradients read behind
// it): the length that fills the SMs' slots in the fewest rounds of run +
// kStart tokens, kStart being what a thread takes to begin; a round that is
// not full counts for 0.4 plus 0.6 of its fill.  slots_of(runs): how many times
// that many runs a sequence fill the slots.  `lengths` are not seen here: a
// ragged batch gets a full one's run length.
constexpr int kStart = 8;
template <typename F>
int best_run(int L, int behind, F slots_of) {
  int best = 8 - behind;
  float least = 3e38f;
  for (int m = 8; m <= 72; m += 8) {
    const int run = m - behind;
    const float x = slots_of((L + run - 1) / run), full = floorf(x);
    const float cost = (full + (x > full ? 0.4f + 0.6f * (x - full) : 0.f)) * (float)(run + kStart);
    if (cost < least) {
      least = cost;
      best = run;
    }
    if (run >= L) break;
  }
  return best;
}
// Five CTAs an SM: what bfloat16 at K = 4 and float32 up to K = 3 hold; the others hold four.
int fwd_run(int B, int L, int D) {
  return best_run(L, 0, [&](int runs) { return (float)B * runs * ((D + 3) / 4) / (float)(kSmCount * 5 * 128); });
}

// CTAs along the runs in the gradients: at most what the SMs hold at once.
int conv_parts(int B, int L, int D, int run) {
  const int across = (D + 127) / 128, most = std::max(1, 2 * kSmCount / across);
  const long long want = ((long long)B * ((L + run - 1) / run) + kBwdRows - 1) / kBwdRows;
  return (int)std::min<long long>(want, most);
}
int bwd_run(int B, int L, int D, int K) {
  const int across = (D + 127) / 128, most = std::max(1, 2 * kSmCount / across);
  return best_run(L, K - 1, [&](int runs) {
    const float turns = ceilf((float)B * runs / (float)(most * kBwdRows));   // a CTA's lines follow one another
    return turns <= 1.f ? (float)B * runs / (float)(most * kBwdRows) : turns;
  });
}

}  // namespace

size_t conv_bwd_workspace_bytes(int B, int L, int D, int K) {
  return sizeof(float) * (size_t)conv_parts(B, L, D, bwd_run(B, L, D, K)) * D * (K + 1);
}

cudaError_t launch_conv_fwd(const lion_conv_args& a, cudaStream_t s) {
  ConvP p = {};
  p.x = a.x;
  p.weight = a.weight;
  p.bias = a.bias;
  p.state = a.state;
  p.lengths = a.lengths;
  p.out = a.y;
  p.state_out = a.state_out;
  p.x_ld = a.x_token ? a.x_token : a.D;
  p.B = a.B;
  p.L = a.L;
  p.D = a.D;
  p.act = a.act;
  p.reverse = a.reverse;
  p.w_wide = rows_wide(a.weight, 0, 4);
  p.nvec = (a.D + 3) / 4;
  p.run = fwd_run(a.B, a.L, a.D);
  p.runs = (a.L + p.run - 1) / p.run;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.x_wide = rows_wide(a.x, p.x_ld, es);
  p.o_wide = rows_wide(a.y, a.D, es);
  p.s_wide = rows_wide(a.state, a.D, es) && rows_wide(a.state_out, a.D, es);
  return LION_CONV_DISPATCH(run_fwd, a.dtype, a.K, p, s);
}

cudaError_t launch_conv_bwd(const lion_conv_bwd_args& a, void* ws, cudaStream_t s) {
  ConvP p = {};
  p.x = a.x;
  p.dy = a.dy;
  p.weight = a.weight;
  p.bias = a.bias;
  p.state = a.state;
  p.lengths = a.lengths;
  p.out = a.dx;
  p.state_out = a.dstate;
  p.part = static_cast<float*>(ws);
  p.x_ld = a.x_token ? a.x_token : a.D;
  p.B = a.B;
  p.L = a.L;
  p.D = a.D;
  p.act = a.act;
  p.reverse = a.reverse;
  p.w_wide = rows_wide(a.weight, 0, 4);
  p.nvec = (a.D + 3) / 4;
  p.run = bwd_run(a.B, a.L, a.D, a.K);
  p.runs = (a.L + p.run - 1) / p.run;
  const int es = a.dtype == DT_BF16 ? 2 : 4;
  p.x_wide = rows_wide(a.x, p.x_ld, es);
  p.o_wide = rows_wide(a.dx, a.D, es) && rows_wide(a.dy, a.D, es);
  p.s_wide = rows_wide(a.state, a.D, es) && rows_wide(a.dstate, a.D, es);
  const int parts = conv_parts(a.B, a.L, a.D, p.run);
  cudaError_t e = LION_CONV_DISPATCH(run_bwd, a.dtype, a.K, p, parts, s);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(p.part, parts, (long long)a.D * (a.K + 1), (long long)a.D * a.K, a.dweight, a.D, a.dbias, 0,
                          nullptr, s);
}

cudaError_t launch_conv_step(const void* x, void* state, const float* weight, const float* bias, void* y, int B, int D,
                             int K, int act, int dtype, cudaStream_t s) {
  return LION_CONV_DISPATCH(run_step, dtype, K, x, state, weight, bias, y, B, D, act, s);
}

}  // namespace lion
