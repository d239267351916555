// delta_internal.h -- what the gated delta rule's files share on the host: the
// layout of what a forward call keeps, and the parameters of its kernels.
#pragma once

#include "delta_common.cuh"

namespace lion {

// Per head and chunk of 32 tokens the planes of T and P and the coefficients;
// with `save`, as the gradients take it, P in as many planes as T, then R of
// every token and the state before every 64th.
struct DeltaLayout {
  size_t tp_chunk, R, states, bytes;
  int nc, nc64;
};
inline DeltaLayout delta_layout(int B, int L, int Hv, int dk, int dv, int dtype, bool save) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  DeltaLayout l;
  const size_t es = dtype == DT_BF16 ? 2 : 4, heads = (size_t)B * Hv;
  const int mid = dtype == DT_BF16 ? Planes<__nv_bfloat16>::mid : Planes<float>::mid;
  const int planes = mid + (save || dtype != DT_BF16 ? mid : 1);
  l.nc = (L + kChunk - 1) / kChunk;
  l.nc64 = (L + kStateChunk - 1) / kStateChunk;
  l.tp_chunk = (size_t)planes * kTile + kCoefs * sizeof(float);
  l.R = up(heads * l.nc * l.tp_chunk);
  l.states = l.R + (save ? up(heads * l.nc * kChunk * dv * es) : 0);
  l.bytes = l.states + (save ? up(heads * l.nc64 * dv * dk * es) : 0);
  return l;
}

template <typename Args>
DeltaP delta_params(const Args& a, void* kept, bool save) {
  const DeltaLayout l = delta_layout(a.B, a.L, a.Hv, a.dk, a.dv, a.dtype, save);
  DeltaP p = {};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.g = a.g;
  p.beta = a.beta;
  p.lengths = a.lengths;
  p.h0 = a.h0;
  p.tp = kept;
  p.tp_chunk = (long long)l.tp_chunk;
  if (save) {
    p.R = static_cast<char*>(kept) + l.R;
    p.states = static_cast<char*>(kept) + l.states;
  }
  p.q_ld = a.q_token ? a.q_token : (long long)a.Hk * a.dk;
  p.k_ld = a.k_token ? a.k_token : (long long)a.Hk * a.dk;
  p.v_ld = a.v_token ? a.v_token : (long long)a.Hv * a.dv;
  p.g_ld = a.g_token ? a.g_token : a.Hv;
  p.beta_ld = a.beta_token ? a.beta_token : a.Hv;
  p.B = a.B;
  p.L = a.L;
  p.Hk = a.Hk;
  p.Hv = a.Hv;
  p.dk = a.dk;
  p.dv = a.dv;
  p.nc = l.nc;
  p.nc64 = l.nc64;
  p.slices = (a.dv + kSlice - 1) / kSlice;
  p.scale = a.scale;
  p.reverse = a.reverse;
  const int es = a.dtype == DT_BF16 ? 2 : 4;   // heads lie on 16 bytes where tokens do: sizes are multiples of 8
  p.q_wide = rows_wide(a.q, p.q_ld, es);
  p.k_wide = rows_wide(a.k, p.k_ld, es);
  p.v_wide = rows_wide(a.v, p.v_ld, es);
  return p;
}

// T, P and the decays of every chunk, then the chain; p.R and p.states where `save`.
cudaError_t launch_delta_chain(const DeltaP& p, int dtype, bool save, cudaStream_t s);

}  // namespace lion
