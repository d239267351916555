// delta_internal.h -- what the gated delta rule's files share on the host: the
// layout of what a forward call keeps, and the parameters of its kernels.
#pragma once

#include <algorithm>

#include "delta_common.cuh"

namespace lion {

// Every chunk's ChunkData; with `save`, as the gradients take them, then R of
// every token and the state before every 64th.  Beside these U, and where the
// walk is cut into segments what they make of a state and the states before them.
struct DeltaLayout {
  size_t R, states, bytes;        // offsets of R and the states, and all of it
  size_t moves, starts, raised, beside;   // the same of U's neighbours
  int nc, nc64, dvp, nseg, seglen;
};
template <typename T, int DK, bool SAVE>
constexpr size_t chunk_bytes() {
  return ChunkData<T, DK, SAVE, sizeof(T) == 4>::bytes;
}
inline DeltaLayout delta_layout(int B, int L, int Hv, int dk, int dv, int dtype, bool save) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  DeltaLayout l;
  const bool bf16 = dtype == DT_BF16;
  const size_t es = bf16 ? 2 : 4, heads = (size_t)B * Hv, DK = dk <= 64 ? 64 : 128;
  const size_t chunk =
      bf16 ? (DK == 64 ? (save ? chunk_bytes<__nv_bfloat16, 64, true>() : chunk_bytes<__nv_bfloat16, 64, false>())
                       : (save ? chunk_bytes<__nv_bfloat16, 128, true>() : chunk_bytes<__nv_bfloat16, 128, false>()))
           : (DK == 64 ? (save ? chunk_bytes<float, 64, true>() : chunk_bytes<float, 64, false>())
                       : (save ? chunk_bytes<float, 128, true>() : chunk_bytes<float, 128, false>()));
  l.nc = (L + kChunk - 1) / kChunk;
  l.nc64 = (L + kStateChunk - 1) / kStateChunk;
  l.dvp = (dv + 15) / 16 * 16;
  // Segments: as many as fill two places an SM, of 16 chunks at least, three of
  // them at least, for walks on a quarter of the SMs or less.  A training step's
  // kernels whole and cut, us (of 128 a head has two walks):
  //   heads of 64, L = 24337   24: 1893 1126   38: 2165 1669   48: 2370 2157   64: 2697 3030
  //   heads of 64, L = 4096                    38:  381  336   48:  419  426   64:  476  556
  //   heads of 128, L = 16384  12: 1804 1223   19: 1997 1706   24: 2143 2220   32: 2372 3001
  const long long ctas = (long long)heads * ((dv + kSlice - 1) / kSlice);
  const long long most = bf16 && 4 * ctas <= kSmCount ? std::min<long long>(2 * kSmCount / ctas, l.nc / 16) : 1;
  l.seglen = most >= 3 ? (int)((l.nc + most - 1) / most) : l.nc;
  l.nseg = (l.nc + l.seglen - 1) / l.seglen;
  const size_t cut = l.nseg > 1 ? heads * l.nseg * dk * sizeof(float) : 0;
  l.moves = up(heads * l.nc * l.dvp * kChunk * sizeof(float));
  l.starts = l.moves + up(cut * (l.dvp + dk));
  l.raised = l.starts + up(cut * dv);
  l.beside = l.raised + (l.nseg > 1 ? up(heads * l.nseg * sizeof(int)) : 0);
  l.R = up(heads * l.nc * chunk);
  l.states = l.R + (save ? up(heads * l.nc * kChunk * l.dvp * es) : 0);
  l.bytes = l.states + (save ? up(heads * l.nc64 * l.dvp * DK * es) : 0);
  return l;
}

// kept: `bytes` of the layout, beside: its `beside`.
template <typename Args>
DeltaP delta_params(const Args& a, char* kept, char* beside, bool save) {
  const DeltaLayout l = delta_layout(a.B, a.L, a.Hv, a.dk, a.dv, a.dtype, save);
  DeltaP p = {};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.g = a.g;
  p.beta = a.beta;
  p.lengths = a.lengths;
  p.h0 = a.h0;
  p.chunks = kept;
  p.U = reinterpret_cast<float*>(beside);
  p.moves = reinterpret_cast<float*>(beside + l.moves);
  p.starts = reinterpret_cast<float*>(beside + l.starts);
  p.raised = reinterpret_cast<int*>(beside + l.raised);
  p.nseg = l.nseg;
  p.seglen = l.seglen;
  if (save) {
    p.R = kept + l.R;
    p.states = kept + l.states;
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
  p.dvp = l.dvp;
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

// Whether the walks' CTAs are more than two an SM.
inline bool crowded(const DeltaP& p) { return (long long)p.B * p.Hv * p.slices > 2 * kSmCount; }
// Whether CTAs of 32 columns are no more than the SMs.
inline bool few(const DeltaP& p) { return (long long)p.B * p.Hv * p.nseg * ((p.dv + 31) / 32) <= kSmCount; }

// Every chunk's ChunkData and U, then the chain; R and states where `save`.
cudaError_t launch_delta_chain(const DeltaP& p, int dtype, bool save, cudaStream_t s);

}  // namespace lion
