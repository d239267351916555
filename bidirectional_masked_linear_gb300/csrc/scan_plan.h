// scan_plan.h -- how the selective scan's launches cut the work (plain C++, no
// CUDA): channels into CTAs' blocks, sequences into segments.
#pragma once

#include <algorithm>

namespace lion {

constexpr int kSmCount = 152;

// Warps and channels of a CTA: forward (one warp: CTAs of one spread best, 64 x 197 x 1536 x 16 529 -> 525 us both
// ways against four) and gradients.
constexpr int kScanFwdWarps = 1, kScanBwdWarps = 4;
constexpr int scan_fwd_channels(int N) { return kScanFwdWarps * (N == 8 ? 128 : 1024 / N); }
constexpr int scan_bwd_channels(int N) { return kScanBwdWarps * (N == 8 ? 32 : 512 / N); }

struct ScanPlan {
  int nblk, nseg, seglen;   // channel blocks of a group; segments of a sequence and their tokens
};

// Cuts sequences into segments so that the SMs' slots for CTAs are filled in
// whole rounds.  The cost, in tokens of a round: rounds x (a segment's tokens +
// what a CTA takes to start), a round that is not full counting for 0.4 plus
// 0.6 of its fill (fewer CTAs on an SM run faster), plus the chain over the
// segments and their states' way through HBM; a sequence left whole is spared
// the pass over the segments' own contributions and costs `whole` of that.  Ragged sequences, whose lengths
// the host does not see, are taken to fill half of the tokens in CTAs that end
// at any time: only the last one's time counts in full, which asks for short
// segments (16 prompts of up to 4096 tokens x 1024 channels: 509 us with two
// whole rounds, 322 to 335 us so; the same batch with every length full takes
// 510 us, and 500 without lengths).  Up to kMaxSegments, of 64 tokens at least.
inline ScanPlan scan_plan(int B, int L, int D, int N, int G, int cta_channels, int slots, float whole, bool ragged) {
  constexpr int kMaxSegments = 512;
  ScanPlan r;
  r.nblk = (D / G + cta_channels - 1) / cta_channels;
  const long long ctas = (long long)B * G * r.nblk;
  auto rounds = [&](long long n) {
    if (ragged) return 0.5f * (float)n / (float)slots + 0.8f;
    const long long full = n / slots, rest = n % slots;
    return (float)full + (rest ? 0.4f + 0.6f * (float)rest / (float)slots : 0.f);
  };
  // a token of a round is some 0.85 us; a segment's states cross HBM four times
  const float states = 4.f * 4.f * (float)B * (float)D * (float)N / (6.7e6f * 0.85f);
  r.nseg = 1;
  r.seglen = (L + 15) / 16 * 16;
  float best = whole * rounds(ctas) * ((float)L + 6.f);
  const int most = std::min(kMaxSegments, L / 64);
  for (int n = 2; n <= most; ++n) {
    const int len = ((L + n - 1) / n + 15) / 16 * 16, real = (L - 1) / len + 1;   // whole tiles
    if (real != n) continue;
    const float cost = rounds(ctas * n) * ((float)len + 6.f) + (0.18f + states) * (float)n;
    if (cost < best) {
      best = cost;
      r.nseg = n;
      r.seglen = len;
    }
  }
  return r;
}

// The slots are those of the measured bfloat16 cases.  The forward's warps an SM hold for every type and N but float32
// at N = 16 (11 of 12) and N = 32 (9 of 12), the gradients' two CTAs but for float32 at N = 16 and N = 64 (one): those
// take more rounds than are counted here.
inline ScanPlan scan_fwd_plan(int B, int L, int D, int N, int G, bool ragged) {
  return scan_plan(B, L, D, N, G, scan_fwd_channels(N), kSmCount * (N == 64 ? 8 : 12) / kScanFwdWarps, 0.6f, ragged);
}
inline ScanPlan scan_bwd_plan(int B, int L, int D, int N, int G, bool ragged) {
  return scan_plan(B, L, D, N, G, scan_bwd_channels(N), 2 * kSmCount, 0.85f, ragged);
}

}  // namespace lion
