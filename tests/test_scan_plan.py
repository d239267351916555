"""The scan's plan (scan_plan.h, compiled here with the host compiler): channel
blocks and segments cover every channel and token once."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def plans(tmp_path, cases):
    """[(forward, gradients)] of cases (B, L, D, N, G, ragged), each (blocks, segments, tokens of a segment,
    channels of a block)."""
    src = tmp_path / "plan.cpp"
    src.write_text(
        '#include <cstdio>\n#include "scan_plan.h"\n'
        "int main() { int B, L, D, N, G, r;\n"
        '  while (scanf("%d %d %d %d %d %d", &B, &L, &D, &N, &G, &r) == 6) {\n'
        "    const lion::ScanPlan f = lion::scan_fwd_plan(B, L, D, N, G, r), b = lion::scan_bwd_plan(B, L, D, N, G, r);\n"
        '    printf("%d %d %d %d %d %d %d %d\\n", f.nblk, f.nseg, f.seglen, lion::scan_fwd_channels(N), b.nblk, b.nseg,\n'
        "           b.seglen, lion::scan_bwd_channels(N)); } }\n")
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "bidirectional_masked_linear_gb300", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    text = "\n".join(" ".join(str(int(v)) for v in c) for c in cases)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.strip().split("\n")]
    return [(r[:4], r[4:]) for r in rows]


def test_blocks_and_segments_cover_everything(tmp_path):
    cases = [(B, L, D, N, G, ragged) for B in (1, 3, 64) for L in (1, 15, 16, 127, 128, 1021, 24337, 10 ** 6)
             for D in (6, 96, 330, 2048) for N in (8, 16, 32, 64) for G in (1, 3) if D % G == 0
             for ragged in (False, True)]
    for (B, L, D, N, G, _), both in zip(cases, plans(tmp_path, cases)):
        for nblk, nseg, seglen, channels in both:
            assert (nblk - 1) * channels < D // G <= nblk * channels
            assert seglen % 16 == 0 and (nseg - 1) * seglen < L <= nseg * seglen
            assert nseg == 1 or seglen >= 64
