"""How a product of 8-bit matrices is split, compiled for the host from the kernel's source: every plan is one
that its launch can run, with no more of the contraction in an accumulator than it may hold."""

import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "matrix_optimizer_owner_gb300", "csrc", "gemm_fp8.cu")

HARNESS = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
%s
int main() {
  const int64_t sides[] = {1, 2, 16, 17, 64, 65, 100, 128, 129, 256, 300, 513, 768, 1024, 1536, 2304, 4096,
                           9216, 9472, 14336, 40000};
  const int64_t ks[] = {1, 128, 129, 1000, 1920, 2048, 4096, 8192, 8193, 16256, 16384, 16385, 17000, 20480,
                        32768, 65536, 65537, 131072, 200000, 524288, 600000, 4000000};
  long counts[3] = {0, 0, 0};
  for (int64_t m : sides)
    for (int64_t n : sides)
      for (int64_t k : ks)
        for (int bf16 : {0, 1})
          for (int acc : {0, 1}) {
            const Gemm8Plan p = plan_gemm(m, n, k, bf16, acc);
            const int nkb = (int)((k + kB8 - 1) / kB8), most = most_blocks(bf16);
            const int64_t tiles = ((m + 255) / 256) * ((n + 255) / 256);
            bool ok = !(p.narrow && p.halves);
            if (p.narrow)
              ok = ok && p.splits >= 1 && p.splits <= 8 && p.kb_split <= most &&
                   (int64_t)p.splits * p.kb_split >= nkb && std::min(m, n) <= (p.nt < 128 ? p.nt : 1 << 30);
            if (p.halves)
              ok = ok && p.kb_split > 0 && p.kb_split < nkb && p.kb_split %% 8 == 0 && p.kb_split <= most &&
                   nkb - p.kb_split <= most && 2 * tiles <= kClusters[4];   // (one CTA an SM)
            ++counts[p.halves ? 2 : p.narrow ? 1 : 0];
            if (!ok) {
              std::printf("%%lld x %%lld x %%lld %%s%%s: narrow %%d halves %%d splits %%d of %%d blocks\n", (long long)m,
                          (long long)n, (long long)k, bf16 ? "bf16" : "f32", acc ? " added" : "", p.narrow,
                          p.halves, p.splits, p.kb_split);
              return 1;
            }
          }
  return counts[0] && counts[1] && counts[2] ? 0 : 2;
}
"""


def test_plans_are_runnable(tmp_path):
    text = open(SRC).read()
    parts = [re.search(r"constexpr int kB8 = \d+;", text).group(0),
             re.search(r"constexpr int kChunk8 = \d+;", text).group(0),
             re.search(r"constexpr int kPairs = .*?\nGemm8Plan plan_gemm.*?\n}\n", text, re.S).group(0)]
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(HARNESS % "\n".join(parts))
    subprocess.run(["g++", "-std=c++17", "-O1", str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
