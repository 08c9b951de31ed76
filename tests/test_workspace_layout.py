"""Where the parts of the workspaces lie: compiled from the library's own header, no GPU needed."""
import os
import random
import shutil
import subprocess

import pytest

from paged_gqa_gb300 import build as B

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "workspace.cuh"
int pgqa::q_amax_parts(int sms) { return 2 * sms; }
int main(int argc, char** argv) {
  using namespace pgqa;
  std::printf("%zu %zu\n", kWsEpochOff, kWsHead);
  for (int i = 1; i + 4 < argc; i += 5) {
    const WsLayout L = make_layout(atoi(argv[i]), atoi(argv[i + 1]), atoi(argv[i + 2]), atoi(argv[i + 3]), atoi(argv[i + 4]));
    for (int c = 0; c < kNumClasses; ++c)
      for (int j = 0; j < 7; ++j) std::printf("%zu ", L.off[c][j]);
    std::printf("%zu %zu\n", L.q_amax_off, L.total);
    const PromptLayout P = prompt_layout(1 + atoi(argv[i]) % (atoi(argv[i + 4]) / 2));
    std::printf("%zu %zu %zu %zu\n", P.part_o, P.part_lse, P.counters, P.total);
  }
}
"""


def test_the_first_bytes_of_every_layout_are_the_epoch_words(tmp_path):
    cxx = shutil.which("g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(B.nvcc())), "include")
    if not cxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "layout.cpp", tmp_path / "layout"
    src.write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", f"-I{B.CSRC}", f"-I{cuda}", f"-I{os.path.join(B.ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    r = random.Random(1)
    args = []
    for _ in range(40):
        hkv = r.choice([1, 2, 4, 5])
        args += [r.choice([1, 3, 64, 256, 5000]), r.choice([1, 4, 256, 16384]), hkv * r.choice([1, 8, 16]), hkv, r.choice([2, 148, 152])]
    lines = subprocess.run([str(exe), *map(str, args)], check=True, capture_output=True, text=True).stdout.splitlines()
    epoch, head = map(int, lines[0].split())
    assert epoch == 0 and head >= 8
    assert len(lines) == 1 + 2 * 40
    for line in lines[1:]:
        *parts, total = map(int, line.split())
        assert min(parts) >= head and all(p % 256 == 0 for p in parts) and parts == sorted(parts)
        assert total >= parts[-1]
