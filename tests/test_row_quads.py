"""Which words of a row the samplers' kernels load, on CPU: the struct that says
so (csrc/sampling.cu, Quads), compiled for the host, over every small row. A word
past the row's end is dropped by the kernel, so no result could show one."""
import os
import re
import shutil
import subprocess

import pytest

import gemm_w4a16_group_gb300 as w4

SOURCE = os.path.join(os.path.dirname(os.path.abspath(w4.__file__)), "csrc", "sampling.cu")

MAIN = """
#include <algorithm>
#include <cstdint>
#include <cstdio>
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
%s
int main() {
  int bad = 0;
  for (int n = 1; n <= 200; ++n)
    for (int shift = 0; shift < 4; ++shift)
      for (int log2 = 0; log2 <= 8; ++log2) {
        int next = 0;
        for (uint32_t i = 0; i < 1u << log2; ++i) {
          const Quads q(n, shift, i, log2);
          for (int k = q.lo; k < q.hi; ++k, ++next) {  // every quad is in one part, and whole or one of its two ends
            const int at = 4 * k - shift;
            bad += k != next || q.is_whole(k) != (at >= 0 && at + 4 <= n);
            bad += (int)q.is_whole(k) + (q.end(0) == k) + (q.end(1) == k) != 1;
            bad += at + 4 <= 0 || at >= n;
          }
          for (int off = 0; off < 4; ++off) {
            auto in_word = [&](int k) { return k >= q.whole_lo && k < q.words_end(off); };
            for (int k = q.lo; q.lo < q.hi && k < q.hi + 2; ++k) {
              const int at = 4 * k - shift - off;  // the word's first element
              if (in_word(k) && (at + 4 <= 0 || at >= n)) {
                if (!bad++) std::printf("n %%d shift %%d off %%d part %%u of 2^%%d: word %%d at element %%d\\n", n, shift, off, i, log2, k, at);
              }
              if (q.is_whole(k)) bad += !in_word(k) || (off && !in_word(k + 1));
            }
          }
        }
        bad += next != (shift + n + 3) / 4;
      }
  return bad != 0;
}
"""


def test_words_of_a_row(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    with open(SOURCE) as f:
        text = f.read()
    quads = re.search(r"^struct Quads \{.*?^\};", text, re.M | re.S).group(0)
    source, program = tmp_path / "quads.cpp", tmp_path / "quads"
    source.write_text(MAIN % quads)
    subprocess.run([cxx, "-std=c++17", "-O1", "-o", str(program), str(source)], check=True)
    run = subprocess.run([str(program)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
