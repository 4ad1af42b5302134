"""The estimate of a packed batch's pieces that the choice of a kernel goes by, compiled from the
library's own header on the CPU."""
import os
import shutil
import subprocess
from fractions import Fraction

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "depth_aware_attention_b200", "csrc")
CUDA = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
SOURCE = r"""
#include <cstdio>
#include "moda_internal.h"
int main() {
  int hkv, t, nseq, unit;
  while (scanf("%d %d %d %d", &hkv, &t, &nseq, &unit) == 4) {
    moda::Problem p{1, hkv, hkv, t, 0, 64, 1, 1, 1.f};
    p.nseq = nseq;
    printf("%lld\n", moda::packed_pieces_estimate(p, unit));
  }
}
"""
# KV heads, tokens, sequences, tokens of a piece
CASES = [(64, 255, 1, 128), (64, 256, 1, 128), (64, 257, 1, 128), (1, 1, 1, 128), (48, 127, 3, 128),
         (4, 600, 3, 128), (4, 3000, 20, 128), (4, 6000, 10, 128), (4, 8000, 60, 128),
         (40, 95, 1, 32), (40, 95, 3, 32), (16, 37, 1000, 8), (65535, 1 << 14, 1 << 30, 128),
         (1, 1 << 30, 1 << 30, 1), (2, 5009, 37, 84)]


@pytest.fixture(scope="module")
def estimates(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA, "include", "cuda.h")):
        pytest.skip("no host compiler or CUDA headers")
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(SOURCE)
    subprocess.check_call([gxx, "-std=c++17", "-I", CSRC, "-I", os.path.join(CUDA, "include"),
                           str(d / "rules.cpp"), "-o", str(d / "rules")])
    out = subprocess.run([str(d / "rules")], input="\n".join("%d %d %d %d" % c for c in CASES),
                         capture_output=True, text=True, check=True).stdout
    return dict(zip(CASES, map(int, out.split())))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_pieces_estimate(case, estimates):
    hkv, tokens, nseq, unit = case
    if nseq == 1:
        want = hkv * -(-tokens // unit)
    else:  # half a piece for each sequence that can hold a token, rounded down once at the end
        want = int(hkv * (Fraction(tokens, unit) + Fraction(min(nseq, tokens), 2)))
    assert estimates[case] == want
