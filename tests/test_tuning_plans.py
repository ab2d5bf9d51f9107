"""Workspace layouts and launch plans of the tuning operators, on the CPU: the
host-only headers are compiled by themselves and their numbers held to what
the kernels address."""
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sub_bit_weight_lb_amd", "csrc")


def compile_plan(folder, header, body):
    """A program that includes `header` and, for each line of integers it is
    given, runs `body` on x[0], x[1], .. and prints what that puts into `out`."""
    src, exe = folder / "plan.cpp", folder / "plan"
    src.write_text(f"""
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>
#include "{header}"
int main() {{
  using namespace nq;
  std::string line;
  while (std::getline(std::cin, line)) {{
    std::istringstream in(line);
    std::vector<long long> x, out;
    for (long long v; in >> v;) x.push_back(v);
    {body}
    for (long long v : out) printf("%lld ", v);
    printf("\\n");
  }}
}}
""")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)])

    def ask(rows):
        text = "".join(" ".join(str(int(v)) for v in r) + "\n" for r in rows)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [[int(v) for v in line.split()] for line in out.splitlines()]
    return ask


def log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(np.exp(rng.uniform(np.log(lo), np.log(hi + 1))))))


# ---------------------------------------------------------------- loss over a vocabulary

@pytest.fixture(scope="module")
def vocab_plan(tmp_path_factory):
    return compile_plan(tmp_path_factory.mktemp("vocab"), "vocab_plan.h", """
    const vocab::Plan p = vocab::plan_for(x[0], x[1], x[2], (int)x[3], true);
    out = {p.piece, p.npieces, p.nz, p.kz, p.part, p.bytes};""")


# (tokens, words, columns) whose last slice of dH, in a vocabulary rounded up to
# 256 words, would start past the words that there are
SHORT = [(1024, 1600, 1280), (1024, 2049, 1024), (1024, 2100, 1024), (65, 30522, 1152),
         (300, 30522, 384), (256, 28996, 896), (12, 36223, 960), (325, 16314, 384), (1232, 1821, 973)]


def test_the_first_piece_writes_every_slice_of_dh(vocab_plan):
    """dH joins nz slices: each must have a share of the first piece, whose
    products write it; later pieces may leave slices out, never have more."""
    rng = random.Random(1)
    shapes = SHORT + [(log_uniform(rng, 1, 8192), log_uniform(rng, 1, 1 << 18), log_uniform(rng, 1, 16384))
                      for _ in range(20000)]
    rows = [s + (t,) for s in shapes for t in range(3)]
    for (T, V, d, t), (piece, npieces, nz, kz, part, total) in zip(rows, vocab_plan(rows)):
        assert piece % 256 == 0 and (npieces - 1) * piece < V <= npieces * piece
        assert kz % 64 == 0 and nz >= 1
        share = [-(-(-(-min(piece, V - v0) // 64) * 64) // kz) for v0 in range(0, V, piece)]
        assert share[0] == nz, (T, V, d, t)
        assert max(share) == nz
        assert total - part >= 4 * nz * T * (-(-d // 4) * 4)
