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
    out = {p.piece, p.npieces, p.nz, p.kz, p.part, p.bytes, p.tp, p.dp, p.wp, p.G};""")


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
    for (T, V, d, t), (piece, npieces, nz, kz, part, total, *_) in zip(rows, vocab_plan(rows)):
        assert piece % 256 == 0 and (npieces - 1) * piece < V <= npieces * piece
        assert kz % 64 == 0 and nz >= 1
        share = [-(-(-(-min(piece, V - v0) // 64) * 64) // kz) for v0 in range(0, V, piece)]
        assert share[0] == nz, (T, V, d, t)
        assert max(share) == nz
        each = 2 if t and d >= 8 and T <= 32 else 1     # of sums per token: G's terms, 16-bit types
        assert total - part >= 4 * nz * T * each * (-(-d // 4) * 4)


def test_pieces_of_the_vocabulary_bound_the_workspace(vocab_plan):
    """G and the copy of W's piece, as they lie there (tokens and columns rounded
    up), hold at most 2^26 values each per term, but for pieces of 2048 words,
    the least; tokens are rounded up to the products' 256 rows, or 64 where
    score_kernel writes G."""
    rng = random.Random(3)
    shapes = [(1, 1 << 24, 64), (1, 1 << 24, 1), (1, 1 << 24, 8), (64, 1 << 24, 64), (65, 1 << 24, 64),
              (1, 1 << 24, 1 << 18), (1 << 14, 1 << 24, 64)]
    shapes += [(log_uniform(rng, 1, 1 << 20), log_uniform(rng, 1, 1 << 18), log_uniform(rng, 1, 1 << 18))
               for _ in range(5000)]
    rows = [s + (t,) for s in shapes for t in range(3)]
    for (T, V, d, t), (piece, _, _, _, part, _, tp, dp, wp, G) in zip(rows, vocab_plan(rows)):
        terms = 2 if t == 0 else 1
        few = d >= 8 and T <= (64 if t == 0 else 32)
        assert tp == -(-T // (64 if few else 256)) * (64 if few else 256) and dp == -(-d // 64) * 64
        assert piece <= max(2048, (1 << 26) // max(tp, dp))
        assert G - wp >= 2 * terms * piece * dp and part - G >= 2 * terms * piece * tp


def test_the_workspace_of_one_token_is_not_that_of_many():
    """Documented sizes: one token and a vocabulary of 2^24 words."""
    import sub_bit_weight_lb_amd as nq
    import torch
    for d in (1, 8, 64):
        got = nq.vocab_loss_work_bytes(1, 1 << 24, d, torch.float32, True)
        # two terms of 2 bytes for 2^26 values of G and of W; the rest is small
        assert got <= 2 * 4 * (1 << 26) + (1 << 24), (d, got)


# ---------------------------------------------------------------- packed layer's gradient

@pytest.fixture(scope="module")
def layer_plan(tmp_path_factory):
    return compile_plan(tmp_path_factory.mktemp("layer"), "binback_plan.h", """
    using namespace binback;
    const Plan p = plan_for(x[0], x[1], x[2], x[3]);
    out = {p.planes[0], p.steps[0], p.planes[1], p.steps[1], p.bytes, thin_tiles(x[3]),
           kThinMax, kDigit, 16 * row_tiles(kProj), 16 * row_tiles(kGrad)};""")


def test_the_digit_planes_cover_what_the_products_read(layer_plan):
    """A thin launch reads the digits of all 16-row tiles of its kernel, a wide
    one those of all rows of its workgroups' two wave rows, whatever T is: both
    must lie inside the chain's planes, in front of its steps. Blocks of 2048
    bytes a digit hold 16 rows and 128 columns, whole groups of four blocks a
    row; the first products have four digits of the chain's columns, the second
    three of the rank's."""
    rng = random.Random(2)
    shapes = [(11008, 4096, 1536), (28672, 8192, 512), (28672, 8192, 64), (8111, 1249, 147),
              (65, 300, 129), (1, 1, 1)]
    shapes += [tuple(log_uniform(rng, 1, 30000) for _ in range(3)) for _ in range(60)]
    rows = [s + (T,) for s in shapes for T in list(range(1, 130)) + [500, 513, 8191]]
    for (m, n, r, T), v in zip(rows, layer_plan(rows)):
        at, end, total, tiles, thin_max, digit = (v[0], v[2]), (v[1], v[3]), v[4], v[5], v[6], v[7]
        for c, K in enumerate((n, m)):
            for nd, cols, wave_rows in ((4, K, v[8]), (3, r, v[9])):
                group = -(-cols // 512) * 4 * nd * digit      # bytes of 16 rows
                if T <= thin_max:
                    groups = tiles
                else:
                    groups = -(-T // (2 * wave_rows)) * 2 * wave_rows // 16
                assert 16 * groups >= T
                assert at[c] + groups * group <= end[c] <= total, (m, n, r, T)


# ---------------------------------------------------------------- inline assembly

def test_assembly_names_the_registers_that_it_writes():
    """Each scalar register that a block of assembly names as a destination is
    among its clobbers, m0 and the carry of a scalar add too."""
    import re
    blocks = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".hip", ".h")):
            continue
        text = open(os.path.join(CSRC, name)).read()
        for block in re.findall(r"asm\s+volatile\s*\((.*?)\);", text, re.S):
            code = "".join(re.findall(r'"([^"]*)"', block)).replace("\\n", " ").replace("\\t", " ")
            writes = set(re.findall(r"\bs_(?:mov|add|sub|or|and|lsh[lr])\w*\s+(m0|s\d+)\b", code))
            if re.search(r"\bs_(?:add|sub|or|and|lsh[lr])\w*\s", code):
                writes.add("scc")
            named = set(re.findall(r'"(m0|s\d+|scc)"', block))
            assert writes <= named, (name, writes - named)
            blocks += bool(writes)
    assert blocks >= 2
