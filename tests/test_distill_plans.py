"""The workspace of a divergence's gradient, on the CPU: the host-only header is compiled by
itself, its places are held to what the kernels address, and the library's sizes to both. One
plan serves a call with the loss's logits and one that computes them again."""
import random

import pytest
import torch

import sub_bit_weight_lb_amd as nq
from test_tuning_plans import compile_plan, log_uniform

TYPES = (torch.float32, torch.bfloat16, torch.float16)
FIELDS = "few rows tp dp piece npieces nz kz hp wp G part products labels share wr val bytes".split()


@pytest.fixture(scope="module")
def distill_plan(tmp_path_factory):
    ask = compile_plan(tmp_path_factory.mktemp("distill"), "vocab_plan.h", """
    const vocab::Plan p = vocab::distill_plan(x[0], x[1], x[2], (int)x[3]);
    const vocab::SharePlan s = vocab::share_plan(x[0], x[1], x[2], (int)x[3], x[4]);
    out = {vocab::few(x[0], x[2], (int)x[3]), vocab::distill_rows(x[0], x[1], x[2], (int)x[3]), p.tp, p.dp, p.piece,
           p.npieces, p.nz, p.kz, p.hp, p.wp, p.G, p.part, p.bytes, s.labels, s.share, s.wr, s.val, s.bytes};""")
    return lambda rows: [dict(zip(FIELDS, got)) for got in ask(rows)]


def up(x, n):
    return -(-x // n) * n


# (tokens, words, columns) of which one row of G per token makes longer pieces of W than two rows, and
# so a larger copy of W and a larger G
LONGER = [(129, 151936, 320), (129, 262144, 256), (192, 256000, 256), (129, 131073, 64), (300, 131072, 8), (150, 131073, 72)]


def test_a_gradient_has_room_with_and_without_kept_logits(distill_plan):
    rng = random.Random(7)
    shapes = LONGER + [(T, V, d) for T in (33, 64, 65, 128, 129, 192, 193, 300, 1024, 8192)
                       for V in (40, 4999, 65536, 131072, 131073, 1 << 18, 1 << 20) for d in (1, 7, 8, 64, 256, 320, 515)]
    shapes += [(log_uniform(rng, 1, 8192), log_uniform(rng, 1, 1 << 20), log_uniform(rng, 1, 4096)) for _ in range(5000)]
    rows = [s + (t, 1 + i % 128) for i, s in enumerate(shapes) for t in range(3)]
    for (T, V, d, t, K), p in zip(rows, distill_plan(rows)):
        assert p["bytes"] == nq.vocab_distill_work_bytes(T, V, d, TYPES[t], K, True)
        assert p["share"] - p["labels"] >= 4 * T and p["wr"] - p["share"] >= 4 * T and p["val"] - p["wr"] >= 4 * T
        assert p["bytes"] - p["val"] >= 4 * T * K
        if p["few"]:
            continue
        terms, forms = (2, 2) if t == 0 else (1, 2 if t == 2 else 1)
        lines = p["rows"] * T                                  # of G and of dH's sums
        assert p["rows"] in (1, 2) and (p["rows"] == 1 or t)
        assert p["npieces"] * p["piece"] >= V and p["piece"] % 256 == 0
        # H's copies have each token's row as often as G; the products read whole tiles' rows of G as far
        # as it has any, kGrad writes those of a tile's tokens, kGradTwo and kept_kernel to the next 64
        assert p["tp"] >= up(lines, 64) and p["tp"] >= (up(T, 256) if p["rows"] == 1 else 0)
        assert p["wp"] - p["hp"] >= 2 * terms * forms * p["tp"] * p["dp"]
        assert p["G"] - p["wp"] >= 2 * terms * p["piece"] * p["dp"]
        assert p["part"] - p["G"] >= 2 * terms * p["tp"] * p["piece"]
        assert p["products"] - p["part"] >= 4 * p["nz"] * lines * up(d, 4)
        assert p["labels"] >= p["products"]
        assert all(p[f] % 256 == 0 for f in ("hp", "wp", "G", "part", "labels", "share", "wr", "val"))
