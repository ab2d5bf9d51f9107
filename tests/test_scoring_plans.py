"""What the operators on single logits keep, on the CPU: the host-only header is
compiled by itself and its numbers held to what the kernels address."""
import random

import pytest

from test_tuning_plans import compile_plan, log_uniform


FIELDS = ("few tile group groups block first step marked lds ldz own piece zs ws stat tops z slot marks places zl best thr "
          "bytes").split()


@pytest.fixture(scope="module")
def keep_plan(tmp_path_factory):
    ask = compile_plan(tmp_path_factory.mktemp("keep"), "vocab_plan.h", """
    const vocab::KeepPlan k = vocab::keep_plan(x[0], x[1], x[2], (int)x[3], x[4], x[5]);
    out = {k.few, k.tile, k.group, k.groups, k.block, k.first, k.step, k.marked, k.lds, k.ldz, k.p.bytes, k.p.piece, k.zs,
           k.ws, k.stat,
           k.tops, k.z, k.slot, k.marks, k.places, k.zl, k.best, k.thr, k.bytes};""")
    return lambda rows: [dict(zip(FIELDS, got)) for got in ask(rows)]


def test_everything_kept_has_its_place(keep_plan):
    rng = random.Random(5)
    shapes = [(1, 1, 1, 1, 0, 1), (1, 1 << 24, 8, 1, 128, 128), (33, 1 << 24, 64, 1, 128, 128),
              (1 << 20, 1 << 18, 64, 1, 128, 128), (1 << 14, 1 << 24, 1 << 18, 0, 128, 128),
              (8193, 131072, 4096, 1, 128, 0), (256, 500, 64, 2, 1, 128), (5, 1 << 24, 64, 1, 128, 0)]
    shapes += [(log_uniform(rng, 1, 1 << 20), log_uniform(rng, 1, 1 << 18), log_uniform(rng, 1, 1 << 14),
                rng.randint(0, 2), rng.randint(0, 128), rng.randint(0, 128)) for _ in range(20000)]
    for (T, V, d, t, listed, top), k in zip(shapes, keep_plan(shapes)):
        few, group, block = k["few"], k["group"], k["block"]
        assert few == (d >= 8 and T <= (64 if t == 0 else 32))
        assert group == (64 if few else k["tile"] // 2) and k["groups"] == -(-V // group) and group in (32, 64, 128)
        assert block == T or (block % 256 == 0 and block < T)
        assert k["marked"] == (listed > 0 and not few)
        assert k["lds"] >= k["groups"] and k["lds"] % 16 == 0
        if few:
            assert block == T and k["ldz"] % 64 == 0 and k["ldz"] >= V
        elif top:
            # (a step's last group is whole; its parts come in fours)
            whole = -(-V // 256) * 256
            assert k["first"] % 256 == 0 and k["step"] % 256 == 0 and 0 < k["first"] <= k["step"] == k["ldz"] <= whole
            assert k["first"] >= min(whole, 2 * top * group)
        # what is kept, in order and without overlaps
        need = [("own", None)]
        if t == 0 and not few:
            need += [("zs", 4 * T), ("ws", 4 * k["piece"])]
            assert k["piece"] % 256 == 0
        need.append(("stat", 16 * block * k["groups"]))
        if top:
            need.append(("tops", 16 * block * k["groups"]))
        need.append(("z", 4 * block * k["ldz"]))
        if k["marked"]:
            need += [("slot", block * k["lds"]), ("marks", 32 * block * listed), ("places", block * listed),
                     ("zl", 4 * block * listed)]
        need += [("best", 8 * block * top), ("thr", 4 * block), ("bytes", 0)]
        for (a, size), (b, _) in zip(need, need[1:]):
            assert k[b] % 256 == 0 or b == "bytes"
            assert size is None and k[a] <= k[b] or size is not None and k[b] - k[a] >= size


def test_what_is_kept_does_not_grow_with_the_tokens(keep_plan):
    """Beside the operands and per-token words, 2^27 values of a kind (or those of 256
    tokens, the least)."""
    for V in (1000, 50021, 131072, 1 << 18):
        for t in (0, 1):
            for listed, top in ((128, 128), (1, 64), (128, 0)):
                k = keep_plan([(1 << 20, V, 64, t, listed, top)])[0]
                assert k["bytes"] - k["stat"] <= 4.1 * 4 * (1 << 27) + (1 << 20) * 1100
