"""What the operators on single logits keep, on the CPU: the host-only header is
compiled by itself and its numbers held to what the kernels address."""
import random

import pytest

from test_tuning_plans import compile_plan, log_uniform


@pytest.fixture(scope="module")
def keep_plan(tmp_path_factory):
    return compile_plan(tmp_path_factory.mktemp("keep"), "vocab_plan.h", """
    const vocab::KeepPlan k = vocab::keep_plan(x[0], x[1], x[2], (int)x[3], x[4], x[5]);
    out = {k.few, k.tile, k.group, k.groups, k.block, k.first, k.step, k.lds, k.ldz, k.p.bytes, k.stat, k.z,
           k.slot, k.zslot, k.best, k.thr, k.bytes, k.tops};""")


def test_everything_kept_has_its_place(keep_plan):
    rng = random.Random(5)
    shapes = [(1, 1, 1, 1, 0, 1), (1, 1 << 24, 8, 1, 128, 128), (33, 1 << 24, 64, 1, 128, 128),
              (1 << 20, 1 << 18, 64, 1, 128, 128), (1 << 14, 1 << 24, 1 << 18, 0, 128, 128),
              (8193, 131072, 4096, 1, 128, 0), (256, 500, 64, 2, 1, 128)]
    shapes += [(log_uniform(rng, 1, 1 << 20), log_uniform(rng, 1, 1 << 18), log_uniform(rng, 1, 1 << 14),
                rng.randint(0, 2), rng.randint(0, 128), rng.randint(0, 128)) for _ in range(20000)]
    for (T, V, d, t, listed, top), got in zip(shapes, keep_plan(shapes)):
        few, tile, group, groups, block, first, step, lds, ldz, own, stat, z, slot, zslot, best, thr, total, tops = got
        assert few == (d >= 8 and T <= (64 if t == 0 else 32))
        assert group == (64 if few else tile // 2) and groups == -(-V // group) and group in (32, 64, 128)
        assert block == T or (block % 256 == 0 and block < T)
        assert lds >= groups and lds % 16 == 0
        # in order, without overlaps, aligned to whole groups of 16 bytes
        assert own <= stat and all(v % 256 == 0 for v in (stat, z, best, thr))
        assert (tops if top else z) - stat >= 16 * block * groups
        assert not top or (tops % 256 == 0 and z - tops >= 16 * block * groups)
        if few:
            assert ldz % 64 == 0 and ldz >= V and block == T
            assert best - z >= 4 * T * ldz
        else:
            if top:
                assert first % 256 == 0 and step % 256 == 0 and 0 < first <= step
                assert ldz == step and (slot if listed else best) - z >= 4 * block * ldz
                # (a step's last group is whole)
                assert step >= min(-(-V // 256) * 256, 8192)
            if listed:
                assert slot % 256 == 0 and zslot % 256 == 0
                assert zslot - slot >= block * lds and best - zslot >= 4 * block * listed * group
        assert thr - best >= 8 * block * top and total - thr >= 4 * block


def test_what_is_kept_does_not_grow_with_the_tokens(keep_plan):
    """Beside the operands and per-token words, 2^27 values of a kind (or those of 256
    tokens, the least)."""
    for V in (1000, 50021, 131072, 1 << 18):
        for t in (0, 1):
            for listed, top in ((128, 128), (1, 64), (128, 0)):
                few, *_, own, stat, z, slot, zslot, best, thr, total, _ = keep_plan([(1 << 20, V, 64, t, listed, top)])[0]
                assert total - stat <= 2.1 * 4 * (1 << 27) + 4 * (1 << 27) + (1 << 20) * 1100
