"""GPU tests of the tuning operators where their launches, workspaces and number
ranges have edges; bounds as in test_gpu_tuning.py."""
import numpy as np
import pytest

from test_gpu_tuning import TYPES, Head, dt

pytestmark = pytest.mark.gpu


def dirty(nbytes, dev):
    """A workspace of just that size, every float in it a NaN."""
    import torch
    return torch.full((nbytes,), 255, dtype=torch.uint8, device=dev)


# ---------------------------------------------------------------- loss

@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", [(1024, 1600, 1280), (325, 16314, 384), (65, 30522, 1152),
                                     (12, 36223, 960), (40, 2100, 72), (3, 64, 130)])
def test_gradient_reads_nothing_that_it_did_not_write(gpu, name, T, V, d):
    """A workspace of NaNs; the vocabularies end so that the last slice of dH
    would start past them if it were cut from the words rounded up to 256."""
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    L = Head(T + V, T, V, d, name, gpu)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels,
                              work=dirty(nq.vocab_loss_work_bytes(T, V, d, dt(name)), gpu))
    L.check_loss(loss, lse)
    L.check_grad(*nq.vocab_loss_backward(
        L.H, L.W, L.labels, lse, L.dl,
        work=dirty(nq.vocab_loss_work_bytes(T, V, d, dt(name), True), gpu)))
