"""GPU tests of the tuning operators where their launches, workspaces and number
ranges have edges; bounds as in test_gpu_tuning.py."""
import numpy as np
import pytest

from test_gpu_tuning import TYPES, Head, Layer, dt

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


# ---------------------------------------------------------------- packed layer's gradient

@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, m, n, r", [(33, 2100, 1500, 64), (35, 8111, 1249, 147), (40, 4096, 600, 300),
                                        (48, 700, 5000, 33), (17, 3000, 900, 90), (65, 1500, 2100, 200),
                                        (300, 700, 1300, 150), (600, 515, 700, 70)])
def test_layer_gradient_in_a_workspace_of_nans(gpu, name, T, m, n, r):
    """Rows of digits past the last token are read but not used; sums and joins
    hold nothing that the call has not written."""
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} {m}x{n} r={r} {name}", flush=True)
    L = Layer(T + m, T, m, n, r, name, gpu)
    work = dirty(nq.binary_matmul_backward_work_bytes(T, m, n, r), gpu)
    L.check(*nq.binary_matmul_backward(*L.args(), work=work))
