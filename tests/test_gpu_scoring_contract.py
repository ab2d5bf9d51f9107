"""What the declarations of the scoring operators say of values that are not finite, of words past the
vocabulary and of lists of more than all mass, on both sides of the sizes where the kernels change."""
import numpy as np
import pytest

from test_gpu_distill_exact import Exact, dt, half

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [4, 32, 70, 300])
def test_a_word_past_the_vocabulary_is_one_whatever_its_mass(gpu, name, T, tail):
    """Lists padded with the vocabulary's size and no mass: NaN in the loss as in the gradient."""
    import torch
    L = Exact(3, T, 300, 64, 6, name, gpu, tail=tail)
    L.ids[:, :2] = torch.arange(T, device=gpu)[:, None].int() % 300
    ok, _ = L.loss()
    L.ids[1, 4], L.logq[1, 4] = 300, -float("inf")
    L.ids[2, 5], L.logq[2, 5] = 2 ** 31 - 1, -float("inf")
    loss, q = L.loss()
    rest = [t for t in range(T) if t not in (1, 2)]
    assert loss[1:3].isnan().all() and torch.equal(loss[rest], ok[rest])
    assert torch.isfinite(q.lse).all() and q.hit[1, 4].isnan() and q.hit[2, 5].isnan()
    dH, dW = L.grad(q)
    assert dH[1:3].isnan().all() and torch.isfinite(dH[rest]).all() and dW.isnan().all()


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("mass", [True, False])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [1, 4, 32, 33, 70, 300])
def test_a_listed_logit_of_minus_infinity(gpu, name, T, mass, tail):
    """An infinity in the row of W of a word that the tokens list, alone or with all words of its group:
    NaN in loss and lse, whether the teacher has any mass there."""
    L = Exact(4, T, 300, 64, 128, name, gpu, tail=tail)
    L.ids[:] = -1
    L.ids[:, 7] = 5                                                     # alone
    for t in range(0, T, 2):
        L.ids[t, 100:102] = L.ids[t, 7].new_tensor([5, 150])            # twice, and with another
    if T > 2:
        import torch
        L.ids[2] = torch.arange(128, device=gpu).int()                  # all of its group, of any size
    L.logq[:] = -20.0
    L.logq[:, ::3] = -5.0
    if not mass:
        L.logq[L.ids == 5] = -float("inf")
        if T > 2:
            L.logq[2] = -float("inf")
            L.logq[2, 100] = -1.0
    L.H[:, 3] = 0.5
    L.W[5, 3] = -float("inf")
    loss, q = L.loss()
    hit = q.hit[:, 7][L.ids[:, 7] == 5]
    if name == "float32":     # (of its operands' terms one is 0, and 0 times infinity NaN)
        assert hit.isnan().all()
    else:
        assert (hit == -float("inf")).all()
    assert q.lse.isnan().all() and loss.isnan().all()
    dH, dW = L.grad(q)
    assert dH.isnan().all() and dW.isnan().all()
