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


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T", [4, 70, 300])
def test_logits_that_their_scale_takes_past_fp32(gpu, T, sign):
    """Sums that are finite, and not after their scale: a vocabulary of one group, and one of several of
    which one is past the type's lowest value."""
    import torch
    import sub_bit_weight_lb_amd as nq
    for V, first in ((20, 0), (300, 0), (300, 256)):
        W = torch.zeros((V, 64), device=gpu)
        W[first:first + 128, 0] = sign * 2.0 ** 20
        W[0, 1] = 1.0
        Hh = torch.zeros((T, 64), device=gpu)
        Hh[0, 0] = 2.0 ** 20
        Hh[1, 1] = 2.0 ** -100
        Hh, W = Hh.bfloat16(), W.bfloat16()
        ids = torch.full((T, 2), V - 1, dtype=torch.int32, device=gpu)
        r = nq.vocab_logprobs(Hh, W, ids, 3, scale=2.0 ** 100)
        assert r.lse[0].isnan() and r.entropy[0].isnan() and r.logprobs[0].isnan().all()
        assert r.top_logprobs[0].isnan().all() and (r.top_ids[0] == -1).all()
        assert torch.isfinite(r.lse[1:]).all() and torch.isfinite(r.entropy[1:]).all() and (r.top_ids[1:] >= 0).all()
        for tail in (True, False):
            for keep in (True, False):
                logq = torch.full((T, 2), -2.0, device=gpu)
                loss, q = nq.vocab_distill(Hh, W, ids, logq, scale=2.0 ** 100, tail=tail, keep=keep)
                assert loss[0].isnan() and q.lse[0].isnan() and torch.isfinite(loss[1:]).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", [(5, 500, 72), (70, 500, 72), (300, 2049, 136), (1100, 3000, 40)])
def test_lists_of_more_than_all_mass(gpu, name, T, V, d):
    """Log probabilities whose sum is far above one, with a tail: there is no rest of them, and the gradient is
    the formula's, beside tokens whose lists are ordinary."""
    import torch
    L = Exact(T + 1, T, V, d, 9, name, gpu)
    L.logq[::2] += 5.0
    L.logq[1::4] += 0.5
    if T > 5:
        L.logq[7] += 11.0
    L.dl[5::7] *= 2.0 ** -6
    L.exact()
    loss, q = L.loss()
    L.check_loss(loss, q)
    for state in (q, L.loss(keep=False)[1]):
        L.check(*L.grad(state), 2)


def tied(V, T, gpu):
    """W and hidden states on a grid: rows whose logits are all equal, equal but for a few better ones at either
    end or all over, in two, three and nine values, rising and falling in long runs."""
    import torch
    W = torch.zeros((V, 64), device=gpu)
    v = torch.arange(V, device=gpu)
    W[:, 0] = (v % 2).float()
    W[:, 1] = (v % 3).float()
    W[:, 2] = (v * 7919 % 9).float()
    W[:, 3] = (v // 1024 % 128).float()
    W[:11, 4] = 1.0
    W[-11:, 5] = 1.0
    W[::997, 6] = 1.0
    W[V // 2:, 7] = 1.0
    Hh = torch.zeros((T, 64), device=gpu)
    for t in range(T):
        n = t % 17
        if n:
            Hh[t, (n - 1) // 2] = 1.0 if n % 2 else -1.0
    return Hh, W


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V", [(17, 131072), (40, 131072), (90, 50021), (600, 130001)])
def test_best_words_of_rows_with_many_equal_logits(gpu, name, T, V):
    import torch
    import sub_bit_weight_lb_amd as nq
    Hh, W = tied(V, T, gpu)
    z = Hh[:17].double() @ W.double().t()
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices
    for k in (1, 20, 128):
        r = nq.vocab_logprobs(Hh.to(dt(name)), W.to(dt(name)), k=k)
        for a in range(0, T, 17):
            assert torch.equal(r.top_ids[a:a + 17].long(), ids[:len(r.top_ids[a:a + 17]), :k])


def test_rows_of_padding_take_no_longer(gpu):
    """Hidden states of zeros, whose logits are all equal, against random ones: a few rounds of the search more,
    not one for every few hundred words (8 times the time allowed; 45 were taken)."""
    import torch
    import sub_bit_weight_lb_amd as nq
    g = torch.Generator(device=gpu).manual_seed(8)
    W = torch.randn((131072, 1024), generator=g, device=gpu).bfloat16()
    Hh = torch.randn((1, 1024), generator=g, device=gpu).bfloat16()

    def least(h):
        out = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(5):
                nq.vocab_logprobs(h, W, k=20)
            b.record()
            torch.cuda.synchronize()
            out.append(a.elapsed_time(b))
        return min(out)

    random = least(Hh)
    assert least(torch.zeros_like(Hh)) <= 8 * random
