"""Refusals of the scoring and distilling operators, on the CPU: by the binding
(the library loader fails, so a check that let a call through would show) and
by the C ABI (status codes before any device work, with pointers that are never
read)."""
import ctypes as C
import os

import pytest
import torch

import sub_bit_weight_lb_amd as nq
from sub_bit_weight_lb_amd import _lib as L

I32, F32 = torch.int32, torch.float32


@pytest.fixture
def no_library(monkeypatch):
    def boom():
        raise AssertionError("the library was called")
    monkeypatch.setattr(L, "load", boom)


# ---------------------------------------------------------------- binding

def head(T=3, V=50, d=20):
    return dict(H=torch.zeros((T, d)), W=torch.zeros((V, d)))


HEADS = [
    dict(H=torch.zeros(20)), dict(H=torch.zeros((3, 20), dtype=torch.float64)),
    dict(H=torch.zeros((3, 21))), dict(H=torch.zeros((3, 40))[:, ::2]),
    dict(W=torch.zeros((50, 20), dtype=torch.bfloat16)), dict(W=torch.zeros((0, 20))),
    dict(W=torch.zeros((1, 20)).expand(50, 20)), dict(H=torch.zeros((3, 0)), W=torch.zeros((50, 0))),
    dict(H=[[0.0] * 20] * 3),
]


@pytest.mark.parametrize("change", HEADS + [
    dict(k=-1), dict(k=129), dict(k=51), dict(W=torch.zeros((4, 20)), k=5),
    dict(tokens=torch.zeros(4, dtype=I32)), dict(tokens=torch.zeros(3, dtype=torch.int64)),
    dict(tokens=torch.zeros((4, 2), dtype=I32)), dict(tokens=torch.zeros((3, 129), dtype=I32)),
    dict(tokens=torch.zeros((3, 4), dtype=I32)[:, ::2]), dict(tokens=torch.zeros((3, 2))),
    dict(tokens=torch.zeros((3, 2, 1), dtype=I32)), dict(tokens=[1, 2, 3]),
    dict(out=(1, 2)), dict(),                                   # (not on a GPU)
])
def test_logprobs_refuses(no_library, change):
    a = dict(head(), tokens=torch.zeros(3, dtype=I32), k=2)
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_logprobs(**a)


@pytest.mark.parametrize("change", [
    dict(logprobs=torch.zeros(4)), dict(logprobs=None), dict(entropy=torch.zeros(3, dtype=I32)),
    dict(lse=torch.zeros(6)[::2]), dict(top_ids=torch.zeros((3, 2))),
    dict(top_ids=torch.zeros((3, 3), dtype=I32)), dict(top_logprobs=torch.zeros((3, 4))[:, ::2]),
])
def test_logprobs_refuses_outputs_of_another_shape(no_library, change):
    out = dict(logprobs=torch.zeros(3), entropy=torch.zeros(3), lse=torch.zeros(3),
               top_ids=torch.zeros((3, 2), dtype=I32), top_logprobs=torch.zeros((3, 2)))
    out.update(change)
    with pytest.raises(ValueError if "top_ids" not in change else (ValueError, TypeError)) if \
            "entropy" not in change else pytest.raises(TypeError):
        nq.vocab_logprobs(**head(), tokens=torch.zeros(3, dtype=I32), k=2, out=nq.VocabLogprobs(**out))


def distill_args(T=3, K=4):
    return dict(head(T), ids=torch.zeros((T, K), dtype=I32), logq=torch.zeros((T, K)))


def state(T=3, K=4, **change):
    a = dict(lse=torch.zeros(T), rest=torch.zeros(T), hit=torch.zeros((T, K)))
    a.update(change)
    return nq.VocabDistill(**a)


@pytest.mark.parametrize("change", HEADS + [
    dict(ids=torch.zeros(3, dtype=I32)), dict(ids=torch.zeros((3, 4), dtype=torch.int64)),
    dict(ids=torch.zeros((2, 4), dtype=I32)), dict(ids=torch.zeros((3, 8), dtype=I32)[:, ::2]),
    dict(ids=torch.zeros((3, 0), dtype=I32), logq=torch.zeros((3, 0))),
    dict(ids=torch.zeros((3, 129), dtype=I32), logq=torch.zeros((3, 129))),
    dict(logq=torch.zeros((3, 5))), dict(logq=torch.zeros((3, 4), dtype=torch.float64)),
    dict(logq=torch.zeros((1, 4)).expand(3, 4)), dict(),
])
def test_distill_refuses(no_library, change):
    a = dict(distill_args())
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_distill(**a)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_distill_backward(**a, state=state(), dloss=torch.zeros(3))


@pytest.mark.parametrize("change", [
    dict(state=None), dict(state=state(lse=torch.zeros(4))), dict(state=state(hit=torch.zeros((3, 5)))),
    dict(state=state(rest=torch.zeros(3, dtype=torch.float64))), dict(dloss=torch.zeros(2)),
    dict(state=state(logits=torch.zeros((3, 50)))), dict(state=state(logits=torch.zeros(385)[1:])),
    dict(dloss=torch.zeros(3, dtype=torch.bfloat16)), dict(dH=torch.zeros((3, 21))),
    dict(dW=torch.zeros((50, 20), dtype=torch.float16)), dict(want_dH=False, want_dW=False),
])
def test_distill_backward_refuses(no_library, change):
    a = dict(distill_args(), state=state(), dloss=torch.zeros(3))
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_distill_backward(**a)


def test_distill_refuses_outputs_of_another_shape(no_library):
    for bad in (dict(loss=torch.zeros(2)), dict(state=state(rest=torch.zeros(2))), dict(state=(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            nq.vocab_distill(**distill_args(), **bad)


# ---------------------------------------------------------------- C ABI

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.fail("libnq.so is not built; run __graft_entry__.build() first")
    return L.load()


PTR = C.c_void_p(4096)    # never read: every call below is refused first
ODD = C.c_void_p(4098)
BIG = 1 << 40


def logprobs(lib, **k):
    a = dict(H=PTR, ldh=20, W=PTR, ldw=20, dtype=0, T=3, V=50, d=20, tokens=PTR, ldt=2, G=2, k=4,
             scale=1.0, logprobs=PTR, entropy=PTR, lse=PTR, top_ids=PTR, top_logprobs=PTR, work=PTR)
    a.update(k)
    return lib.nq_vocab_logprobs(*a.values(), None)


def distill(lib, **k):
    a = dict(H=PTR, ldh=20, W=PTR, ldw=20, dtype=0, T=3, V=50, d=20, ids=PTR, ldi=4, logq=PTR, ldq=4,
             K=4, scale=1.0, tail=1, loss=PTR, lse=PTR, rest=PTR, hit=PTR, logits=None, work=PTR)
    a.update(k)
    return lib.nq_vocab_distill(*a.values(), None)


def backward(lib, **k):
    a = dict(H=PTR, ldh=20, W=PTR, ldw=20, dtype=0, T=3, V=50, d=20, ids=PTR, ldi=4, logq=PTR, ldq=4,
             K=4, scale=1.0, tail=1, lse=PTR, rest=PTR, hit=PTR, logits=None, dloss=PTR, dH=PTR,
             lddh=20, dW=PTR, lddw=20, work=PTR)
    a.update(k)
    return lib.nq_vocab_distill_backward(*a.values(), None)


@pytest.mark.parametrize("call", [logprobs, distill, backward])
@pytest.mark.parametrize("bad", [dict(H=None), dict(W=None), dict(work=None), dict(ldh=19),
                                 dict(ldw=19), dict(dtype=3), dict(T=-1), dict(T=(1 << 20) + 1),
                                 dict(V=0), dict(V=BIG), dict(d=0), dict(ldw=BIG),
                                 dict(d=(1 << 18) + 1, ldh=1 << 19, ldw=1 << 19),
                                 dict(T=1 << 20, V=(1 << 18) + 1), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(H=ODD), dict(work=C.c_void_p(4104)),
                                 dict(lse=None), dict(lse=ODD)])
def test_head_status(lib, call, bad):
    assert call(lib, **bad) == L.NQ_ERR_INVALID_ARG
    assert lib.nq_last_error_message().decode()


@pytest.mark.parametrize("bad", [dict(G=-1), dict(G=129, ldt=129), dict(ldt=1), dict(ldt=BIG),
                                 dict(k=-1), dict(k=129, V=500), dict(k=51), dict(tokens=None),
                                 dict(logprobs=None), dict(entropy=None), dict(top_ids=None),
                                 dict(top_logprobs=None), dict(tokens=ODD), dict(top_ids=ODD)])
def test_logprobs_status(lib, bad):
    assert logprobs(lib, **bad) == L.NQ_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [distill, backward])
@pytest.mark.parametrize("bad", [dict(ids=None), dict(logq=None), dict(K=0), dict(K=129, ldi=129, ldq=129),
                                 dict(ldi=3), dict(ldq=3), dict(ldi=BIG), dict(ids=ODD), dict(logq=ODD),
                                 dict(rest=None), dict(hit=None), dict(hit=ODD),
                                 dict(logits=C.c_void_p(4104))])
def test_distill_status(lib, call, bad):
    assert call(lib, **bad) == L.NQ_ERR_INVALID_ARG


def test_distill_backward_status(lib):
    for bad in (dict(dloss=None), dict(dH=None, dW=None), dict(lddh=19), dict(lddw=19), dict(dW=ODD),
                dict(dloss=ODD), dict(T=0)):
        assert backward(lib, **bad) == L.NQ_ERR_INVALID_ARG
    assert distill(lib, loss=None) == L.NQ_ERR_INVALID_ARG


def test_no_tokens_is_a_noop(lib):
    assert logprobs(lib, T=0, H=None, lse=None) == L.NQ_OK
    assert distill(lib, T=0, H=None, ids=None) == L.NQ_OK
    assert backward(lib, T=0, dW=None) == L.NQ_OK


def test_workspaces(lib):
    f, g = lib.nq_vocab_logprobs_work_bytes, lib.nq_vocab_distill_work_bytes
    assert f(1, 0, 4, 0, 1, 0) == f(1, 4, 4, 9, 1, 1) == f(1, 4, 4, 0, 129, 1) == f(1, 4, 4, 0, 1, 5) == -1
    assert f(1, 4, 4, 0, -1, 0) == f(-1, 4, 4, 0, 1, 1) == f(1 << 20, (1 << 18) + 1, 8, 1, 1, 1) == -1
    assert g(1, 4, 4, 0, 0, 0) == g(1, 4, 4, 0, 129, 0) == g(1, 4, 4, 3, 1, 1) == -1
    assert f(0, 4, 4, 0, 1, 1) == g(0, 4, 4, 0, 1, 0) == 0
    for dt in (0, 1, 2):
        assert f(300, 5000, 515, dt, 4, 20) > 0 and g(300, 5000, 515, dt, 20, 0) > 0
        # the loss's own gradient is a part of it
        assert g(300, 5000, 515, dt, 20, 1) > lib.nq_vocab_loss_work_bytes(300, 5000, 515, dt, 1)
    # logits that are kept
    h = lib.nq_vocab_distill_logits
    assert h(3, 50, 20, 0) == 3 * 128 and h(64, 1000, 8, 0) == 64 * 1024 and h(32, 1000, 8, 1) == 32 * 1024
    assert h(8192, 131072, 4096, 1) == 1 << 30 and h(8193, 131072, 4096, 1) == 0
    assert h(4096, 131072, 1000, 1) == 0 and h(4096, 131072, 1000, 0) == 1 << 29
    assert h(128, 1000, 8, 2) == 128 * 1024 and h(3, 1000, 7, 1) == 3 * 1024
    assert h(65, 1000, 8, 0) == h(8192, 131072, 8, 2) == h(3, 1000, 7, 0) == h(0, 5, 8, 0) == 0
    assert h(1, 0, 8, 0) == h(1, 5, 8, 3) == -1
    # of any number of tokens and words: three kinds of 2^27 values, beside the operands' copies
    for T, V in ((1 << 20, 1 << 18), (1 << 14, 1 << 24), (8192, 131072)):
        own = f(T, V, 64, 1, 128, 128)
        assert own < 3 * 4 * (1 << 27) * 1.3 + 2 * 64 * (1 << 20) + 2 * (1 << 26) + (1 << 28), (T, V, own)
