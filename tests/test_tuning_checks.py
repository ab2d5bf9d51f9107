"""Refusals of the tuning operators, on the CPU: by the binding (sizes, types
and strides that the C ABI cannot see; the library loader fails, so a check
that let a call through would show) and by the C ABI (status codes before any
device work, with pointers that are never read)."""
import ctypes as C
import os

import pytest
import torch

import sub_bit_weight_lb_amd as nq
from sub_bit_weight_lb_amd import _lib as L

I32, F32, U8, I8 = torch.int32, torch.float32, torch.uint8, torch.int8


@pytest.fixture
def no_library(monkeypatch):
    def boom():
        raise AssertionError("the library was called")
    monkeypatch.setattr(L, "load", boom)


def act8(rows, cols):
    return nq.Act8(torch.zeros((rows, cols), dtype=I8),
                   torch.zeros((rows, -(-cols // 32)), dtype=U8))


# ---------------------------------------------------------------- binding

@pytest.mark.parametrize("X, error", [
    (torch.zeros(5), ValueError),                                # not a matrix
    (torch.zeros((4, 6), dtype=torch.float64), TypeError),
    (torch.zeros((4, 6), dtype=I32), TypeError),
    (torch.zeros((4, 12))[:, ::2], ValueError),                  # column stride 2
    (torch.zeros((1, 6)).expand(4, 6), ValueError),              # rows overlap
    (torch.zeros((4, 6)), TypeError),                            # not on a GPU
])
def test_quantize_refuses(no_library, X, error):
    with pytest.raises(error):
        nq.act8_quantize(X)


@pytest.mark.parametrize("q", [
    act8(4, 65), act8(5, 64),
    nq.Act8(torch.zeros((4, 64), dtype=U8), torch.zeros((4, 2), dtype=U8)),
    nq.Act8(torch.zeros((4, 64), dtype=I8), torch.zeros((4, 3), dtype=U8)),
    nq.Act8(torch.zeros((4, 64), dtype=I8), torch.zeros((3, 2), dtype=U8)),
    nq.Act8(torch.zeros((4, 128), dtype=I8)[:, ::2], torch.zeros((4, 2), dtype=U8)),
    "not a checkpoint",
])
def test_quantize_refuses_buffers_of_another_shape(no_library, q):
    with pytest.raises((ValueError, TypeError)):
        nq.act8_quantize(torch.zeros((4, 64)), q)


def test_dequantize_refuses(no_library):
    q = act8(4, 64)
    for out in (torch.zeros((4, 63)), torch.zeros((3, 64)), torch.zeros((4, 128))[:, ::2]):
        with pytest.raises(ValueError):
            nq.act8_dequantize(q, out=out)
    with pytest.raises(TypeError):
        nq.act8_dequantize(q, dtype=torch.float64)
    with pytest.raises(TypeError):
        nq.act8_dequantize(q, out=torch.zeros((4, 64)), dtype=torch.float16)


def backward_args(m=40, n=70, r=33, T=3, dtype=F32):
    w = lambda k: (k + 31) // 32  # noqa: E731
    return dict(U_bits=torch.zeros((m, w(r)), dtype=I32), Ut_bits=torch.zeros((r, w(m)), dtype=I32),
                V_bits=torch.zeros((n, w(r)), dtype=I32), Vt_bits=torch.zeros((r, w(n)), dtype=I32),
                s1=torch.ones(m), s2=torch.ones(n), X=act8(T, n),
                dY=torch.zeros((T, m), dtype=dtype), r=r)


@pytest.mark.parametrize("change", [
    dict(U_bits=torch.zeros((40, 1), dtype=I32)),
    dict(Ut_bits=torch.zeros((33, 1), dtype=I32)),
    dict(Ut_bits=torch.zeros((32, 2), dtype=I32)),
    dict(V_bits=torch.zeros((69, 2), dtype=I32)),
    dict(Vt_bits=torch.zeros((33, 2), dtype=I32)),
    dict(Vt_bits=torch.zeros((33, 3), dtype=torch.int64)),
    dict(s1=torch.ones(39)), dict(s2=torch.ones(71)), dict(s2=torch.ones(70, dtype=torch.float64)),
    dict(X=act8(4, 70)), dict(X=act8(3, 71)), dict(X=torch.zeros((3, 70))),
    dict(dY=torch.zeros((3, 41))), dict(dY=torch.zeros((3, 40), dtype=torch.float64)),
    dict(dY=torch.zeros((3, 80))[:, ::2]),
    dict(dX=torch.zeros((3, 69))), dict(dX=torch.zeros((3, 70), dtype=torch.bfloat16)),
    dict(ds1=torch.zeros(39)), dict(ds2=torch.zeros(140)[::2]), dict(r=65),
])
def test_backward_refuses(no_library, change):
    a = backward_args()
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        nq.binary_matmul_backward(**a)


def test_backward_refuses_a_short_or_skewed_workspace():
    need = nq.binary_matmul_backward_work_bytes(3, 40, 70, 33)
    assert need > 0
    with pytest.raises(ValueError, match="work"):
        nq._workspace(torch.zeros(need - 1, dtype=U8), need, None)
    buf = torch.zeros(need + 32, dtype=U8)
    skew = buf[1:] if buf.data_ptr() % 16 == 0 else buf
    with pytest.raises(ValueError, match="aligned"):
        nq._workspace(skew, need, None)
    with pytest.raises(ValueError, match="contiguous"):
        nq._workspace(torch.zeros(2 * need, dtype=U8)[::2], need, None)


def loss_args(T=3, V=50, d=20, dtype=F32):
    return dict(H=torch.zeros((T, d), dtype=dtype), W=torch.zeros((V, d), dtype=dtype),
                labels=torch.zeros(T, dtype=I32))


@pytest.mark.parametrize("change", [
    dict(H=torch.zeros((3, 21))), dict(H=torch.zeros((3, 20), dtype=torch.float16)),
    dict(H=torch.zeros((3, 40))[:, ::2]), dict(W=torch.zeros((0, 20))),
    dict(H=torch.zeros((3, 20), dtype=torch.float64), W=torch.zeros((50, 20), dtype=torch.float64)),
    dict(labels=torch.zeros(3, dtype=torch.int64)), dict(labels=torch.zeros(4, dtype=I32)),
    dict(labels=torch.zeros(6, dtype=I32)[::2]),
])
def test_loss_refuses(no_library, change):
    a = loss_args()
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_loss(**a)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_loss_backward(**a, lse=torch.zeros(3), dloss=torch.zeros(3))


@pytest.mark.parametrize("change", [
    dict(lse=torch.zeros(4)), dict(dloss=torch.zeros(3, dtype=torch.float64)),
    dict(dH=torch.zeros((3, 21))), dict(dW=torch.zeros((50, 20), dtype=torch.bfloat16)),
    dict(dW=torch.zeros((49, 20))), dict(want_dH=False, want_dW=False),
])
def test_loss_backward_refuses(no_library, change):
    a = dict(loss_args(), lse=torch.zeros(3), dloss=torch.zeros(3))
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        nq.vocab_loss_backward(**a)


def test_loss_refuses_outputs_of_another_shape(no_library):
    for bad in (dict(loss=torch.zeros(2)), dict(lse=torch.zeros(3, dtype=torch.float64))):
        with pytest.raises((ValueError, TypeError)):
            nq.vocab_loss(**loss_args(), **bad)


def test_tensors_must_share_a_gpu():
    class Fake:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
    with pytest.raises(ValueError, match="c is on cuda:1"):
        nq._on_device("a b c", Fake(0), None, Fake(1))
    with pytest.raises(TypeError, match="b must be a CUDA"):
        nq._on_device("a b", None, torch.zeros(1))


# ---------------------------------------------------------------- C ABI

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.fail("libnq.so is not built; run __graft_entry__.build() first")
    return L.load()


PTR = C.c_void_p(4096)    # never read: every call below is refused first
BIG = 1 << 40


def quantize(lib, **k):
    a = dict(X=PTR, dtype=0, rows=4, cols=64, ldx=64, codes=PTR, ldc=64, exps=PTR, lde=2)
    a.update(k)
    return lib.nq_act8_quantize(*a.values(), None)


def dequantize(lib, **k):
    a = dict(codes=PTR, ldc=64, exps=PTR, lde=2, rows=4, cols=64, X=PTR, dtype=0, ldx=64)
    a.update(k)
    return lib.nq_act8_dequantize(*a.values(), None)


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=BIG),
                                 dict(X=None), dict(ldx=63), dict(codes=None), dict(exps=None),
                                 dict(ldc=63), dict(lde=1), dict(X=C.c_void_p(4098))])
def test_act8_status(lib, call, bad):
    assert call(lib, **bad) == L.NQ_ERR_INVALID_ARG
    assert lib.nq_last_error_message().decode()


def test_act8_empty_is_a_noop(lib):
    assert quantize(lib, rows=0, X=None, codes=None, exps=None) == L.NQ_OK
    assert dequantize(lib, cols=0, X=None) == L.NQ_OK
    assert lib.nq_act8_steps(None, 0, 0, 0, None, 0, None) == L.NQ_OK
    assert lib.nq_act8_steps(PTR, 1, 4, 2, PTR, 2, None) == L.NQ_ERR_INVALID_ARG
    assert lib.nq_act8_steps(None, 2, 4, 2, PTR, 2, None) == L.NQ_ERR_INVALID_ARG


def backward(lib, **k):
    a = dict(u=PTR, ldu=2, ut=PTR, ldut=2, v=PTR, ldv=2, vt=PTR, ldvt=3, m=40, n=70, r=33, s1=PTR,
             s2=PTR, codes=PTR, ldc=70, exps=PTR, lde=3, T=3, dY=PTR, dtype=0, lddy=40, dX=PTR,
             lddx=70, ds1=PTR, ds2=PTR, work=PTR)
    a.update(k)
    return lib.nq_binary_matmul_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(u=None), dict(ut=None), dict(v=None), dict(vt=None),
                                 dict(ldu=1), dict(ldut=1), dict(ldv=1), dict(ldvt=2), dict(m=0),
                                 dict(n=-1), dict(r=0), dict(m=BIG), dict(s1=None), dict(s2=None),
                                 dict(codes=None), dict(exps=None), dict(ldc=69), dict(lde=2),
                                 dict(T=-1), dict(T=BIG), dict(dY=None), dict(dtype=7),
                                 dict(lddy=39), dict(lddx=69), dict(ds1=None), dict(ds2=None),
                                 dict(work=None), dict(work=C.c_void_p(4104)),
                                 dict(dY=C.c_void_p(4097))])
def test_backward_status(lib, bad):
    assert backward(lib, **bad) == L.NQ_ERR_INVALID_ARG


def test_backward_workspace(lib):
    f = lib.nq_binary_matmul_backward_work_bytes
    assert f(-1, 4, 4, 4) == f(1, BIG, 4, 4) == -1
    assert f(0, 4, 4, 4) == 0
    assert f(1, 4096, 4096, 2048) < f(64, 4096, 4096, 2048) < f(8192, 4096, 4096, 2048) < 1 << 30


def test_backward_refuses_more_values_than_a_launch_covers(lib):
    f = lib.nq_binary_matmul_backward_work_bytes
    for T, m, n, r in [((1 << 24) + 1, 1, 1, 1), (1 << 20, 65537, 8, 8), (1 << 20, 8, 65537, 8),
                       (1 << 20, 8, 8, 65537)]:
        assert f(T, m, n, r) == -1
        assert backward(lib, T=T, m=m, n=n, r=r, ldu=4096, ldut=4096, ldv=4096, ldvt=4096,
                        ldc=n, lde=4096, lddy=m, lddx=n) == L.NQ_ERR_INVALID_ARG
    assert f(1 << 20, 65536, 4096, 512) > 0


def vloss(lib, **k):
    a = dict(H=PTR, ldh=20, W=PTR, ldw=20, dtype=0, T=3, V=50, d=20, labels=PTR, scale=1.0,
             loss=PTR, lse=PTR, work=PTR)
    a.update(k)
    return lib.nq_vocab_loss(*a.values(), None)


def vback(lib, **k):
    a = dict(H=PTR, ldh=20, W=PTR, ldw=20, dtype=0, T=3, V=50, d=20, labels=PTR, scale=1.0,
             lse=PTR, dloss=PTR, dH=PTR, lddh=20, dW=PTR, lddw=20, work=PTR)
    a.update(k)
    return lib.nq_vocab_loss_backward(*a.values(), None)


@pytest.mark.parametrize("call", [vloss, vback])
@pytest.mark.parametrize("bad", [dict(H=None), dict(W=None), dict(labels=None), dict(work=None),
                                 dict(lse=None), dict(ldh=19), dict(ldw=19), dict(dtype=3),
                                 dict(T=-1), dict(T=(1 << 20) + 1), dict(V=0), dict(V=BIG),
                                 dict(d=0), dict(d=(1 << 18) + 1, ldh=1 << 19, ldw=1 << 19),
                                 dict(ldw=BIG), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(H=C.c_void_p(4098)),
                                 dict(work=C.c_void_p(4104))])
def test_vocab_status(lib, call, bad):
    assert call(lib, **bad) == L.NQ_ERR_INVALID_ARG


def test_vocab_backward_status(lib):
    for bad in (dict(dloss=None), dict(dH=None, dW=None), dict(lddh=19), dict(lddw=19),
                dict(dW=C.c_void_p(4098)), dict(T=0)):
        assert vback(lib, **bad) == L.NQ_ERR_INVALID_ARG
    assert vback(lib, T=0, dW=None) == L.NQ_OK
    assert vloss(lib, T=0, H=None, loss=None) == L.NQ_OK


def test_vocab_workspace(lib):
    f = lib.nq_vocab_loss_work_bytes
    assert f(1, 0, 4, 0, 0) == f(1, 4, 4, 9, 0) == f(-1, 4, 4, 0, 0) == -1
    assert f(0, 4, 4, 0, 1) == 0
    # the logits of 4096 tokens and 131072 words would be 2 GiB in fp32
    assert f(4096, 131072, 4096, 1, 0) < 1 << 31
    for dt in (0, 1, 2):
        for grad in (0, 1):
            assert f(300, 5000, 515, dt, grad) > 0


def test_loss_refuses_more_logits_than_a_launch_covers(lib):
    for call in (vloss, vback):
        assert call(lib, T=1 << 20, V=(1 << 18) + 1) == L.NQ_ERR_INVALID_ARG
    for grad in (0, 1):
        assert lib.nq_vocab_loss_work_bytes(1 << 20, (1 << 18) + 1, 8, 1, grad) == -1
        assert lib.nq_vocab_loss_work_bytes(1 << 20, 1 << 18, 8, 1, grad) > 0


def test_ste_step_from_a_checkpoint_status(lib):
    assert lib.nq_ste_step_act8(None, PTR, 64, PTR, 2, PTR, 64, None, 4, 1e-4,
                                None) == L.NQ_ERR_INVALID_ARG
