"""GPU parity of the operators that tune a packed model against the float64
oracle (oracle/tuning.py), each difference held to a bound worked out from the
roundings that the operator documents.

With u = 2^-24 (half a unit of fp32) and h(t) half a unit of the output type
(torch.finfo(t).eps / 2: fp32 u, bf16 2^-8, fp16 2^-11):

checkpoint   nothing rounds but the codes: equal to the oracle.
layer        a and s1 dy: two fp32 roundings each at most (2 u), then fixed
             point, 2^-31 of the row's largest; sums of digits are exact and
             joined by ND - 1 fp32 multiply-adds and a conversion each (ND = 4,
             then 3), whose roundings are u of the partial results, at most
             |p| plus the lower digits' sums, K 2^-8 max|a| together; p, dp:
             fixed point, 2^-23 of the row's largest. So with A = sum_c |a_c|
             over a row: |dp| <= 2 u A + K 2^-31 max|a| + 8 u (|p| + K 2^-7
             max|a|), |dq| <= sum_k |dp_k| + r 2^-23 max|p| + 6 u (|q| + r 2^-7
             max|p|). dx adds u and h(t);
             ds1, ds2 sum at most 24 rounded fp32 terms in a row before fp64
             takes over (16 in a lane, 4 lanes, 2 halves, the product).
loss         z: an fp32 sum of d exact products, (d + 2) u sum |h_k w_k|, for
             fp32 operands (two fp16 terms: a value to 2^-24 of itself or
             2^-39 of the largest, the product of the second terms left out,
             2^-24) 2^-22 more of it and d 2^-38 of the largest product; exp and
             log within 4 units; sums of V positive terms V u. G is rounded
             once, h(t); dH and dW sum V and T rounded terms in fp32.
"""
import numpy as np
import pytest

from oracle import tuning as O
from oracle.lbadmm import pack_signs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ["float32", "bfloat16", "float16"]


def dt(name):
    import torch
    return getattr(torch, name)


def H(t):
    return t.detach().double().cpu().numpy()


def half(name):
    import torch
    return torch.finfo(dt(name)).eps / 2


def least(name):
    """The spacing of subnormals of a type: what rounds to nothing."""
    import torch
    return 2.0 ** -149 if name == "float32" else 2.0 ** -133 if name == "bfloat16" else 2.0 ** -24


def put(x, dev, name="float32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev).to(dt(name))


def strided(t, extra, lead=0):
    """t with `extra` columns after each row and `lead` elements before the
    first, so that rows are not aligned to 16 bytes."""
    import torch
    buf = torch.full((t.shape[0] * (t.shape[1] + extra) + lead,), 77, dtype=t.dtype, device=t.device)
    v = buf[lead:].view(t.shape[0], t.shape[1] + extra)[:, :t.shape[1]]
    v.copy_(t)
    return v


def activations(rng, rows, cols):
    mag = np.exp(0.6 * rng.standard_normal(cols))
    mag[rng.random(cols) < 0.01] *= 100.0
    return rng.standard_normal((rows, cols)) * mag


# ---------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows, cols", [(1, 1), (3, 31), (4, 32), (5, 33), (2, 47), (7, 1000),
                                        (64, 4096), (130, 8193), (1, 28672), (0, 5), (5, 0)])
def test_checkpoint_equals_oracle(gpu, name, rows, cols):
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case {rows}x{cols} {name}", flush=True)
    rng = np.random.default_rng(rows * 7 + cols)
    X = put(activations(rng, rows, cols) if cols else np.zeros((rows, 0)), gpu, name)
    want_c, want_e = O.act8_quantize(H(X), 9 if name == "float16" else 121)
    q = nq.act8_quantize(X)
    assert np.array_equal(q.codes.cpu().numpy(), want_c)
    assert np.array_equal(q.exps.cpu().numpy(), want_e)
    got = nq.act8_dequantize(q)
    assert got.dtype == X.dtype
    assert np.array_equal(H(got), O.act8_values(want_c, want_e))
    assert np.array_equal(H(nq.act8_dequantize(q, dtype=torch.float32)), O.act8_values(want_c, want_e))
    assert np.array_equal(H(nq.act8_steps(q)), O.act8_steps(want_e))


@pytest.mark.parametrize("name", TYPES)
def test_checkpoint_of_hard_values(gpu, name):
    import torch
    import sub_bit_weight_lb_amd as nq
    f = torch.finfo(dt(name))
    rows = []
    # zeros of both signs, the least and largest values, ties, one code over a
    # border, values that are not finite, groups of one column
    for lead in (0.0, -0.0, f.tiny, f.smallest_normal / 2, f.max, -f.max, 127.0, 127.5, 1.9921875,
                 float("nan"), float("inf"), -float("inf")):
        r = torch.zeros(65)
        r[0], r[1], r[2], r[40], r[64] = lead, 0.5, 62.5, 1.0, lead
        rows.append(r)
    X = torch.stack(rows).to(gpu).to(dt(name))
    want_c, want_e = O.act8_quantize(H(X), 9 if name == "float16" else 121)
    q = nq.act8_quantize(X)
    assert np.array_equal(q.exps.cpu().numpy(), want_e)
    assert np.array_equal(q.codes.cpu().numpy(), want_c)
    got = H(nq.act8_dequantize(q))
    assert np.array_equal(got, O.act8_values(want_c, want_e), equal_nan=True)
    finite = np.isfinite(O.act8_values(want_c, want_e))
    assert np.isfinite(got[finite]).all()


@pytest.mark.parametrize("name", TYPES)
def test_checkpoint_of_values_past_the_last_level_cache(gpu, name):
    """Above 256 MB of values the accesses change; nothing else does."""
    import torch
    import sub_bit_weight_lb_amd as nq
    rows, cols = 9001, 7501 if name == "float32" else 15001
    X = torch.randn(rows, cols, device=gpu).mul_(3).to(dt(name))
    assert X.numel() * X.element_size() > 256 << 20
    q = nq.act8_quantize(X)
    got = nq.act8_dequantize(q)
    for r in (slice(0, 4500), slice(4500, rows)):
        part = nq.act8_quantize(X[r])
        assert torch.equal(part.codes, q.codes[r]) and torch.equal(part.exps, q.exps[r])
        assert torch.equal(nq.act8_dequantize(part), got[r])


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("cols, extra, lead", [(33, 5, 1), (64, 1, 3), (1000, 7, 1), (4096, 9, 0)])
def test_checkpoint_of_views_writes_nothing_else(gpu, name, cols, extra, lead):
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case {cols}+{extra} lead {lead} {name}", flush=True)
    rng = np.random.default_rng(cols)
    X = strided(put(activations(rng, 9, cols), gpu, name), extra, lead)
    cb = torch.full((9, cols + 3), 99, dtype=torch.int8, device=gpu)
    eb = torch.full((9, -(-cols // 32) + 2), 99, dtype=torch.uint8, device=gpu)
    q = nq.act8_quantize(X, nq.Act8(cb[:, 1:1 + cols], eb[:, 1:-1]))
    want_c, want_e = O.act8_quantize(H(X), 9 if name == "float16" else 121)
    assert np.array_equal(q.codes.cpu().numpy(), want_c) and np.array_equal(q.exps.cpu().numpy(), want_e)
    assert (cb[:, 0] == 99).all() and (cb[:, 1 + cols:] == 99).all()
    assert (eb[:, 0] == 99).all() and (eb[:, -1] == 99).all()
    out = strided(torch.zeros_like(X), extra, lead)
    nq.act8_dequantize(q, out=out)
    assert np.array_equal(H(out), O.act8_values(want_c, want_e))
    if extra:
        gap = out.as_strided((9, extra), (cols + extra, 1), lead + cols)[:-1]
        assert (gap == 77).all()


# ---------------------------------------------------------------- packed layer's gradient

class Layer:
    def __init__(self, seed, T, m, n, r, name, dev):
        import torch
        rng = np.random.default_rng(seed)
        self.SU, self.SV = (np.where(rng.random(s) < 0.5, 1.0, -1.0) for s in ((m, r), (n, r)))
        bits = lambda S: torch.from_numpy(pack_signs(S).astype(np.uint32).view(np.int32)).to(dev)  # noqa: E731
        self.U, self.Ut, self.V, self.Vt = (bits(S) for S in (self.SU, self.SU.T, self.SV, self.SV.T))
        self.s1 = put(rng.uniform(0.005, 0.03, m), dev)
        self.s2 = put(rng.uniform(0.005, 0.03, n), dev)
        c, e = O.act8_quantize(activations(rng, T, n))
        import sub_bit_weight_lb_amd as nq
        self.q = nq.Act8(torch.from_numpy(c).to(dev), torch.from_numpy(e).to(dev))
        self.x = O.act8_values(c, e)
        self.dY = put(activations(rng, T, m) * 1e-2, dev, name)
        self.name, self.r = name, r

    def args(self):
        return (self.U, self.Ut, self.V, self.Vt, self.s1, self.s2, self.q, self.dY, self.r)

    def check(self, dX, ds1, ds2):
        s1, s2, dy, x = H(self.s1), H(self.s2), H(self.dY), self.x
        r, h = self.r, half(self.name)
        want = O.layer_backward(self.SU, self.SV, s1, s2, x, dy)

        def chain(a, S, S2):
            """(values, bounds) of the product a S S2^T"""
            p = a @ S
            K, big = a.shape[1], np.abs(a).max(1)
            ep = (2 * U * np.abs(a).sum(1) + K * 2.0 ** -31 * big)[:, None]
            ep = ep + 8 * U * (np.abs(p) + (K * 2.0 ** -7 * big)[:, None])
            q, big = p @ S2.T, (np.abs(p) + ep).max(1)
            eq = (ep.sum(1) + r * 2.0 ** -23 * big)[:, None]
            eq = eq + 6 * U * (np.abs(q) + (r * 2.0 ** -7 * big)[:, None])
            return q, eq

        q, eq = chain(x * s2, self.SV, self.SU)
        da, eda = chain(dy * s1, self.SU, self.SV)
        near = lambda got, ref, tol, what: np.testing.assert_array_less(  # noqa: E731
            np.abs(H(got) - ref), 1.01 * tol + 1e-300, err_msg=what)
        if dX is not None:
            near(dX, want[0], s2 * eda + (U + h) * np.abs(want[0]) + least(self.name), "dX")
        near(ds1, want[1], (np.abs(dy) * eq).sum(0) + 24 * U * (np.abs(dy * q)).sum(0), "ds1")
        near(ds2, want[2], (np.abs(x) * eda).sum(0) + 24 * U * (np.abs(da * x)).sum(0), "ds2")


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, m, n, r", [
    (1, 1, 1, 1), (1, 40, 70, 33), (3, 129, 31, 128), (16, 200, 257, 96), (17, 33, 64, 5),
    (32, 130, 130, 130), (33, 65, 300, 129), (64, 512, 256, 64), (65, 100, 90, 40),
    (128, 127, 129, 33), (129, 257, 100, 160), (300, 513, 640, 200), (700, 96, 1100, 257)])
def test_backward_matches_oracle(gpu, name, T, m, n, r):
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} {m}x{n} r={r} {name}", flush=True)
    L = Layer(T + m, T, m, n, r, name, gpu)
    got = nq.binary_matmul_backward(*L.args())
    L.check(*got)
    again = nq.binary_matmul_backward(*L.args())
    assert all((a == b).all() for a, b in zip(got, again))


def test_backward_of_a_long_layer(gpu):
    """Few row tiles and many columns: the first products are split over the
    columns."""
    import sub_bit_weight_lb_amd as nq
    L = Layer(5, 70, 6000, 9000, 70, "float32", gpu)
    L.check(*nq.binary_matmul_backward(*L.args()))


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("name", TYPES)
def test_backward_of_views_writes_nothing_else(gpu, name, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} {name}", flush=True)
    m, n, r = 77, 101, 45
    L = Layer(9, T, m, n, r, name, gpu)
    wide = lambda t: strided(t, 3, 1)  # noqa: E731
    L.U, L.Ut, L.V, L.Vt = (wide(t) for t in (L.U, L.Ut, L.V, L.Vt))
    # set bits past a row's columns meet zero digits
    for t, cols in ((L.U, r), (L.Ut, m), (L.V, r), (L.Vt, n)):
        t[:, -1] |= ~((1 << (cols % 32)) - 1)
    L.q = nq.Act8(wide(L.q.codes), wide(L.q.exps))
    L.dY = wide(L.dY)
    dX = wide(torch.zeros((T, n), dtype=dt(name), device=gpu))
    got = nq.binary_matmul_backward(*L.args(), dX=dX)
    L.check(*got)
    gap = dX.as_strided((T, 3), (n + 3, 1), 1 + n)[:-1]
    assert (gap == 77).all()
    none, ds1, ds2 = nq.binary_matmul_backward(*L.args(), want_dX=False)
    assert none is None and (ds1 == got[1]).all() and (ds2 == got[2]).all()


@pytest.mark.parametrize("T", [6, 150])
def test_backward_rows_that_are_not_finite(gpu, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Layer(11, T, 70, 90, 40, "float32", gpu)
    clean = nq.binary_matmul_backward(*L.args())
    L.dY[2, 3] = float("inf")
    L.q.exps[4, 1] = 255
    dX, ds1, ds2 = nq.binary_matmul_backward(*L.args())
    assert dX[2].isnan().all()
    rest = [t for t in range(T) if t != 2]
    assert (dX[rest] == clean[0][rest]).all()
    assert ds1.isnan().all() and ds2.isnan().all()
    L.dY[2] = 0     # a zero row and an all-zero checkpoint row are ordinary
    L.q.exps[4] = 1
    L.q.codes[4] = 0
    assert all(torch.isfinite(t).all() for t in nq.binary_matmul_backward(*L.args()))


def test_backward_of_no_tokens(gpu):
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Layer(1, 2, 33, 40, 8, "bfloat16", gpu)
    q = nq.Act8(L.q.codes[:0], L.q.exps[:0])
    dX, ds1, ds2 = nq.binary_matmul_backward(*L.args()[:6], q, L.dY[:0], 8,
                                             ds1=torch.ones(33, device=gpu))
    assert dX.shape == (0, 40) and (ds1 == 0).all() and (ds2 == 0).all()


# ---------------------------------------------------------------- loss

class Head:
    def __init__(self, seed, T, V, d, name, dev, scale=1.0, ignored=0.2):
        import torch
        rng = np.random.default_rng(seed)
        self.H = put(rng.standard_normal((T, d)), dev, name)
        self.W = put(rng.standard_normal((V, d)) * 1.5 / np.sqrt(d), dev, name)
        lab = rng.integers(0, V, T)
        lab[rng.random(T) < ignored] = -100
        self.labels = torch.from_numpy(lab.astype(np.int32)).to(dev)
        dl = rng.standard_normal(T)
        self.dl = put(dl, dev)
        self.name, self.scale = name, scale

    def zbound(self):
        Hh, W = np.abs(H(self.H)), np.abs(H(self.W))
        Hh[self.labels.cpu().numpy() < 0] = 0
        d, fp32 = Hh.shape[1], self.name == "float32"
        tiny = d * 2.0 ** -38 * Hh.max() * W.max() if fp32 else 0.0
        return abs(self.scale) * (((d + 2) * U + (2.0 ** -22 if fp32 else 0.0)) * (Hh @ W.T) + tiny)

    def check_loss(self, loss, lse):
        V = self.W.shape[0]
        lab = self.labels.cpu().numpy()
        Hh = H(self.H)
        Hh[lab < 0] = 0
        want, want_lse = O.vocab_loss(Hh, H(self.W), lab, self.scale)
        ez = self.zbound().max(1)
        tol = 1.01 * (ez + (V + 8) * U + 4 * U * np.abs(want_lse)) * (lab >= 0)
        np.testing.assert_array_less(np.abs(H(lse) - want_lse), tol + 1e-300)
        np.testing.assert_array_less(np.abs(H(loss) - want), 2 * tol + 1e-300)

    def check_grad(self, dH, dW):
        T, V = self.H.shape[0], self.W.shape[0]
        lab, h = self.labels.cpu().numpy(), half(self.name)
        Hh, W, dl = H(self.H), H(self.W), H(self.dl)
        Hh[lab < 0] = 0
        use = lab >= 0
        wantH, wantW, G = O.vocab_loss_backward(Hh, W, lab, dl, self.scale)
        ez = self.zbound()[use]
        p = np.exp(self.scale * Hh[use] @ W.T - O.vocab_loss(Hh, W, lab, self.scale)[1][use][:, None])
        # of p: its exponent is off by z's and lse's bounds and its own
        # rounding, exp by 4 units; then the subtraction, dloss / max and
        # the rounding of G, which for fp16 is kept in 2^15 steps
        ee = ez + ez.max(1, keepdims=True) + (V + 16) * U + 16 * U * np.abs(np.log(np.maximum(p, 1e-30)))
        big = np.abs(dl[use]).max() if use.any() else 0.0
        eg = (p * (np.expm1(ee) + 8 * U)) * np.abs(dl[use])[:, None] * abs(self.scale)
        eg += (h + 4 * U) * np.abs(G)
        if self.name != "bfloat16":
            # (fp16's subnormals; fp32's second term, and the terms left out)
            eg += 2.0 ** -25 / 2 ** 15 * big * abs(self.scale)
        sumH = (np.abs(G) + eg) @ np.abs(W)
        sumW = (np.abs(G) + eg).T @ np.abs(Hh[use])
        tH = eg @ np.abs(W) + ((V + 40) * U + (2.0 ** -22 if self.name == "float32" else 0)) * sumH
        tW = eg.T @ np.abs(Hh[use]) + ((T + 40) * U + (2.0 ** -22 if self.name == "float32" else 0)) * sumW
        if self.name == "float32":   # operands to 2^-39 of the largest, V or T of them
            tH += V * 2.0 ** -38 * (np.abs(G).max() if G.size else 0.0) * np.abs(W).max()
            tW += T * 2.0 ** -38 * (np.abs(G).max() if G.size else 0.0) * np.abs(Hh).max()
        if dH is not None:
            np.testing.assert_array_less(np.abs(H(dH)[use] - wantH[use]),
                                         1.01 * tH + h * np.abs(wantH[use]) + least(self.name))
            assert (H(dH)[~use] == 0).all()
        if dW is not None:
            np.testing.assert_array_less(np.abs(H(dW) - wantW),
                                         1.01 * tW + h * np.abs(wantW) + least(self.name))


CASES = [(1, 1, 1), (1, 2, 7), (2, 63, 64), (16, 64, 130), (17, 65, 8), (33, 257, 515),
         (64, 1000, 96), (65, 500, 72), (300, 1000, 64), (257, 2049, 200), (513, 300, 129)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", CASES)
def test_loss_and_gradient_match_oracle(gpu, name, T, V, d):
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    L = Head(T + V + d, T, V, d, name, gpu)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    L.check_loss(loss, lse)
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    L.check_grad(dH, dW)
    l2, s2 = nq.vocab_loss(L.H, L.W, L.labels)
    h2, w2 = nq.vocab_loss_backward(L.H, L.W, L.labels, s2, L.dl)
    assert (l2 == loss).all() and (h2 == dH).all() and (w2 == dW).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", [(600, 4100, 200), (600, 4100, 1100), (1100, 12100, 1100),
                                     (700, 10300, 2000),
                                     (70, 4100, 2052), (2, 3, 4)])
def test_loss_and_gradient_in_tiles_of_every_size(gpu, name, T, V, d):
    """128 x 128 tiles with few and with many k, 256 x 256 tiles in every
    product, 64 x 64 tiles with many k, fewer columns than a load takes."""
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    L = Head(T + V + d, T, V, d, name, gpu)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    L.check_loss(loss, lse)
    L.check_grad(*nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, d", [(15, 200), (16, 72), (31, 136), (32, 1000), (33, 129), (48, 64),
                                  (63, 40), (64, 515)])
def test_loss_of_few_tokens(gpu, name, T, d):
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} d={d} {name}", flush=True)
    L = Head(T + d, T, 1500 + T, d, name, gpu)
    L.check_loss(*nq.vocab_loss(L.H, L.W, L.labels))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [9, 40, 140])
def test_loss_of_views_and_a_temperature(gpu, name, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} {name}", flush=True)
    V, d = 301, 77
    L = Head(3, T, V, d, name, gpu, scale=0.4)
    L.H, L.W = strided(L.H, 5, 1), strided(L.W, 2, 3)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels, scale=0.4)
    L.check_loss(loss, lse)
    dH, dW = strided(torch.zeros_like(L.H), 3, 1), strided(torch.zeros_like(L.W), 1, 1)
    nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl, scale=0.4, dH=dH, dW=dW)
    L.check_grad(dH, dW)
    for t, extra in ((dH, 3), (dW, 1)):
        gap = t.as_strided((t.shape[0], extra), (d + extra, 1), 1 + d)[:-1]
        assert (gap == 77).all()
    # one of the two alone is the same
    a, none = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl, scale=0.4, want_dW=False)
    assert none is None and (a == dH).all()
    none, b = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl, scale=0.4, want_dH=False)
    assert none is None and (b == dW).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [8, 130])
def test_ignored_tokens_may_hold_anything(gpu, name, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Head(4, T, 200, 72, name, gpu, ignored=0.5)
    off = L.labels < 0
    assert off.any() and not off.all()
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    grads = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    L.H[off] = float("nan")
    L.dl[off] = float("inf")
    bad_lse = torch.where(off, torch.full_like(lse, float("nan")), lse)
    l2, s2 = nq.vocab_loss(L.H, L.W, L.labels)
    g2 = nq.vocab_loss_backward(L.H, L.W, L.labels, bad_lse, L.dl)
    assert (l2 == loss).all() and (s2 == lse).all() and (l2[off] == 0).all()
    assert all((a == b).all() for a, b in zip(grads, g2))
    # all of them ignored
    L.labels.fill_(-1)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    assert (loss == 0).all() and (lse == 0).all() and (dH == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("T", [8, 130])
def test_labels_past_the_vocabulary_and_rows_that_are_not_finite(gpu, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Head(6, T, 200, 64, "bfloat16", gpu, ignored=0.0)
    ok, _ = nq.vocab_loss(L.H, L.W, L.labels)
    L.labels[1] = 200
    L.H[3, 5] = float("inf")
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    rest = [t for t in range(T) if t not in (1, 3)]
    assert loss[1].isnan() and torch.isfinite(lse[1]) and loss[3].isnan()
    assert (loss[rest] == ok[rest]).all()
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    assert dH[1].isnan().all() and dH[3].isnan().all() and dW.isnan().all()
    assert torch.isfinite(dH[rest]).all()


@pytest.mark.parametrize("name", TYPES)
def test_upstream_gradients_of_any_size(gpu, name):
    """dloss of zero, of a mean over very many tokens, and of mixed sizes."""
    import sub_bit_weight_lb_amd as nq
    L = Head(8, 70, 400, 64, name, gpu)
    _, lse = nq.vocab_loss(L.H, L.W, L.labels)
    keep = L.dl.clone()
    for f in (0.0, 2.0 ** -20, 1e3):
        L.dl = keep * f
        dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
        L.check_grad(dH, dW)
    L.dl = keep.clone()
    L.dl[::2] *= 1e-4
    L.check_grad(*nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl))


def test_extreme_logits(gpu):
    """Logits in the hundreds: nothing overflows, a token that is certain of
    its label has loss 0."""
    import torch
    import sub_bit_weight_lb_amd as nq
    W = torch.eye(64, device=gpu).repeat(5, 1)[:300].contiguous().to(torch.bfloat16)
    Hh = torch.zeros((70, 64), device=gpu, dtype=torch.bfloat16)
    Hh[:, 0], Hh[:, 1] = 500.0, -500.0
    labels = torch.zeros(70, dtype=torch.int32, device=gpu)
    labels[1] = 1
    for T in (70, 4):
        loss, lse = nq.vocab_loss(Hh[:T], W, labels[:T])
        # words 0, 64, .. 256 share the largest logit
        assert abs(float(lse[0]) - (500.0 + np.log(5))) < 1e-3
        assert abs(float(loss[0]) - np.log(5)) < 1e-3 and abs(float(loss[1]) - 1000.0 - np.log(5)) < 1e-3
        dH, dW = nq.vocab_loss_backward(Hh[:T], W, labels[:T], lse, torch.ones(T, device=gpu))
        assert torch.isfinite(dH).all() and torch.isfinite(dW).all()


def test_several_pieces_of_the_vocabulary(gpu):
    """A hidden size so large that the vocabulary is taken in pieces of 2048
    words, the last one short; against a float64 product on the GPU."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d = 20, 5000, 33000
    g = torch.Generator(device=gpu).manual_seed(1)
    Hh = torch.randn((T, d), generator=g, device=gpu).bfloat16()
    W = (torch.randn((V, d), generator=g, device=gpu) * (1.5 / d ** 0.5)).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device=gpu, dtype=torch.int32)
    labels[3] = -1
    dl = torch.randn(T, generator=g, device=gpu)
    loss, lse = nq.vocab_loss(Hh, W, labels)
    dH, dW = nq.vocab_loss_backward(Hh, W, labels, lse, dl)
    H64, W64 = Hh.double(), W.double()
    z = torch.mm(H64, W64.t())
    use = labels >= 0
    ref = torch.logsumexp(z, 1)
    zb = (d + 2) * U * torch.mm(H64.abs(), W64.abs().t()).max()
    assert ((lse.double() - ref).abs()[use] <= zb + (V + 64) * U).all()
    G = torch.softmax(z, 1)
    G[torch.arange(T, device=gpu), labels.long().clamp(min=0)] -= 1
    G *= (dl.double() * use).unsqueeze(1)
    # relative to the sums of magnitudes: G's rounding (2^-8), the exponent's
    # bound, fp32 sums over V or T terms; then the output's rounding
    rel = 2.0 ** -8 + float(torch.expm1(2 * zb + (V + 64) * U)) + (V + 64) * U
    for got, ref, mag in ((dH, torch.mm(G, W64), torch.mm(G.abs(), W64.abs())),
                          (dW, torch.mm(G.t(), H64), torch.mm(G.abs().t(), H64.abs()))):
        assert ((got.double() - ref).abs() <= rel * mag + 2.0 ** -8 * ref.abs() + 1e-30).all()


# ---------------------------------------------------------------- together

def test_scale_gradients_of_a_packed_model(gpu):
    """Forward through a packed layer, the loss over its outputs, and back to
    the layer's scales from an 8-bit checkpoint: against the float64 formulas,
    and those against central differences along a random direction."""
    import torch
    import sub_bit_weight_lb_amd as nq
    rng = np.random.default_rng(12)
    T, n, m, r, V = 90, 96, 128, 64, 500
    L = Layer(13, T, m, n, r, "float32", gpu)
    W = put(rng.standard_normal((V, m)) / np.sqrt(m), gpu)
    labels = torch.from_numpy(rng.integers(-20, V, T).astype(np.int32)).to(gpu)
    s1 = L.s1 * 4
    used = labels >= 0
    dl = used.float() / used.sum()
    X = put(activations(rng, T, n), gpu)
    q = nq.act8_quantize(X)
    x = nq.act8_dequantize(q)
    Y = nq.binary_matmul(L.U, L.Vt, s1, L.s2, x, r)
    loss, lse = nq.vocab_loss(Y, W, labels)
    dY, dW = nq.vocab_loss_backward(Y, W, labels, lse, dl)
    dX, ds1, ds2 = nq.binary_matmul_backward(L.U, L.Ut, L.V, L.Vt, s1, L.s2, q, dY, r)

    lab = labels.cpu().numpy()
    x64, W64, dl64 = H(x), H(W), H(dl)

    def forward(a1, a2, xx):
        y = a1 * (((xx * a2) @ L.SV) @ L.SU.T)
        return y, (dl64 * O.vocab_loss(y, W64, lab)[0]).sum()

    a1, a2 = H(s1), H(L.s2)
    y, total = forward(a1, a2, x64)
    dy = O.vocab_loss_backward(y, W64, lab, dl64)[0]
    want = O.layer_backward(L.SU, L.SV, a1, a2, x64, dy)
    assert abs(float((dl * loss).sum()) - total) <= 1e-5 * abs(total)
    for got, ref in zip((dX, ds1, ds2), want):
        # each step is within 1e-5 of its norm (fp32 throughout); they chain
        assert np.linalg.norm(H(got) - ref) <= 1e-4 * np.linalg.norm(ref)
    v = [rng.standard_normal(t.shape) for t in (x64, a1, a2)]
    h = 1e-6
    up = forward(a1 + h * v[1], a2 + h * v[2], x64 + h * v[0])[1]
    dn = forward(a1 - h * v[1], a2 - h * v[2], x64 - h * v[0])[1]
    slope = sum((g * d).sum() for g, d in zip((want[0], want[1], want[2]), v))
    assert abs((up - dn) / (2 * h) - slope) <= 1e-4 * (1 + abs(slope))


def test_captured_passes_replay(gpu):
    """A checkpoint, the loss and both gradients captured into a graph: every
    replay equals the eager result on the same inputs, with eager work between
    the replays; a second graph that shares the workspace runs after it."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, m, n, r, V = 150, 128, 160, 64, 700
    L = Layer(21, T, m, n, r, "bfloat16", gpu)
    Hd = Head(22, T, V, m, "bfloat16", gpu)
    X = put(activations(np.random.default_rng(1), T, n), gpu, "bfloat16")
    work = torch.empty(max(nq.binary_matmul_backward_work_bytes(T, m, n, r),
                           nq.vocab_loss_work_bytes(T, V, m, torch.bfloat16, True)),
                       dtype=torch.uint8, device=gpu)

    def run():
        q = nq.act8_quantize(X)
        loss, lse = nq.vocab_loss(Hd.H, Hd.W, Hd.labels, work=work)
        dH, dW = nq.vocab_loss_backward(Hd.H, Hd.W, Hd.labels, lse, Hd.dl, work=work)
        return (nq.act8_dequantize(q), loss, dH, dW) + nq.binary_matmul_backward(
            L.U, L.Ut, L.V, L.Vt, L.s1, L.s2, q, dH, r, work=work)

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for k in range(3):
        gen = torch.Generator(device=gpu).manual_seed(k)
        X.copy_(torch.randn(X.shape, generator=gen, device=gpu))
        Hd.H.copy_(torch.randn(Hd.H.shape, generator=gen, device=gpu))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for out in outs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_calls_on_two_streams_at_once(gpu):
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Layer(31, 200, 256, 320, 96, "float32", gpu)
    Hd = Head(32, 200, 900, 128, "float16", gpu)
    X = put(activations(np.random.default_rng(2), 200, 320), gpu)
    want = (nq.act8_quantize(X).codes, *nq.vocab_loss(Hd.H, Hd.W, Hd.labels),
            *nq.binary_matmul_backward(*L.args()))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((nq.act8_quantize(X).codes, *nq.vocab_loss(Hd.H, Hd.W, Hd.labels),
                            *nq.binary_matmul_backward(*L.args())))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_what_a_call_allocates_belongs_to_the_stream_it_is_given(gpu):
    """Calls on a stream passed by its handle, while the current stream takes
    and fills memory of the sizes that the calls have just let go."""
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Layer(33, 300, 384, 320, 96, "float32", gpu)
    Hd = Head(34, 300, 5000, 256, "float32", gpu)

    def run(**kw):
        loss, lse = nq.vocab_loss(Hd.H, Hd.W, Hd.labels, **kw)
        return (loss, *nq.vocab_loss_backward(Hd.H, Hd.W, Hd.labels, lse, Hd.dl, **kw),
                *nq.binary_matmul_backward(*L.args(), **kw),
                nq.act8_dequantize(nq.act8_quantize(Hd.W, **kw), **kw))

    want = run()
    sizes = [nq.vocab_loss_work_bytes(300, 5000, 256, torch.float32, g) for g in (False, True)]
    sizes.append(nq.binary_matmul_backward_work_bytes(300, 384, 320, 96))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    for _ in range(3):
        got = run(stream=side.cuda_stream)
        assert torch.cuda.current_stream() == here
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=gpu).fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = run(stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refinement_from_a_checkpoint_is_the_same_step(gpu):
    """STERefiner on a checkpoint of its inputs equals, bit for bit, the steps
    on the values that the checkpoint stands for."""
    import torch
    import sub_bit_weight_lb_amd as nq
    m, n, r, N, bt = 130, 100, 40, 300, 120
    rng = np.random.default_rng(5)
    X = put(activations(rng, N, n), gpu)
    q = nq.act8_quantize(X)
    W = put(0.02 * rng.standard_normal((m, n)), gpu)
    Y = X @ W.t()
    Uf, Vf = put(0.1 * rng.standard_normal((m, r)), gpu), put(0.1 * rng.standard_normal((n, r)), gpu)
    s1, s2 = put(rng.uniform(0.01, 0.03, m), gpu), put(rng.uniform(0.01, 0.03, n), gpu)
    batches = [torch.from_numpy(rng.permutation(N)[:bt].astype(np.int32)).to(gpu) for _ in range(3)]
    out = []
    for src in (nq.act8_dequantize(q), q):
        with nq.STERefiner(m, n, r, bt) as h:
            h.set_params(Uf, Vf, s1, s2)
            losses = h.refine(src, Y, batches)
            out.append((losses, h.params()))
    assert out[0][0] == out[1][0]
    assert all(torch.equal(a, b) for a, b in zip(out[0][1], out[1][1]))
