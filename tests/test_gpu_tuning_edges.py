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


@pytest.mark.parametrize("T", [6, 50, 150, 600])
@pytest.mark.parametrize("down", [60, 90, 100])
def test_layer_gradient_of_small_numbers(gpu, T, down):
    """fp32 gradients and activations 2^-down as large: rows keep all digits of
    their fixed point until fp32's own subnormals, 2^-149, end them. (dY and the
    values of X are 2^-7 and 1, s1 and s2 2^-6: at 2^-100 the products s1 dY begin
    to be subnormal, off by 2^-150 each, 2^-37 of a row's largest.)"""
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} 2^-{down}", flush=True)
    L = Layer(T, T, 200, 300, 70, "float32", gpu)
    L.dY *= 2.0 ** -down
    L.check(*nq.binary_matmul_backward(*L.args()))
    L = Layer(T, T, 200, 300, 70, "float32", gpu)
    L.q.exps -= down
    L.x = L.x * 2.0 ** -down
    L.check(*nq.binary_matmul_backward(*L.args()))


# ---------------------------------------------------------------- the loss and its gradient together

U = 2.0 ** -24


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [1, 5, 16, 17, 32, 33, 64, 65, 128])
def test_probabilities_of_the_gradient_sum_to_one(gpu, name, T):
    """sum_v G_tv = 0: read in dH at a column where every word holds 1 and every
    token 0. Columns that cancel in pairs make z's partial sums a thousand times
    its value, so z is off by 1e-4 and more, and probabilities add up to one
    only if the gradient's z are those that lse came from. With the same z, with
    y_v = z_v - lse <= 0 and gaps a_v = max z - z_v, what is left is
      lse: U |lse| of its last sum, 2 U log V of the logarithm, and of the sum of
        exponentials 24 U (its depth, exp's 2 units) and 4 U sum_v p_v a_v;
      exp in the gradient: sum_v p_v (4 U + 4 U |y_v|);
      G: 2 U and its rounding to its type, half() or 2^-22 of fp32's terms, and
        dH's fp32 sum over the words, (V + 40) U, of sum_v |G_v|, and dH's own
        rounding."""
    import torch
    import sub_bit_weight_lb_amd as nq
    from test_gpu_tuning import H as host, half, put
    print(f"case T={T} {name}", flush=True)
    V, d = 300, 512
    rng = np.random.default_rng(T)
    W = rng.standard_normal((V, d)) * 0.1
    X = rng.standard_normal((T, d)) * 0.3
    labels = rng.integers(0, V, T)
    X[:, 256:] += 4.0 * W[labels, 256:]          # most tokens are sure of their label
    W[:, 0], X[:, 0] = 1.0, 0.0                  # where the sum is read
    W[:, 128] = 0.0
    W[:, 1:128] *= 100.0
    X[:, 1:128] *= 300.0
    W[:, 129:256], X[:, 129:256] = W[:, 1:128], -X[:, 1:128]
    Hd, Wd = put(X, gpu, name), put(W, gpu, name)
    lab = torch.from_numpy(labels.astype(np.int32)).to(gpu)
    dl = put(rng.uniform(0.5, 1.0, T), gpu)
    _, lse = nq.vocab_loss(Hd, Wd, lab)
    dH, _ = nq.vocab_loss_backward(Hd, Wd, lab, lse, dl)

    z = host(Hd) @ host(Wd).T
    top = z.max(1, keepdims=True)
    lse64 = (top + np.log(np.exp(z - top).sum(1, keepdims=True)))[:, 0]
    p = np.exp(z - lse64[:, None])
    G = p.copy()
    G[np.arange(T), labels] -= 1.0
    # (the z that are used differ from these by a part in a hundred at most)
    absG, gaps, y = 1.1 * np.abs(G).sum(1), (p * (top - z)).sum(1), (p * (lse64[:, None] - z)).sum(1)
    g_type = 2.0 ** -22 if name == "float32" else half(name)
    tol = U * (np.abs(lse64) + 2 * np.log(V) + 24 + 4 * gaps + 4 + 4 * y)
    tol = tol + (2 * U + g_type + (V + 40) * U) * absG
    tol = 1.1 * host(dl) * tol * (1 + half(name))
    got = np.abs(host(dH)[:, 0])
    print("largest share of the bound", float((got / tol).max()), flush=True)
    np.testing.assert_array_less(got, tol)


@pytest.mark.parametrize("tokens", [(1, 2, 8, 16), (17, 24, 30, 32), (33, 40, 48, 64), (65, 80, 100, 128)])
def test_fp32_gradients_are_as_exact_as_the_plain_form(gpu, tokens):
    """Against float64, over some batches together, the error (relative, in the
    norm) of dH, dW and lse is at most 1.5 times that of the same formulas in
    fp32 torch products. Both round every partial sum once to fp32, in orders
    of their own, so that the two errors are samples of one size: a sum in
    three passes over k, the largest first, rounds three times as often at full
    size and comes out at twice it; logits that differ from those of lse at ten
    times it."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d = 700, 4096
    own, plain = np.zeros(3), np.zeros(3)
    for T in tokens:
        print(f"case T={T}", flush=True)
        g = torch.Generator(device=gpu).manual_seed(T)
        W = 0.02 * torch.randn((V, d), generator=g, device=gpu)
        labels = torch.randint(0, V, (T,), generator=g, device=gpu)
        lean = (torch.arange(T, device=gpu) % 2).float().unsqueeze(1) * (10.0 / (0.0004 * d))
        X = torch.randn((T, d), generator=g, device=gpu) + lean * W[labels]
        dl = torch.full((T,), 1.0 / T, device=gpu)

        def formulas(X, W, dl):
            z = torch.mm(X, W.t())
            top = z.amax(1, keepdim=True)
            lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
            G = torch.exp(z - lse.unsqueeze(1))
            G[torch.arange(T, device=gpu), labels] -= 1.0
            G = G * dl.unsqueeze(1)
            return torch.mm(G, W), torch.mm(G.t(), X), lse

        _, lse = nq.vocab_loss(X, W, labels.int())
        got = (*nq.vocab_loss_backward(X, W, labels.int(), lse, dl), lse)
        want = formulas(X.double(), W.double(), dl.double())
        for e, values in ((own, got), (plain, formulas(X, W, dl))):
            e += [float((a.double() - b).norm() / b.norm()) ** 2 for a, b in zip(values, want)]
    ratio = np.sqrt(own / plain)
    print("own", np.sqrt(own), "plain", np.sqrt(plain), flush=True)
    assert (ratio[:2] <= 1.5).all(), ratio
    assert ratio[2] <= 2.0, ratio     # (lse adds one sum of a handful of large terms)


@pytest.mark.parametrize("T", [9, 64, 65, 300])
def test_a_loud_token_costs_the_others_nothing(gpu, T):
    """fp32 hidden states of one token 1e8 times the rest: the others' loss, lse
    and dH keep every bit."""
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Head(41, T, 700, 200, "float32", gpu, ignored=0.0)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    L.check_loss(loss, lse)
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    L.check_grad(dH, dW)
    L.H[3] *= 1e8
    loud = nq.vocab_loss(L.H, L.W, L.labels)
    rest = [t for t in range(T) if t != 3]
    assert torch.equal(loud[0][rest], loss[rest]) and torch.equal(loud[1][rest], lse[rest])
    got, _ = nq.vocab_loss_backward(L.H, L.W, L.labels, loud[1], L.dl)
    assert torch.equal(got[rest], dH[rest])
    # ignored, it does not count for dW either
    L.labels[3] = -1
    without, _ = nq.vocab_loss(L.H, L.W, L.labels)
    assert torch.equal(without[rest], loss[rest])
    L.check_grad(*nq.vocab_loss_backward(L.H, L.W, L.labels, loud[1], L.dl))


def check_rows_of_dh(L, dH):
    """dH's rows to bounds that scale with the row's own dloss, as in
    Head.check_grad but for what is left of G's range: fp16 terms of G hold
    (p - [label]) f 2^15 with 1/2 <= |f| < 1, so a probability to 2^-25 of 2^14
    at least, 2^-39; fp16 keeps up to 10 bits of the tokens' differences in it,
    2^-29; bf16's exponents reach further than any of these. W's terms hold
    2^-39 of its largest."""
    from oracle import tuning as O
    from test_gpu_tuning import H as host, half, least
    lab, h, V = L.labels.cpu().numpy(), half(L.name), L.W.shape[0]
    use = lab >= 0
    Hh, W, dl = host(L.H), host(L.W), host(L.dl)
    Hh[~use] = 0
    want, _, G = O.vocab_loss_backward(Hh, W, lab, dl, L.scale)
    size = np.abs(dl[use])[:, None] * abs(L.scale)
    ez = L.zbound()[use]
    p = np.exp(L.scale * Hh[use] @ W.T - O.vocab_loss(Hh, W, lab, L.scale)[1][use][:, None])
    ee = ez + ez.max(1, keepdims=True) + (V + 16) * U + 16 * U * np.abs(np.log(np.maximum(p, 1e-30)))
    eg = p * (np.expm1(ee) + 8 * U) * size + (h + 4 * U) * np.abs(G)
    eg += {"float32": 2.0 ** -39, "float16": 2.0 ** -29, "bfloat16": 0.0}[L.name] * size
    more = 2.0 ** -22 if L.name == "float32" else 0.0
    tol = eg @ np.abs(W) + ((V + 40) * U + more) * ((np.abs(G) + eg) @ np.abs(W))
    if L.name == "float32":
        tol += V * 2.0 ** -38 * size * np.abs(W).max()
    got = host(dH)
    np.testing.assert_array_less(np.abs(got[use] - want[use]),
                                 1.01 * tol + h * np.abs(want[use]) + least(L.name))
    assert (got[~use] == 0).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V", [(9, 400), (30, 5000), (64, 700), (70, 5000), (300, 700)])
def test_a_token_of_small_weight_keeps_its_gradient(gpu, name, T, V):
    """dloss from 1 to 1e-7 of the largest: each row of dH is as exact as if it
    were alone. (fp16's subnormals end at 2^-24: its dloss are 2^10 times as
    large, so that what is asked for can be written.)"""
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} {name}", flush=True)
    L = Head(51, T, V, 96, name, gpu)
    _, lse = nq.vocab_loss(L.H, L.W, L.labels)
    for k in range(T):
        L.dl[k] = (-1.0) ** k * 10.0 ** -(k % 8) * (1.0 + 0.1 * (k % 5)) * (1024 if name == "float16" else 1)
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    check_rows_of_dh(L, dH)
    L.check_grad(None, dW)
    only, none = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl, want_dW=False)
    assert none is None and (only == dH).all()
    none, only = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl, want_dH=False)
    assert none is None and (only == dW).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [9, 70])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_dloss_that_is_not_finite_stays_in_its_row(gpu, name, T, bad):
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Head(52, T, 400, 64, name, gpu, ignored=0.0)
    _, lse = nq.vocab_loss(L.H, L.W, L.labels)
    L.dl[2] = 0.0
    want, _ = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    assert (want[2] == 0).all()
    L.dl[2] = bad
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    rest = [t for t in range(T) if t != 2]
    assert torch.equal(dH[rest], want[rest])
    assert not torch.isfinite(dH[2]).any() and not torch.isfinite(dW).all()
    L.dl.fill_(bad)
    dH, _ = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    assert not torch.isfinite(dH).any()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", [(9, 300, 64), (40, 300, 129), (70, 300, 64), (300, 1200, 200)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_word_that_is_not_finite_shows_in_every_loss(gpu, name, T, V, d, bad):
    """Also where its logit is -infinity, which exp would make a zero."""
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Head(61, T, V, d, name, gpu)
    L.labels[L.labels == 7] = 8
    L.W[7, 5] = bad
    used = L.labels >= 0
    assert (L.H[used, 5] > 0).any() and (L.H[used, 5] < 0).any()
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels)
    assert loss[used].isnan().all() and lse[used].isnan().all()
    assert (loss[~used] == 0).all() and (lse[~used] == 0).all()
    dH, dW = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    assert dH[used].isnan().all() and (dH[~used] == 0).all() and dW.isnan().all()


@pytest.mark.parametrize("name", ["bfloat16", "float16"])
@pytest.mark.parametrize("T, V, d", [(1, 5000, 1000), (1, 32000, 512), (2, 700, 4096), (5, 32000, 512),
                                     (16, 5000, 1000), (32, 32000, 512), (33, 32000, 512), (300, 5000, 1000)])
def test_16_bit_gradients_against_the_plain_form(gpu, name, T, V, d):
    """The error of dH and dW (relative, in the norm) against that of the formulas in
    fp32, rounded once at the end. Up to 32 tokens G has two terms, 16 bits of it
    or more, and what is left is the outputs' rounding: 1 + 2^-8 of its square
    and the fp32 sums, 1.05 with room. With more it is rounded to the type itself,
    half a unit as the outputs are: two roundings of one size, 2^0.5 of one, 1.5
    with room for their samples."""
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    for seed in range(6):
        g = torch.Generator(device=gpu).manual_seed(100 * seed + T)
        W = 0.02 * torch.randn((V, d), generator=g, device=gpu)
        labels = torch.randint(0, V, (T,), generator=g, device=gpu)
        lean = (torch.rand((T, 1), generator=g, device=gpu) < 0.5) * (10.0 / (0.0004 * d))
        X = (torch.randn((T, d), generator=g, device=gpu) + lean * W[labels]).to(dt(name))
        W = W.to(dt(name))
        dl = torch.full((T,), 1.0 / T, device=gpu)

        def formulas(X, W, dl):
            z = torch.mm(X, W.t())
            G = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
            G[torch.arange(T, device=gpu), labels] -= 1.0
            G = G * dl.unsqueeze(1)
            return torch.mm(G, W), torch.mm(G.t(), X)

        _, lse = nq.vocab_loss(X, W, labels.int())
        got = nq.vocab_loss_backward(X, W, labels.int(), lse, dl)
        plain = [v.to(dt(name)) for v in formulas(X.float(), W.float(), dl)]
        for a, p, e in zip(got, plain, formulas(X.double(), W.double(), dl.double())):
            own, ref = (float((v.double() - e).norm() / e.norm()) for v in (a, p))
            assert own <= (1.05 if T <= 32 else 1.5) * ref, (seed, own, ref)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", [(1, 1, 8), (2, 1, 40), (32, 1, 16), (33, 1, 16), (5, 3, 9), (32, 65, 8),
                                     (64, 129, 31), (16, 63, 7)])
@pytest.mark.parametrize("scale", [1.0, -0.7, 0.0])
def test_smallest_vocabularies_and_scales_of_any_sign(gpu, name, T, V, d, scale):
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} scale={scale} {name}", flush=True)
    L = Head(T + V, T, V, d, name, gpu, scale=scale)
    loss, lse = nq.vocab_loss(L.H, L.W, L.labels, scale=scale,
                              work=dirty(nq.vocab_loss_work_bytes(T, V, d, dt(name)), gpu))
    L.check_loss(loss, lse)
    L.check_grad(*nq.vocab_loss_backward(
        L.H, L.W, L.labels, lse, L.dl, scale=scale,
        work=dirty(nq.vocab_loss_work_bytes(T, V, d, dt(name), True), gpu)))


@pytest.mark.parametrize("name, k", [("float32", 90), ("float32", -90), ("bfloat16", 90),
                                     ("bfloat16", -90), ("float16", 3)])
@pytest.mark.parametrize("T", [7, 40, 90])
def test_gradients_scale_with_dloss_to_the_bit(gpu, name, k, T):
    """All dloss times a power of two give the same gradient times it, where no
    output leaves its type's normal numbers."""
    import torch
    import sub_bit_weight_lb_amd as nq
    L = Head(71, T, 300, 72, name, gpu)
    L.labels[L.labels >= 0] %= 7          # many tokens share a label
    _, lse = nq.vocab_loss(L.H, L.W, L.labels)
    a = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl)
    L.check_grad(*a)
    b = nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl * 2.0 ** k)
    for x, y in zip(a, b):
        x, y = x.float(), y.float()
        least = 4 * torch.finfo(dt(name)).smallest_normal
        normal = ((x.abs() > least) & (y.abs() > least)) | ((x == 0) & (y == 0))
        assert normal.float().mean() > 0.9
        assert torch.equal(x[normal] * 2.0 ** k, y[normal])


@pytest.mark.parametrize("name", TYPES)
def test_captured_gradients_of_few_tokens_replay(gpu, name):
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d = 11, 900, 136
    L = Head(81, T, V, d, name, gpu)
    work = torch.empty(nq.vocab_loss_work_bytes(T, V, d, dt(name), True), dtype=torch.uint8, device=gpu)

    def run():
        loss, lse = nq.vocab_loss(L.H, L.W, L.labels, work=work)
        return (loss, lse, *nq.vocab_loss_backward(L.H, L.W, L.labels, lse, L.dl, work=work))

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(3):
        gen = torch.Generator(device=gpu).manual_seed(k)
        L.H.copy_(torch.randn(L.H.shape, generator=gen, device=gpu))
        L.dl.copy_(torch.randn(L.dl.shape, generator=gen, device=gpu))
        work.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
