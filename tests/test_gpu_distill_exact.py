"""The gradient of a divergence from a teacher's words where its size alone bounds the logits'
error too loosely to say anything: here hidden states and weights are small integers times a
power of two, whose logits are exact in any order of summing (fp32's second terms are zero). What
is left, with u = 2^-24 and h half a unit of the output type:

S, lse     the sum of a group of up to 128 words, 32 in a lane and 6 more additions, each word's exp to 4 u and
           2 u |y| of its argument's rounding; the groups' joins, of which a sum goes through V / 128 / 256 in a
           thread and 8 more, each with an exp, two products and a sum (8 u): (48 + 8 (V / 32768 + 9)) u and
           2 u sum p |y| of S, and u |lse| and u |z| more of lse and rest (`dl`)
G          lse and rest once each, the exponential 4 u and 2 u |y|: (2 dl + 16 u (1 + |y|)) of Q p + r p', p' the
           softmax of the words that are not listed; a 16-bit G's rounding, h of |G| in one term and 2 h^2 in two (one
           more u for its factor); fp16's least value at its scale, 2^-24 / 2^14 of the largest dloss
dH, dW     their sums' own roundings, n + 40 of them, and h of the result

Each test says how large the bound is beside the gradient: one of zeros, or one that leaves a piece of the vocabulary
out, does not pass.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def dt(name):
    import torch
    return getattr(torch, name)


def half(name):
    import torch
    return torch.finfo(dt(name)).eps / 2


def least(name):
    return 2.0 ** -149 if name == "float32" else 2.0 ** -133 if name == "bfloat16" else 2.0 ** -24


def grid(shape, gen, dev, step, name):
    """Integers of -3 .. 3 times `step`."""
    import torch
    return torch.randint(-3, 4, shape, generator=gen, device=dev, dtype=torch.int8).to(dt(name)).mul_(step)


class Exact:
    def __init__(self, seed, T, V, d, K, name, dev, scale=0.5, tail=True):
        import torch
        g = torch.Generator(device=dev).manual_seed(seed)
        # z of standard deviation 1 to 2: 4 sqrt(d) steps
        fine = 2.0 ** -int(np.ceil(np.log2(2 * np.sqrt(d))))
        self.H = grid((T, d), g, dev, 0.5, name)
        self.W = grid((V, d), g, dev, 2 * fine, name)
        ids = torch.randint(0, V, (T, K), generator=g, device=dev)
        logq = torch.log_softmax(2 * torch.randn((T, K + 1), generator=g, device=dev), 1)[:, :K].contiguous()
        ids[torch.rand((T, K), generator=g, device=dev) < 0.1] = -1
        if T > 4:
            ids[3] = -1
        ids[:, 0], ids[0, 0] = torch.where(ids[:, 0] >= 0, V - 1, ids[:, 0]), 0
        self.ids, self.logq = ids.int(), logq
        self.dl = torch.randn(T, generator=g, device=dev)
        self.T, self.V, self.d, self.K = T, V, d, K
        self.name, self.scale, self.tail, self.dev = name, scale, tail, dev

    def loss(self, **kw):
        import sub_bit_weight_lb_amd as nq
        return nq.vocab_distill(self.H, self.W, self.ids, self.logq, scale=self.scale, tail=self.tail, **kw)

    def grad(self, q, **kw):
        import sub_bit_weight_lb_amd as nq
        return nq.vocab_distill_backward(self.H, self.W, self.ids, self.logq, q, self.dl, scale=self.scale,
                                         tail=self.tail, **kw)

    def logits(self):
        import torch
        h = self.H.double() * self.scale
        return torch.cat([torch.mm(h, self.W[a:a + 16384].double().t()) for a in range(0, self.V, 16384)], 1)

    def exact(self):
        """loss, lse, rest, hit, G and the bounds of lse and of G (but for its rounding)."""
        import torch
        z = self.logits()
        ids, logq, V = self.ids.long(), self.logq.double(), self.V
        on = ids >= 0
        self.used = used = on.any(1)
        if not self.tail:
            logq = torch.log_softmax(torch.where(on, logq, -1e300), 1)
        q = torch.where(on, torch.exp(logq), 0.0)
        at = torch.where(on, ids, V)
        inside = torch.zeros((self.T, V + 1), dtype=torch.bool, device=self.dev).scatter_(1, at, True)[:, :V]
        target = torch.zeros((self.T, V + 1), dtype=torch.float64, device=self.dev).scatter_add_(1, at, q)[:, :V]
        lse = torch.logsumexp(z, 1)
        hit = torch.where(on, z.gather(1, ids.clamp(min=0)), 0.0)
        loss = torch.where(on & (q > 0), q * (logq - hit + lse[:, None]), 0.0).sum(1)
        p = torch.softmax(z, 1)
        rest, r, part = lse, torch.zeros_like(lse), None
        if self.tail:
            r = (1 - q.sum(1)).clamp(min=0)
            others = z.masked_fill(inside, -float("inf"))
            rest = torch.logsumexp(others, 1)
            loss = loss + torch.where(r > 0, r * (torch.log(r) - rest + lse), 0.0)
            part = r[:, None] * torch.softmax(others, 1)
        y = (z - z.amax(1, keepdim=True)).abs()
        size = z.abs().amax(1)
        self.edl = ((48 + 8 * (V / 32768 + 9)) * U + 2 * U * (p * y).sum(1) + 2 * U * (lse.abs() + rest.abs() + size))
        whole = (q.sum(1) + r)[:, None]
        f = torch.where(used, self.dl.double() * self.scale, 0.0)[:, None]
        mag = whole * p
        G = mag - target
        if part is not None:
            G, mag = G - part, mag + part
        self.eG = mag * f.abs() * (2 * self.edl[:, None] + 16 * U * (1 + y + 2 * size[:, None]))
        self.G, self.q, self.r = G * f, q, r
        self.want = loss, lse, rest, hit
        return self

    def check_loss(self, loss, q):
        import torch
        u = self.used
        want, lse, rest, hit = self.want
        assert ((q.lse.double() - lse).abs() <= self.edl)[u].all()
        assert ((q.rest.double() - rest).abs() <= self.edl)[u].all()
        assert ((q.hit.double() - hit).abs() <= U * hit.abs())[u].all()       # (exact: rounded at most)
        tol = (self.q.sum(1) + self.r) * 2 * self.edl + 4 * U * want.abs()
        assert ((loss.double() - want).abs() <= tol)[u].all()
        assert all((t[~u] == 0).all() for t in (loss, q.lse, q.rest, q.hit))

    def check(self, dH, dW, terms, rows=slice(None), cols=slice(None), pieces=()):
        """terms of a 16-bit G; rows of dW, columns of both; pieces of the vocabulary that dH must show."""
        import torch
        h = half(self.name)
        more = 2.0 ** -21 if self.name == "float32" else h if terms == 1 else 2 * h * h
        whole = self.q.sum(1) + self.r        # (G is scaled by it where it is more than 1)
        big = float((self.dl.double().abs() * self.used * torch.where(whole < 1.5, 1.0, 2 * whole)).max()) * abs(self.scale)
        eG = self.eG + (more + 2 * U) * self.G.abs()
        if self.name != "bfloat16":
            eG = eG + 2.0 ** -38 * big
        mag = self.G.abs() + eG
        W, H = self.W[:, cols], self.H[:, cols].double()

        def over(a, b):          # a @ W of columns, in parts
            return sum(torch.mm(a[:, i:i + 16384], b(W[i:i + 16384].double())) for i in range(0, self.V, 16384))
        extra = 2.0 ** -21 if self.name == "float32" else 0.0    # (the terms that fp32's passes leave out)
        if dH is not None:
            ref, tol = over(self.G, lambda w: w), over(eG + ((self.V + 40) * U + extra) * mag, torch.abs)
            tol = tol + h * ref.abs() + least(self.name)
            assert ((dH[:, cols].double() - ref).abs() <= tol).all()
            assert (dH[~self.used] == 0).all()
            u = self.used
            assert (ref.abs() > 2 * tol)[u].double().mean() > 0.5            # (zeros would not pass)
            for a, b in pieces:
                one = torch.mm(self.G[:, a:b], W[a:b].double())
                assert (one.abs() > 2 * tol)[u].any(), (a, b)                # (nor a piece left out or taken twice)
        if dW is not None:
            ref, tol = self.G[:, rows].t() @ H, (eG + ((self.T + 40) * U + extra) * mag)[:, rows].t() @ H.abs()
            tol = tol + h * ref.abs() + least(self.name)
            assert ((dW[rows][:, cols].double() - ref).abs() <= tol).all()
            assert (ref.abs() > 2 * tol).double().mean() > 0.5


# ---------------------------------------------------------------- without kept logits

@pytest.mark.parametrize("name", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("T, V, d", [(129, 151936, 320), (192, 131073, 64), (150, 262144, 72), (300, 131072, 8)])
def test_a_gradient_that_computes_its_logits_keeps_to_its_workspace(gpu, name, T, V, d):
    """Vocabularies so long that pieces of them are copied and G has a second term or none: a
    workspace of the stated size, with nothing written behind it."""
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    L = Exact(T + V, T, V, d, 9, name, gpu).exact()
    need = nq.vocab_distill_work_bytes(T, V, d, dt(name), 9, True)
    guard = torch.full((need + (1 << 26),), 255, dtype=torch.uint8, device=gpu)
    loss, q = L.loss(keep=False)
    assert q.logits is None
    L.check_loss(loss, q)
    dH, dW = L.grad(q, work=guard[:need])
    assert (guard[need:] == 255).all()
    L.check(dH, dW, 2 if T <= 192 else 1)


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("name", ["bfloat16", "float16"])
@pytest.mark.parametrize("T, V, d", [(33, 700, 72), (40, 500, 515), (65, 300, 328), (129, 257, 77), (192, 400, 264)])
def test_16_bit_gradients_have_both_terms_with_and_without_the_logits(gpu, name, T, V, d, keep):
    """33 to 192 tokens, rows in place and copied (d = 77, 515), either result alone: the same bounds."""
    import torch
    print(f"case T={T} V={V} d={d} {name} keep={keep}", flush=True)
    L = Exact(T + V + d, T, V, d, 9, name, gpu).exact()
    loss, q = L.loss(keep=keep)
    assert (q.logits is not None) == keep
    dH, dW = L.grad(q)
    L.check(dH, dW, 2)
    assert torch.equal(L.grad(q, want_dW=False)[0], dH)
    assert torch.equal(L.grad(q, want_dH=False)[1], dW)


@pytest.mark.parametrize("name", ["bfloat16", "float16"])
@pytest.mark.parametrize("T, V, d", [(300, 500, 4000), (800, 700, 1000), (301, 4999, 515), (2000, 300, 72)])
def test_short_products_have_both_terms(gpu, name, T, V, d):
    """More tokens, where T V d is 2^32 at most: what a second term costs is little there."""
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    assert T > 192 and T * V * d <= 1 << 32
    L = Exact(T + V + d, T, V, d, 9, name, gpu).exact()
    for keep in (True, False):
        _, q = L.loss(keep=keep)
        L.check(*L.grad(q), 2)


# ---------------------------------------------------------------- large sizes

@pytest.mark.parametrize("name, T, keep", [("bfloat16", 40, True), ("bfloat16", 40, False), ("float16", 200, True),
                                           ("float16", 200, False), ("float32", 70, True), ("float32", 70, False),
                                           ("float32", 5, True)])
def test_a_hidden_size_that_takes_the_vocabulary_in_pieces(gpu, name, T, keep):
    """Each of the pieces in which W is copied shows in dH, and words of all of them in dW."""
    V, d = 5000, 33001
    print(f"case T={T} {name} keep={keep}", flush=True)
    L = Exact(11, T, V, d, 30, name, gpu).exact()
    loss, q = L.loss(keep=keep)
    assert (q.logits is not None) == keep
    L.check_loss(loss, q)
    dH, dW = L.grad(q)
    L.check(dH, dW, 1 if T == 200 else 2, pieces=[(0, 1792), (1792, 3584), (3584, V)])


@pytest.mark.parametrize("T, tail", [(3, True), (3, False), (70, True), (70, False), (300, True)])
def test_gradients_of_a_vocabulary_past_32_bits(gpu, T, tail):
    """W of more than 2^32 bytes: dW's first and last words, the first and last columns of both, and the
    words past 2^31 and 2^32 bytes in dH."""
    V, d = 140001, 16384
    first = [(1 << n) // (2 * d) for n in (31, 32)]
    print(f"case T={T} tail={tail}", flush=True)
    L = Exact(6, T, V, d, 4, "bfloat16", gpu, tail=tail)
    L.ids[1, 1:3] = L.ids.new_tensor(first) + 7
    L.exact()
    loss, q = L.loss()
    L.check_loss(loss, q)
    terms = 2 if T <= 192 else 1
    for state, cols in ((q, slice(0, 64)), (q, slice(d - 64, d)), (L.loss(keep=False)[1], slice(d - 64, d))):
        dH, dW = L.grad(state)
        for rows in (slice(0, 200), slice(first[0] - 100, first[0] + 100), slice(first[1] - 100, first[1] + 100),
                     slice(V - 200, V)):
            L.check(None, dW, terms, rows=rows, cols=cols)
        L.check(dH, None, terms, cols=cols, pieces=[(0, first[0]), (first[0], first[1]), (first[1], V)])
