"""GPU parity of log probabilities over a vocabulary and of the divergence from a
teacher's words with its gradient, against the float64 oracle (oracle/scoring.py).
Each difference is held to a bound worked out from the roundings, with u = 2^-24
and h(t) half a unit of the output type:

z            an fp32 sum of d exact products, (d + 2) u sum |h_k w_k|; fp32
             operands (two fp16 terms) 2^-22 of it and d 2^-38 of the largest
             product more. Its scaling rounds once (in the 2).
S, lse       exp to 4 units and (its argument times log2 e, rounded) 2 u |y| e^y:
             weighted with p, y^2 <= 2 e^-y .. so the sums' own bound is (V + 64) u of S
             plus 2 u sum p |y|. lse: ez + that + 2 u |lse|.
entropy      d entropy = -sum p (log p + entropy) dz, at most 2 entropy ez; U adds
             2 u sum p y^2 and (V + 64) u of itself.
loss         sum q <= 1 (+ r): ez and lse's bound each once, rest's like lse's; the
             entries' part is taken in 64 bits, so that one rounding is left.
gradient     G of a word: the exponent's bound on its exponentials, then the
             roundings of the products that the loss over a vocabulary has.
"""
import numpy as np
import pytest

from oracle import scoring as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ["float32", "bfloat16", "float16"]


def dt(name):
    import torch
    return getattr(torch, name)


def H64(t):
    return t.detach().double().cpu().numpy()


def half(name):
    import torch
    return torch.finfo(dt(name)).eps / 2


def least(name):
    return 2.0 ** -149 if name == "float32" else 2.0 ** -133 if name == "bfloat16" else 2.0 ** -24


def put(x, dev, name="float32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev).to(dt(name))


def ints(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)


def strided(t, extra, lead=0):
    """t with `extra` columns after each row and `lead` elements before the first."""
    import torch
    buf = torch.full((t.shape[0] * (t.shape[1] + extra) + lead,), 77, dtype=t.dtype, device=t.device)
    v = buf[lead:].view(t.shape[0], t.shape[1] + extra)[:, :t.shape[1]]
    v.copy_(t)
    return v


def less(err, tol):
    np.testing.assert_array_less(err, np.broadcast_to(tol, np.shape(err)) + 1e-300)


class Head:
    """H, W and the bounds of z and its sums."""

    def __init__(self, seed, T, V, d, name, dev, scale=1.0):
        self.rng = np.random.default_rng(seed)
        self.H = put(self.rng.standard_normal((T, d)), dev, name)
        self.W = put(self.rng.standard_normal((V, d)) * 2.0 / np.sqrt(d), dev, name)
        self.name, self.scale, self.dev = name, scale, dev
        self.T, self.V, self.d = T, V, d

    def exact(self):
        """z, the bound of z per row (of its largest), and of lse"""
        h, w = H64(self.H), H64(self.W)
        fp32 = self.name == "float32"
        z = self.scale * (h @ w.T)
        rel = (self.d + 2) * U + (2.0 ** -22 if fp32 else 0.0)
        tiny = self.d * 2.0 ** -38 * np.abs(h).max(1, keepdims=True) * np.abs(w).max() if fp32 else 0.0
        self.z = z
        self.ezs = abs(self.scale) * (rel * (np.abs(h) @ np.abs(w).T) + tiny)
        self.ez = self.ezs.max(1)
        self.lse = O.lse_of(z)
        y = z - z.max(1, keepdims=True)
        p = np.exp(z - self.lse[:, None])
        self.sums = (self.V + 64) * U + 2 * U * (p * np.abs(y)).sum(1)
        self.elog = 1.01 * (self.ez + self.sums + 2 * U * np.abs(self.lse) + 2 * U * np.abs(z).max(1))
        self.second = (p * y * y).sum(1)
        return self


# ---------------------------------------------------------------- log probabilities

def check_logprobs(L, tokens, k, r):
    L.exact()
    want = O.vocab_logprobs(H64(L.H), H64(L.W), None if tokens is None else tokens.cpu().numpy(), k, L.scale)
    less(np.abs(H64(r.lse) - L.lse), L.elog)
    ent = want[1]
    less(np.abs(H64(r.entropy) - ent),
         1.01 * (2 * ent * L.ez + 2 * U * L.second + 2 * L.sums * (1 + ent) + 4 * U * (1 + ent)))
    both = L.elog + L.ez + 2 * U * np.abs(L.z).max(1)
    if tokens is not None:
        got, ref = H64(r.logprobs).reshape(L.T, -1), want[0].reshape(L.T, -1)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = ~np.isnan(ref)
        assert (got[ok & (ref == 0)] == 0).all() or L.V == 1
        less(np.where(ok, np.abs(got - ref), 0), both[:, None])
    if not k:
        return
    ids = r.top_ids.cpu().numpy()
    assert ids.dtype == np.int32 and ids.min() >= 0 and ids.max() < L.V
    rows = np.arange(L.T)[:, None]
    assert all(len(set(i)) == k for i in ids.tolist())
    zi = L.z[rows, ids]
    # in order, and none left out that is better, but for what z is off by
    less(zi[:, 1:] - zi[:, :-1], 2 * L.ez[:, None] + 1e-12)
    others = L.z.copy()
    others[rows, ids] = -np.inf
    less(others.max(1) - zi[:, -1], 2 * L.ez + 1e-12)
    less(np.abs(H64(r.top_logprobs) - (zi - L.lse[:, None])), both[:, None])


CASES = [(1, 1, 1, 1), (1, 2, 7, 2), (2, 63, 64, 63), (16, 64, 130, 20), (17, 65, 8, 1), (33, 257, 515, 128),
         (64, 1000, 96, 5), (65, 500, 72, 100), (300, 1000, 64, 7), (257, 2049, 200, 33), (513, 300, 129, 128)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d, k", CASES)
def test_logprobs_match_oracle(gpu, name, T, V, d, k):
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} k={k} {name}", flush=True)
    L = Head(T + V + d, T, V, d, name, gpu)
    tokens = ints(L.rng.integers(-2, V, (T, 3)), gpu)
    r = nq.vocab_logprobs(L.H, L.W, tokens, k)
    check_logprobs(L, tokens, k, r)
    again = nq.vocab_logprobs(L.H, L.W, tokens, k)
    for f in ("logprobs", "entropy", "lse", "top_ids", "top_logprobs"):
        assert torch.equal(getattr(r, f), getattr(again, f))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d, k", [(600, 4100, 200, 20), (600, 4100, 1100, 20), (1100, 12100, 1100, 64),
                                        (700, 30000, 136, 128), (70, 4100, 2052, 3), (40, 70001, 100, 50)])
def test_logprobs_in_tiles_of_every_size_and_several_steps(gpu, name, T, V, d, k):
    """128 x 128, 256 x 256 and 64 x 64 tiles; vocabularies past the first step."""
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} k={k} {name}", flush=True)
    L = Head(T + V + d, T, V, d, name, gpu)
    tokens = ints(L.rng.integers(0, V, T), gpu)
    check_logprobs(L, tokens, k, nq.vocab_logprobs(L.H, L.W, tokens, k))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [5, 70, 300])
def test_logprobs_of_parts(gpu, name, T):
    """Any of the outputs without the others, given tokens in one or two dimensions,
    strided inputs, a negative scale, outputs of the caller's."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d, k = 9001, 77, 11
    L = Head(3, T, V, d, name, gpu, scale=-0.4)
    L.H, L.W = strided(L.H, 5, 1), strided(L.W, 2, 3)
    tokens = strided(ints(L.rng.integers(-1, V, (T, 5)), gpu), 3, 1)
    all_ = nq.vocab_logprobs(L.H, L.W, tokens, k, scale=-0.4)
    check_logprobs(L, tokens, k, all_)
    one = nq.vocab_logprobs(L.H, L.W, tokens[:, 0].contiguous(), scale=-0.4)
    assert one.logprobs.shape == (T,) and one.top_ids.shape == (T, 0)
    none = nq.vocab_logprobs(L.H, L.W, k=k, scale=-0.4)
    assert none.logprobs is None
    bare = nq.vocab_logprobs(L.H, L.W, scale=-0.4)
    for r in (one, none, bare):
        assert torch.equal(r.lse, all_.lse) and torch.equal(r.entropy, all_.entropy)
    assert torch.equal(one.logprobs, all_.logprobs[:, 0])
    assert torch.equal(none.top_ids, all_.top_ids) and torch.equal(none.top_logprobs, all_.top_logprobs)
    need = nq.vocab_logprobs_work_bytes(T, V, d, dt(name), 5, k)
    out = nq.VocabLogprobs(*(torch.full_like(getattr(all_, f), 77) for f in
                             ("logprobs", "entropy", "lse", "top_ids", "top_logprobs")))
    guard = torch.full((need + 4096,), 255, dtype=torch.uint8, device=gpu)
    got = nq.vocab_logprobs(L.H, L.W, tokens, k, scale=-0.4, out=out, work=guard[:need])
    assert got is out and (guard[need:] == 255).all()
    for f in ("logprobs", "entropy", "lse", "top_ids", "top_logprobs"):
        assert torch.equal(getattr(out, f), getattr(all_, f))
    # fewer best words are the first of more
    few = nq.vocab_logprobs(L.H, L.W, k=1, scale=-0.4)
    assert torch.equal(few.top_ids[:, 0], all_.top_ids[:, 0])


@pytest.mark.parametrize("T", [1, 3, 40, 130, 600])
@pytest.mark.parametrize("k", [1, 20, 128])
def test_equal_logits_go_to_the_lower_word(gpu, T, k):
    """Logits of a few values, exact in any order of summing: words repeat, rows of
    zeros, and values that rise or fall along the vocabulary."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d = 20011, 64
    rng = np.random.default_rng(T + k)
    W = rng.integers(-1, 2, (V, d)).astype(np.float32)
    W[:, 0] = np.arange(V) // 79 - 128          # (254 levels: exact in bf16)
    h = rng.integers(-2, 3, (T, d)).astype(np.float32)
    h[:, 0] = 0
    h[0] = 0                                    # all equal
    if T > 2:
        h[1], h[2] = 0, 0
        h[1, 0], h[2, 0] = 1, -1                # rising and falling
    Wd, Hd = put(W, gpu, "bfloat16"), put(h, gpu, "bfloat16")
    r = nq.vocab_logprobs(Hd, Wd, k=k)
    z = h.astype(np.float64) @ W.astype(np.float64).T
    want = np.argsort(-z, axis=1, kind="stable")[:, :k]
    assert np.array_equal(r.top_ids.cpu().numpy(), want)
    assert r.top_ids[0].tolist() == list(range(k))
    assert abs(float(r.entropy[0]) - np.log(V)) <= (V + 64) * U + 4 * U * np.log(V)


@pytest.mark.parametrize("name", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [6, 70, 300])
def test_logprobs_of_rows_that_are_not_finite(gpu, name, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d, k = 9000, 64, 6
    L = Head(6, T, V, d, name, gpu)
    tokens = ints(np.stack([L.rng.integers(0, V, T), np.full(T, -1), np.full(T, V)], 1), gpu)
    ok = nq.vocab_logprobs(L.H, L.W, tokens, k)
    assert (ok.logprobs[:, 1] == 0).all() and ok.logprobs[:, 2].isnan().all()
    L.H[1, 3], L.H[3, 5], L.H[4] = float("nan"), float("inf"), -float("inf")
    r = nq.vocab_logprobs(L.H, L.W, tokens, k)
    bad = [1, 3, 4]
    rest = [t for t in range(T) if t not in bad]
    for f in ("entropy", "lse", "top_logprobs", "top_ids"):
        assert torch.equal(getattr(r, f)[rest], getattr(ok, f)[rest])
    assert torch.equal(r.logprobs[rest, :2], ok.logprobs[rest, :2])
    assert r.lse[bad].isnan().all() and r.entropy[bad].isnan().all() and r.top_logprobs[bad].isnan().all()
    assert (r.top_ids[bad] == -1).all() and r.logprobs[bad, 0].isnan().all() and (r.logprobs[bad, 1] == 0).all()
    # one word of W: every row
    L.H[bad] = 0.25
    L.W[V - 1, 7] = -float("inf")
    r = nq.vocab_logprobs(L.H, L.W, tokens, k)
    assert r.lse.isnan().all() and (r.top_ids == -1).all()


def test_certain_rows(gpu):
    """Logits in the hundreds: entropy and log probabilities of rows that are all but
    certain, and of words that are all but impossible."""
    import torch
    import sub_bit_weight_lb_amd as nq
    W = torch.zeros((400, 64), device=gpu)
    W[7, 0], W[300, 1], W[301, 1] = 1.0, 1.0, 1.0
    for T in (3, 80):
        for name in TYPES:
            Hh = torch.zeros((T, 64), device=gpu)
            Hh[0, 0], Hh[1, 1], Hh[2, 0] = 500.0, 500.0, 12.0
            tokens = torch.full((T, 2), 7, dtype=torch.int32, device=gpu)
            tokens[:, 1] = 301
            r = nq.vocab_logprobs(Hh.to(dt(name)), W.to(dt(name)), tokens, 2)
            lp, ent = H64(r.logprobs), H64(r.entropy)
            assert lp[0, 0] == 0 and lp[0, 1] == -500 and ent[0] == 0
            assert abs(lp[1, 1] + np.log(2)) < 4 * U and lp[1, 0] == pytest.approx(-500 - np.log(2), abs=500 * 2 * U)
            assert abs(ent[1] - np.log(2)) < 4 * U and r.top_ids[1].tolist() == [300, 301]
            rest = 399 * np.exp(-12.0)
            want = np.log1p(rest) + 12 * rest / (1 + rest)
            # (exp of 12: 2 u 12 and 4 units of the rest's share; log's argument u)
            assert abs(ent[2] - want) <= 32 * U * 12 * rest + 2 * U


def test_logprobs_of_no_rows(gpu):
    import torch
    import sub_bit_weight_lb_amd as nq
    W = torch.zeros((10, 8), device=gpu)
    r = nq.vocab_logprobs(W[:0], W, torch.zeros((0, 2), dtype=torch.int32, device=gpu), 3)
    assert r.logprobs.shape == (0, 2) and r.lse.shape == (0,) and r.top_ids.shape == (0, 3)
    r = nq.vocab_logprobs(W, W, torch.zeros((10, 0), dtype=torch.int32, device=gpu), 0)
    assert r.logprobs.shape == (10, 0) and abs(float(r.lse[0]) - np.log(10)) < 8 * U * 3


@pytest.mark.parametrize("name", ["bfloat16", "float32"])
@pytest.mark.parametrize("k", [1, 20, 64, 128])
def test_vocabularies_in_several_steps(gpu, name, k):
    """More logits than are kept whole: the best words of a step at a time. Values on a
    grid, whose logits are exact in any order of summing, so that equal ones are many;
    rows of one value, and rows that rise or fall along the vocabulary."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d = 520, 130003, 64
    assert T * V > 1 << 26
    g = torch.Generator(device=gpu).manual_seed(k)
    W = torch.randint(-3, 4, (V, d), generator=g, device=gpu).float()
    W[:, 0] = (torch.arange(V, device=gpu) // 512 - 127).float()
    Hh = torch.randint(-3, 4, (T, d), generator=g, device=gpu).float() / 8
    Hh[:, 0] = 0
    Hh[0] = 0
    Hh[1], Hh[2], Hh[1, 0], Hh[2, 0] = 0, 0, 0.125, -0.125
    tokens = torch.randint(0, V, (T, 2), generator=g, device=gpu, dtype=torch.int32)
    r = nq.vocab_logprobs(Hh.to(dt(name)), W.to(dt(name)), tokens, k)
    z = torch.mm(Hh.double(), W.double().t())
    lse = torch.logsumexp(z, 1)
    for a in range(0, T, 130):
        best, ids = torch.sort(z[a:a + 130], dim=1, descending=True, stable=True)
        assert torch.equal(r.top_ids[a:a + 130].long(), ids[:, :k])
        tol = (V + 64) * U + 8 * U * best.abs().max()
        assert ((r.top_logprobs[a:a + 130].double() - (best[:, :k] - lse[a:a + 130, None])).abs() <= tol).all()
    tol = (V + 64) * U + 8 * U * z.abs().max()
    assert ((r.lse.double() - lse).abs() <= tol).all()
    assert ((r.logprobs.double() - (z.gather(1, tokens.long()) - lse[:, None])).abs() <= tol).all()


def test_steps_and_blocks_are_one_result(gpu):
    """More tokens than a block holds, with a list so long that blocks are short: the rows'
    results are those of calls on parts of them."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d, k, G = 50000, 3000, 32, 20, 128
    g = torch.Generator(device=gpu).manual_seed(4)
    Hh = torch.randn((T, d), generator=g, device=gpu).bfloat16()
    W = torch.randn((V, d), generator=g, device=gpu).bfloat16()
    tokens = torch.randint(-3, V, (T, G), generator=g, device=gpu, dtype=torch.int32)
    logq = torch.log_softmax(torch.randn((T, G), generator=g, device=gpu), 1) - 0.1
    r = nq.vocab_logprobs(Hh, W, tokens, k)
    loss, q = nq.vocab_distill(Hh, W, tokens, logq)
    for rows in (slice(0, 2000), slice(43000, 45000), slice(49000, T)):
        p = nq.vocab_logprobs(Hh[rows], W, tokens[rows], k)
        # (tiles of another size join the words in another order: lse to rounding, z the same)
        assert torch.equal(p.top_ids, r.top_ids[rows])
        assert (p.lse - r.lse[rows]).abs().max() <= 2 * (V + 64) * U
        assert (p.logprobs - r.logprobs[rows]).abs().max() <= 4 * (V + 64) * U
        l2, q2 = nq.vocab_distill(Hh[rows], W, tokens[rows], logq[rows])
        assert torch.equal(q2.hit, q.hit[rows])
        assert (l2 - loss[rows]).abs().max() <= 8 * (V + 64) * U


# ---------------------------------------------------------------- divergence

class Taught(Head):
    def __init__(self, seed, T, V, d, K, name, dev, scale=1.0, tail=True):
        super().__init__(seed, T, V, d, name, dev, scale)
        rng = self.rng
        ids = np.stack([rng.choice(V, K, replace=V < K) for _ in range(T)])
        logq = np.log(rng.dirichlet(np.ones(K + 1), T)[:, :K] + 1e-9)
        ids[rng.random((T, K)) < 0.1] = -1
        if T > 1:
            ids[rng.random(T) < 0.2] = -1
        self.K, self.tail = K, tail
        self.ids, self.logq = ints(ids, dev), put(logq, dev)
        self.dl = put(rng.standard_normal(T), dev)

    def loss(self, **kw):
        import sub_bit_weight_lb_amd as nq
        return nq.vocab_distill(self.H, self.W, self.ids, self.logq, scale=self.scale, tail=self.tail, **kw)

    def grad(self, q, **kw):
        import sub_bit_weight_lb_amd as nq
        return nq.vocab_distill_backward(self.H, self.W, self.ids, self.logq, q, self.dl, scale=self.scale,
                                         tail=self.tail, **kw)

    def exact(self):
        super().exact()
        self.i, self.lq = self.ids.cpu().numpy(), H64(self.logq)
        self.used = (self.i >= 0).any(1)
        self.q, _, self.r = O.teacher(self.i, self.lq, self.tail)
        return self

    def check_loss(self, loss, q):
        self.exact()
        want, lse, rest, hit = O.vocab_distill(H64(self.H), H64(self.W), self.i, self.lq, self.scale, self.tail)
        u = self.used
        less(np.abs(H64(q.lse) - lse)[u], self.elog[u])
        fin = np.isfinite(rest)
        assert np.array_equal(H64(q.rest)[~fin], rest[~fin])
        less(np.abs(H64(q.rest) - rest)[u & fin], (self.elog + 2 * U * np.abs(np.where(fin, rest, 0)))[u & fin])
        less(np.abs(H64(q.hit) - hit)[u], (self.ez + 2 * U * np.abs(self.z).max(1))[u, None])
        tol = (self.q.sum(1) + self.r) * (2 * self.elog + self.ez) + 4 * U * np.abs(want)
        less(np.abs(H64(loss) - want)[u], 1.01 * tol[u])
        for t in (loss, q.lse, q.rest, q.hit):
            assert (H64(t)[~u] == 0).all()

    def check_grad(self, dH, dW):
        self.exact()
        T, V, h, fp32 = self.T, self.V, half(self.name), self.name == "float32"
        Hh, W, dl = H64(self.H), H64(self.W), H64(self.dl)
        wantH, wantW, G = O.vocab_distill_backward(Hh, W, self.i, self.lq, dl, self.scale, self.tail)
        use = self.used
        f = np.abs(dl * self.scale)[use][:, None]
        p = np.exp(self.z - self.lse[:, None])[use]
        whole = (self.q.sum(1) + self.r)[use][:, None]
        # the exponent of p and of exp(z - rest) (r of it), off by z, lse or rest, and its own
        # rounding; exp by 4 units
        ee = (self.ezs[use] + 2 * self.elog[use][:, None]
              + 16 * U * (1 + np.abs(np.log(np.maximum(p, 1e-30)))))
        listed = np.zeros((T, V), bool)
        for t in range(T):
            listed[t, self.i[t][self.i[t] >= 0]] = True
        share = np.where(listed[use], whole * p, np.abs(whole * p) + np.abs(whole * p * f - G[use] * np.sign(
            dl * self.scale)[use][:, None]) / np.maximum(f, 1e-300))
        eg = share * (np.expm1(ee) + 8 * U) * f
        eg += (h + 8 * U) * np.abs(G[use])
        big = np.abs(dl[use]).max() if use.any() else 0.0
        if self.name != "bfloat16":   # (fp16's subnormals; fp32's second term, and the terms left out)
            eg += 2.0 ** -25 / 2 ** 15 * big * abs(self.scale) * 2
        more = 2.0 ** -22 if fp32 else 0.0
        mag = np.abs(G[use]) + eg
        tH = eg @ np.abs(W) + ((V + 40) * U + more) * (mag @ np.abs(W))
        tW = eg.T @ np.abs(Hh[use]) + ((T + 40) * U + more) * (mag.T @ np.abs(Hh[use]))
        if fp32:
            top = np.abs(G).max() if G.size else 0.0
            tH += V * 2.0 ** -38 * top * np.abs(W).max()
            tW += T * 2.0 ** -38 * top * np.abs(Hh).max()
        if dH is not None:
            less(np.abs(H64(dH) - wantH)[use], 1.01 * tH + h * np.abs(wantH[use]) + least(self.name))
            assert (H64(dH)[~use] == 0).all()
        if dW is not None:
            less(np.abs(H64(dW) - wantW), 1.01 * tW + h * np.abs(wantW) + least(self.name))


NEAR = [(1, 1, 1, 1), (1, 2, 7, 1), (2, 63, 64, 5), (16, 64, 130, 64), (17, 65, 8, 3), (33, 257, 515, 128),
        (64, 1000, 96, 20), (65, 500, 72, 100), (300, 1000, 64, 7), (257, 2049, 200, 33), (513, 300, 129, 128)]


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d, K", NEAR)
def test_divergence_and_gradient_match_oracle(gpu, name, T, V, d, K, tail):
    import torch
    print(f"case T={T} V={V} d={d} K={K} {name} tail={tail}", flush=True)
    L = Taught(T + V + d, T, V, d, K, name, gpu, 0.5 if T % 2 else 1.0, tail)
    loss, q = L.loss()
    L.check_loss(loss, q)
    dH, dW = L.grad(q)
    L.check_grad(dH, dW)
    l2, q2 = L.loss()
    h2, w2 = L.grad(q2)
    assert torch.equal(l2, loss) and torch.equal(q2.rest, q.rest) and torch.equal(q2.hit, q.hit)
    assert torch.equal(h2, dH) and torch.equal(w2, dW)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d, K", [(600, 4100, 200, 20), (600, 4100, 1100, 20), (1100, 12100, 300, 64),
                                        (70, 4100, 2052, 3), (40, 30011, 100, 50)])
def test_divergence_in_tiles_of_every_size(gpu, name, T, V, d, K):
    print(f"case T={T} V={V} d={d} K={K} {name}", flush=True)
    L = Taught(T + V + d, T, V, d, K, name, gpu)
    loss, q = L.loss()
    L.check_loss(loss, q)
    L.check_grad(*L.grad(q))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d, K", [(70, 4100, 800, 100), (300, 2049, 1100, 33), (513, 300, 900, 128),
                                        (65, 40, 768, 64), (129, 70000, 770, 5)])
def test_gradient_with_and_without_the_logits(gpu, name, T, V, d, K):
    """Logits that the loss kept, and computed again: the same bits of z, so gradients
    that differ by the rounding of its exponential alone."""
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} K={K} {name}", flush=True)
    L = Taught(T + V, T, V, d, K, name, gpu)
    loss, q = L.loss()
    assert q.logits.shape == (T, -(-V // 128) * 128)
    L.check_loss(loss, q)
    L.exact()
    less(np.abs(H64(q.logits)[L.used, :V] - L.z[L.used]), (L.ez + 2 * U * np.abs(L.z).max(1))[L.used, None])
    dH, dW = L.grad(q)
    L.check_grad(dH, dW)
    l2, bare = L.loss(keep=False)
    assert bare.logits is None and torch.equal(loss, l2)
    assert all(torch.equal(getattr(q, f), getattr(bare, f)) for f in ("lse", "rest", "hit"))
    L.check_grad(*L.grad(bare))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [9, 40, 140])
def test_divergence_of_views(gpu, name, T):
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d, K = 301, 77, 9
    L = Taught(3, T, V, d, K, name, gpu, 0.4)
    L.H, L.W, L.ids, L.logq = strided(L.H, 5, 1), strided(L.W, 2, 3), strided(L.ids, 4, 1), strided(L.logq, 1, 2)
    need = nq.vocab_distill_work_bytes(T, V, d, dt(name), K)
    guard = torch.full((need + 4096,), 255, dtype=torch.uint8, device=gpu)
    given = torch.full((T,), 77.0, device=gpu)
    state = nq.VocabDistill(torch.zeros(T, device=gpu), torch.zeros(T, device=gpu), torch.zeros(T, K, device=gpu))
    loss, q = L.loss(work=guard[:need], loss=given, state=state)
    assert loss is given and q is state and (guard[need:] == 255).all()
    L.check_loss(loss, q)
    dH, dW = strided(torch.zeros_like(L.H), 3, 1), strided(torch.zeros_like(L.W), 1, 1)
    need = nq.vocab_distill_work_bytes(T, V, d, dt(name), K, True)
    guard = torch.full((need + 4096,), 255, dtype=torch.uint8, device=gpu)
    L.grad(q, dH=dH, dW=dW, work=guard[:need])
    assert (guard[need:] == 255).all()
    L.check_grad(dH, dW)
    for t, extra in ((dH, 3), (dW, 1)):
        gap = t.as_strided((t.shape[0], extra), (d + extra, 1), 1 + d)[:-1]
        assert (gap == 77).all()
    a, none = L.grad(q, want_dW=False)
    assert none is None and torch.equal(a, dH)
    none, b = L.grad(q, want_dH=False)
    assert none is None and torch.equal(b, dW)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("T", [5, 70])
def test_words_listed_twice_and_whole_vocabularies(gpu, T, tail):
    """A word's entries add up; with every word listed there is no rest; entries of no
    probability; one entry with all of it."""
    import torch
    V, d, K = 40, 32, 64
    L = Taught(9, T, V, d, K, "float32", gpu, 1.0, tail)
    ids = np.full((T, K), -1)
    lq = np.full((T, K), -np.inf)
    rng = np.random.default_rng(0)
    ids[0, :V], lq[0, :V] = rng.permutation(V), np.log(rng.dirichlet(np.ones(V)))      # every word
    ids[1, :] = rng.integers(0, 5, K)                                                   # five words, many times
    lq[1, :] = np.log(rng.dirichlet(np.ones(K + 3))[:K])
    ids[2, 3], lq[2, 3] = 17, 0.0                                                       # certain
    ids[3, :4], lq[3, 0] = [1, 2, 3, 2], np.log(0.6)                                    # words of no probability
    ids[4, 60:64], lq[4, 60:64] = [39, 0, 39, 39], np.log([0.1, 0.2, 0.3, 0.1])
    L.ids, L.logq = ints(ids, gpu), put(lq, gpu)
    loss, q = L.loss()
    L.check_loss(loss, q)
    if tail:
        assert q.rest[0] == -float("inf")
    L.check_grad(*L.grad(q))


@pytest.mark.parametrize("T", [8, 130])
@pytest.mark.parametrize("name", TYPES)
def test_ignored_tokens_may_hold_anything(gpu, name, T):
    import torch
    L = Taught(4, T, 200, 72, 6, name, gpu)
    L.ids[::3] = -1
    off = (L.ids < 0).all(1)
    loss, q = L.loss()
    grads = L.grad(q)
    L.H[off], L.logq[off], L.dl[off] = float("nan"), float("nan"), float("inf")
    L.logq[L.ids < 0] = float("nan")
    l2, q2 = L.loss()
    assert torch.equal(loss, l2) and (l2[off] == 0).all()
    for f in ("lse", "rest", "hit"):
        assert torch.equal(getattr(q, f), getattr(q2, f))
    q2.lse[off] = q2.rest[off] = float("nan")
    q2.hit[L.ids < 0] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip(grads, L.grad(q2)))
    L.ids.fill_(-1)
    loss, q = L.loss()
    dH, dW = L.grad(q)
    assert all((t == 0).all() for t in (loss, q.lse, q.rest, q.hit, dH, dW))


@pytest.mark.parametrize("T", [8, 130])
def test_words_past_the_vocabulary_and_rows_that_are_not_finite(gpu, T):
    import torch
    L = Taught(6, T, 200, 64, 5, "bfloat16", gpu)
    L.ids[:6, 0] = 3
    ok, _ = L.loss()
    L.ids[1, 4] = 200
    L.H[3, 5] = float("inf")
    L.logq[4, 0] = float("nan")
    loss, q = L.loss()
    bad = [1, 3, 4]
    rest = [t for t in range(T) if t not in bad]
    assert loss[bad].isnan().all() and torch.isfinite(q.lse[1]) and q.hit[1, 4].isnan() and q.lse[3].isnan()
    assert torch.equal(loss[rest], ok[rest])
    dH, dW = L.grad(q)
    assert dH[bad].isnan().all() and dW.isnan().all() and torch.isfinite(dH[rest]).all()


@pytest.mark.parametrize("name", TYPES)
def test_upstream_gradients_of_any_size(gpu, name):
    L = Taught(8, 70, 400, 64, 10, name, gpu)
    _, q = L.loss()
    keep = L.dl.clone()
    for f in (0.0, 2.0 ** -20, 1e3):
        L.dl = keep * f
        L.check_grad(*L.grad(q))
    L.dl = keep.clone()
    L.dl[::2] *= 1e-4
    L.check_grad(*L.grad(q))


@pytest.mark.parametrize("T", [4, 70])
def test_a_rest_that_is_next_to_nothing(gpu, T):
    """The listed words hold all but 2^-40 of the student's mass and half of the
    teacher's: rest is a sum of its own, and the divergence and its gradient are large."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d = 1500, 64
    for name in TYPES:
        L = Taught(10, T, V, d, 2, name, gpu)
        W = torch.randn((V, d), generator=torch.Generator(device=gpu).manual_seed(1), device=gpu) * 0.01
        W[5, 0], W[800, 0] = 4.0, 3.75
        Hh = torch.randn((T, d), generator=torch.Generator(device=gpu).manual_seed(2), device=gpu)
        Hh[:, 0] = 9.0
        L.H, L.W = Hh.to(dt(name)), W.to(dt(name))
        L.ids = torch.tensor([[5, 800]] * T, dtype=torch.int32, device=gpu)
        L.logq = torch.full((T, 2), float(np.log(0.25)), device=gpu)
        loss, q = L.loss()
        L.check_loss(loss, q)
        assert (H64(q.rest) - H64(q.lse) < -20).all() and (loss > 10).all()
        L.check_grad(*L.grad(q))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T, V, d", [(1, 5000, 4100), (3, 70000, 64), (7, 333, 8), (16, 900, 1000), (19, 2100, 130),
                                     (32, 4099, 515)])
def test_gradient_of_few_tokens(gpu, name, T, V, d):
    """With the loss's logits and without them; slices of the words, columns and words
    past whole blocks, one output alone."""
    import torch
    import sub_bit_weight_lb_amd as nq
    print(f"case T={T} V={V} d={d} {name}", flush=True)
    L = Taught(T + V, T, V, d, 17, name, gpu)
    loss, q = L.loss()
    assert q.logits.shape == (T, -(-V // 128) * 128)
    L.check_loss(loss, q)
    dH, dW = L.grad(q)
    L.check_grad(dH, dW)
    bare = nq.VocabDistill(q.lse, q.rest, q.hit)
    l2, _ = L.loss(state=bare)
    assert torch.equal(loss, l2)
    assert all(torch.equal(a, b) for a, b in zip((dH, dW), L.grad(bare)))
    assert torch.equal(L.grad(q, want_dW=False)[0], dH) and torch.equal(L.grad(q, want_dH=False)[1], dW)


@pytest.mark.parametrize("name, T, keep", [("bfloat16", 40, True), ("bfloat16", 40, False), ("float16", 200, True),
                                           ("float32", 70, True), ("float32", 70, False), ("float32", 5, True)])
def test_several_pieces_of_the_vocabulary(gpu, name, T, keep):
    """A hidden size so large that W is copied and taken in pieces: against float64 on
    the GPU."""
    import torch
    V, d, K = 5000, 33001, 30
    L = Taught(11, T, V, d, K, name, gpu)
    loss, q = L.loss(keep=keep)
    assert (q.logits is None) == (not keep)
    dH, dW = L.grad(q)
    z = torch.mm(L.H.double(), L.W.double().t())
    more = 2.0 ** -22 if name == "float32" else 0.0
    zb = ((d + 2) * U + more) * float(torch.mm(L.H.double().abs(), L.W.double().abs().t()).max())
    h = half(name)
    ids = L.ids.long()
    on = ids >= 0
    used = on.any(1)
    qk = torch.where(on, torch.exp(L.logq.double()), 0.0)
    r = (1 - qk.sum(1)).clamp(min=0)
    at = torch.where(on, ids, V)
    inside = torch.zeros((T, V + 1), dtype=torch.bool, device=gpu).scatter_(1, at, True)[:, :V]
    target = torch.zeros((T, V + 1), dtype=torch.float64, device=gpu).scatter_add_(1, at, qk)[:, :V]
    rest = torch.logsumexp(z.masked_fill(inside, -float("inf")), 1)
    tol = 2 * zb + 2 * (V + 64) * U
    assert ((q.lse.double() - torch.logsumexp(z, 1)).abs()[used] <= tol).all()
    assert ((q.rest.double() - rest).abs()[used] <= tol).all()
    assert ((q.hit.double() - torch.where(on, z.gather(1, ids.clamp(min=0)), 0.0)).abs() <= tol).all()
    G = (qk.sum(1) + r).unsqueeze(1) * torch.softmax(z, 1) - target
    part = r.unsqueeze(1) * torch.softmax(z.masked_fill(inside, -float("inf")), 1)
    f = (L.dl.double() * used).unsqueeze(1)
    mag = ((qk.sum(1) + r).unsqueeze(1) * torch.softmax(z, 1) + target + part) * f.abs()
    G = (G - part) * f
    # (G's rounding, or its second term's end)
    rel = h + 2.0 ** -21 + more + float(np.expm1(3 * tol)) + (V + 64) * U
    for got, ref, m in ((dH, torch.mm(G, L.W.double()), torch.mm(mag, L.W.double().abs())),
                        (dW, torch.mm(G.t().contiguous(), L.H.double()),
                         torch.mm(mag.t().contiguous(), L.H.double().abs()))):
        assert ((got.double() - ref).abs() <= rel * m + h * ref.abs() + V * 2.0 ** -38 + least(name)).all()


# ---------------------------------------------------------------- together

def packed(seed, m, n, r, dev):
    from oracle.lbadmm import pack_signs
    import torch
    import sub_bit_weight_lb_amd as nq
    rng = np.random.default_rng(seed)
    SU, SV = (np.where(rng.random(s) < 0.5, -1.0, 1.0) for s in ((m, r), (n, r)))
    U_, V_ = (torch.from_numpy(pack_signs(x).view(np.int32)).to(dev) for x in (SU, SV))
    return SU, SV, U_, V_, nq.transpose_signs(U_, m, r), nq.transpose_signs(V_, n, r)


def test_a_packed_layer_is_tuned_towards_its_model(gpu):
    """The original layer's best words are written down, the packed layer's divergence from
    them and its scales' gradient follow: against the float64 formulas, and those against
    central differences."""
    import torch
    import sub_bit_weight_lb_amd as nq
    from oracle import tuning as OT
    rng = np.random.default_rng(12)
    T, n, m, r, V, K, tau = 90, 96, 128, 64, 500, 24, 2.0
    SU, SV, Ub, Vb, Ut, Vt = packed(13, m, n, r, gpu)
    s1, s2 = put(rng.uniform(0.02, 0.06, m), gpu), put(rng.uniform(0.5, 1.5, n), gpu)
    head = put(rng.standard_normal((V, m)) / np.sqrt(m), gpu)
    X = put(rng.standard_normal((T, n)), gpu)
    q8 = nq.act8_quantize(X)
    x = nq.act8_dequantize(q8)
    layer = put(rng.standard_normal((m, n)) / np.sqrt(n), gpu)         # the original
    taught = nq.vocab_logprobs((x.double() @ layer.double().t()).float(), head, k=K, scale=1 / tau)
    assert (torch.exp(taught.top_logprobs).sum(1) < 1).all()
    Y = nq.binary_matmul(Ub, Vt, s1, s2, x, r)
    loss, state = nq.vocab_distill(Y, head, taught.top_ids, taught.top_logprobs, scale=1 / tau)
    dl = torch.full((T,), tau * tau / T, device=gpu)
    dY, _ = nq.vocab_distill_backward(Y, head, taught.top_ids, taught.top_logprobs, state, dl, scale=1 / tau)
    got = nq.binary_matmul_backward(Ub, Ut, Vb, Vt, s1, s2, q8, dY, r)
    ids, lq, x64, W64, dl64 = taught.top_ids.cpu().numpy(), H64(taught.top_logprobs), H64(x), H64(head), H64(dl)

    def forward(a1, a2):
        y = a1 * (((x64 * a2) @ SV) @ SU.T)
        return y, (dl64 * O.vocab_distill(y, W64, ids, lq, 1 / tau)[0]).sum()

    a1, a2 = H64(s1), H64(s2)
    y, total = forward(a1, a2)
    want = OT.layer_backward(SU, SV, a1, a2, x64, O.vocab_distill_backward(y, W64, ids, lq, dl64, 1 / tau)[0])
    assert abs(float((dl * loss).sum()) - total) <= 1e-5 * abs(total)
    for a, b in zip(got, want):
        assert np.linalg.norm(H64(a) - b) <= 1e-4 * np.linalg.norm(b)
    v, h = [rng.standard_normal(t.shape) for t in (a1, a2)], 1e-6
    slope = sum((g * d).sum() for g, d in zip(want[1:], v))
    up, dn = (forward(a1 + s * h * v[0], a2 + s * h * v[1])[1] for s in (1, -1))
    assert abs((up - dn) / (2 * h) - slope) <= 1e-4 * (1 + abs(slope))
    # nothing to learn from itself: the divergence is 0 and its gradient what rounding leaves
    own = nq.vocab_logprobs(Y, head, k=K, scale=1 / tau)
    zero, st = nq.vocab_distill(Y, head, own.top_ids, own.top_logprobs, scale=1 / tau)
    assert zero.abs().max() <= 64 * U
    d0, _ = nq.vocab_distill_backward(Y, head, own.top_ids, own.top_logprobs, st, dl, scale=1 / tau)
    assert float(d0.norm()) <= 1e-4 * float(dY.norm())


@pytest.mark.parametrize("T", [6, 150])
def test_captured_passes_replay(gpu, T):
    """Log probabilities, divergence and gradient in two graphs that share a workspace:
    every replay equals the eager result, with eager work in between."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d, K = 9000, 128, 12
    L = Taught(21, T, V, d, K, "bfloat16", gpu)
    work = torch.empty(max(nq.vocab_logprobs_work_bytes(T, V, d, torch.bfloat16, K, K),
                           nq.vocab_distill_work_bytes(T, V, d, torch.bfloat16, K),
                           nq.vocab_distill_work_bytes(T, V, d, torch.bfloat16, K, True)),
                       dtype=torch.uint8, device=gpu)

    def run():
        p = nq.vocab_logprobs(L.H, L.W, L.ids, K, work=work)
        loss, q = nq.vocab_distill(L.H, L.W, p.top_ids, L.logq, work=work)
        dH, dW = nq.vocab_distill_backward(L.H, L.W, p.top_ids, L.logq, q, L.dl, work=work)
        return p.logprobs, p.entropy, p.top_ids, p.top_logprobs, loss, q.rest, q.hit, dH, dW

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for k in range(3):
        gen = torch.Generator(device=gpu).manual_seed(k)
        L.H.copy_(torch.randn(L.H.shape, generator=gen, device=gpu))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_calls_on_other_streams(gpu):
    """Two streams at once, and a stream given by its handle while the current one takes
    and fills memory that the calls have let go."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d, K = 200, 9000, 128, 20
    L = Taught(32, T, V, d, K, "float16", gpu)

    def run(**kw):
        p = nq.vocab_logprobs(L.H, L.W, L.ids, K, **kw)
        loss, q = L.loss(**kw)
        return (p.logprobs, p.top_ids, p.top_logprobs, loss, q.rest, *L.grad(q, **kw))

    want = run()
    sizes = [nq.vocab_logprobs_work_bytes(T, V, d, torch.float16, K, K)]
    sizes += [nq.vocab_distill_work_bytes(T, V, d, torch.float16, K, g) for g in (False, True)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for _ in range(3):
        got.append(run(stream=streams[0].cuda_stream))
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=gpu).fill_(255)
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---------------------------------------------------------------- ends of the ranges

@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T", [3, 70, 300])
def test_a_scale_of_zero(gpu, name, T):
    """All logits 0: p = 1 / V, the lowest words first, no gradient."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d, K = 5003, 72, 9
    L = Taught(41, T, V, d, K, name, gpu, scale=0.0)
    r = nq.vocab_logprobs(L.H, L.W, L.ids, K, scale=0.0)
    # (V terms of 1: exact; log rounds by an ulp of 8.5 at most, and is exact to 4 u elsewhere)
    tol = 4 * U * np.log(V)
    assert (np.abs(H64(r.lse) - np.log(V)) <= tol).all() and (np.abs(H64(r.entropy) - np.log(V)) <= tol).all()
    assert (r.top_ids == torch.arange(K, device=gpu, dtype=torch.int32)).all()
    assert (np.abs(H64(r.top_logprobs) + np.log(V)) <= 2 * tol).all()
    loss, q = L.loss()
    dH, dW = L.grad(q)
    assert (q.hit == 0).all() and (dH == 0).all() and (dW == 0).all()


def softmaxed(z, ids, logq):
    """Divergence without a tail and its gradient by z, in float64 on the GPU."""
    import torch
    lse = torch.logsumexp(z, 1, keepdim=True)
    lq = torch.log_softmax(logq.double(), 1)
    loss = (lq.exp() * (lq - z.gather(1, ids.long()) + lse)).sum(1)
    return loss, lse[:, 0], torch.exp(z - lse).scatter_add_(1, ids.long(), -lq.exp())


@pytest.mark.parametrize("name", ["bfloat16", "float32"])
def test_very_many_tokens(gpu, name):
    """More tokens than the second axis of a grid holds."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d, K = 100001, 130, 24, 5
    g = torch.Generator(device=gpu).manual_seed(5)
    Hh = torch.randn((T, d), generator=g, device=gpu).to(dt(name))
    W = torch.randn((V, d), generator=g, device=gpu).to(dt(name))
    ids = torch.randint(0, V, (T, K), generator=g, device=gpu, dtype=torch.int32)
    logq = torch.randn((T, K), generator=g, device=gpu)
    dl = torch.randn(T, generator=g, device=gpu)
    z = Hh.double() @ W.double().t()
    loss, lse, G = softmaxed(z, ids, logq)
    more = 2.0 ** -22 if name == "float32" else 0.0
    zb = ((d + 2) * U + more) * float((Hh.double().abs() @ W.double().abs().t()).max()) + 2 * U * float(z.abs().max())
    tol = 2 * zb + 2 * (V + 64) * U + 4 * U * float(loss.abs().max())
    r = nq.vocab_logprobs(Hh, W, ids, K)
    assert ((r.lse.double() - lse).abs() <= tol).all()
    assert ((r.logprobs.double() - (z.gather(1, ids.long()) - lse[:, None])).abs() <= tol).all()
    best = torch.topk(z, K, 1).values
    assert ((z.gather(1, r.top_ids.long()) - best).abs() <= 2 * zb).all()
    got, q = nq.vocab_distill(Hh, W, ids, logq, tail=False)
    assert ((got.double() - loss).abs() <= tol).all()
    dH, dW = nq.vocab_distill_backward(Hh, W, ids, logq, q, dl, tail=False)
    G *= dl.double()[:, None]
    mag = G.abs() + torch.exp(z - lse[:, None]) * dl.double().abs()[:, None]
    h = half(name)
    for out, ref, m, n in ((dH, G @ W.double(), mag @ W.double().abs(), V),
                           (dW, G.t() @ Hh.double(), mag.t() @ Hh.double().abs(), T)):
        rel = h + more + float(np.expm1(3 * tol)) + (n + 64) * U
        assert ((out.double() - ref).abs() <= rel * m + h * ref.abs() + n * 2.0 ** -38 + least(name)).all()


@pytest.mark.parametrize("T", [3, 70])
def test_a_vocabulary_past_32_bits(gpu, T):
    """W of more than 2^32 bytes: the last words and columns."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, d, K = 140001, 16384, 4
    assert 2 * V * d > 1 << 32
    g = torch.Generator(device=gpu).manual_seed(6)
    W = torch.empty((V, d), dtype=torch.bfloat16, device=gpu)
    W.normal_(0.0, 1 / 64, generator=g)
    Hh = torch.randn((T, d), generator=g, device=gpu).bfloat16()
    z = torch.cat([Hh.double() @ W[a:a + 20000].double().t() for a in range(0, V, 20000)], 1)
    ids = torch.cat([torch.randint(0, V, (T, K - 1), generator=g, device=gpu, dtype=torch.int32),
                     torch.full((T, 1), V - 1, dtype=torch.int32, device=gpu)], 1)
    logq = torch.randn((T, K), generator=g, device=gpu)
    dl = torch.randn(T, generator=g, device=gpu)
    loss, lse, G = softmaxed(z, ids, logq)
    size = max(float((Hh.double().abs() @ W[a:a + 20000].double().abs().t()).max()) for a in range(0, V, 20000))
    zb = (d + 2) * U * size
    tol = 2 * zb + 2 * (V + 64) * U
    r = nq.vocab_logprobs(Hh, W, ids, K)
    assert ((r.lse.double() - lse).abs() <= tol).all()
    assert ((r.logprobs.double() - (z.gather(1, ids.long()) - lse[:, None])).abs() <= tol).all()
    assert ((z.gather(1, r.top_ids.long()) - torch.topk(z, K, 1).values).abs() <= 2 * zb).all()
    got, q = nq.vocab_distill(Hh, W, ids, logq, tail=False)
    assert ((got.double() - loss).abs() <= tol).all()
    dH, dW = nq.vocab_distill_backward(Hh, W, ids, logq, q, dl, tail=False)
    G *= dl.double()[:, None]
    mag = G.abs() + torch.exp(z - lse[:, None]) * dl.double().abs()[:, None]
    h = half("bfloat16")
    rel = h + float(np.expm1(3 * tol)) + (V + 64) * U
    cols = torch.cat([torch.arange(64, device=gpu), torch.arange(d - 64, d, device=gpu)])
    near = W[:, cols].double()
    assert ((dH[:, cols].double() - G @ near).abs() <= rel * (mag @ near.abs()) + h * (G @ near).abs()).all()
    for rows in (slice(0, 200), slice(V - 200, V)):
        ref, m = G[:, rows].t() @ Hh.double(), mag[:, rows].t() @ Hh.double().abs()
        assert ((dW[rows].double() - ref).abs() <= rel * m + h * ref.abs() + least("bfloat16")).all()


def test_kept_logits_past_31_bits(gpu):
    """Kept logits of more than 2^31 bytes, in several pieces for the gradient."""
    import torch
    import sub_bit_weight_lb_amd as nq
    T, V, d, K = 4100, 140001, 1024, 3
    g = torch.Generator(device=gpu).manual_seed(7)
    W = torch.randn((V, d), generator=g, device=gpu).mul_(1 / 16).bfloat16()
    Hh = torch.randn((T, d), generator=g, device=gpu).bfloat16()
    ids = torch.randint(0, V, (T, K), generator=g, device=gpu, dtype=torch.int32)
    logq = torch.randn((T, K), generator=g, device=gpu)
    dl = torch.randn(T, generator=g, device=gpu)
    got, q = nq.vocab_distill(Hh, W, ids, logq, tail=False)
    assert q.logits is not None and 4 * q.logits.numel() > 1 << 31
    dH, dW = nq.vocab_distill_backward(Hh, W, ids, logq, q, dl, tail=False)
    z = Hh.double() @ W.double().t()
    loss, lse, G = softmaxed(z, ids, logq)
    zb = (d + 2) * U * float((Hh[:256].double().abs() @ W.double().abs().t()).max()) * 1.5
    tol = 2 * zb + 2 * (V + 64) * U
    assert ((got.double() - loss).abs() <= tol).all()
    G *= dl.double()[:, None]
    mag = torch.exp(z - lse[:, None]).mul_(dl.double().abs()[:, None]).add_(G.abs())
    h = half("bfloat16")
    rel = h + float(np.expm1(3 * tol)) + (V + 64) * U
    w, x = W.double(), Hh.double()
    assert ((dH.double() - G @ w).abs() <= rel * (mag @ w.abs()) + h * (G @ w).abs()).all()
    for rows in (slice(0, 300), slice(V // 2, V // 2 + 300), slice(V - 300, V)):
        ref, m = G[:, rows].t() @ x, mag[:, rows].t() @ x.abs()
        assert ((dW[rows].double() - ref).abs() <= rel * m + h * ref.abs() + least("bfloat16")).all()


@pytest.mark.parametrize("T", [5, 140])
def test_lists_with_entries_of_no_mass(gpu, T):
    """Log probabilities of -infinity: in a part of a list they add nothing; as all of it they
    leave the rest alone (with a tail) or no softmax (without)."""
    import torch
    V, d, K = 700, 40, 6
    for tail in (True, False):
        L = Taught(43, T, V, d, K, "float32", gpu, tail=tail)
        L.logq[:, 1::2] = -float("inf")
        L.logq[2] = -float("inf")
        ids = L.ids.cpu().numpy()
        loss, q = L.loss()
        dH, dW = L.grad(q)
        z = H64(L.H) @ H64(L.W).T
        lse = O.lse_of(z)
        if tail:
            rest = np.array([O.lse_of(np.delete(z[t], np.unique(ids[t][ids[t] >= 0]))[None])[0] for t in range(T)])
            # (z's sums of 40 products, lse, rest: (d + 2) u |h| |w|, (V + 64) u of each sum)
            tol = 4 * ((d + 2) * U + 2.0 ** -22) * (np.abs(H64(L.H)) @ np.abs(H64(L.W)).T).max() + 2 * (V + 64) * U
            if (ids[2] >= 0).any():
                assert abs(float(loss[2]) - (lse[2] - rest[2])) <= tol
            assert torch.isfinite(loss).all() and torch.isfinite(dH).all() and torch.isfinite(dW).all()
        else:
            some = torch.arange(T, device=gpu) != 2
            assert (ids[2] < 0).all() or (loss[2].isnan() and dH[2].isnan().all())
            assert torch.isfinite(loss[some]).all() and torch.isfinite(dH[some]).all()


@pytest.mark.parametrize("name", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [7, 90, 700])
@pytest.mark.parametrize("V", [128, 129, 700, 1000, 1700, 2100, 3000, 3300, 6000, 9000, 33000])
def test_best_words_of_short_and_long_vocabularies(gpu, name, T, V):
    """128 and 100 best words where the vocabulary has fewer parts than that, about as many, and
    more: words, single parts and four parts at a time bound them. Logits on a grid, exact in any
    order of summing."""
    import torch
    import sub_bit_weight_lb_amd as nq
    g = torch.Generator(device=gpu).manual_seed(V)
    W = torch.randint(-3, 4, (V, 64), generator=g, device=gpu).float()
    Hh = torch.randint(-3, 4, (T, 64), generator=g, device=gpu).float() / 8
    Hh[0] = 0
    z = torch.mm(Hh.double(), W.double().t())
    best, ids = torch.sort(z, dim=1, descending=True, stable=True)
    for k in (100, 128):
        r = nq.vocab_logprobs(Hh.to(dt(name)), W.to(dt(name)), k=k)
        assert torch.equal(r.top_ids.long(), ids[:, :k])
        want = best[:, :k] - torch.logsumexp(z, 1)[:, None]
        assert ((r.top_logprobs.double() - want).abs() <= (V + 64) * U + 8 * U * best.abs().max()).all()


@pytest.mark.parametrize("name", ["bfloat16", "float16"])
@pytest.mark.parametrize("T", [1, 4, 17, 32])
@pytest.mark.parametrize("d, lead", [(8, 1), (9, 0), (33, 1), (333, 0), (514, 1), (515, 1)])
def test_rows_at_odd_addresses(gpu, name, T, d, lead):
    """Rows of W and H at every address that 16-bit values can have: the results are those of
    aligned copies."""
    import torch
    import sub_bit_weight_lb_amd as nq
    V, K = 777, 9
    L = Taught(61, T, V, d, K, name, gpu)
    pad = 8 - d % 8
    H1, W1 = (strided(x, pad) for x in (L.H, L.W))
    want = nq.vocab_logprobs(H1, W1, L.ids, K)
    loss, q = nq.vocab_distill(H1, W1, L.ids, L.logq)
    for h, w in ((strided(L.H, 0, lead), strided(L.W, 0, lead)), (strided(L.H, 1, 1), W1), (H1, strided(L.W, 1, 1)),
                 (strided(L.H, 2, 1), strided(L.W, 3, 2))):
        r = nq.vocab_logprobs(h, w, L.ids, K)
        assert all(torch.equal(getattr(r, f), getattr(want, f)) for f in ("logprobs", "lse", "entropy", "top_ids"))
        l2, q2 = nq.vocab_distill(h, w, L.ids, L.logq)
        assert torch.equal(l2, loss) and torch.equal(q2.hit, q.hit)
