"""Cases of the operators that score a packed model and tune it towards the
model it was made from: log probabilities with their entropy and the best
alternatives, and the divergence from a teacher's top words with its gradient.
`run` computes them in plain torch, or with `own` set through
sub_bit_weight_lb_amd. Logits are z = scale H W^T throughout.

  logprobs      vocab_logprobs: lse_t = log sum_v exp z_tv; z - lse of the
                tokens that are given per row (0 where one is negative: none);
                the entropy of softmax(z_t); the k largest z with their words,
                the lower word first where two are equal.
  distill       vocab_distill: KL(q || p) of p = softmax(z_t) from a teacher's
                K words (a negative one: no entry; a row without any is
                ignored) and their log probabilities. With `tail` the rest of
                the teacher's mass r = 1 - sum q is one outcome more, of
                probability exp(rest - lse) for the student, rest = log sum
                exp z over the words that are not listed; without, q is
                normalised over the row's entries.
  distill_grad  vocab_distill and vocab_distill_backward: the loss, then dH
                and dW of sum_t dloss_t loss_t.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # a small head and a handful of tokens: latency alone
        dict(name="logprobs-small", op="logprobs", tokens=5, vocab=1003, d=256, given=1, k=3, type="fp32"),
        # one generated token with its alternatives: W is the traffic
        dict(name="logprobs-token", op="logprobs", tokens=1, vocab=32000, d=4096, given=1, k=20, type="bf16"),
        # multiple-choice questions: four answers' log probabilities at each ragged question's end
        dict(name="logprobs-choices", op="logprobs", tokens=509, vocab=50021, d=1000, given=4, k=5, type="fp16"),
        # the original model's top words over two 2048-token samples, to tune its packed form by
        dict(name="logprobs-teacher", op="logprobs", tokens=4096, vocab=131072, d=4096, given=1, k=64, type="bf16"),
        # a prompt's last tokens against a teacher
        dict(name="distill-tokens", op="distill", tokens=7, vocab=32000, d=4096, k=20, tail=True, type="bf16"),
        # a ragged batch, odd vocabulary, a long list
        dict(name="distill-odd", op="distill", tokens=777, vocab=50021, d=1000, k=100, tail=True, type="fp16"),
        # an fp32 head against a list that is taken for the whole distribution
        dict(name="distill-fp32", op="distill", tokens=512, vocab=32000, d=2048, k=32, tail=False, type="fp32"),
        # one token's step: W is read, dW written
        dict(name="grad-token", op="distill_grad", tokens=1, vocab=32000, d=4096, k=20, tail=True, type="bf16"),
        # a short ragged batch with rows of W that are not 16-byte aligned
        dict(name="grad-odd", op="distill_grad", tokens=301, vocab=4999, d=515, k=33, tail=True, type="fp16"),
        # an fp32 head in training
        dict(name="grad-fp32", op="distill_grad", tokens=1024, vocab=32000, d=2048, k=64, tail=False, type="fp32"),
        # two 2048-token samples, a 131072-word vocabulary
        dict(name="grad-large", op="distill_grad", tokens=4096, vocab=131072, d=4096, k=64, tail=True, type="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["logprobs", "distill", "distill_grad"])
    kind = rng.choice(["fp32", "bf16", "fp16"])
    vocab, d = _log_uniform(rng, 500, 131072), _log_uniform(rng, 64, 8192)
    d = d if rng.random() < 0.3 else max(64, d // 64 * 64)
    # (an fp32 head costs several times a bf16 one)
    most = (1 << 41) // (vocab * d) // (8 if kind == "fp32" else 2)
    case = dict(op=op, tokens=_log_uniform(rng, 1, max(1, min(8192, most))), vocab=vocab, d=d,
                k=_log_uniform(rng, 1, 128), type=kind)
    if op == "logprobs":
        return dict(case, given=rng.randint(1, 8))
    return dict(case, tail=rng.random() < 0.7)


# ---------------------------------------------------------------- inputs

def _grid(x, step):
    """x in 8 bits of a step that is a power of two. Every order of summing
    gives the same logits of such values, and so the same best words."""
    return (x / step).round().clamp(-127, 127) * step


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    t = TYPES[case["type"]]
    T, V, d, k = case["tokens"], case["vocab"], case["d"], case["k"]
    W = 0.02 * torch.randn(V, d, generator=gen, device=DEV)
    H = torch.randn(T, d, generator=gen, device=DEV)
    lean = 10.0 / (0.0004 * d)
    if case["op"] == "logprobs":
        # hidden states and a head that were kept in 8 bits; half of the tokens are predicted well
        W = _grid(W, 2.0 ** -11)
        tokens = torch.randint(0, V, (T, case["given"]), generator=gen, device=DEV)
        sure = (torch.rand(T, 1, generator=gen, device=DEV) < 0.5) * lean
        H = _grid(H + sure * W[tokens[:, 0]], 2.0 ** -4)
        if T > 1:  # some have fewer answers
            tokens = torch.where(torch.rand(tokens.shape, generator=gen, device=DEV) < 0.12, -1, tokens)
        return dict(case=case, H=H.to(t), W=W.to(t), tokens=tokens.to(torch.int32), scale=1.0)
    # a teacher's distinct words, probabilities that fall with the rank, 1 % to 30 % of its mass elsewhere
    gaps = torch.randint(1, max(2, V // k), (T, k), generator=gen, device=DEV)
    ids = gaps.cumsum(1) - 1
    ids = ids.gather(1, torch.rand(T, k, generator=gen, device=DEV).argsort(1))
    rank = torch.arange(1, k + 1, device=DEV)
    steep = 0.5 + 1.5 * torch.rand(T, 1, generator=gen, device=DEV)
    logits = -steep * torch.log(rank) + 0.2 * torch.randn(T, k, generator=gen, device=DEV)
    mass = 0.7 + 0.29 * torch.rand(T, 1, generator=gen, device=DEV)
    share = torch.exp(logits) / torch.exp(logits).sum(1, keepdim=True)
    logq = torch.log(mass * share)
    # a student that leans to the same words, not as far, at a temperature of 2
    for j in range(k):
        H += (1.5 * lean * share[:, j:j + 1].sqrt() * torch.rand(T, 1, generator=gen, device=DEV)) * W[ids[:, j]]
    if T > 1:  # some lists are shorter; some tokens are padding or a prompt
        ids = torch.where((torch.rand(T, 1, generator=gen, device=DEV) < 0.1) & (rank > (k + 1) // 2), -1, ids)
        ids = torch.where(torch.rand(T, 1, generator=gen, device=DEV) < 0.12, -1, ids)
    used = (ids >= 0).any(1).float()
    return dict(case=case, H=H.to(t), W=W.to(t), ids=ids.to(torch.int32), logq=logq, scale=0.5,
                dloss=used / used.sum().clamp(min=1.0))


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import sub_bit_weight_lb_amd as nq
    case = s["case"]
    if case["op"] == "logprobs":
        r = nq.vocab_logprobs(s["H"], s["W"], s["tokens"], case["k"], scale=s["scale"])
        return dict(logprobs=r.logprobs, entropy=r.entropy, lse=r.lse, top_ids=r.top_ids,
                    top_logprobs=r.top_logprobs)
    loss, q = nq.vocab_distill(s["H"], s["W"], s["ids"], s["logq"], scale=s["scale"], tail=case["tail"])
    out = dict(loss=loss, lse=q.lse, rest=q.rest, hit=q.hit)
    if case["op"] == "distill":
        return out
    dH, dW = nq.vocab_distill_backward(s["H"], s["W"], s["ids"], s["logq"], q, s["dloss"],
                                       scale=s["scale"], tail=case["tail"])
    return dict(out, dH=dH, dW=dW)


def _lse(z):
    top = z.amax(1, keepdim=True)
    return torch.log(torch.exp(z - top).sum(1)) + top[:, 0]


def _plain(s):
    case, scale = s["case"], s["scale"]
    H, W = s["H"].float(), s["W"].float()
    z = scale * (H @ W.t()) + 0.0  # (no zero below zero)
    lse = _lse(z)
    if case["op"] == "logprobs":
        tokens = s["tokens"].long()
        logprobs = z.gather(1, tokens.clamp(min=0)) - lse.unsqueeze(1)
        logprobs = torch.where(tokens >= 0, logprobs, torch.zeros_like(logprobs))
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - top)
        total = e.sum(1)
        entropy = torch.log(total) - (e * (z - top)).sum(1) / total
        del e
        # the order of z, and the lower word first among equals, in one integer
        bits = z.view(torch.int32)
        bits = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
        word = z.shape[1] - 1 - torch.arange(z.shape[1], device=z.device)
        best = torch.topk((bits << 32) + word, case["k"], dim=1).values
        ids = z.shape[1] - 1 - (best & 0xffffffff)
        return dict(logprobs=logprobs, entropy=entropy, lse=lse, top_ids=ids.to(torch.int32),
                    top_logprobs=z.gather(1, ids) - lse.unsqueeze(1))
    ids, logq, tail = s["ids"].long(), s["logq"], case["tail"]
    entry = ids >= 0
    used = entry.any(1)
    hit = z.gather(1, ids.clamp(min=0))
    q = torch.where(entry, torch.exp(logq), torch.zeros_like(logq))
    if not tail:
        q = q / q.sum(1, keepdim=True).clamp(min=1e-30)
        logq = torch.log(q)
    loss = torch.where(q > 0, q * (logq - (hit - lse.unsqueeze(1))), torch.zeros_like(q)).sum(1)
    rest, r = lse, torch.zeros_like(lse)
    if tail:
        inside = torch.zeros(z.shape[0], z.shape[1] + 1, dtype=torch.bool, device=z.device)
        inside.scatter_(1, torch.where(entry, ids, torch.full_like(ids, z.shape[1])), True)
        inside = inside[:, :-1]
        r = (1.0 - q.double().sum(1)).clamp(min=0).float()
        rest = _lse(torch.where(inside, torch.full_like(z, -math.inf), z))
        loss = loss + torch.where(r > 0, r * (torch.log(r) - (rest - lse)), torch.zeros_like(r))
    none = torch.zeros_like(lse)
    out = dict(loss=torch.where(used, loss, none), lse=torch.where(used, lse, none),
               rest=torch.where(used, rest, none), hit=torch.where(entry, hit, torch.zeros_like(hit)))
    if case["op"] == "distill":
        return out
    whole = (q.sum(1) + r).unsqueeze(1)
    if tail:
        part = (whole[:, 0] * torch.exp(rest - lse) - r).unsqueeze(1)
        G = torch.where(inside, whole * torch.exp(z - lse.unsqueeze(1)), torch.exp(z - rest.unsqueeze(1)) * part)
    else:
        G = whole * torch.exp(z - lse.unsqueeze(1))
    G.scatter_add_(1, ids.clamp(min=0), -q)
    G = torch.where(used.unsqueeze(1), G * (s["dloss"] * scale).unsqueeze(1), torch.zeros_like(G))
    t = TYPES[case["type"]]
    return dict(out, dH=(G @ W).to(t), dW=(G.t() @ H).to(t))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    b = SIZE[case["type"]]
    T, V, d, k = case["tokens"], case["vocab"], case["d"], case["k"]
    if case["op"] == "logprobs":
        return dict(bytes=b * d * (T + V) + 4 * T * (2 * case["given"] + 2 + 2 * k), flops=2.0 * T * V * d)
    grad = case["op"] == "distill_grad"
    return dict(bytes=(2 if grad else 1) * b * d * (T + V) + 4 * T * (3 * k + 4), flops=(6.0 if grad else 2.0) * T * V * d)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    H, W = s["H"].to(f64) * s["scale"], s["W"].to(f64)
    some = max(1, min(512, (1 << 26) // case["vocab"]))
    parts = []
    dW = torch.zeros_like(W) if case["op"] == "distill_grad" else None
    for a in range(0, H.shape[0], some):
        rows = slice(a, a + some)
        z = torch.mm(H[rows], W.t())
        if case["op"] == "logprobs":
            parts.append(_exact_logprobs(z, s["tokens"][rows].long(), case["k"]))
            continue
        p, G = _exact_distill(z, s["ids"][rows].long(), s["logq"][rows].to(f64), case["tail"])
        if dW is not None:
            G *= s["dloss"][rows].to(f64).unsqueeze(1)
            p["dH"] = torch.mm(G, W) * s["scale"]
            dW += torch.mm(G.t().contiguous(), H[rows])
        parts.append(p)
    out = {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
    return out if dW is None else dict(out, dW=dW)


def _exact_logprobs(z, tokens, k):
    logp = torch.log_softmax(z, 1)
    best, ids = torch.sort(logp, dim=1, descending=True, stable=True)
    given = torch.where(tokens >= 0, logp.gather(1, tokens.clamp(min=0)), 0.0)
    return dict(logprobs=given, entropy=-(torch.exp(logp) * logp).sum(1), lse=torch.logsumexp(z, 1),
                top_ids=ids[:, :k].to(torch.int32), top_logprobs=best[:, :k])


def _exact_distill(z, ids, logq, tail):
    """The outputs of the loss, and its derivative by z."""
    V = z.shape[1]
    entry = ids >= 0
    used = entry.any(1)
    lse = torch.logsumexp(z, 1)
    if not tail:
        logq = torch.log_softmax(torch.where(entry, logq, -1e300), 1)
    q = torch.where(entry, torch.exp(logq), 0.0)
    # the teacher's probability of each word, the last one for entries that are none
    at = torch.where(entry, ids, V)
    target = torch.zeros(z.shape[0], V + 1, dtype=z.dtype, device=z.device).scatter_add_(1, at, q)[:, :V]
    listed_ = torch.zeros(z.shape[0], V + 1, dtype=torch.bool, device=z.device).scatter_(1, at, True)[:, :V]
    hit = torch.where(entry, z.gather(1, ids.clamp(min=0)), 0.0)
    loss = torch.where(entry, q * (logq - hit + lse.unsqueeze(1)), 0.0).sum(1)
    rest = lse
    G = torch.softmax(z, 1)
    if tail:
        others = z.masked_fill(listed_, -math.inf)
        rest = torch.logsumexp(others, 1)
        r = (1.0 - q.sum(1)).clamp(min=0.0)
        loss = loss + torch.where(r > 0, r * (torch.log(r) - rest + lse), 0.0)
        G = G * (q.sum(1) + r).unsqueeze(1) - r.unsqueeze(1) * torch.softmax(others, 1)
    G = torch.where(used.unsqueeze(1), G - target, 0.0)
    return dict(loss=torch.where(used, loss, 0.0), lse=torch.where(used, lse, 0.0),
                rest=torch.where(used, rest, 0.0), hit=hit), G
