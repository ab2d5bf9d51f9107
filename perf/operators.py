"""Cases of the operators that tune a packed low-rank binary model: 8-bit
activation checkpoints, the gradient of a packed layer from such a
checkpoint, and the softmax cross entropy over a large vocabulary with its
gradient. `run` computes them in plain torch, or with `own` set through
sub_bit_weight_lb_amd.

  checkpoint  act8_quantize, then act8_dequantize: X -> (codes, exponents) -> X^
              Groups of 32 columns of a row share the step 2^e, e the least
              integer with max|x| <= 127 2^e (-126 <= e <= 121, at most 9 for
              fp16, so that X^ stays finite); code = round-to-even(x / 2^e)
              in -127 .. 127.
  scales      binary_matmul_backward: for Y = X^ W^T, W = diag(s1) S_U S_V^T
              diag(s2), and dL/dY: dX, ds1 and ds2, with X^ the checkpoint.
  loss        vocab_loss: lse_t = log sum_v exp(h_t . w_v), loss_t = lse_t -
              h_t . w_label (0 where the label is negative: ignored).
  loss_grad   vocab_loss and vocab_loss_backward: the loss, then dH and dW of
              sum_t dloss_t loss_t.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # one token's activations of a 4096-wide layer: latency alone
        dict(name="checkpoint-token", op="checkpoint", rows=1, cols=4096, type="fp32"),
        # a ragged batch whose rows are not 16-byte aligned and end inside a group
        dict(name="checkpoint-odd", op="checkpoint", rows=1021, cols=11007, type="fp16"),
        # a quarter of a calibration set of 128 x 2048 tokens at one 4096-wide layer
        dict(name="checkpoint-calibration", op="checkpoint", rows=65536, cols=4096, type="bf16"),
        # one token through a 4096 x 4096 layer at 1 bit per weight: the signs are the traffic
        dict(name="scales-token", op="scales", tokens=1, m=4096, n=4096, r=2048, type="fp32"),
        # a small layer, every size odd
        dict(name="scales-odd", op="scales", tokens=777, m=1001, n=1501, r=333, type="fp16"),
        # one 2048-token sample through an 11008 x 4096 layer of rank 1536, bf16 gradients
        dict(name="scales-sample", op="scales", tokens=2048, m=11008, n=4096, r=1536, type="bf16"),
        # a batch of four 2048-token samples through a 4096 x 4096 layer, fp32 gradients
        dict(name="scales-batch", op="scales", tokens=8192, m=4096, n=4096, r=2048, type="fp32"),
        # scoring one token against a 32000-word vocabulary: W is the traffic
        dict(name="loss-token", op="loss", tokens=1, vocab=32000, d=4096, type="bf16"),
        # scoring a ragged batch, odd vocabulary
        dict(name="loss-odd", op="loss", tokens=509, vocab=50021, d=1000, type="fp16"),
        # a short ragged batch with rows of W that are not 16-byte aligned
        dict(name="grad-odd", op="loss_grad", tokens=301, vocab=4999, d=515, type="bf16"),
        # an fp32 head in training
        dict(name="grad-fp32", op="loss_grad", tokens=1024, vocab=32000, d=2048, type="fp32"),
        # two 2048-token samples, a 131072-word vocabulary: logits of 1 GiB in bf16 that are not kept
        dict(name="grad-large", op="loss_grad", tokens=4096, vocab=131072, d=4096, type="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["checkpoint", "scales", "loss", "loss_grad"])
    kind = rng.choice(["fp32", "bf16", "fp16"])
    if op == "checkpoint":
        cols = _log_uniform(rng, 1, 28672)
        return dict(op=op, rows=_log_uniform(rng, 1, max(1, 65536 * 2048 // cols)), cols=cols, type=kind)
    if op == "scales":
        m, n = _log_uniform(rng, 32, 11008), _log_uniform(rng, 32, 11008)
        r = _log_uniform(rng, 8, max(8, min(m, n, 2048)))
        most = 8192 * 2048 * 8192 // (r * (m + n))
        return dict(op=op, tokens=_log_uniform(rng, 1, max(1, min(8192, most))), m=m, n=n, r=r, type=kind)
    vocab, d = _log_uniform(rng, 500, 131072), _log_uniform(rng, 64, 8192)
    d = d if rng.random() < 0.3 else max(64, d // 64 * 64)
    # (an fp32 head costs several times a bf16 one)
    most = (1 << 41) // (vocab * d) // (8 if kind == "fp32" else 2)
    return dict(op=op, tokens=_log_uniform(rng, 1, max(1, min(8192, most))), vocab=vocab, d=d, type=kind)


# ---------------------------------------------------------------- inputs

def _activations(rows, cols, gen):
    """Activations with a spread of channel magnitudes and a few channels far
    above the rest, as hidden states have them."""
    mag = torch.exp(0.6 * torch.randn(cols, generator=gen, device=DEV))
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.002
    mag = torch.where(loud, 30.0 * mag, mag)
    return torch.randn(rows, cols, generator=gen, device=DEV) * mag


def _steps(x, kind):
    """e of each group of 32 columns (rows x groups, int32) for x in fp32."""
    rows, cols = x.shape
    pad = -cols % 32
    a = torch.nn.functional.pad(x.abs(), (0, pad)).view(rows, (cols + pad) // 32, 32).amax(-1)
    mant, ex = torch.frexp(a.double())
    e = torch.where(mant <= 127.0 / 128.0, ex - 7, ex - 6)
    e = torch.where(a == 0, torch.full_like(e, -126), e)
    return e.clamp(-126, 9 if kind == "fp16" else 121)


def _codes(x, e):
    """Codes of x for the exponents e (each step a power of two, so that the
    quotient is exact in 64 bits)."""
    step = torch.exp2(e.double()).repeat_interleave(32, 1)[:, :x.shape[1]]
    return torch.round(x.double() / step).clamp(-127, 127).to(torch.int8)


def _signs(rows, cols, gen):
    return torch.rand(rows, cols, generator=gen, device=DEV) < 0.5


def _pack(s):
    """Bit k of word w of row i = s[i, 32 w + k]."""
    rows, cols = s.shape
    s = torch.nn.functional.pad(s, (0, -cols % 32)).view(rows, -1, 32).long()
    w = (s << torch.arange(32, device=s.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    kind = case["type"]
    t = TYPES[kind]
    if case["op"] == "checkpoint":
        return dict(case=case, X=_activations(case["rows"], case["cols"], gen).to(t))
    if case["op"] == "scales":
        T, m, n, r = case["tokens"], case["m"], case["n"], case["r"]
        x = _activations(T, n, gen)
        e = _steps(x, kind)
        su, sv = _signs(m, r, gen), _signs(n, r, gen)
        return dict(
            case=case, codes=_codes(x, e), exps=(e + 127).to(torch.uint8),
            U_bits=_pack(su), Ut_bits=_pack(su.t()), V_bits=_pack(sv), Vt_bits=_pack(sv.t()),
            s1=0.02 * torch.rand(m, generator=gen, device=DEV) + 0.01,
            s2=0.02 * torch.rand(n, generator=gen, device=DEV) + 0.01,
            dY=(0.01 * torch.randn(T, m, generator=gen, device=DEV)).to(t))
    T, V, d = case["tokens"], case["vocab"], case["d"]
    W = 0.02 * torch.randn(V, d, generator=gen, device=DEV)
    labels = torch.randint(0, V, (T,), generator=gen, device=DEV)
    # half of the tokens are predicted well: their hidden state leans to the label
    lean = (torch.rand(T, 1, generator=gen, device=DEV) < 0.5) * (10.0 / (0.0004 * d))
    H = torch.randn(T, d, generator=gen, device=DEV) + lean * W[labels]
    if T > 1:  # some tokens are padding or a prompt
        labels = torch.where(torch.rand(T, generator=gen, device=DEV) < 0.12, torch.full_like(labels, -100), labels)
    used = (labels >= 0).float()
    return dict(case=case, H=H.to(t), W=W.to(t), labels=labels.to(torch.int32),
                dloss=used / used.sum().clamp(min=1.0))


# ---------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import sub_bit_weight_lb_amd as nq
    op = s["case"]["op"]
    if op == "checkpoint":
        q = nq.act8_quantize(s["X"])
        return dict(x=nq.act8_dequantize(q), step=nq.act8_steps(q))
    if op == "scales":
        q = nq.Act8(s["codes"], s["exps"])
        dX, ds1, ds2 = nq.binary_matmul_backward(
            s["U_bits"], s["Ut_bits"], s["V_bits"], s["Vt_bits"], s["s1"], s["s2"], q, s["dY"],
            s["case"]["r"])
        return dict(dX=dX, ds1=ds1, ds2=ds2)
    loss, lse = nq.vocab_loss(s["H"], s["W"], s["labels"])
    if op == "loss":
        return dict(loss=loss, lse=lse)
    dH, dW = nq.vocab_loss_backward(s["H"], s["W"], s["labels"], lse, s["dloss"])
    return dict(loss=loss, lse=lse, dH=dH, dW=dW)


def _unpack(bits, cols):
    """+-1 in fp32 from packed signs."""
    b = (bits.unsqueeze(-1) >> torch.arange(32, device=bits.device, dtype=torch.int32)) & 1
    return (2 * b - 1).view(bits.shape[0], -1)[:, :cols].float()


def _plain(s):
    op, kind = s["case"]["op"], s["case"]["type"]
    t = TYPES[kind]
    if op == "checkpoint":
        x = s["X"].float()
        e = _steps(x, kind)
        step = torch.exp2(e.double())
        x8 = _codes(x, e) * step.repeat_interleave(32, 1)[:, :x.shape[1]]
        return dict(x=x8.to(t), step=step.float())
    if op == "scales":
        r, n = s["case"]["r"], s["case"]["n"]
        su, sv = _unpack(s["U_bits"], r), _unpack(s["V_bits"], r)
        step = torch.exp2(s["exps"].float() - 127.0).repeat_interleave(32, 1)[:, :n]
        x, dy = s["codes"].float() * step, s["dY"].float()
        q = ((x * s["s2"]) @ sv) @ su.t()
        da = ((dy * s["s1"]) @ su) @ sv.t()
        return dict(dX=(da * s["s2"]).to(t), ds1=(dy * q).sum(0), ds2=(da * x).sum(0))
    H, W, labels = s["H"].float(), s["W"].float(), s["labels"].long()
    used = labels >= 0
    logits = H @ W.t()
    top = logits.amax(1, keepdim=True)
    lse = torch.log(torch.exp(logits - top).sum(1)) + top[:, 0]
    hit = logits.gather(1, labels.clamp(min=0).unsqueeze(1))[:, 0]
    lse = torch.where(used, lse, torch.zeros_like(lse))
    loss = torch.where(used, lse - hit, torch.zeros_like(lse))
    if op == "loss":
        return dict(loss=loss, lse=lse)
    G = torch.exp(logits - lse.unsqueeze(1))
    G.scatter_add_(1, labels.clamp(min=0).unsqueeze(1), torch.full_like(lse, -1.0).unsqueeze(1))
    G = torch.where(used.unsqueeze(1), G * s["dloss"].unsqueeze(1), torch.zeros_like(G))
    return dict(loss=loss, lse=lse, dH=(G @ W).to(t), dW=(G.t() @ H).to(t))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    b = SIZE[case["type"]]
    if case["op"] == "checkpoint":
        rows, cols = case["rows"], case["cols"]
        groups = rows * -(-cols // 32)
        # X read, X^ and the steps written; the codes and exponents in between written and read
        return dict(bytes=rows * cols * (2 * b + 2) + groups * (4 + 2), flops=4 * rows * cols)
    if case["op"] == "scales":
        T, m, n, r = case["tokens"], case["m"], case["n"], case["r"]
        return dict(bytes=T * (n + -(-n // 32)) + b * T * (m + n) + r * (m + n) / 8 + 8 * (m + n),
                    flops=4.0 * T * r * (m + n))
    T, V, d = case["tokens"], case["vocab"], case["d"]
    grad = case["op"] == "loss_grad"
    return dict(bytes=(2 if grad else 1) * b * d * (T + V) + 16 * T,
                flops=(6.0 if grad else 2.0) * T * V * d)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _exact_checkpoint(s["X"], case["type"])
    if case["op"] == "scales":
        return _exact_scales(s, case)
    return _exact_loss(s, case["op"] == "loss_grad")


def _exact_checkpoint(X, kind):
    X = X.cpu().numpy() if X.dtype != torch.bfloat16 else X.float().cpu().numpy()
    rows, cols = X.shape
    out = np.empty((rows, cols), np.float32)
    groups = -(-cols // 32)
    steps = np.empty((rows, groups), np.float32)
    some = max(1, (1 << 24) // cols)
    for a in range(0, rows, some):
        x = X[a:a + some].astype(np.float64)
        g = np.zeros((x.shape[0], groups * 32))
        g[:, :cols] = x
        g = g.reshape(x.shape[0], groups, 32)
        big = np.abs(g).max(-1)
        e = np.ceil(np.log2(np.maximum(big, 2.0 ** -140) / 127.0))
        e += big > np.ldexp(127.0, e.astype(int))          # (the logarithm may be off by a unit at a border)
        e -= big <= np.ldexp(127.0, e.astype(int) - 1)
        e = np.clip(e, -126, 9 if kind == "fp16" else 121).astype(int)[..., None]
        c = np.clip(np.rint(np.ldexp(g, -e)), -127, 127)
        out[a:a + some] = np.ldexp(c, e).reshape(x.shape[0], -1)[:, :cols]
        steps[a:a + some] = np.ldexp(1.0, e[..., 0])
    return dict(x=torch.from_numpy(out), step=torch.from_numpy(steps))


def _exact_scales(s, case):
    f64 = torch.float64
    n, r = case["n"], case["r"]
    col = torch.arange(r, device=DEV)
    su = ((s["U_bits"][:, col // 32] >> (col % 32).int()) & 1).to(f64).mul_(2).sub_(1)
    sv = ((s["V_bits"][:, col // 32] >> (col % 32).int()) & 1).to(f64).mul_(2).sub_(1)
    group = torch.arange(n, device=DEV) // 32
    x = torch.ldexp(s["codes"].to(f64), s["exps"][:, group].int() - 127)
    dy, s1, s2 = s["dY"].to(f64), s["s1"].to(f64), s["s2"].to(f64)
    ds1 = torch.einsum("ti,ti->i", dy, torch.mm(torch.mm(x * s2, sv), su.t().contiguous()))
    da = torch.mm(torch.mm(dy * s1, su), sv.t().contiguous())
    return dict(dX=da * s2, ds1=ds1, ds2=torch.einsum("tj,tj->j", da, x))


def _exact_loss(s, grad):
    f64 = torch.float64
    H, W, labels = s["H"].to(f64), s["W"].to(f64), s["labels"].long()
    T = H.shape[0]
    lse, loss = H.new_zeros(T), H.new_zeros(T)
    dH, dW = (torch.zeros_like(H), torch.zeros_like(W)) if grad else (None, None)
    for a in range(0, T, 1024):
        rows = torch.arange(a, min(T, a + 1024), device=DEV)
        rows = rows[labels[rows] >= 0]
        if not len(rows):
            continue
        z = torch.mm(H[rows], W.t())
        lse[rows] = torch.logsumexp(z, 1)
        at = torch.arange(len(rows), device=DEV), labels[rows]
        loss[rows] = lse[rows] - z[at]
        if grad:
            p = torch.softmax(z, 1)
            p[at] -= 1.0
            p *= s["dloss"][rows].to(f64).unsqueeze(1)
            dH[rows] = torch.mm(p, W)
            dW += torch.mm(p.t(), H[rows])
    out = dict(loss=loss, lse=lse)
    return dict(out, dH=dH, dW=dW) if grad else out
