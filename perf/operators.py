"""Cases of the language-model operators that feed the optimizer step.

A training step in front of the ZeRO step starts and ends in the same table
of the flat parameter vector when the embedding is tied to the output layer:

  embed, embed_grad   the scaled row lookup, and its gradient summed per token
                      into the table's part of a gradient buffer;
  norm, norm_grad     the root-mean-square norm of (activation + residual)
                      that keeps its input as an 8-bit checkpoint, the
                      normalised activation rebuilt from that checkpoint, and
                      the gradient computed from it;
  xent, xent_grad     the softmax cross entropy over the vocabulary without
                      kept logits, and the gradients of the activations and of
                      the table.

listed() and draw() say which sizes, prepare() makes what a program has in
hand, run() is one pass (in elementary torch operations, or with `own` through
the library), work() what the pass cannot do without, and exact() its result
in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128               # elements that share one scale of the 8-bit checkpoint
TINY = 1e-30              # a block whose largest magnitude is below this is kept as zeros
EPS = 1e-5


# ---------------------------------------------------------------- the cases --

def listed():
    """Sizes of the GPT-2-small-shaped set (vocabulary 50257, hidden 768) and
    of the Llama-3.2-1B-shaped one (128256, 2048; 8192 inside the
    feed-forward part)."""
    return [
        # a handful of prompts' first tokens: the latency of one lookup
        {"name": "embed_small", "op": "embed", "T": 77, "V": 50257, "D": 768},
        # 16 sequences of 4096 tokens
        {"name": "embed_large", "op": "embed", "T": 65536, "V": 128256, "D": 2048},
        # one short sequence into an untied table: every row of the gradient is written
        {"name": "embed_grad_small", "op": "embed_grad", "T": 1023, "V": 50257, "D": 768, "accumulate": False},
        # a full micro-batch added to the output layer's gradient of a tied table
        {"name": "embed_grad_tied", "op": "embed_grad", "T": 32768, "V": 128256, "D": 2048, "accumulate": True},
        # one short sequence through one norm
        {"name": "norm_small", "op": "norm", "T": 333, "D": 768},
        # a full micro-batch through one norm
        {"name": "norm_large", "op": "norm", "T": 32768, "D": 2048},
        {"name": "norm_grad_small", "op": "norm_grad", "T": 333, "D": 768},
        {"name": "norm_grad_large", "op": "norm_grad", "T": 32768, "D": 2048},
        # the loss of a few tokens: the table is read for very few rows
        {"name": "xent_few", "op": "xent", "T": 17, "V": 50257, "D": 768},
        # two sequences of 4096 tokens
        {"name": "xent_large", "op": "xent", "T": 8192, "V": 128256, "D": 2048},
        # one ragged sequence with ignored tokens
        {"name": "xent_grad_ragged", "op": "xent_grad", "T": 1001, "V": 50257, "D": 768},
        {"name": "xent_grad_large", "op": "xent_grad", "T": 8192, "V": 128256, "D": 2048},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "norm", "norm_grad", "xent", "xent_grad"))
    if op.startswith("norm"):
        D = _log(rng, 64, 8192, 8)
        return {"op": op, "T": _log(rng, 1, (32768 * 2048) // D), "D": D}
    D = _log(rng, 64, 2048, 8)
    V = _log(rng, 1000, 128256)
    if op.startswith("xent"):
        return {"op": op, "T": _log(rng, 1, 8192), "V": V, "D": D}
    case = {"op": op, "T": _log(rng, 1, 32768), "V": V, "D": D}
    if op == "embed_grad":
        case["accumulate"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------- the inputs --

def _tokens(g, T, V, masked):
    """Token ids whose frequency falls as one over their rank, as in text; a
    part of them -1 (padding that takes part in nothing)."""
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1)).floor().long() - 1).clamp_(0, V - 1)
    hole = torch.rand(T, generator=g, device="cuda") < masked
    return torch.where(hole, torch.full_like(t, -1), t)


def _normal(g, shape, sigma, dtype=torch.bfloat16):
    """N(0, sigma), made in pieces so that no large 32-bit copy is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 26):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * sigma)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, D = case["op"], case["T"], case["D"]
    s = {"op": op, "T": T, "D": D, "V": case.get("V", 0)}
    if op.startswith("norm"):
        s["weight"] = (1 + _normal(g, (D,), 0.1).float()).to(torch.bfloat16)
        x = _normal(g, (T, D), 1.0)
        res = _normal(g, (T, D), 2.0)
        if op == "norm":
            return s | {"x": x, "res": res}
        # what the forward pass has kept, and the gradients that come back
        codes, scales, rstd = [], [], []
        for a, b in zip(x.split(4096), res.split(4096)):
            kept = _keep(a.float() + b.float())
            for to, v in zip((codes, scales, rstd), kept):
                to.append(v)
        s |= {"codes": torch.cat(codes), "scales": torch.cat(scales), "rstd": torch.cat(rstd)}
        del x, res
        return s | {"dy": _normal(g, (T, D), 1e-3), "dsum": _normal(g, (T, D), 1e-3)}
    V = s["V"]
    s["scale"] = math.sqrt(D) if op.startswith("embed") else 1.0
    s["tokens"] = _tokens(g, T, V, 0.03)
    if op == "embed":
        return s | {"table": _normal(g, (V, D), 0.02)}
    if op == "embed_grad":
        s["accumulate"] = case["accumulate"]
        return s | {"dy": _normal(g, (T, D), 1e-3), "grad": _normal(g, (V, D), 1e-3)}
    s["table"] = _normal(g, (V, D), 0.02)
    s["h"] = _normal(g, (T, D), 1.0)
    if op == "xent_grad":
        lse = [torch.logsumexp(part.float() @ s["table"].float().T, 1) for part in s["h"].split(1024)]
        s["lse"] = torch.cat(lse)
        # the mean over the tokens that count, as the upstream gradient of each
        s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


def _keep(total):
    """The 8-bit checkpoint of a 32-bit activation: codes, one scale for each
    block of 128 elements, and the row's reciprocal root mean square."""
    T, D = total.shape
    nb = -(-D // BLOCK)
    pad = torch.nn.functional.pad(total, (0, nb * BLOCK - D)).view(T, nb, BLOCK)
    amax = pad.abs().amax(2)
    full = torch.full_like(amax, 127.0)
    used = amax >= TINY
    scales = torch.where(used, amax / full, torch.zeros_like(amax))
    inverse = torch.where(used, full / amax, torch.zeros_like(amax))
    codes = torch.round(pad * inverse[:, :, None]).to(torch.int8).view(T, nb * BLOCK)[:, :D]
    rstd = 1 / torch.sqrt((total * total).mean(1) + EPS)
    return codes.contiguous(), scales, rstd


def _normed(codes, scales, rstd):
    """The normalised activation (before the weight) that a checkpoint stands for."""
    spread = scales.repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]
    return codes.to(scales.dtype) * spread * rstd[:, None]


# ----------------------------------------------------------------- one pass --

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        t = s["tokens"]
        rows = s["table"][t.clamp(min=0)].float() * s["scale"]
        return (rows * (t >= 0)[:, None]).to(torch.bfloat16)
    if op == "embed_grad":
        t, grad = s["tokens"], s["grad"]
        part = s["dy"].float() * ((t >= 0).float() * s["scale"])[:, None]
        total = grad.float() if s["accumulate"] else torch.zeros(grad.shape, device=grad.device)
        total.index_add_(0, t.clamp(min=0), part)
        grad.copy_(total)
        return grad
    if op == "norm":
        total = s["x"].float() + s["res"].float()
        codes, scales, rstd = _keep(total)
        y = total * rstd[:, None] * s["weight"].float()
        again = _normed(codes, scales, rstd) * s["weight"].float()
        return {"y": y.to(torch.bfloat16), "sum": total.to(torch.bfloat16), "rstd": rstd, "scales": scales,
                "replayed": again.to(torch.bfloat16)}
    if op == "norm_grad":
        dy, xhat = s["dy"].float(), _normed(s["codes"], s["scales"], s["rstd"])
        dxhat = dy * s["weight"].float()
        dx = (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)) * s["rstd"][:, None] + s["dsum"].float()
        return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xhat).sum(0).to(torch.bfloat16)}
    t, T = s["tokens"], s["T"]
    counts = t >= 0
    logits = s["h"].float() @ s["table"].float().T
    if op == "xent":
        top = logits.amax(1)
        lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
        at = logits.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return {"loss": torch.where(counts, lse - at, torch.zeros_like(lse)), "lse": lse}
    p = torch.exp(logits - s["lse"][:, None])
    p[torch.arange(T, device=p.device), t.clamp(min=0)] -= 1
    p *= (s["dloss"] * counts)[:, None]
    return {"dh": (p @ s["table"].float()).to(torch.bfloat16), "dtable": (p.T @ s["h"].float()).to(torch.bfloat16)}


def _run_own(s):
    import zero_optimizer_step_rs_gb300 as z
    op, T, D, V = s["op"], s["T"], s["D"], s["V"]

    def kept(name, shape, dtype=torch.bfloat16):
        """A buffer that the program makes once and uses for every pass."""
        if name not in s:
            s[name] = torch.empty(shape, dtype=dtype, device="cuda")
        return s[name]

    def scratch(size, *args):
        if "scratch" not in s:
            s["scratch"] = torch.empty(max(16, size(*args)), dtype=torch.uint8, device="cuda")
        return s["scratch"]

    if op == "embed":
        out = kept("out", (T, D))
        z.zero_embed(s["table"], s["tokens"], out, scale=s["scale"])
        return out
    if op == "embed_grad":
        z.zero_embed_grad(s["dy"], s["tokens"], s["grad"], scratch(z.zero_embed_grad_scratch_bytes, T, V, D),
                          scale=s["scale"], accumulate=s["accumulate"])
        return s["grad"]
    if op == "norm":
        y, total, again = kept("y", (T, D)), kept("sum", (T, D)), kept("again", (T, D))
        codes = kept("codes", (T, D), torch.int8)
        scales = kept("scales", (T, -(-D // BLOCK)), torch.float32)
        rstd = kept("rstd", (T,), torch.float32)
        z.zero_norm(s["x"], s["weight"], y, codes, scales, rstd, residual=s["res"], sum_out=total, eps=EPS)
        z.zero_norm_replay(codes, scales, rstd, s["weight"], again)
        return {"y": y, "sum": total, "rstd": rstd, "scales": scales, "replayed": again}
    if op == "norm_grad":
        dx, dweight = kept("dx", (T, D)), kept("dweight", (D,))
        z.zero_norm_grad(s["dy"], s["codes"], s["scales"], s["rstd"], s["weight"], dx, dweight,
                         scratch(z.zero_norm_grad_scratch_bytes, T, D), dsum=s["dsum"])
        return {"dx": dx, "dweight": dweight}
    if op == "xent":
        loss, lse = kept("loss", (T,), torch.float32), kept("lse", (T,), torch.float32)
        z.zero_xent(s["h"], s["table"], s["tokens"], loss, lse, scratch(z.zero_xent_scratch_bytes, T, V, D))
        return {"loss": loss, "lse": lse}
    dh, dtable = kept("dh", (T, D)), kept("dtable", (V, D))
    z.zero_xent_grad(s["h"], s["table"], s["tokens"], s["lse"], s["dloss"], dh, dtable,
                     scratch(z.zero_xent_grad_scratch_bytes, T, V, D))
    return {"dh": dh, "dtable": dtable}


# ------------------------------------------------------- what it cannot avoid --

def _rows_met(T, V):
    """The expected number of different rows among T tokens of _tokens()."""
    edge = np.log(np.arange(1, V + 2)) / math.log(V + 1)
    return float(-np.expm1(0.97 * T * np.log1p(-np.minimum(np.diff(edge), 0.999))).sum())


def work(case):
    op, T, D, V = case["op"], case["T"], case["D"], case.get("V", 0)
    if op == "embed":
        return {"bytes": 2 * D * (_rows_met(T, V) + T) + 8 * T, "flops": T * D}
    if op == "embed_grad":
        rows = 2 * _rows_met(T, V) if case["accumulate"] else V
        return {"bytes": 2 * D * (T + rows) + 8 * T, "flops": T * D}
    kept = T * D + 4 * T * -(-D // BLOCK) + 4 * T
    if op == "norm":       # x, residual, y, sum; the checkpoint written and read; the replayed activation
        return {"bytes": T * D * (2 + 2 + 2 + 2) + 2 * kept + 2 * T * D + 2 * D, "flops": 12 * T * D}
    if op == "norm_grad":  # dy, dsum, the checkpoint, dx
        return {"bytes": T * D * (2 + 2 + 2) + kept + 4 * D, "flops": 12 * T * D}
    if op == "xent":       # one product of the activations with the table
        return {"bytes": 2 * D * (T + V) + 16 * T, "flops": 2 * T * D * V + 4 * T * V}
    # the logits again (only their log-sum was kept), and one product for each gradient
    return {"bytes": 4 * D * (T + V) + 16 * T, "flops": 6 * T * D * V + 4 * T * V}


# -------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    op, T, D, V = case["op"], case["T"], case["D"], case.get("V", 0)
    if op.startswith("xent") and work(case)["flops"] > 8e12:
        return None        # 64-bit products run at about 1 TFLOP/s
    s = prepare(case, seed)
    f = torch.float64
    if op == "embed":
        out = torch.zeros((T, D), dtype=f, device="cuda")
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        out[at] = s["table"].index_select(0, s["tokens"][at]).to(f) * s["scale"]
        return out
    if op == "embed_grad":
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        out = s["grad"].to(f) if s["accumulate"] else torch.zeros((V, D), dtype=f, device="cuda")
        return out.index_put_((s["tokens"][at],), s["dy"][at].to(f) * s["scale"], accumulate=True)
    if op == "norm":
        total = s["x"].to(f).add_(s["res"])
        rstd = (total.square().mean(1) + EPS).rsqrt()
        y = total * rstd[:, None] * s["weight"].to(f)
        blocks = [total[:, b:b + BLOCK] for b in range(0, D, BLOCK)]
        scales = torch.stack([b.abs().amax(1) / 127 for b in blocks], 1)
        # a value half-way between two codes may go to either: what is rebuilt has no one value there
        return {"y": y, "sum": total, "rstd": rstd, "scales": scales, "replayed": None}
    if op == "norm_grad":
        dy, w, r = s["dy"].to(f), s["weight"].to(f), s["rstd"].to(f)[:, None]
        xhat = torch.empty((T, D), dtype=f, device="cuda")
        for b in range(s["scales"].shape[1]):
            cut = slice(b * BLOCK, (b + 1) * BLOCK)
            xhat[:, cut] = s["codes"][:, cut].to(f) * s["scales"][:, b:b + 1].to(f) * r
        inner = torch.einsum("td,td,d->t", dy, xhat, w) / D
        dx = r * (dy * w - xhat * inner[:, None]) + s["dsum"].to(f)
        return {"dx": dx, "dweight": torch.einsum("td,td->d", dy, xhat)}
    h, table, t = s["h"].to(f), s["table"].to(f), s["tokens"]
    logits = torch.matmul(h, table.t())
    ok = t >= 0
    if op == "xent":
        lse = torch.logsumexp(logits, 1)
        loss = torch.zeros(T, dtype=f, device="cuda")
        loss[ok] = lse[ok] - logits[ok, t[ok]]
        return {"loss": loss, "lse": lse}
    d = logits.sub_(s["lse"].to(f)[:, None]).exp_()
    d[ok, t[ok]] -= 1.0
    d.mul_(torch.where(ok, s["dloss"].to(f), torch.zeros_like(s["dloss"], dtype=f))[:, None])
    return {"dh": torch.matmul(d, table), "dtable": torch.matmul(d.t(), h)}
