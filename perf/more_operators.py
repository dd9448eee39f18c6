"""Cases of the operators between the cross entropy and the optimizer step.

Training on preferences or rewards, and the last pass over gradients that were
made elsewhere:

  layer_norm, layer_norm_grad   the norm of (activation + residual) with mean,
                      weight and bias, and its gradients;
  preference          the loss of pairs of sequences from their tokens' losses
                      (log ratios against a reference), and the gradient of
                      each token's loss;
  policy              the clipped policy loss with a KL term over packed
                      sequences, and the gradient of each token's loss;
  grad_norm           the 2-norm of many tensors, each one's and of all;
  grad_clip           that norm, and the tensors scaled into gradient buffers.

listed() and draw() say which sizes, prepare() makes what a program has in
hand, run() is one pass (in elementary torch operations, or with `own` through
the library), work() what the pass cannot do without, and exact() its result
in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-5
BETA = 0.1                # of the preference loss
SMOOTHING = 0.05
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
KL_COEF = 0.04
MAX_NORM = 1.0
F = torch.float64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases --

def listed():
    """Sizes of the GPT-2-small-shaped set (hidden 768), of the
    Llama-3.2-1B-shaped one (hidden 2048, 146 tensors) and of the set of 37
    odd-sized tensors."""
    return [
        # one short sequence through one norm
        {"name": "layer_norm_small", "op": "layer_norm", "T": 333, "D": 768, "residual": True},
        # a full micro-batch through one norm
        {"name": "layer_norm_large", "op": "layer_norm", "T": 32768, "D": 2048, "residual": True},
        # a short sequence through a norm without a residual beside it
        {"name": "layer_norm_grad_small", "op": "layer_norm_grad", "T": 333, "D": 768, "residual": False},
        {"name": "layer_norm_grad_large", "op": "layer_norm_grad", "T": 32768, "D": 2048, "residual": True},
        # four pairs of short answers
        {"name": "preference_small", "op": "preference", "T": 999, "P": 4, "kind": "sigmoid", "average": False},
        # a batch of 256 pairs of answers of about 2000 tokens, by their mean log ratio
        {"name": "preference_large", "op": "preference", "T": 1048575, "P": 256, "kind": "ipo", "average": True},
        # one group of 16 short answers
        {"name": "policy_small", "op": "policy", "T": 1501, "S": 16, "per_token": False, "average": True},
        # 512 answers of about 2000 tokens, an advantage for each token
        {"name": "policy_large", "op": "policy", "T": 1048575, "S": 512, "per_token": True, "average": False},
        # a small model's 37 odd-sized tensors, views of one flat buffer
        {"name": "grad_norm_small", "op": "grad_norm", "tensors": 37, "numel": 1000007, "type": "bf16"},
        # the 1B set's 146 gradients
        {"name": "grad_norm_large", "op": "grad_norm", "layers": 16, "type": "bf16"},
        # gradients summed in 32 bits elsewhere, clipped into the 16-bit buffers of the step
        {"name": "grad_clip_small", "op": "grad_clip", "tensors": 37, "numel": 1000007, "type": "fp32",
         "to": "bf16", "norm": 7.0},
        {"name": "grad_clip_large", "op": "grad_clip", "layers": 16, "type": "fp32", "to": "bf16", "norm": 7.0},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_grad", "preference", "policy", "grad_norm", "grad_clip"))
    if op.startswith("layer_norm"):
        D = _log(rng, 64, 8192, 8)
        return {"op": op, "T": _log(rng, 1, (32768 * 2048) // D), "D": D, "residual": rng.random() < 0.7}
    if op == "preference":
        T = _log(rng, 2, (1 << 20) - 1)
        return {"op": op, "T": T, "P": _log(rng, 1, min(1024, T)),
                "kind": rng.choice(("sigmoid", "hinge", "ipo")), "average": rng.random() < 0.5}
    if op == "policy":
        T = _log(rng, 1, (1 << 20) - 1)
        return {"op": op, "T": T, "S": _log(rng, 1, min(2048, T)), "per_token": rng.random() < 0.5,
                "average": rng.random() < 0.5}
    kind = rng.choice(tuple(TYPES))
    case = {"op": op, "tensors": _log(rng, 1, 400), "numel": _log(rng, 10000, 1 << (29 if kind == "fp32" else 30)),
            "type": kind}
    if op == "grad_clip":
        # in 16 bits the type stays, 32 bits may be kept or rounded
        case |= {"to": rng.choice(("fp32", "bf16")) if case["type"] == "fp32" else case["type"],
                 "norm": rng.choice((0.5, 7.0))}
    return case


def _sizes(case):
    """The tensors' sizes: of the 1B-shaped set, or ragged ones that sum to numel."""
    if "layers" in case:
        d, ff, kv, V = 2048, 8192, 512, 128256
        layer = [d * d, d * kv, d * kv, d * d, d * ff, d * ff, ff * d, d, d]
        return [V * d] + layer * case["layers"] + [d]
    n, total = case["tensors"], case["numel"]
    r = random.Random(n * 1000003 + total)
    w = [math.exp(r.uniform(0, 6)) for _ in range(n)]
    sizes = [int(total * x / sum(w)) for x in w]
    sizes[0] += total - sum(sizes)
    return sizes


# --------------------------------------------------------------- the inputs --

def _normal(g, shape, sigma, dtype=torch.bfloat16):
    """N(0, sigma), made in pieces so that no large 32-bit copy is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 26):
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * sigma)
    return out


def _packed(g, T, S):
    """S ragged sequences packed one behind the other (a few empty ones where
    there are many), and their tokens' ids: a prompt of about a quarter that
    takes part in nothing, and single holes."""
    w = torch.rand(S, generator=g, device="cuda", dtype=F) ** 2 + 0.02
    ends = (torch.cumsum(w, 0) / w.sum() * T).round().long()
    ends[-1] = T
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    at = torch.arange(T, device="cuda")
    s = torch.searchsorted(offsets, at, right=True) - 1
    length = (offsets[1:] - offsets[:-1])[s]
    prompt = (at - offsets[s]).float() < torch.rand(S, generator=g, device="cuda")[s] * 0.5 * length
    hole = prompt | (torch.rand(T, generator=g, device="cuda") < 0.02)
    ids = torch.randint(0, 50257, (T,), generator=g, device="cuda")
    return offsets, torch.where(hole, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op.startswith("layer_norm"):
        T, D = case["T"], case["D"]
        s["weight"] = (1 + _normal(g, (D,), 0.1).float()).to(torch.bfloat16)
        s["bias"] = _normal(g, (D,), 0.1)
        # a residual stream whose channels have offsets of their own
        x = _normal(g, (T, D), 2.0).add_(_normal(g, (D,), 1.0))
        if op == "layer_norm":
            return s | {"x": x, "res": _normal(g, (T, D), 1.0) if case["residual"] else None}
        mean, rstd = [], []
        for part in x.split(4096):
            m = part.float().mean(1)
            mean.append(m)
            rstd.append(1 / torch.sqrt((part.float() - m[:, None]).square().mean(1) + EPS))
        s |= {"x": x, "mean": torch.cat(mean), "rstd": torch.cat(rstd), "dy": _normal(g, (T, D), 1e-3)}
        return s | {"dsum": _normal(g, (T, D), 1e-3) if case["residual"] else None}
    if op in ("preference", "policy"):
        T = case["T"]
        S = 2 * case["P"] if op == "preference" else case["S"]
        s["offsets"], s["targets"] = _packed(g, T, S)
        counts = s["targets"] >= 0

        def logs(base, sigma):
            """Losses of another model or of an earlier state: near the first one's."""
            x = base + torch.randn(T, generator=g, device="cuda") * sigma
            return torch.where(counts, x.clamp(min=1e-6), torch.zeros_like(x))
        nll = torch.rand(T, generator=g, device="cuda").clamp(min=1e-6).log().neg() * 1.5
        s["nll"] = logs(nll, 0.0)
        s["ref_nll"] = logs(nll, 0.3)
        if op == "preference":
            # the mean over the pairs, as the upstream gradient of each
            return s | {"dloss": torch.full((case["P"],), 1.0 / case["P"], device="cuda")}
        s["old_nll"] = logs(nll, 0.15)
        s["advantages"] = torch.randn(T if case["per_token"] else S, generator=g, device="cuda")
        return s | {"dloss": torch.full((S,), 1.0 / (S if case["average"] else T), device="cuda")}
    sizes = _sizes(case)
    N, dtype = sum(sizes), TYPES[case["type"]]
    flat = _normal(g, (N,), case.get("norm", 7.0) / math.sqrt(N), dtype)
    s["grads"] = list(flat.split(sizes))
    if op == "grad_clip":
        # the tensors' places in a flat gradient buffer
        s["flat"] = torch.empty(N, dtype=TYPES[case["to"]], device="cuda")
        s["outs"] = list(s["flat"].split(sizes))
    return s


# ----------------------------------------------------------------- one pass --

def run(state):
    return (_run_own if own else _run_plain)(state)


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _run_plain(s):
    op = s["op"]
    if op == "layer_norm":
        total = s["x"].float()
        if s["res"] is not None:
            total = total + s["res"].float()
        mean = total.mean(1)
        centred = total - mean[:, None]
        rstd = 1 / torch.sqrt(centred.square().mean(1) + EPS)
        y = centred * rstd[:, None] * s["weight"].float() + s["bias"].float()
        out = {"y": y.to(torch.bfloat16), "mean": mean, "rstd": rstd}
        return out if s["res"] is None else out | {"sum": total.to(torch.bfloat16)}
    if op == "layer_norm_grad":
        dy, r = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * r
        u = dy * s["weight"].float()
        dx = (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True)) * r
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xhat).sum(0).to(torch.bfloat16),
                "dbias": dy.sum(0).to(torch.bfloat16)}
    if op in ("preference", "policy"):
        return _plain_loss(s)
    parts = [g.float().square().sum(dtype=F) for g in s["grads"]]   # sums of up to 2^30 terms
    norms = torch.sqrt(torch.stack(parts))
    norm = torch.sqrt(torch.stack(parts).sum())
    if op == "grad_norm":
        return {"norm": norm.float().view(1), "norms": norms.float()}
    coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    for g, out in zip(s["grads"], s["outs"]):
        out.copy_(g.float() * coef)
    return {"norm": norm.float().view(1), "out": s["flat"]}


def _plain_loss(s):
    T, off = s["T"], s["offsets"]
    S = off.numel() - 1
    live = s["targets"] >= 0
    seq = torch.searchsorted(off, torch.arange(T, device=off.device), right=True) - 1

    def sums(x):
        """Over each sequence's tokens that count; in 64 bits, as they may be long."""
        return torch.zeros(S, dtype=F, device=off.device).index_add_(0, seq, torch.where(live, x.to(F), 0.0))
    counts = sums(torch.ones_like(s["nll"]))
    share = 1 / counts.clamp(min=1) if s["average"] else torch.ones_like(counts)
    if s["op"] == "preference":
        ratios = sums(s["ref_nll"].to(F) - s["nll"].to(F)) * share
        d = ratios[0::2] - ratios[1::2]
        if s["kind"] == "sigmoid":
            zz = BETA * d
            loss = (1 - SMOOTHING) * _softplus(-zz) + SMOOTHING * _softplus(zz)
            slope = BETA * (SMOOTHING / (1 + torch.exp(-zz)) - (1 - SMOOTHING) / (1 + torch.exp(zz)))
        elif s["kind"] == "hinge":
            loss, slope = (1 - BETA * d).clamp(min=0), -BETA * (BETA * d < 1).to(F)
        else:
            loss, slope = (d - 1 / (2 * BETA)).square(), 2 * (d - 1 / (2 * BETA))
        back = torch.stack([-slope * s["dloss"], slope * s["dloss"]], 1).view(S) * share
        dnll = torch.where(live, back[seq], 0.0)
        return {"loss": loss.float(), "ratios": ratios.float(), "counts": counts.to(torch.int32),
                "dnll": dnll.float()}
    # which tokens are clipped, and the estimator's small differences, in 64 bits
    change = s["old_nll"].to(F) - s["nll"].to(F)
    drift = s["nll"].to(F) - s["ref_nll"].to(F)
    a = (s["advantages"] if s["per_token"] else s["advantages"][seq]).to(F)
    ratio = torch.exp(change)
    bounded = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    clipped = ((a > 0) & (ratio > 1 + CLIP_HIGH)) | ((a < 0) & (ratio < 1 - CLIP_LOW))
    k = torch.exp(drift) - drift - 1
    loss = sums(KL_COEF * k - torch.minimum(ratio * a, bounded * a)) * share
    slope = torch.where(clipped, 0.0, ratio * a) + KL_COEF * (torch.exp(drift) - 1)
    dnll = torch.where(live, slope * (s["dloss"] * share)[seq], 0.0)
    return {"loss": loss.float(), "kl": (sums(k) * share).float(), "clipped": sums(clipped).to(torch.int32),
            "counts": counts.to(torch.int32), "dnll": dnll.float()}


def _run_own(s):
    import zero_optimizer_step_rs_gb300 as z
    op = s["op"]

    def kept(name, shape, dtype=torch.float32):
        """A buffer that the program makes once and uses for every pass."""
        name = "own_" + name
        if name not in s:
            s[name] = torch.empty(shape, dtype=dtype, device="cuda")
        return s[name]

    def scratch(size, *args):
        if "scratch" not in s:
            s["scratch"] = torch.empty(max(16, size(*args)), dtype=torch.uint8, device="cuda")
        return s["scratch"]

    if op.startswith("layer_norm"):
        T, D, bf = s["T"], s["D"], torch.bfloat16
        if op == "layer_norm":
            y, mean, rstd = kept("y", (T, D), bf), kept("mean", (T,)), kept("rstd", (T,))
            total = None if s["res"] is None else kept("sum", (T, D), bf)
            z.zero_layer_norm(s["x"], s["weight"], s["bias"], y, mean, rstd, residual=s["res"], sum_out=total,
                              eps=EPS)
            out = {"y": y, "mean": mean, "rstd": rstd}
            return out if total is None else out | {"sum": total}
        dx, dw, db = kept("dx", (T, D), bf), kept("dw", (D,), bf), kept("db", (D,), bf)
        z.zero_layer_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], dx, dw, db,
                               scratch(z.zero_layer_norm_grad_scratch_bytes, T, D), dsum=s["dsum"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "preference":
        T, P = s["T"], s["P"]
        loss, slope, dnll = kept("loss", (P,)), kept("slope", (P,)), kept("dnll", (T,))
        ratios, counts = kept("ratios", (2 * P,)), kept("counts", (2 * P,), torch.int32)
        kind = {"sigmoid": z.ZERO_PREF_SIGMOID, "hinge": z.ZERO_PREF_HINGE, "ipo": z.ZERO_PREF_IPO}[s["kind"]]
        z.zero_preference(s["nll"], s["ref_nll"], s["targets"], s["offsets"], loss, slope, ratios, counts,
                          scratch(z.zero_preference_scratch_bytes, T, P), kind=kind, beta=BETA,
                          smoothing=SMOOTHING if s["kind"] == "sigmoid" else 0.0, average=s["average"])
        z.zero_preference_grad(s["targets"], s["offsets"], slope, counts, s["dloss"], dnll, average=s["average"])
        return {"loss": loss, "ratios": ratios, "counts": counts, "dnll": dnll}
    if op == "policy":
        T, S = s["T"], s["S"]
        loss, kl, dnll = kept("loss", (S,)), kept("kl", (S,)), kept("dnll", (T,))
        clipped, counts = kept("clipped", (S,), torch.int32), kept("counts", (S,), torch.int32)
        how = dict(per_token=s["per_token"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF,
                   average=s["average"])
        z.zero_policy(s["nll"], s["old_nll"], s["ref_nll"], s["advantages"], s["targets"], s["offsets"], loss, kl,
                      clipped, counts, scratch(z.zero_policy_scratch_bytes, T, S), **how)
        z.zero_policy_grad(s["nll"], s["old_nll"], s["ref_nll"], s["advantages"], s["targets"], s["offsets"],
                           counts, s["dloss"], dnll, **how)
        return {"loss": loss, "kl": kl, "clipped": clipped, "counts": counts, "dnll": dnll}
    n = len(s["grads"])
    norm, norms = kept("norm", (1,)), kept("norms", (n,))
    room = scratch(z.zero_grad_norm_scratch_bytes, n)
    if op == "grad_norm":
        z.zero_grad_norm(s["grads"], norm, room, norms=norms)
        return {"norm": norm, "norms": norms}
    z.zero_grad_norm(s["grads"], norm, room)
    z.zero_grad_clip(s["grads"], norm, MAX_NORM, outs=s["outs"])
    return {"norm": norm, "out": s["flat"]}


# ------------------------------------------------------- what it cannot avoid --

def work(case):
    op = case["op"]
    if op.startswith("layer_norm"):
        T, D = case["T"], case["D"]
        if op == "layer_norm":       # x, y; the residual and the sum
            return {"bytes": T * D * (8 if case["residual"] else 4) + 8 * T + 4 * D, "flops": 10 * T * D}
        return {"bytes": T * D * (8 if case["residual"] else 6) + 8 * T + 6 * D, "flops": 16 * T * D}
    if op == "preference":           # two losses and the id of each token; the gradient
        return {"bytes": case["T"] * (4 + 4 + 8 + 4) + 8 * 2 * case["P"] + 32 * case["P"], "flops": 4 * case["T"]}
    if op == "policy":               # three losses and the id, the advantages; the gradient
        T, S = case["T"], case["S"]
        return {"bytes": T * (12 + 8 + 4) + 4 * (T if case["per_token"] else S) + 28 * S, "flops": 40 * T}
    N, size = sum(_sizes(case)), torch.empty(0, dtype=TYPES[case["type"]]).element_size()
    if op == "grad_norm":
        return {"bytes": N * size, "flops": 2 * N}
    return {"bytes": N * (size + torch.empty(0, dtype=TYPES[case["to"]]).element_size()), "flops": 3 * N}


# -------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "layer_norm":
        t = s["x"].to(F)
        if s["res"] is not None:
            t = t.add_(s["res"])
        var, mean = torch.var_mean(t, 1, correction=0)
        rstd = (var + EPS).rsqrt()
        y = torch.addcmul(s["bias"].to(F), (t - mean[:, None]).mul_(rstd[:, None]), s["weight"].to(F))
        return {"y": y, "mean": mean, "rstd": rstd} | ({} if s["res"] is None else {"sum": t})
    if op == "layer_norm_grad":
        dy, w, r = s["dy"].to(F), s["weight"].to(F), s["rstd"].to(F)[:, None]
        xhat = s["x"].to(F).sub_(s["mean"][:, None]).mul_(r)
        one = torch.einsum("td,d->t", dy, w) / case["D"]
        two = torch.einsum("td,td,d->t", dy, xhat, w) / case["D"]
        dx = (dy * w).sub_(one[:, None]).sub_(xhat * two[:, None]).mul_(r)
        if s["dsum"] is not None:
            dx.add_(s["dsum"])
        return {"dx": dx, "dweight": torch.einsum("td,td->d", dy, xhat), "dbias": dy.sum(0)}
    if op in ("preference", "policy"):
        return _exact_loss(s)
    total, norms = 0.0, []
    for g in s["grads"]:
        part = sum(float(torch.dot(c, c)) for c in (p.to(F) for p in g.split(1 << 27)))
        norms.append(math.sqrt(part))
        total += part
    norm = torch.tensor([math.sqrt(total)], dtype=F, device="cuda")
    if op == "grad_norm":
        return {"norm": norm, "norms": torch.tensor(norms, dtype=F, device="cuda")}
    coef = min(1.0, MAX_NORM / (math.sqrt(total) + 1e-6))
    return {"norm": norm, "out": torch.cat([g.to(F) * coef for g in s["grads"]])}


def _exact_loss(s):
    """Sequence by sequence, from its tokens that count."""
    off = s["offsets"].tolist()
    pieces = {k: s[k].to(F) for k in ("nll", "ref_nll", "old_nll") if k in s}
    rows = {k: [] for k in ("loss", "kl", "clipped", "counts", "ratios")}
    dnll = torch.zeros(s["T"], dtype=F, device="cuda")
    adv = s["advantages"].to(F) if "advantages" in s else None
    at = [torch.nonzero(t >= 0)[:, 0] + lo for lo, t in zip(off, (s["targets"][a:b] for a, b in zip(off, off[1:])))]
    zero = torch.zeros((), dtype=F, device="cuda")
    if s["op"] == "policy":
        for i, t in enumerate(at):
            n = max(1, t.numel()) if s["average"] else 1
            rows["counts"].append(t.numel())
            a = adv[t] if s["per_token"] else adv[i].expand(t.numel())
            p, q = -pieces["nll"][t], -pieces["old_nll"][t]
            r = torch.exp(p - q)
            edge = torch.where(a > 0, torch.full_like(r, 1 + CLIP_HIGH), torch.full_like(r, 1 - CLIP_LOW))
            over = torch.where(a > 0, r > edge, (r < edge) & (a < 0))
            gap = -pieces["ref_nll"][t] - p
            k3 = torch.expm1(gap) - gap
            rows["loss"].append((torch.where(over, edge, r) * -a + KL_COEF * k3).sum() / n if t.numel() else zero)
            rows["kl"].append(k3.sum() / n if t.numel() else zero)
            rows["clipped"].append(over.sum())
            dnll[t] = (torch.where(over, torch.zeros_like(r), r * a) + KL_COEF * torch.expm1(gap)) * (s["dloss"][i].to(F) / n)
        return {"loss": torch.stack(rows["loss"]), "kl": torch.stack(rows["kl"]),
                "clipped": torch.stack(rows["clipped"]).to(torch.int32),
                "counts": torch.tensor(rows["counts"], dtype=torch.int32, device="cuda"), "dnll": dnll}
    for t in at:
        n = max(1, t.numel()) if s["average"] else 1
        rows["counts"].append(t.numel())
        rows["ratios"].append((pieces["ref_nll"][t] - pieces["nll"][t]).sum() / n)
    for i in range(s["P"]):
        d = rows["ratios"][2 * i] - rows["ratios"][2 * i + 1]
        x = BETA * d
        if s["kind"] == "sigmoid":
            loss = -(1 - SMOOTHING) * torch.nn.functional.logsigmoid(x) - SMOOTHING * torch.nn.functional.logsigmoid(-x)
            slope = BETA * (torch.sigmoid(x) - 1 + SMOOTHING)
        elif s["kind"] == "hinge":
            loss, slope = torch.relu(1 - x), torch.where(x < 1, -BETA, 0.0).to(F)
        else:
            loss, slope = (d - 0.5 / BETA) ** 2, 2 * d - 1 / BETA
        rows["loss"].append(loss)
        for j, sign in ((2 * i, -1), (2 * i + 1, 1)):
            n = max(1, at[j].numel()) if s["average"] else 1
            dnll[at[j]] = sign * slope * s["dloss"][i].to(F) / n
    return {"loss": torch.stack(rows["loss"]), "ratios": torch.stack(rows["ratios"]),
            "counts": torch.tensor(rows["counts"], dtype=torch.int32, device="cuda"), "dnll": dnll}
