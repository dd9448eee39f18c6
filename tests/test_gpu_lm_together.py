"""The operators together as a training step uses them: a small model with a layer norm and a
tied table, trained on preferences or with the policy loss, its gradients clipped into the
step's buffers.  The gradients against 64-bit automatic differentiation."""
import pytest
import torch

import zero_optimizer_step_rs_gb300 as z
from tests import lm_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Model:
    """x = scale table[tok], h = layer_norm(x + r), nll = xent(h table^T); the parameters are one
    flat vector (an odd number of other elements first, so that the tensors lie anywhere)."""

    def __init__(self, V=300, D=136, lengths=(40, 25, 0, 31, 7, 60), seed=1):
        g = R.gen(seed)
        self.V, self.D, self.T = V, D, sum(lengths) + 5       # (five tokens of no sequence)
        self.scale = 3.0
        off = [3]
        for n in lengths:
            off.append(off[-1] + n)
        self.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        self.seqs = list(zip(off, off[1:]))
        self.plan = z.Plan([V * D, D, D], R=2, M=1, stage=2)
        flat = torch.randn(self.plan.N, generator=g, device="cuda") * 0.3
        flat[V * D:V * D + D] += 1
        self.replicas = [flat.to(BF) for _ in range(2)]
        self.master = torch.zeros(self.plan.padded, device="cuda")
        self.master[:self.plan.N] = flat
        T = self.T
        self.tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.targets[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
        self.res = R.bf16(g, (T, D))
        self.near = torch.randn(T, generator=g, device="cuda") * 0.3
        self.adv = torch.randn(len(lengths), generator=g, device="cuda")
        bf, f = dict(dtype=BF, device="cuda"), dict(device="cuda")
        self.x, self.s, self.h, self.dh, self.ds = (torch.zeros((T, D), **bf) for _ in range(5))
        self.mean, self.rstd, self.nll, self.lse, self.dnll = (torch.zeros(T, **f) for _ in range(5))
        size = max(z.zero_embed_grad_scratch_bytes(T, V, D), z.zero_layer_norm_grad_scratch_bytes(T, D),
                   z.zero_xent_scratch_bytes(T, V, D), z.zero_xent_grad_scratch_bytes(T, V, D),
                   z.zero_policy_scratch_bytes(T, len(lengths)), z.zero_grad_norm_scratch_bytes(3))
        self.scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.grad = torch.zeros(self.plan.N, **bf)
        self.clipped = [torch.zeros(self.plan.N, **bf) for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        S = len(lengths)
        self.loss, self.slope = torch.zeros(S // 2, **f), torch.zeros(S // 2, **f)
        self.ratios, self.kl, self.seq_loss = (torch.zeros(S, **f) for _ in range(3))
        self.counts, self.cut = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
        self.d_pair, self.d_seq = torch.ones(S // 2, **f) / (S // 2), torch.ones(S, **f) / S
        self.norm, self.norms = torch.zeros(1, **f), torch.zeros(3, **f)

    def views(self, flat):
        a, b, c, d = self.plan.tensor_offsets()
        return flat[a:b].view(self.V, self.D), flat[b:c], flat[c:d]

    def forward(self):
        table, w, b = self.views(self.replicas[0])
        z.zero_embed(table, self.tokens, self.x, scale=self.scale, dev_status=self.status)
        z.zero_layer_norm(self.x, w, b, self.h, self.mean, self.rstd, residual=self.res, sum_out=self.s)
        z.zero_xent(self.h, table, self.targets, self.nll, self.lse, self.scratch,
                    dev_status=self.status)

    def backward(self, dnll):
        table, w, _ = self.views(self.replicas[0])
        d_table, d_w, d_b = self.views(self.grad)
        z.zero_xent_grad(self.h, table, self.targets, self.lse, dnll, self.dh, d_table, self.scratch)
        z.zero_layer_norm_grad(self.dh, self.s, self.mean, self.rstd, w, self.ds, d_w, d_b, self.scratch)
        z.zero_embed_grad(self.ds, self.tokens, d_table, self.scratch, scale=self.scale, accumulate=True)

    def clip(self, most):
        grads = list(self.views(self.grad))
        z.zero_grad_norm(grads, self.norm, self.scratch, norms=self.norms, dev_status=self.status)
        for flat in self.clipped:
            z.zero_grad_clip(grads, self.norm, most, outs=list(self.views(flat)))

    def preference(self, ref):
        args = (self.targets, self.offsets)
        z.zero_preference(self.nll, ref, *args, self.loss, self.slope, self.ratios, self.counts,
                          self.scratch, beta=0.3, smoothing=0.1, dev_status=self.status)
        z.zero_preference_grad(*args, self.slope, self.counts, self.d_pair, self.dnll)

    def policy(self, old, ref):
        how = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1, average=True)
        args = (self.nll, old, ref, self.adv, self.targets, self.offsets)
        z.zero_policy(*args, self.seq_loss, self.kl, self.cut, self.counts, self.scratch,
                      dev_status=self.status, **how)
        z.zero_policy_grad(*args, self.counts, self.d_seq, self.dnll, **how)

    def exact(self, loss_of):
        """The parameters' gradients of loss_of(nll, each sequence's tokens that count)."""
        table, w, b = (p.to(R.F).requires_grad_() for p in self.views(self.replicas[0]))
        s = table[self.tokens] * self.scale + self.res.to(R.F)
        m = s.mean(1, keepdim=True)
        h = (s - m) / ((s - m).square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b
        l = h @ table.T
        at = l.gather(1, self.targets.clamp(min=0)[:, None])[:, 0]
        nll = torch.logsumexp(l, 1) - at
        live = [lo + (self.targets[lo:hi] >= 0).nonzero()[:, 0] for lo, hi in self.seqs]
        loss = loss_of(nll, live)
        loss.backward()
        return loss, nll.detach(), [p.grad for p in (table, w, b)]


# What is rounded to bf16 on the way (x, s, h, P, dh, ds) is off by U16 / sqrt(3) in norm each:
# 0.006 together.  h's rounding moves a logit, of size 0.3 sqrt(136) = 3.5, by 0.008, and so a
# token's loss: r of the policy by 0.008 of itself, z of a pair of 40 tokens by 0.3 * 0.008 *
# sqrt(40) = 0.015 and the pair's slope by about as much of itself.  0.03 leaves room for
# their sum; a wrong term is off by its whole size.
CLOSE = 0.03


def check(m, loss, want_loss, grads):
    assert abs(loss - want_loss.item()) <= CLOSE * (abs(want_loss.item()) + 0.1)
    for got, want in zip(m.views(m.grad), grads):
        R.norm_close(got, want, CLOSE)
    m.clip(1e-3)
    each = torch.stack([g.to(R.F).norm() for g in m.views(m.grad)])
    R.within(m.norms, each, each * 64 * R.U32)
    coef = torch.tensor(1e-3).double() / (m.norm.cpu().double() + 1e-6)
    want = m.grad if coef >= 1 else (m.grad.float() * coef.float().item()).to(BF)
    assert all(torch.equal(c, want) for c in m.clipped)
    assert z.zero_get_device_status(m.status) == (0, 0)


def test_preference_step():
    m = Model()
    m.forward()
    # the reference's losses: near the model's, with anything where nothing counts
    ref = torch.where(m.targets >= 0, m.nll + m.near, torch.full_like(m.nll, float("nan")))
    ref[:3] = ref[-2:] = float("inf")
    m.dnll[:3] = m.dnll[-2:] = 0                              # tokens of no sequence stay as they are
    m.preference(ref)
    m.targets[:3] = m.targets[-2:] = -1
    m.backward(m.dnll)

    def loss_of(nll, live):
        q = torch.stack([(ref[t].to(R.F) - nll[t]).sum() for t in live])
        d = 0.3 * (q[0::2] - q[1::2])
        return (0.9 * torch.nn.functional.softplus(-d) + 0.1 * torch.nn.functional.softplus(d)).mean()
    want, _, grads = m.exact(loss_of)
    check(m, m.loss.mean().item(), want, grads)


def test_policy_step_and_optimizer():
    m = Model(seed=4)
    m.forward()
    nll = m.nll.clone()
    old, ref = nll + 0.5 * m.near, nll - m.near
    m.dnll.zero_()
    m.policy(old, ref)
    m.targets[:3] = m.targets[-2:] = -1
    m.backward(m.dnll)

    def loss_of(x, live):
        terms = []
        for i, t in enumerate(live):
            r = torch.exp(old[t].to(R.F) - x[t])
            d = x[t] - ref[t].to(R.F)
            A = m.adv[i].to(R.F)
            # (which tokens are clipped is decided at the kernel's own losses)
            at = torch.exp(old[t].to(R.F) - nll[t].to(R.F))
            cut = (at > 1.3) if A > 0 else (at < 0.8)
            bound = 1.3 if A > 0 else 0.8
            e = -torch.where(cut, torch.full_like(r, bound), r) * A + 0.1 * (torch.expm1(d) - d)
            terms.append(e.mean() if t.numel() else e.sum())
        return torch.stack(terms).mean()
    want, _, grads = m.exact(loss_of)
    check(m, m.seq_loss.mean().item(), want, grads)
    assert 0 < int(m.cut.sum()) < int(m.counts.sum())
    before = m.replicas[0].clone()
    state = [torch.zeros_like(m.master) for _ in range(2)]
    z.zero_step(m.plan, m.clipped, m.master, *state, m.replicas, z.hparams(lr=1e-2), 1)
    assert torch.equal(m.replicas[0], m.replicas[1]) and not torch.equal(before, m.replicas[0])


def test_the_whole_step_in_a_graph():
    """Captured once, replayed on other tokens and advantages: the eager calls' bits."""
    m = Model(seed=7)

    def step():
        m.forward()
        m.dnll.zero_()
        m.policy(old, ref)
        m.backward(m.dnll)
        m.clip(1e-3)
    old, ref = torch.zeros(m.T, device="cuda"), torch.zeros(m.T, device="cuda")
    m.forward()
    old.copy_(m.nll + 0.5 * m.near)
    ref.copy_(m.nll - m.near)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        step()
    g = R.gen(11)
    for _ in range(3):
        m.tokens.copy_(torch.randint(0, m.V, (m.T,), generator=g, device="cuda"))
        m.adv.copy_(torch.randn(m.adv.numel(), generator=g, device="cuda"))
        step()
        want = [t.clone() for t in (m.grad, m.clipped[0], m.seq_loss, m.kl, m.norm, m.dnll)]
        for t in (m.grad, m.clipped[0], m.seq_loss, m.kl, m.norm):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in
                   zip((m.grad, m.clipped[0], m.seq_loss, m.kl, m.norm, m.dnll), want))
