"""One training loop from token ids to the optimizer step, on one GPU.

The smallest model that uses every operator: the sum of a token's and a
position's embedding, one root-mean-square norm that keeps an 8-bit
checkpoint, and the softmax cross entropy against the same (tied) token table.

    x = scale * table[tok], r = wpe[pos]; h = norm(x + r); loss = xent(h table^T)

The parameters are one flat bf16 vector per data-parallel rank, and every
gradient is written into its tensor's part of the rank's flat gradient buffer:
the table's by zero_xent_grad first, then zero_embed_grad adds to it.  zero_step
reduces the ranks' gradients, updates the sharded state and writes all replicas.

    python examples/tied_lm_step.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_optimizer_step_rs_gb300 as z  # noqa: E402


class TiedModel:
    def __init__(self, V=1000, D=256, ctx=64, batch=8, R=2, seed=0):
        self.V, self.D, self.ctx, self.T, self.R = V, D, ctx, batch * ctx, R
        self.scale = math.sqrt(D)
        self.plan = z.Plan([V * D, ctx * D, D], R=R, M=1, stage=2)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n, dev = self.plan.N, "cuda"
        start = torch.randn(n, generator=g, device=dev) * 0.02
        start[-D:] = 1.0                                        # the norm's weight
        self.replicas = [start.to(torch.bfloat16) for _ in range(R)]
        self.grads = [torch.zeros(n, dtype=torch.bfloat16, device=dev) for _ in range(R)]
        self.master = torch.zeros(self.plan.padded, device=dev)
        self.master[:n] = start
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.pos = torch.arange(ctx, device=dev).repeat(batch)

        # buffers that every pass uses again
        T = self.T
        bf = lambda: torch.empty((T, D), dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.x, self.r, self.h, self.dh, self.dx = bf(), bf(), bf(), bf(), bf()
        self.codes = torch.empty((T, D), dtype=torch.int8, device=dev)
        self.scales = torch.empty((T, -(-D // z.ZERO_NORM_BLOCK)), device=dev)
        self.rstd, self.loss, self.lse, self.dloss = (torch.empty(T, device=dev) for _ in range(4))
        size = max(z.zero_embed_grad_scratch_bytes(T, max(V, ctx), D),
                   z.zero_norm_grad_scratch_bytes(T, D), z.zero_xent_scratch_bytes(T, V, D),
                   z.zero_xent_grad_scratch_bytes(T, V, D))
        self.scratch = torch.empty(size, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def views(self, flat):
        """The token table, the position table and the norm's weight of a flat vector."""
        a, b, c, d = self.plan.tensor_offsets()
        return flat[a:b].view(self.V, self.D), flat[b:c].view(self.ctx, self.D), flat[c:d]

    def backward(self, rank, tokens, targets):
        """The rank's gradients, in its flat buffer; the mean loss of its tokens."""
        table, wpe, w = self.views(self.replicas[rank])
        d_table, d_wpe, d_w = self.views(self.grads[rank])
        s = self.scratch
        z.zero_embed(table, tokens, self.x, scale=self.scale, dev_status=self.status)
        z.zero_embed(wpe, self.pos, self.r)
        z.zero_norm(self.x, w, self.h, self.codes, self.scales, self.rstd, residual=self.r)
        z.zero_xent(self.h, table, targets, self.loss, self.lse, s, dev_status=self.status)
        count = (targets >= 0).sum().clamp(min=1)
        self.dloss.copy_(1.0 / count)
        # self.h could be given up here: the backward pass makes it again
        z.zero_norm_replay(self.codes, self.scales, self.rstd, w, self.h)
        z.zero_xent_grad(self.h, table, targets, self.lse, self.dloss, self.dh, d_table, s)
        z.zero_norm_grad(self.dh, self.codes, self.scales, self.rstd, w, self.dx, d_w, s)
        z.zero_embed_grad(self.dx, tokens, d_table, s, scale=self.scale, accumulate=True)
        z.zero_embed_grad(self.dx, self.pos, d_wpe, s)
        return self.loss.sum() / count

    def step(self, t, batches, lr=3e-3):
        """One optimizer step over the ranks' (tokens, targets); the mean loss, on the GPU."""
        losses = [self.backward(r, *batches[r]) for r in range(self.R)]
        z.zero_step(self.plan, self.grads, self.master, self.m, self.v, self.replicas,
                    z.hparams(lr=lr), step=t, dev_status=self.status)
        return torch.stack(losses).mean()


def synthetic(model, seed):
    """Sequences whose next token follows from the one before; a few targets ignored."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    tokens = torch.randint(0, model.V, (model.T,), generator=g, device="cuda")
    targets = (tokens * 7 + 3) % model.V
    targets[torch.rand(model.T, generator=g, device="cuda") < 0.1] = -1
    return tokens, targets


def main(steps=60):
    model = TiedModel()
    for t in range(1, steps + 1):
        loss = model.step(t, [synthetic(model, 2 * t + r) for r in range(model.R)])
        if t == 1 or t % 10 == 0:
            print(f"step {t}: loss {loss.item():.4f}")
    code, word = z.zero_get_device_status(model.status)
    print(f"device status {word} ({z.zero_status_string(code)})")


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
