"""A small language model trained with every optimizer operator of the library.

Muon steps the hidden matrices (int8 momentum, Newton-Schulz), AdamW the rest:
embedding and head with 8-bit states, norm gains with 32-bit states.  One
global norm over all gradients gives the clip factor; the Muon gradients are
scaled by it in place, the AdamW step takes it as an argument.  A batch whose
norm is not finite is left out as a whole: the AdamW step would write nothing
by itself, but the Muon step reads its gradients whatever they hold, so the
program looks at the factor before it.  The embedding's rows and its gradient
are the library's as well.

The data are synthetic: a fixed random permutation of the vocabulary, each
token followed by its image, so a model that learns reaches a loss near 0.

    python examples/train_lm.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_momentum_newton_amd as q  # noqa: E402

VOCAB, WIDTH, HIDDEN, LAYERS, BATCH = 512, 256, 512, 2, 1024


class Embedding(torch.autograd.Function):
    """Rows of the table; their gradients are added to the table's buffer, in
    an order that the tokens determine.  The buffer is the one that the table
    has when the rows are taken.  Autograd itself is told of no gradient: hooks
    on the table and torch.autograd.grad see none."""

    @staticmethod
    def forward(ctx, table, tokens):
        ctx.save_for_backward(tokens)
        ctx.grad = table.grad
        return q.embedding_lookup(tokens, table.detach())

    @staticmethod
    def backward(ctx, dy):
        q.embedding_grad(*ctx.saved_tensors, dy.contiguous(), ctx.grad, accumulate=True)
        return None, None


class Model:
    """Residual blocks x + W2 relu(W1 (g * norm(x))), fp32 weights; each weight
    has a gradient buffer of its own that backward accumulates into."""

    def __init__(self, device, seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.weights = {}

        def param(name, *shape, std):
            w = torch.randn(*shape, generator=gen, device=device) * std if std else torch.ones(*shape, device=device)
            self.weights[name] = w.requires_grad_()
            w.grad = torch.zeros_like(w)

        param("embedding", VOCAB, WIDTH, std=0.5)
        for k in range(LAYERS):
            param(f"gain{k}", WIDTH, std=0)
            param(f"up{k}", HIDDEN, WIDTH, std=WIDTH ** -0.5)
            param(f"down{k}", WIDTH, HIDDEN, std=HIDDEN ** -0.5)
        param("gain_out", WIDTH, std=0)
        param("head", VOCAB, WIDTH, std=0.02)

    def loss(self, tokens, targets):
        w = self.weights

        def norm(x, gain):
            return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain

        x = Embedding.apply(w["embedding"], tokens)
        for k in range(LAYERS):
            x = x + torch.relu(norm(x, w[f"gain{k}"]) @ w[f"up{k}"].t()) @ w[f"down{k}"].t()
        logits = norm(x, w["gain_out"]) @ w["head"].t()
        return torch.nn.functional.cross_entropy(logits, targets)


class Optimizer:
    def __init__(self, model, lr_muon=0.01, lr_adamw=3e-3, max_norm=1.0):
        w = {k: (p.detach(), p.grad) for k, p in model.weights.items()}
        self.lr_adamw, self.max_norm, self.steps = lr_adamw, max_norm, 0
        muon = [k for k in w if k.startswith(("up", "down"))]
        rest = [k for k in w if k not in muon]
        # every gradient: one norm
        self.all_grads = q.GradPlan([g for _, g in w.values()])
        self.muon_grads = q.GradPlan([w[k][1] for k in muon])
        self.ws = self.all_grads.workspace()
        self.norm, self.coef = (torch.zeros(1, device=self.all_grads.device) for _ in range(2))
        # Muon: int8 momentum, one norm group per matrix
        triples, self.mats, segments = [], [], []
        for i, k in enumerate(muon):
            weight, grad = w[k]
            codes = torch.zeros(weight.numel(), dtype=torch.int8, device=weight.device)
            absmax = torch.zeros(-(-weight.numel() // q.BLOCK), device=weight.device)
            triples.append((codes, absmax, grad.view(-1)))
            self.mats.append((*weight.shape, *weight.shape, weight))
            segments.append((i, 0, weight.numel(), i))
        self.muon_plan = q.Plan(triples, segments, len(muon))
        self.muon_hp = q.make_hparams(lr_full=lr_muon, period=1, precision="bf16", weight_decay=0.01)
        self.muon_ws = torch.empty(q.muon_step_workspace_bytes(self.muon_plan, None, self.mats, hparams=self.muon_hp),
                                   dtype=torch.uint8, device=self.all_grads.device)
        # AdamW: 8-bit states for the two large tables, 32-bit ones for the gains
        entries = []
        for k in rest:
            weight, grad = w[k]
            table = weight.dim() == 2
            state = q.AdamWState(weight.numel(), bits=8 if table else 32, device=weight.device)
            entries.append((weight, grad, state, None, 1.0, 0.01 if table else 0.0))
        self.adamw_plan = q.AdamWPlan(entries)

    def step(self):
        """One step; False, with no weight or state written, where the
        gradients' norm is not finite."""
        q.grad_norm(self.all_grads, self.max_norm, norm=self.norm, coef=self.coef, ws=self.ws)
        if self.coef.isnan().item():      # the host waits for the norm
            return False
        self.steps += 1
        q.grad_scale(self.muon_grads, self.coef)
        q.muon_step(self.muon_plan, None, self.mats, self.steps, self.muon_hp, ws=self.muon_ws)
        q.adamw_step(self.adamw_plan, self.steps, lr=self.lr_adamw, betas=(0.9, 0.99), grad_scale=self.coef,
                     rounding="stochastic", seed=1)
        return True


def main(steps=120, device="cuda", report=print):
    """Trains and returns the losses."""
    gen = torch.Generator(device=device)
    gen.manual_seed(7)
    follows = torch.randperm(VOCAB, generator=gen, device=device)
    model = Model(device)
    opt = Optimizer(model)
    losses = []
    for t in range(steps):
        tokens = torch.randint(0, VOCAB, (BATCH,), generator=gen, device=device)
        for p in model.weights.values():
            p.grad.zero_()
        loss = model.loss(tokens, follows[tokens])
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and t % 20 == 0:
            report(f"step {t}: loss {loss.item():.4f}, gradient norm {opt.norm.item():.4f}")
    losses = torch.stack(losses).tolist()
    if report:
        report(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
