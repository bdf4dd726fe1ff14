"""A training step with every parameter of a model updated on the GPU.

A small next-token model learns a synthetic Markov chain.  Its weights are
bf16 with fp32 masters.  After the backward pass one call takes the global
norm of all gradients; its clip factor stays on the GPU and goes into both
updates: Dion3 for the square hidden matrices (one stack per shape), AdamW
for the embedding, the head and the vectors.  Nothing in the step waits for
the GPU, and a step whose gradients are not finite changes nothing.

    python examples/train_step.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gram_newton_schulz_amd as gns  # noqa: E402
from gram_newton_schulz_amd import synth  # noqa: E402

VOCAB, CONTEXT, WIDTH, BLOCKS, BATCH = 256, 4, 512, 6, 1024


class Model(torch.nn.Module):
    """Embeddings of the last CONTEXT tokens, residual blocks of two square
    matrices each, a head."""

    def __init__(self, generator):
        super().__init__()

        def weight(*shape, scale):
            return torch.nn.Parameter((torch.randn(*shape, generator=generator) * scale).bfloat16())

        self.embedding = weight(VOCAB, WIDTH // CONTEXT, scale=1.0)
        self.up = torch.nn.ParameterList([weight(WIDTH, WIDTH, scale=WIDTH ** -0.5) for _ in range(BLOCKS)])
        self.down = torch.nn.ParameterList([weight(WIDTH, WIDTH, scale=WIDTH ** -0.5) for _ in range(BLOCKS)])
        self.gain = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(WIDTH, dtype=torch.bfloat16))
                                            for _ in range(BLOCKS)])
        self.head = weight(VOCAB, WIDTH, scale=WIDTH ** -0.5)

    def forward(self, tokens):
        x = self.embedding[tokens].reshape(tokens.shape[0], WIDTH)
        for up, down, gain in zip(self.up, self.down, self.gain):
            h = x * torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6).bfloat16() * gain
            x = x + torch.relu(h @ up.t()) @ down.t()
        return x @ self.head.t()


def grad_buffer(params):
    """One bf16 buffer whose slices are the parameters' gradients."""
    flat = torch.zeros(sum(p.numel() for p in params), dtype=torch.bfloat16, device=params[0].device)
    at = 0
    for p in params:
        p.grad = flat[at:at + p.numel()].view_as(p)
        at += p.numel()
    return flat


class Trainer:
    def __init__(self, model, lr=0.02, adam_lr=3e-3, max_norm=0.5, fraction=0.5):
        self.matrices = list(model.up) + list(model.down)
        self.rest = [model.embedding, model.head] + list(model.gain)
        self.lr, self.adam_lr, self.max_norm = lr, adam_lr, max_norm
        # Dion3's state: the stack of masters, its gradients as one [batch, n, m] tensor
        n = len(self.matrices)
        self.G = grad_buffer(self.matrices).view(n, WIDTH, WIDTH)
        self.W = torch.stack([p.detach().float() for p in self.matrices])
        self.M, self.v = torch.zeros_like(self.W), torch.zeros(n, WIDTH, device=self.W.device)
        self.k = gns.select_count(WIDTH, fraction)
        self.workspace = torch.empty(gns.dion3_workspace_bytes(torch.bfloat16, n, WIDTH, WIDTH, self.k),
                                     dtype=torch.uint8, device=self.W.device)
        # AdamW's state: fp32 masters and moments, and the number of its updates, which is counted on the
        # GPU because only the GPU knows which steps were skipped; every step refreshes the bf16 weights
        self.updates = torch.zeros(1, dtype=torch.int64, device=self.W.device)
        self.flat_rest = grad_buffer(self.rest)
        self.masters = [p.detach().float() for p in self.rest]
        decayed = [1.0 if p.dim() == 2 else 0.0 for p in self.rest]
        self.adamw = gns.adamw_list(self.masters, [p.grad for p in self.rest],
                                    [torch.zeros_like(w) for w in self.masters],
                                    [torch.zeros_like(w) for w in self.masters],
                                    copies=[p.detach() for p in self.rest], wd_scales=decayed)
        # every gradient of the model, for the norm
        self.grads = gns.tensor_list([self.G] + [p.grad for p in self.rest])

    def zero_grad(self):
        self.G.zero_()
        self.flat_rest.zero_()

    def step(self):
        got = gns.grad_norm(self.grads, max_norm=self.max_norm)
        clip = got.clip
        gns.dion3_step(self.W, self.G, self.M, self.v, self.k, synth.NS5_MUON, lr=self.lr, mu=0.9,
                       grad_scale=clip, workspace=self.workspace)
        torch._foreach_copy_([p.detach() for p in self.matrices], list(self.W))
        gns.adamw_step(self.adamw, count=self.updates, lr=self.adam_lr, betas=(0.9, 0.95), weight_decay=0.01,
                       grad_scale=clip)
        return got


def batches(generator, device):
    """Windows of a Markov chain: the next token follows from the last two,
    except once in eight."""
    table = torch.randint(VOCAB, (VOCAB, VOCAB), generator=generator)
    while True:
        seq = torch.randint(VOCAB, (BATCH, CONTEXT + 1), generator=generator)
        seq[:, -3] %= 16
        seq[:, -2] %= 16
        noise = torch.rand(BATCH, generator=generator) < 0.125
        seq[:, -1] = torch.where(noise, seq[:, -1], table[seq[:, -3], seq[:, -2]])
        yield seq[:, :-1].to(device), seq[:, -1].to(device)


def train(steps, seed=0, log=print):
    """(losses, norms) of `steps` steps."""
    gen = torch.Generator().manual_seed(seed)
    model = Model(gen).cuda()
    trainer = Trainer(model)
    losses, norms = [], []
    data = batches(gen, "cuda")
    for i in range(steps):
        tokens, target = next(data)
        trainer.zero_grad()
        loss = torch.nn.functional.cross_entropy(model(tokens).float(), target)
        loss.backward()
        got = trainer.step()
        losses.append(loss.detach())
        norms.append(got.norm)
        if log and (i % 10 == 0 or i == steps - 1):
            log(f"step {i:4d}  loss {float(losses[-1]):.3f}  norm {float(got.norm):.3f}  clip {float(got.clip):.3f}")
    return torch.stack(losses).cpu(), torch.stack(norms).cpu()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)
