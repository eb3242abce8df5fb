"""Trains the adapters that the library serves: a few LoRA adapters over two
frozen linear layers and a frozen head, tokens of all adapters mixed in one
batch, as they are when the adapters are served.

    python examples/train_adapters.py [--steps 40] [--device cuda]

A step is one pass of the library's own calls:

    lora_meta_prepare      which tokens belong to which adapter
    add_lora_linear        each layer's adapters, on top of the frozen product
    lora_cross_entropy     the loss of the head's logits and its gradient
    lora_linear_backward   gradients of A and B, and of the layer's input
    lora_orthogonalize     the momentum of all adapters made orthogonal
                           (the update of the Muon optimiser)

The frozen products are torch matmuls.  Workspaces and buffers are allocated
once.  The data are random: every adapter learns its own map from 512 inputs
to labels.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import expand_gemm_gb300 as eg


class Layer:
    """A frozen linear layer of size hidden x hidden with stacked adapters."""

    def __init__(self, hidden, rank, loras, scale, tokens, device, gen):
        bf16 = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.scale = scale
        self.base = (torch.randn(hidden, hidden, generator=gen) * hidden ** -0.5).to(**bf16)
        # masters in fp32, what the kernels read in bf16; B starts at zero
        self.masters = [(torch.randn(loras, rank, hidden, generator=gen) * hidden ** -0.5).to(**f32),
                        torch.zeros(loras, hidden, rank, **f32)]
        self.weights = [m.to(torch.bfloat16) for m in self.masters]
        self.grads = [torch.empty_like(w) for w in self.weights]
        self.momenta = [torch.zeros_like(m) for m in self.masters]
        self.updates = [torch.empty_like(w) for w in self.weights]
        self.buffer = torch.zeros(1, tokens, rank, **f32)

    def forward(self, x, meta):
        self.x = x
        y = x + x @ self.base.T
        self.buffer.zero_()
        eg.add_lora_linear(y, x, [self.weights[0]], [self.weights[1]], None, self.scale, [y.shape[1]], meta,
                           buffer=self.buffer)
        return y

    def backward(self, dy, meta, workspace):
        """The adapters' gradients; returns the gradient of the input."""
        dx = dy + dy @ self.base
        eg.lora_linear_backward(dy, self.x, self.buffer, [self.weights[0]], [self.weights[1]], self.scale, meta,
                                dx=dx, d_lora_a=[self.grads[0]], d_lora_b=[self.grads[1]], workspace=workspace)
        return dx

    def update(self, lr, beta):
        for master, weight, grad, momentum, update in zip(self.masters, self.weights, self.grads, self.momenta,
                                                          self.updates):
            momentum.mul_(beta).add_(grad)
            # adapters whose momentum is zero get a zero update
            eg.lora_orthogonalize(momentum, update)
            master.sub_(update, alpha=lr)
            weight.copy_(master)


def train(steps=40, tokens=512, hidden=512, vocab=2000, rank=16, loras=4, scale=2.0, lr=0.05, beta=0.9, device="cuda",
          seed=0):
    """The mean loss of every step."""
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, loras, (tokens,), generator=gen, dtype=torch.int32).to(device)
    x = torch.randn(tokens, hidden, generator=gen).to(device, torch.bfloat16)
    head = (torch.randn(vocab, hidden, generator=gen) * hidden ** -0.5).to(device, torch.bfloat16)
    targets = torch.randint(0, vocab, (tokens,), generator=gen, dtype=torch.int32)
    targets[::8] = -100                                   # positions that are not learnt
    learnt = int((targets >= 0).sum())
    targets = targets.to(device)
    weight = torch.full((tokens,), 1.0 / learnt, device=device)
    layers = [Layer(hidden, rank, loras, scale, tokens, device, gen) for _ in range(2)]
    meta = eg.LoRAKernelMeta.make(loras, tokens, device)
    loss = torch.empty(tokens, device=device)
    dh = torch.empty_like(x)
    loss_ws = torch.empty(eg.lora_cross_entropy_workspace(tokens, hidden, vocab, hidden_grad=True, device=device),
                          dtype=torch.uint8, device=device)
    back_ws = torch.empty(eg.lora_linear_backward_workspace(tokens, hidden, [hidden], rank, loras, device=device),
                          dtype=torch.uint8, device=device)
    history = torch.empty(steps, device=device)
    for step in range(steps):
        eg.lora_meta_prepare(ids, meta)
        h = x
        for layer in layers:
            h = layer.forward(h, meta)
        eg.lora_cross_entropy(h, head, targets, loss, token_weight=weight, hidden_grad=dh, workspace=loss_ws)
        history[step] = loss.sum()
        grad = dh
        for layer in reversed(layers):
            grad = layer.backward(grad, meta, back_ws)
        for layer in layers:
            layer.update(lr * (1.0 - step / steps), beta)
    return history.tolist()


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=40)
    parser.add_argument("--device", default="cuda")
    args = parser.parse_args()
    for step, loss in enumerate(train(args.steps, device=args.device)):
        print("step %3d  loss %.4f" % (step, loss))


if __name__ == "__main__":
    main()
