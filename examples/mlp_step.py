"""One training step of the MLP half of a GPT block and its loss, through the
library's operators: up projection with GELU, down projection with dropout
and the residual, cross-entropy over the vocabulary, and every gradient.

    python examples/mlp_step.py [--tokens 8192] [--hidden 6144] [--vocab 128256] [--check]

``--check`` runs a small step and compares it with autograd in 64 bits.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pmm_fc_layer_gb300 as fc  # noqa: E402


class MlpStep:
    """Weights, buffers and workspace of the step; nothing is allocated per
    call.  X [T x H] bf16, labels [T] int32; W1 [H x F], W2 [F x H], head
    [H x V], biases fp32."""

    def __init__(self, T, H, F, V, p=0.1, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        bf = dict(device=device, dtype=torch.bfloat16)
        self.T, self.H, self.F, self.V, self.p = T, H, F, V, p
        self.W1 = torch.randn(H, F, device=device, generator=g).mul_(0.02).to(torch.bfloat16)
        self.W2 = torch.randn(F, H, device=device, generator=g).mul_(0.02).to(torch.bfloat16)
        self.head = torch.randn(H, V, device=device, generator=g).mul_(0.02).to(torch.bfloat16)
        self.b1 = torch.randn(F, device=device, generator=g).mul_(0.1)
        self.b2 = torch.randn(H, device=device, generator=g).mul_(0.1)
        self.rng = torch.tensor([1234, 0], device=device)  # the step's seed and offset
        self.Z1, self.A1, self.dZ1 = (torch.empty(T, F, **bf) for _ in range(3))
        self.Y, self.dY, self.dZ2, self.dX = (torch.empty(T, H, **bf) for _ in range(4))
        self.dW1, self.dW2, self.dhead = (torch.empty_like(w) for w in (self.W1, self.W2, self.head))
        self.db1, self.db2 = torch.empty(F, device=device), torch.empty(H, device=device)
        self.token_loss, self.loss = torch.empty(T, device=device), torch.empty(1, device=device)
        self.kept = torch.empty(1, device=device, dtype=torch.int32)
        need = max(fc.axonn_linear_ce_workspace_size(T, H, V), fc.axonn_epi_workspace_size(T, F),
                   fc.axonn_epi_workspace_size(T, H))
        self.ws = torch.empty(need, device=device, dtype=torch.uint8)

    def __call__(self, X, labels, keep=None):
        T, H, F, up, down = self.T, self.H, self.F, fc.Shape(self.T, self.H, self.F), fc.Shape(self.T, self.F, self.H)
        # forward: A1 = gelu(X W1 + b1);  Y = X + D(A1 W2 + b2);  loss over Y head
        fc.axonn_fc_fwd_epi(X, self.W1, self.A1, up, bias=self.b1, act="gelu_tanh", pre=self.Z1)
        fc.axonn_fc_fwd_epi(self.A1, self.W2, self.Y, down, bias=self.b2, residual=X, p=self.p, rng=self.rng)
        fc.axonn_linear_ce(self.Y, self.head, labels, self.token_loss, self.loss, self.kept, self.ws,
                           keep=keep, dX=self.dY, dW=self.dhead)
        # backward: through the dropout, the down and the up projection, and the residual
        fc.axonn_epi_bwd(self.dY, self.dZ2, dbias=self.db2, p=self.p, rng=self.rng, ws=self.ws)
        fc.axonn_fc_wgrad(self.A1, self.dZ2, self.dW2, down)
        fc.axonn_fc_dgrad_epi(self.dZ2, self.W2, self.dZ1, down, pre=self.Z1, act="gelu_tanh",
                              dbias=self.db1, ws=self.ws)
        fc.axonn_fc_wgrad(X, self.dZ1, self.dW1, up)
        fc.axonn_fc_dgrad_epi(self.dZ1, self.W1, self.dX, up, residual=self.dY)
        return self.loss


def reference(step, X, labels, keep=None):
    """The same step by autograd in 64 bits (the mask read off the library's
    dropout of ones)."""
    ones = torch.ones(step.T, step.H, device=X.device, dtype=torch.bfloat16)
    mask = torch.empty_like(ones)
    fc.axonn_dropout(ones, mask, step.p, step.rng)
    thr = int(65536 * step.p + 0.5)
    mask = (mask != 0).double() * (65536 / (65536 - thr))
    leaf = {n: getattr(step, n).double().requires_grad_(True) for n in ("W1", "W2", "head", "b1", "b2")}
    x = X.double().requires_grad_(True)
    a = torch.nn.functional.gelu(x @ leaf["W1"] + leaf["b1"], approximate="tanh")
    y = x + mask * (a @ leaf["W2"] + leaf["b2"])
    count = (labels >= 0) & (labels < step.V)
    if keep is not None:
        count &= keep != 0
    loss = torch.nn.functional.cross_entropy((y @ leaf["head"])[count], labels[count].long())
    loss.backward()
    return loss.detach(), {"dX": x.grad, **{"d" + n: t.grad for n, t in leaf.items()}}


def check(T=300, H=256, F=1024, V=1003, p=0.1):
    """Relative errors (2-norm) of the loss and of each gradient."""
    step = MlpStep(T, H, F, (V + 7) // 8 * 8, p)
    step.head, step.dhead, step.V = step.head[:, :V], step.dhead[:, :V], V
    X = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    labels = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    labels[::11] = -100
    keep = (torch.rand(T, device="cuda") < 0.5).to(torch.uint8)
    loss = float(step(X, labels, keep))
    fc.axonn_sync_status()
    want, grads = reference(step, X, labels, keep)
    out = {"loss": abs(loss - float(want)) / float(want)}
    for name, ref in grads.items():
        out[name] = float((getattr(step, name).double() - ref).norm() / ref.norm())
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=6144)
    ap.add_argument("--vocab", type=int, default=128256)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--check", action="store_true")
    args = ap.parse_args()
    if args.check:
        for name, err in check().items():
            print(f"{name:6s} {err:.2e}")
        return
    T, H, V = args.tokens, args.hidden, args.vocab
    step = MlpStep(T, H, 4 * H, V)
    X = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    labels = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(3 + args.steps):
        if i == 3:
            begin.record()
        step.rng[1] = i
        step(X, labels)
    end.record()
    fc.axonn_sync_status()
    ms = begin.elapsed_time(end) / args.steps
    flops = 12 * T * H * 4 * H + 6 * T * H * V
    print(f"{ms:.3f} ms a step, {flops / ms / 1e9:.0f} TFLOP/s of {flops:.3e} flops, loss {float(step.loss):.4f}")


if __name__ == "__main__":
    main()
