"""Training steps of a small pre-norm language model on the library's operators: the sparse
feed-forward layer between layer norms, the cross entropy of the vocabulary, and the clipping of
all gradients.

    x_0 = embedding(token);  a = norm(x);  x <- x + ffn(a)  per block;  loss = xent(norm(x) head^T)

Every operator's backward is called by hand, in the order in which the gradients arise; nothing
of the [tokens][vocabulary] logits is kept. The data are synthetic: the next token is a fixed
permutation of the current one, except for a tenth that is random.

    python examples/train_step.py [--steps 30] [--dtype bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_sparse_transformer_up_amd as tw  # noqa: E402

TILE_W, SLOTS = 128, 16


class Model:
    """fp32 master weights; the products read them in ``dtype``."""

    def __init__(self, vocab, d, f, blocks, dtype, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std
        self.dtype, self.blocks = dtype, blocks
        self.emb = randn(vocab, d, std=1.0).to(dtype)
        self.p = {"head": randn(vocab, d, std=d ** -0.5), "norm.w": torch.ones(d, device=device),
                  "norm.b": torch.zeros(d, device=device)}
        for i in range(blocks):
            # about 1 % of the hidden units fire at unit-spread inputs
            self.p.update({f"{i}.w1t": randn(f, d, std=d ** -0.5), f"{i}.b1": torch.full((f,), -2.326, device=device),
                           f"{i}.w2": randn(f, d, std=f ** -0.5), f"{i}.norm.w": torch.ones(d, device=device),
                           f"{i}.norm.b": torch.zeros(d, device=device)})

    def __call__(self, name):
        return self.p[name].to(self.dtype)


def loss_and_gradients(m: Model, tokens, targets, l1_coef=0.0):
    """Mean loss over the tokens with a target (targets >= 0) and the gradients by name."""
    # forward: x is the residual stream, y the last block's output, not yet added to it
    x, y, saved = m.emb[tokens], None, []
    for i in range(m.blocks):
        a, x, mean, rstd = tw.layer_norm_fwd(x, m.p[f"{i}.norm.w"], m.p[f"{i}.norm.b"], residual=y)
        w1t, w2 = m(f"{i}.w1t"), m(f"{i}.w2")
        y, h = tw.twell_ffn_fwd(a, w1t, m.p[f"{i}.b1"], w2, TILE_W, SLOTS, ovf_cap=len(tokens), y_dtype=m.dtype)
        saved.append((a, x, mean, rstd, w1t, w2, h))
    a, x, mean, rstd = tw.layer_norm_fwd(x, m.p["norm.w"], m.p["norm.b"], residual=y)

    # the loss and the way back; dx is the residual stream's gradient
    n = (targets >= 0).sum().clamp(min=1)
    dloss = (1.0 / n).expand(len(tokens)).contiguous()
    grads = {}
    loss, _, da, grads["head"] = tw.linear_xent_fwd_bwd(a, m("head"), targets, dloss)
    dx, grads["norm.w"], grads["norm.b"] = tw.layer_norm_bwd(da, x, m.p["norm.w"], mean, rstd)
    for i in reversed(range(m.blocks)):
        a, x, mean, rstd, w1t, w2, h = saved[i]
        da, grads[f"{i}.w1t"], grads[f"{i}.w2"], grads[f"{i}.b1"] = tw.twell_ffn_bwd(a, w1t, w2, h, dx, l1_coef)
        dx, grads[f"{i}.norm.w"], grads[f"{i}.norm.b"] = tw.layer_norm_bwd(da, x, m.p[f"{i}.norm.w"], mean, rstd, dres=dx)
    return loss.sum() / n, grads


def train_step(m: Model, tokens, targets, lr, max_norm):
    """One clipped gradient descent step in place: (loss, gradient norm)."""
    loss, grads = loss_and_gradients(m, tokens, targets)
    norm, clipped = tw.grad_clip(list(grads.values()), max_norm)
    for name, g in zip(grads, clipped):
        m.p[name].sub_(g, alpha=lr)
    return loss, norm


def batch(vocab, n, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    perm = torch.randperm(vocab, generator=torch.Generator(device=device).manual_seed(1), device=device)
    tokens = torch.randint(0, vocab, (n,), generator=g, device=device)
    noise = torch.rand(n, generator=g, device=device) < 0.1
    targets = torch.where(noise, torch.randint(0, vocab, (n,), generator=g, device=device), perm[tokens])
    targets[:: 16] = -100                                   # positions that are not scored
    return tokens, targets


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--vocab", type=int, default=997)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args(argv)
    m = Model(a.vocab, 256, 1024, 2, torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    losses = []
    for step in range(a.steps):
        tokens, targets = batch(a.vocab, a.tokens, step)
        loss, norm = train_step(m, tokens, targets, lr=10.0, max_norm=0.5)
        losses.append(float(loss))
        print(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}", flush=True)
    return losses


if __name__ == "__main__":
    main()
