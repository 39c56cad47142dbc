"""Training steps of a small pre-norm language model whose feed-forward blocks are dense and gated, on the
library's operators from the embedding to the optimizer.

    x_0 = gelu(embedding(token) w_in^T + b_in);  x <- x + block(norm(x))  per block;  loss = xent(norm(x) head^T)

Every operator's backward is called by hand, in the order in which the gradients arise. The weights are kept
in fp32; the products read copies in ``dtype``, which the AdamW step writes in the same pass. The gradients are
clipped inside the step by the norm over all of them. The data are synthetic: the next token is a fixed
permutation of the current one, except for a tenth that is random.

    python examples/dense_step.py [--steps 30] [--dtype bf16] [--states 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_sparse_transformer_up_amd as tw  # noqa: E402


class Model:
    """fp32 weights by name, and what the products read of them."""

    def __init__(self, vocab, d, f, blocks, dtype, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std
        self.dtype, self.blocks = dtype, blocks
        self.emb = randn(vocab, d, std=1.0).to(dtype)
        self.p = {"head": randn(vocab, d, std=d ** -0.5), "in.w": randn(d, d, std=d ** -0.5),
                  "in.b": torch.zeros(d, device=device), "norm.w": torch.ones(d, device=device),
                  "norm.b": torch.zeros(d, device=device)}
        for i in range(blocks):
            self.p.update({f"{i}.wg": randn(f, d, std=d ** -0.5), f"{i}.wu": randn(f, d, std=d ** -0.5),
                           f"{i}.w2": randn(f, d, std=f ** -0.5), f"{i}.bg": torch.zeros(f, device=device),
                           f"{i}.bu": torch.zeros(f, device=device), f"{i}.norm.w": torch.ones(d, device=device),
                           f"{i}.norm.b": torch.zeros(d, device=device)})
        self.refresh()

    def refresh(self):
        """The matrices as the products read them; vectors stay fp32."""
        self.w = {k: v.to(self.dtype) if v.dim() == 2 else v for k, v in self.p.items()}


def loss_and_gradients(m: Model, tokens, targets):
    """Mean loss over the tokens with a target (targets >= 0) and the gradients by name."""
    w, e = m.w, m.emb[tokens]
    x, pre = tw.linear_fwd(e, w["in.w"], bias=w["in.b"], act="gelu", want_pre=True)
    saved = []
    for i in range(m.blocks):
        a, _, mean, rstd = tw.layer_norm_fwd(x, w[f"{i}.norm.w"], w[f"{i}.norm.b"])
        y, g, u = tw.ffn_gated_dense_fwd(a, w[f"{i}.wg"], w[f"{i}.wu"], w[f"{i}.w2"], bg=w[f"{i}.bg"], bu=w[f"{i}.bu"],
                                         residual=x, act="silu", want_saved=True)
        saved.append((a, x, mean, rstd, g, u))
        x = y
    a, _, mean, rstd = tw.layer_norm_fwd(x, w["norm.w"], w["norm.b"])

    # the loss and the way back; dx is the residual stream's gradient
    n = (targets >= 0).sum().clamp(min=1)
    dloss = (1.0 / n).expand(len(tokens)).contiguous()
    grads = {}
    loss, _, da, grads["head"] = tw.linear_xent_fwd_bwd(a, w["head"], targets, dloss)
    dx, grads["norm.w"], grads["norm.b"] = tw.layer_norm_bwd(da, x, w["norm.w"], mean, rstd)
    for i in reversed(range(m.blocks)):
        a, x, mean, rstd, g, u = saved[i]
        da, grads[f"{i}.wg"], grads[f"{i}.wu"], grads[f"{i}.w2"], grads[f"{i}.bg"], grads[f"{i}.bu"] = tw.ffn_gated_dense_bwd(
            dx, a, w[f"{i}.wg"], w[f"{i}.wu"], w[f"{i}.w2"], g, u, act="silu", want_bias=True)
        dx, grads[f"{i}.norm.w"], grads[f"{i}.norm.b"] = tw.layer_norm_bwd(da, x, w[f"{i}.norm.w"], mean, rstd, dres=dx)
    _, grads["in.w"], grads["in.b"] = tw.linear_bwd(dx, e, w["in.w"], pre=pre, act="gelu", want_dx=False, want_bias=True)
    return loss.sum() / n, grads


class Adam:
    """The optimizer's states, in 32 or in 8 bits, and its step with clipping."""

    def __init__(self, m: Model, lr, states=32, decay=0.01, max_norm=1.0):
        self.names, self.t, self.lr, self.max_norm = list(m.p), 0, lr, max_norm
        p = [m.p[k] for k in self.names]
        if states == 8:
            st = [tw.adamw8_states(x) for x in p]
            self.states = dict(m=[s[0] for s in st], m_scales=[s[1] for s in st], v=[s[2] for s in st], v_scales=[s[3] for s in st])
        else:
            self.states = dict(m=[torch.zeros_like(x) for x in p], v=[torch.zeros_like(x) for x in p])
        self.decay = [decay if x.dim() == 2 else 0.0 for x in p]         # matrices only

    def step(self, m: Model, grads):
        """One step; returns the gradients' norm. bf16 matrices are rewritten by the step itself."""
        self.t += 1
        g = [grads[k] for k in self.names]
        norm = tw.grad_norm(g)
        bf16 = m.dtype == torch.bfloat16
        tw.adamw_step([m.p[k] for k in self.names], g, lr=self.lr, step=self.t, betas=(0.9, 0.95), weight_decay=self.decay, norm=norm,
                      max_norm=self.max_norm, copies=[m.w[k] if m.w[k] is not m.p[k] else None for k in self.names] if bf16 else None,
                      **self.states)
        if not bf16:
            m.refresh()
        return norm


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
    ap.add_argument("--states", type=int, choices=(8, 32), default=32)
    ap.add_argument("--vocab", type=int, default=997)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args(argv)
    m = Model(a.vocab, 256, 1024, 2, torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    opt, losses = Adam(m, lr=3e-3, states=a.states), []
    for step in range(a.steps):
        loss, grads = loss_and_gradients(m, *batch(a.vocab, a.tokens, step))
        norm = opt.step(m, grads)
        losses.append(float(loss))
        print(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}", flush=True)
    return losses


if __name__ == "__main__":
    main()
