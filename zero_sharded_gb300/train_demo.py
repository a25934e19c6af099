"""A training step from tokens to updated weights on the library's operators.

    python -m zero_sharded_gb300.train_demo [--steps N] [--tokens T] [--width D] [--hidden F] [--vocab V] [--layers L]

A residual network of gated blocks predicts each token's successor.  Per block

    u = x W_up^T;  a = silu(u);  y = a W_down^T;  h <- h + gate * norm(y);  x = norm(h)

Kept for the backward pass: x and a of every block and y as 8-bit checkpoints (cz_block_norm_fwd and cz_act_encode
write them), the residual stream in bf16.  The objective is cz_token_logp_fwd's mean log probability with a small entropy
bonus; its gradient (in place of the logits), the norms' gradients, the recomputation of u from x's checkpoint and the weight
gradients straight from the checkpoints into the flat gradient buffer lead to cz_muon_step_ex, which updates the
fp32 masters and the bf16 copies the next forward pass reads.  Plain matrix products are PyTorch's.
"""

from __future__ import annotations

import argparse

import torch

from . import cz

BF16 = torch.bfloat16


class Demo:
    def __init__(self, tokens: int = 1024, width: int = 256, hidden: int = 512, vocab: int = 1000, layers: int = 2,
                 seed: int = 0):
        self.T, self.D, self.F, self.V, self.L = tokens, width, hidden, vocab, layers
        gen = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.shapes = [s for _ in range(layers) for s in ((hidden, width), (width, hidden))] + [(vocab, width)]
        self.offsets = [0]
        for r, c in self.shapes:
            self.offsets.append(self.offsets[-1] + (r * c + 7) // 8 * 8)   # tensors start on 16-byte boundaries
        n = self.offsets.pop()
        flat = torch.zeros(n)
        for o, (r, c) in zip(self.offsets, self.shapes):
            flat[o:o + r * c] = rnd(r * c) / c ** 0.5
        self.P = flat.cuda()                                     # fp32 masters
        self.PB = self.P.to(BF16)                                # what the products read
        self.G, self.M = torch.zeros_like(self.P), torch.zeros_like(self.P)
        numels = [r * c for r, c in self.shapes]
        self.plan = cz.cz_plan_partition(numels, [len(numels)], 1, 1.0)
        self.args = cz.StepArgs(self.offsets, self.shapes)
        self.opts = cz.make_opts(param_bf16=self.PB)
        self.embed = rnd(vocab, width).cuda().to(BF16)           # fixed
        # vectors of the norms (the last input's norm included) and the gates: plain gradient descent
        self.w_post = torch.ones(layers, width, device="cuda")
        self.w_pre = torch.ones(layers + 1, width, device="cuda")
        self.gate = torch.full((layers, width), 0.5, device="cuda")
        new = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        T, D = tokens, width
        self.h = [new(T, D) for _ in range(layers + 1)]
        self.x = new(T, D)
        self.rstd = new(layers + 1, 2, T, t=torch.float32)
        keep = lambda cols: new(cz.cz_act_size(T, cols), t=torch.uint8)  # noqa: E731
        self.x_kept = [keep(D) for _ in range(layers + 1)]
        self.y_kept, self.a_kept = [keep(D) for _ in range(layers)], [keep(hidden) for _ in range(layers)]
        self.logp, self.entropy, self.lse = (new(T, t=torch.float32) for _ in range(3))
        self.top_ids, self.top_logp = new(T, 4, t=torch.int64), new(T, 4, t=torch.float32)
        self.dw_post, self.dw_pre = torch.zeros_like(self.w_post), torch.zeros_like(self.w_pre)
        self.dgate = torch.zeros_like(self.gate)
        self.norm_ws = torch.zeros(cz.cz_block_norm_workspace(T, D), dtype=torch.uint8, device="cuda")
        self.ws = torch.zeros(max(cz.cz_act_wgrad_workspace(new(T, r), c) for r, c in self.shapes), dtype=torch.uint8,
                              device="cuda")

    def weight(self, i: int):
        r, c = self.shapes[i]
        return self.PB[self.offsets[i]:self.offsets[i] + r * c].view(r, c)

    def grad(self, i: int):
        r, c = self.shapes[i]
        return self.G[self.offsets[i]:self.offsets[i] + r * c].view(r, c)

    def forward(self, tokens, targets):
        """Logits; every input that the backward pass needs is kept."""
        self.h[0].copy_(self.embed[tokens])
        # no block before the first input: only the norm in front of a block runs
        cz.cz_block_norm_fwd(self.h[0], self.h[0], None, x=self.x, w_pre=self.w_pre[0], post_norm=False, y_scale=0.0,
                             rstd_pre=self.rstd[0, 1], x_ckpt=self.x_kept[0], stream=torch.cuda.current_stream())
        for i in range(self.L):
            s = torch.cuda.current_stream()
            a = torch.nn.functional.silu(self.x @ self.weight(2 * i).t())
            cz.cz_act_encode(a, self.a_kept[i], stream=s)
            y = a @ self.weight(2 * i + 1).t()
            cz.cz_block_norm_fwd(self.h[i], y, self.h[i + 1], x=self.x, w_post=self.w_post[i], w_pre=self.w_pre[i + 1],
                                 gate=self.gate[i], rstd_post=self.rstd[i + 1, 0], rstd_pre=self.rstd[i + 1, 1],
                                 y_ckpt=self.y_kept[i], x_ckpt=self.x_kept[i + 1], stream=s)
        logits = self.x @ self.weight(2 * self.L).t()
        cz.cz_token_logp_fwd(logits, targets, self.logp, entropy=self.entropy, lse=self.lse, top_ids=self.top_ids,
                             top_logp=self.top_logp, stream=torch.cuda.current_stream())
        return logits

    def backward(self, logits, targets, entropy_bonus: float = 0.0):
        """Gradients of -mean(logp) - entropy_bonus * mean(entropy) into self.G and the vectors' gradients."""
        s = torch.cuda.current_stream()
        g = torch.full((self.T,), -1.0 / self.T, device="cuda")
        cz.cz_token_logp_bwd(logits, targets, self.lse, logits, entropy=self.entropy, g_logp=g, g_entropy=g * entropy_bonus,
                             stream=s)
        top = 2 * self.L
        cz.cz_act_wgrad(logits, self.x_kept[self.L], self.grad(top), workspace=self.ws, stream=s)
        dx = logits @ self.weight(top)
        dh = torch.zeros(self.T, self.D, dtype=BF16, device="cuda")
        dy = torch.empty_like(dh)
        for i in reversed(range(self.L)):
            # dh: in, the gradient of this block's h; out, of the h before it
            cz.cz_block_norm_bwd(self.h[i + 1], None, dx, dh, dh, dy, w_post=self.w_post[i], w_pre=self.w_pre[i + 1],
                                 gate=self.gate[i], rstd_post=self.rstd[i + 1, 0], rstd_pre=self.rstd[i + 1, 1],
                                 y_ckpt=self.y_kept[i], dw_post=self.dw_post[i], dw_pre=self.dw_pre[i + 1],
                                 dgate=self.dgate[i], workspace=self.norm_ws, stream=s)
            cz.cz_act_wgrad(dy, self.a_kept[i], self.grad(2 * i + 1), workspace=self.ws, stream=s)
            da = dy @ self.weight(2 * i + 1)
            x = torch.empty_like(dh)                             # u is computed again from the block's kept input
            cz.cz_act_decode(self.x_kept[i], x, stream=s)
            u = (x @ self.weight(2 * i).t()).float()
            sig = torch.sigmoid(u)
            du = (da.float() * sig * (1 + u * (1 - sig))).to(BF16)
            cz.cz_act_wgrad(du, self.x_kept[i], self.grad(2 * i), workspace=self.ws, stream=s)
            dx = du @ self.weight(2 * i)
        cz.cz_block_norm_bwd(self.h[0], None, dx, dh, dh, None, w_pre=self.w_pre[0], post_norm=False, y_scale=0.0,
                             rstd_pre=self.rstd[0, 1], dw_pre=self.dw_pre[0], workspace=self.norm_ws, stream=s)

    def step(self, tokens, targets, lr: float = 0.02, entropy_bonus: float = 0.0):
        """One training step; returns the mean log probability of the targets before it (a device scalar)."""
        logits = self.forward(tokens, targets)
        self.backward(logits, targets, entropy_bonus)
        for w, g in ((self.w_post, self.dw_post), (self.w_pre, self.dw_pre), (self.gate, self.dgate)):
            w.add_(g, alpha=-lr)
        cz.cz_muon_step_ex(self.plan, 0, self.P, self.G, self.M, self.args, lr, 0.95, 5, torch.cuda.current_stream(), self.opts)
        return self.logp.mean()

    def status(self) -> int:
        """First error that a kernel recorded (CZ_OK if none)."""
        for ws in (self.ws, None):
            st = cz.cz_device_status(torch.cuda.current_stream(), ws)
            if st != cz.CZ_OK:
                return st
        return cz.CZ_OK


def batch(demo: Demo, gen) -> tuple:
    """Tokens and their successors: a fixed rule with some noise, so that there is something to learn."""
    t = torch.randint(0, demo.V, (demo.T,), generator=gen)
    n = (7 * t + 3) % demo.V
    noise = torch.rand(demo.T, generator=gen) < 0.1
    n[noise] = torch.randint(0, demo.V, (int(noise.sum()),), generator=gen)
    return t.cuda(), n.cuda()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 30), ("tokens", 4096), ("width", 256), ("hidden", 512), ("vocab", 1000), ("layers", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    demo = Demo(a.tokens, a.width, a.hidden, a.vocab, a.layers)
    gen = torch.Generator().manual_seed(1)
    for i in range(a.steps):
        logp = demo.step(*batch(demo, gen))
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i}: mean log probability {logp.item():.4f}, entropy {demo.entropy.mean().item():.4f}")
    st = demo.status()
    if st != cz.CZ_OK:
        raise SystemExit(f"device status {st}: {cz.cz_status_string(st)}")


if __name__ == "__main__":
    main()
