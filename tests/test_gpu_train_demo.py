"""The training-step operators together: gradients of the demo's network against autograd, and a few steps that learn.

The demo rounds activations and gradients to bf16 about ten times on the way (2^-9 each, at random) and reads blocks from
8-bit checkpoints (an error of up to 1/127 of a block's largest value, 0.4 % of it on average): together a few percent of
a gradient's norm.  Bound: 5 %."""

import pytest
import torch

from zero_sharded_gb300 import cz
from zero_sharded_gb300 import train_demo as td

pytestmark = pytest.mark.gpu


def _reference(d, tokens, targets, bonus):
    """The same network in fp32 under autograd, from the bf16 weights."""
    w = [d.weight(i).float().requires_grad_() for i in range(len(d.shapes))]
    w_post, w_pre, gate = (t.clone().requires_grad_() for t in (d.w_post, d.w_pre, d.gate))
    norm = lambda v: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    h = d.embed[tokens].float()
    x = norm(h) * w_pre[0]
    for i in range(d.L):
        y = torch.nn.functional.silu(x @ w[2 * i].t()) @ w[2 * i + 1].t()
        h = h + gate[i] * norm(y) * w_post[i]
        x = norm(h) * w_pre[i + 1]
    lp = torch.log_softmax(x @ w[-1].t(), -1)
    logp = lp.gather(1, targets[:, None])[:, 0]
    entropy = -(lp.exp() * lp).sum(-1)
    (-(logp.mean() + bonus * entropy.mean())).backward()
    return [v.grad for v in w], w_post.grad, w_pre.grad, gate.grad, logp.detach(), entropy.detach()


@pytest.mark.parametrize("shape", [(515, 256, 512, 1000, 2), (300, 200, 328, 501, 1)])
def test_gradients_against_autograd(shape):
    d = td.Demo(*shape)
    tokens, targets = td.batch(d, torch.Generator().manual_seed(2))
    logits = d.forward(tokens, targets)
    best = logits.float().max(1)
    assert torch.equal(d.top_ids[:, 0], torch.argmax(logits.float(), 1))
    assert torch.allclose(d.top_logp[:, 0], best.values - d.lse, atol=1e-4)
    d.backward(logits, targets, 0.1)
    assert d.status() == cz.CZ_OK
    w, w_post, w_pre, gate, logp, entropy = _reference(d, tokens, targets, 0.1)
    rel = lambda a, b: float((a - b).norm() / b.norm())  # noqa: E731
    assert rel(d.logp, logp) < 0.02 and rel(d.entropy, entropy) < 0.02
    for i, g in enumerate(w):
        assert rel(d.grad(i), g) < 0.05, (i, rel(d.grad(i), g))
    for a, b in ((d.dw_post, w_post), (d.dw_pre, w_pre), (d.dgate, gate)):
        assert rel(a, b) < 0.05


def test_steps_learn_on_any_stream():
    d = td.Demo(tokens=2048, width=128, hidden=256, vocab=200, layers=2)
    gen = torch.Generator().manual_seed(3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        seen = [float(d.step(*td.batch(d, gen))) for _ in range(25)]
    side.synchronize()
    assert d.status() == cz.CZ_OK
    assert seen[-1] > seen[0] + 1.0, seen
