"""The hybrid model of examples/hybrid_lm.py: its layers' operators together, in
training and from prompt to single tokens."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    spec = importlib.util.spec_from_file_location("hybrid_lm", os.path.join(ROOT, "examples", "hybrid_lm.py"))
    m = importlib.util.module_from_spec(spec)
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    spec.loader.exec_module(m)
    yield m
    torch.backends.cuda.matmul.allow_tf32 = old


def test_single_tokens_continue_the_prompt(lm):
    """Every step's logits equal those of one prompt call over the whole text: fp32 operators and products, three
    blocks deep, on logits of order one; the loosest part is the chunk kernel's, held elsewhere to 1e-4 of the norm."""
    tokens, logits, full = lm.serve()
    assert tokens.shape == (4, 12) and torch.isfinite(full).all()
    assert float((logits - full).abs().max()) <= 1e-3 * float(full.abs().max())


def test_training_fits_counting_sequences(lm):
    losses = lm.train(steps=30)
    assert losses[0] > 3.5 and losses[-1] < 0.8 * losses[0]  # starts near log 97


def test_block_gradient_against_differences(lm):
    """The loss along its gradient, by central differences of the whole model: fp32 losses are good to about 1e-6,
    which over a step of 2e-3 is 5e-4, and the third derivative adds the step's square; the slope is the gradient's
    norm, of order one."""
    m = lm.HybridLM(kinds=("ssm", "ssm"), width=64, seed=3)
    ps = [t.requires_grad_() for t in m.parameters()]
    lens = [20, 3, 45]
    q = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(0, 97, (sum(lens),), generator=q, device="cuda")
    y = torch.randint(0, 97, (sum(lens),), generator=q, device="cuda")
    cu = lm.offsets(lens)
    loss = lambda: torch.nn.functional.cross_entropy(m.logits(x, cu), y)
    grads = torch.autograd.grad(loss(), ps)
    slope = float(torch.sqrt(sum(d.square().sum() for d in grads)))
    h, at = 1e-3, {}
    with torch.no_grad():
        for s in (1, -1):
            for p, d in zip(ps, grads):
                p += s * h / slope * d
            at[s] = float(loss())
            for p, d in zip(ps, grads):
                p -= s * h / slope * d
    assert abs((at[1] - at[-1]) / (2 * h) - slope) <= 0.01 * slope
