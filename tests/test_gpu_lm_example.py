"""The embedding, the vocabulary's loss and the layer's single tokens together, as
examples/hybrid_lm.py uses them."""
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
    spec = importlib.util.spec_from_file_location("hybrid_lm_ends", os.path.join(ROOT, "examples", "hybrid_lm.py"))
    m = importlib.util.module_from_spec(spec)
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    spec.loader.exec_module(m)
    yield m
    torch.backends.cuda.matmul.allow_tf32 = old


def batch(lm, seed, vocab=97):
    lens = [20, 3, 45, 1]
    q = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(0, vocab, (sum(lens),), generator=q, device="cuda")
    y = torch.randint(0, vocab, (sum(lens),), generator=q, device="cuda")
    y[::6] = -100
    return x, y, lm.offsets(lens)


def test_loss_and_its_gradient_are_those_of_the_logits(lm):
    """One backward pass through the whole model: the loss without logits against torch's over the model's logits.  Both
    fp32; the logits are of order ten, so that softmaxes differ by 1e-5 at most."""
    m = lm.HybridLM(kinds=("ssm", "ssm"), width=64, seed=3)
    ps = [t.requires_grad_() for t in m.parameters()]
    x, y, cu = batch(lm, 5)
    a = m.loss(x, y, cu)
    ga = torch.autograd.grad(a, ps)
    b = torch.nn.functional.cross_entropy(m.logits(x, cu), y, ignore_index=-100)
    gb = torch.autograd.grad(b, ps)
    assert abs(float((a - b).detach())) <= 1e-5 * float(b.detach())
    for u, v in zip(ga, gb):
        assert float((u - v).norm()) <= 1e-4 * float(v.norm()) + 1e-7


def test_a_training_step_in_a_graph(lm):
    """Forward and backward captured once and replayed on other tokens, while an eager graph of the same parameters lives."""
    m = lm.HybridLM(kinds=("ssm", "ssm"), width=64, seed=4)
    ps = [t.requires_grad_() for t in m.parameters()]
    x, y, cu = batch(lm, 6)
    x2, y2, _ = batch(lm, 7)
    want = torch.autograd.grad(m.loss(x2, y2, cu), ps)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(m.loss(x, y, cu), ps)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(m.loss(x, y, cu), ps)
    x.copy_(x2)
    y.copy_(y2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_serving_steps_in_a_graph(lm):
    """The step of a batch captured over the caches and replayed gives the eager tokens' logits, padded rows among them."""
    m = lm.HybridLM(seed=5)
    prompts = [torch.arange(n, device="cuda") % 97 for n in (4, 9, 2)]
    slots = torch.tensor([2, 0, 5, -1], dtype=torch.int32, device="cuda")  # one padded row

    def start():
        c = m.caches(6)
        m.prompt(torch.cat(prompts), lm.offsets([4, 9, 2]), c, slots[:3])
        return c
    tok = torch.tensor([1, 2, 3, 0], device="cuda")
    eager = start()
    want = []
    for i in range(5):
        want.append(m.step((tok + i) % 97, eager, slots))
    caches = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(tok, start(), slots)
    torch.cuda.current_stream().wait_stream(side)
    at = tok.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(at, caches, slots)
    for i in range(5):
        at.copy_((tok + i) % 97)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:3], want[i][:3])
