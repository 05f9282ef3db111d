"""The tree serving example: at temperature 0 it gives the target's own greedy continuation, and its books are kept."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("tree_serving", os.path.join(HERE, "..", "examples", "tree_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def prompts():
    g = torch.Generator().manual_seed(3)
    return [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (1, 16, 33, 300)]


def dense_logits(model, tokens):
    """The model over a whole sequence in 64 bits, by plain rotation and attention."""
    n = len(tokens)
    angle = torch.arange(n, device="cuda").double()[:, None] * model.inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turn(x):
        u, w = x.chunk(2, -1)
        return torch.cat((u * cos - w * sin, w * cos + u * sin), -1)

    def attend(layer, q, k, v):
        q, k = turn(q), turn(k)
        k, v = (t.repeat_interleave(model.Hq // model.H, 2).transpose(1, 2) for t in (k, v))
        s = q.transpose(1, 2) @ k.transpose(2, 3) * model.D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
        return (s.softmax(-1) @ v).transpose(1, 2)

    return model.forward(torch.tensor([tokens], device="cuda"), attend)[0]


@pytest.mark.parametrize("levels,width,twin", [(1, 1, False), (4, 3, False), (3, 8, False), (5, 2, True)])
def test_greedy_trees_are_greedy_decoding(example, levels, width, twin):
    target = example.Transformer(1000, 64, 2, 4, 2, 64, torch.float32, 5, first=2)
    drafter = target.first_layers(2, 0) if twin else target.first_layers(1, 0)
    out, rate = example.serve(prompts(), levels=levels, width=width, steps=5, vocab=1000, dtype=torch.float32, pages=400, page_size=8,
                              drafter=drafter, target=target)
    wide = target.first_layers(2, 2)
    for name in ("embed", "head"):
        setattr(wide, name, getattr(target, name).double())
    wide.layers = [tuple(w.double() for w in layer) for layer in target.layers]
    assert len(out) == 4
    for p, tokens in zip(prompts(), out):
        assert 5 <= len(tokens) <= 5 * (levels + 1)
        logits = dense_logits(wide, p + tokens)[len(p) - 1:-1]
        top = logits.topk(2, -1).values
        clear = top[:, 0] - top[:, 1] > 1e-3  # fp32 decides these as 64 bits do
        assert clear.float().mean() > 0.9
        assert (logits.argmax(-1) == torch.tensor(tokens, device="cuda"))[clear].all()
    if twin:  # the drafter is the target: its first choice is what the target draws, to the last level
        assert rate > levels - 0.5


def test_sampled_trees(example):
    out, rate = example.serve(prompts(), levels=3, width=4, steps=6, temperature=0.8, top_k=40, top_p=0.95, vocab=1000)
    assert 0 <= rate <= 3 and len(out) == 4
    for tokens in out:
        assert 6 <= len(tokens) <= 24 and all(0 <= t < 1000 for t in tokens)
