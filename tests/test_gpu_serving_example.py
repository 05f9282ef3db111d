"""The serving example: greedy speculative decoding gives the target's own greedy continuation, and the
sampled path keeps its books."""
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
    spec = importlib.util.spec_from_file_location("speculative_serving",
                                                  os.path.join(HERE, "..", "examples", "speculative_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def prompts():
    g = torch.Generator().manual_seed(3)
    return [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (1, 16, 33, 70)]


def dense_logits(model, tokens):
    """The model over a whole sequence in 64 bits, by plain attention."""
    n = len(tokens)

    def attend(layer, q, k, v):
        if layer is None:
            return torch.arange(n, device="cuda")[None]
        k, v = (t.repeat_interleave(model.Hq // model.H, 2).transpose(1, 2) for t in (k, v))
        s = q.transpose(1, 2) @ k.transpose(2, 3) * model.D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
        return (s.softmax(-1) @ v).transpose(1, 2)

    return model.forward(torch.tensor([tokens], device="cuda"), attend)[0]


@pytest.mark.parametrize("K,good_drafter", [(1, False), (3, True), (4, False)])
def test_greedy_speculation_is_greedy_decoding(example, K, good_drafter):
    make = lambda first, seed, layers: example.Transformer(1000, 64, layers, first, 4, 2, 64, torch.float32, seed)  # noqa: E731
    target = make(1, 5, 2)
    drafter = make(0, 5 if good_drafter else 6, 1)
    out, rate = example.serve(prompts(), N=2, K=K, steps=5, cut_every=3, temperature=0.0, top_k=0, top_p=1.0, vocab=1000,
                              dtype=torch.float32, pages=256, page_size=8, drafter=drafter, target=target)
    wide = make(1, 5, 2)
    for name in ("embed", "place", "head"):
        setattr(wide, name, getattr(target, name).double())
    wide.layers = [tuple(w.double() for w in layer) for layer in target.layers]
    assert {b for b, _, _ in out} == set(range(4))
    for b, tokens, _ in out:
        have = list(prompts()[b])
        logits = dense_logits(wide, have + tokens)[len(have) - 1:-1]
        top = logits.topk(2, -1).values
        clear = top[:, 0] - top[:, 1] > 1e-3  # fp32 decides these as 64 bits do
        assert clear.float().mean() > 0.9
        assert (logits.argmax(-1) == torch.tensor(tokens, device="cuda"))[clear].all()


def test_sampled_serving(example):
    out, rate = example.serve(prompts(), N=4, K=3, steps=6, cut_every=2, vocab=1000, pages=512)
    assert 0 <= rate <= 1 and {b for b, _, _ in out} == set(range(4)) and len(out) < 16
    for _, tokens, score in out:
        assert 6 <= len(tokens) <= 24 and all(0 <= t < 1000 for t in tokens) and score <= 0
    # the same model as drafter: nearly everything is accepted
    twin = [example.Transformer(1000, 64, 1, first, 4, 2, 64, torch.float32, 9) for first in (0, 1)]
    _, rate = example.serve(prompts(), N=4, K=3, steps=6, cut_every=0, vocab=1000, pages=512, dtype=torch.float32,
                            drafter=twin[0], target=twin[1])
    assert rate > 0.97
