"""The decode-step operators together (examples/thought_decode.py)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

import thought_decode as td  # noqa: E402

pytestmark = pytest.mark.gpu


def _prompts(c, lengths):
    g = torch.Generator().manual_seed(7)
    return [torch.randint(c.vocab, (n,), generator=g).tolist() for n in lengths]


def _run(d, prompts, steps):
    """Every step's tokens, log probabilities, entropies and alternatives."""
    out = [d.prefill(prompts)]
    tokens = [d.tokens.clone()]
    for _ in range(steps):
        out.append(d.step())
        tokens.append(d.tokens.clone())
    assert int(d.err) == 0
    return [torch.stack([o[i] for o in out]) for i in range(4)] + [torch.stack(tokens)]


# one token, inside a page, a page and one more, and more rows than the
# few-row attention takes; the steps cross a page's end
LENGTHS = (1, 13, 17, 60)


def test_a_client_does_not_depend_on_the_others(cuda_device):
    c = td.Config()
    prompts = _prompts(c, LENGTHS)
    together = _run(td.Decoder(c, len(prompts)), prompts, 9)
    for i in range(len(prompts)):
        alone = _run(td.Decoder(c, 1), prompts[i:i + 1], 9)
        for a, b in zip(together, alone):
            assert torch.equal(a[:, i], b[:, 0])


def test_values_agree_with_each_other(cuda_device):
    c = td.Config()
    prompts = _prompts(c, LENGTHS)
    logprobs, entropy, top_ids, top_logprobs, tokens = _run(td.Decoder(c, len(prompts)), prompts, 4)
    # the chosen token is the first alternative, and has its log probability
    assert torch.equal(top_ids[:, :, 0], tokens)
    assert torch.equal(top_logprobs[:, :, 0], logprobs)
    assert (top_logprobs[:, :, 1:] <= top_logprobs[:, :, :-1]).all()
    assert (entropy > 0).all() and (entropy < torch.log(torch.tensor(float(c.vocab)))).all()


def test_captured_step(cuda_device):
    c = td.Config()
    prompts = _prompts(c, LENGTHS)
    want = _run(td.Decoder(c, len(prompts)), prompts, 6)
    d = td.Decoder(c, len(prompts))
    d.prefill(prompts)
    d.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d.step()
    for n in range(2, 7):
        graph.replay()
        for i in range(4):
            assert torch.equal(out[i], want[i][n])
        assert torch.equal(d.tokens, want[4][n])
    assert int(d.err) == 0
