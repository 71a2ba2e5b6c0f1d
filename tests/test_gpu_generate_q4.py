"""The generation example with 4-bit projections and scores: its steps agree with a recomputation, and its scores with its logits.

As with fp32 projections, decoding through the cache and prefilling at once are the same function: fp32 sums in
another order alone (1e-4 of the largest logit).
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "generate.py")
    spec = importlib.util.spec_from_file_location("generate_example_q4", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def server(example):
    s = example.Server(3, max_len=120, q4=True)
    yield s
    s.close()


def test_decoding_matches_prefilling_with_4_bit_projections(example, server):
    gen = torch.Generator("cuda").manual_seed(2)
    lens = [1, 17, 60]
    seqs = [torch.randint(0, example.VOCAB, (n + 3,), generator=gen, device="cuda") for n in lens]
    server.reset()
    logits = server.step(torch.cat([s[:n] for s, n in zip(seqs, lens)]), lens)
    for j in range(3):
        logits = server.step(torch.stack([s[n + j] for s, n in zip(seqs, lens)]), [1, 1, 1])
    server.reset()
    whole = server.step(torch.cat(seqs), [n + 3 for n in lens])
    assert float((logits - whole).abs().max()) <= 1e-4 * float(whole.abs().max())


def test_scores_of_the_made_tokens(example, server):
    prompts, scores = [[5], list(range(30)), [7] * 11], []
    ids = example.generate(server, prompts, 6, seed=4, scores=scores, top=5)
    assert torch.equal(ids, example.generate(server, prompts, 6, seed=4)) and len(scores) == 6
    for j, s in enumerate(scores):
        assert (s["logp"] <= 0).all() and (s["entropy"] > 0).all() and (s["rank"] >= 0).all()
        assert (s["top_logp"][:, :-1] >= s["top_logp"][:, 1:]).all()
        for r in range(3):                                     # a token among the best has its rank's place and score
            k = int(s["rank"][r])
            if k < 5:
                assert int(s["top_ids"][r, k]) == int(ids[r, j]) and float(s["top_logp"][r, k]) == float(s["logp"][r])
    greedy = []
    example.generate(server, prompts, 3, temperature=0.0, scores=greedy, top=1)
    assert all((s["rank"] == 0).all() for s in greedy)
