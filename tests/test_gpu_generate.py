"""The generation example: its steps (tables, qkv, attention, experts, sampling) agree with a recomputation.

Decoding through the cache and prefilling the same tokens at once are the same function: fp32, so the
logits may differ by rounding alone (two layers of sums of 64 to 512 products: 1e-4 of the largest).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "generate.py")
    spec = importlib.util.spec_from_file_location("generate_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def server(example):
    s = example.Server(3, max_len=200)
    yield s
    s.close()


def test_decoding_through_the_cache_matches_prefilling_at_once(example, server):
    gen = torch.Generator("cuda").manual_seed(2)
    lens = [1, 17, 60]
    seqs = [torch.randint(0, example.VOCAB, (n + 6,), generator=gen, device="cuda") for n in lens]
    server.reset()
    logits = server.step(torch.cat([s[:n] for s, n in zip(seqs, lens)]), lens)
    for j in range(6):                                          # one token of each request at a time
        logits = server.step(torch.stack([s[n + j] for s, n in zip(seqs, lens)]), [1, 1, 1])
    server.reset()
    whole = server.step(torch.cat(seqs), [n + 6 for n in lens])
    assert float((logits - whole).abs().max()) <= 1e-4 * float(whole.abs().max())
    server.reset()                                              # in chunks of other sizes, one request resting
    server.step(torch.cat([seqs[0][:3], seqs[2][:40]]), [3, 0, 40])
    chunked = server.step(torch.cat([seqs[0][3:], seqs[1], seqs[2][40:]]), [4, 23, 26])
    assert float((chunked - whole).abs().max()) <= 1e-4 * float(whole.abs().max())
    assert server.attn.status() == 0 and server.pool.status() == 0


def test_generation_repeats_and_follows_its_parameters(example, server):
    prompts = [[5], list(range(30)), [7] * 11]
    a = example.generate(server, prompts, 8, seed=4)
    assert torch.equal(a, example.generate(server, prompts, 8, seed=4))
    assert not torch.equal(a, example.generate(server, prompts, 8, seed=5))
    assert int(a.min()) >= 0 and int(a.max()) < example.VOCAB
    greedy = example.generate(server, prompts, 8, temperature=0.0, seed=4)
    assert torch.equal(greedy, example.generate(server, prompts, 8, temperature=1.0, top_k=1, seed=9))
