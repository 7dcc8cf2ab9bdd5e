"""The serving example: plan, projections, cache write, attention and sampling together."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    path = Path(__file__).resolve().parent.parent / "examples" / "serve.py"
    spec = importlib.util.spec_from_file_location("serve_example", path)
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["serve_example"] = mod  # (dataclasses look their module up)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("window", [0, 40])
def test_steps_agree_with_one_pass(serve, window):
    """Tokens drawn greedily one by one are, up to rounding, the likeliest ones of one pass over all of them."""
    model = serve.Model(serve.Config(window=window), seed=1)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (1, 17, 130, 64, 5)]
    new = [6, 9, 4, 9, 1]
    out = serve.generate(model, prompts, new)
    assert [len(o) for o in out] == new
    for o, p, n in zip(out, prompts, new):
        for i in (0, n - 1):
            logits = serve.Server(model, 1).step([p + o[:i]])[0].float()
            # the two ways round some 16 intermediate results to 2^-8 each, in other places
            assert logits[o[i]] >= logits.max() - 16 * 2.0 ** -8 * logits.abs().max()


def test_a_prompt_in_chunks_and_pages_handed_on(serve):
    """A prompt in pieces beside another request's tokens, over pages that a finished request has left."""
    model = serve.Model(serve.Config(pages=24, max_pages=16), seed=3)
    g = torch.Generator().manual_seed(4)
    a, b, c = (torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (200, 90, 150))
    alone = serve.Server(model, 1).step([c])[0].float()
    server = serve.Server(model, 2)
    server.step([a, b])
    with pytest.raises(RuntimeError):
        server.step([c, [1]])
    server.drop([1])
    server.table = torch.cat([server.table, torch.full_like(server.table, -1)])
    server.past.append(0)
    for i in range(0, 150, 50):
        logits = server.step([[7], c[i:i + 50]])
    err = (logits[1].float() - alone).abs().max()
    assert err <= 16 * 2.0 ** -8 * alone.abs().max()


def test_sampled_tokens_follow_the_seed(serve):
    model = serve.Model(serve.Config(), seed=5)
    prompts = [[1, 2, 3], [4] * 40]
    runs = [serve.generate(model, prompts, [12, 12], 0.9, 40, 0.9, 0.05, seed) for seed in (1, 1, 2)]
    assert runs[0] == runs[1] and runs[0] != runs[2]
    assert all(0 <= t < model.cfg.vocab for o in runs[0] for t in o)
