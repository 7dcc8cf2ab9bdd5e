"""The serving example with an 8-bit cache and with trees of drafted tokens: rotary positions, cache store and read-back,
attention and the choice of a path together."""
import importlib.util
import sys
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    path = Path(__file__).resolve().parent.parent / "examples" / "serve.py"
    spec = importlib.util.spec_from_file_location("serve_example_drafts", path)
    mod = importlib.util.module_from_spec(spec)
    sys.modules["serve_example_drafts"] = mod
    spec.loader.exec_module(mod)
    return mod


def prompts_of(model, lengths, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in lengths]


# Logits of the same tokens by another route: some 16 intermediate results rounded to 2^-8 in other places.  Through an
# 8-bit cache nothing else differs: a key or value is quantised from the same 16-bit rows on every route, up to those roundings,
# each of which may move a code by one (int8: 2^-7 of the row's largest, e4m3: 2^-3 of the value).
def slack(cache):
    return {"bf16": 16 * 2.0 ** -8, "int8": 24 * 2.0 ** -8, "e4m3": 0.35}[cache]


@pytest.mark.parametrize("cache", ["int8", "e4m3"])
@pytest.mark.parametrize("window", [0, 40])
def test_steps_agree_with_one_pass(serve, cache, window):
    model = serve.Model(serve.Config(window=window, cache=cache), seed=1)
    prompts = prompts_of(model, (1, 17, 130, 64, 5), 2)
    new = [6, 9, 4, 9, 1]
    out = serve.generate(model, prompts, new)
    assert [len(o) for o in out] == new
    for o, p, n in zip(out, prompts, new):
        for i in (0, n - 1):
            logits = serve.Server(model, 1).step([p + o[:i]])[0].float()
            assert logits[o[i]] >= logits.max() - slack(cache) * logits.abs().max()


def test_an_8_bit_cache_is_near_a_16_bit_one(serve):
    """Logits with 127 steps a row stay near those without quantisation."""
    models = [serve.Model(serve.Config(cache=c), seed=9) for c in ("bf16", "int8")]
    prompt = prompts_of(models[0], (150,), 3)
    a, b = (serve.Server(m, 1).step(prompt)[0].float() for m in models)
    assert (a - b).norm() <= 0.1 * a.norm()


@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_trees_give_the_tokens_of_single_steps(serve, cache):
    """Drafts with the model's own continuation among wrong branches: what verify takes is what single steps give, up to
    rounding, and the cache it leaves serves the steps behind it."""
    model = serve.Model(serve.Config(cache=cache), seed=4)
    prompts = prompts_of(model, (40, 3, 129), 5)
    want = serve.generate(model, prompts, [14] * 3)
    server = serve.Server(model, 3)
    first = server.step(prompts).argmax(-1).tolist()
    got = [[t] for t in first]
    taken = 0
    for _ in range(4):
        trees = []
        for o, full in zip(got, want):
            nodes, tip = [(-1, o[-1])], 0
            for depth in range(3):    # a wrong branch, then the right one, at every depth
                right = full[len(o) + depth] if o == full[:len(o)] and len(o) + depth < len(full) else 7
                nodes += [(tip, (right + 1) % model.cfg.vocab), (tip, right)]
                nodes.append((len(nodes) - 2, right))   # a grandchild on the wrong branch
                tip = len(nodes) - 2
            trees.append(nodes)
        before = list(server.past)
        more = server.verify(trees)
        for o, m, p, q in zip(got, more, before, server.past):
            assert q == p + len(m) and 1 <= len(m) <= 4
            o += m
            taken += len(m)
    assert taken > 3 * 4   # some drafts were taken
    logits = server.step([[o[-1]] for o in got]).float()
    # (servers share the model's caches: what another one does comes last)
    for o, p in zip(got, prompts):
        for i in range(1, len(o)):
            one = serve.Server(model, 1).step([p + o[:i]])[0].float()
            assert one[o[i]] >= one.max() - slack(cache) * one.abs().max()
    # the moved cache: the step over it against one pass over the same tokens
    for r, (o, p) in enumerate(zip(got, prompts)):
        alone = serve.Server(model, 1).step([p + o])[0].float()
        assert (logits[r] - alone).abs().max() <= slack(cache) * alone.abs().max()
    # every page is either free or held by a request
    held = server.table[server.table >= 0].tolist()
    assert sorted(held + server.free) == list(range(model.cfg.pages))
