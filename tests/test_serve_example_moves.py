"""What the serving example's verify() moves in the cache: the rows of an accepted path that do not lie in place, bit for bit,
and nothing else."""
import pytest
import torch

from test_serve_example_drafts import prompts_of, serve  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def state(model):
    """Every layer's keys, values and scales, as bytes a slot."""
    out = []
    for cache in model.caches:
        for t in (*cache.pages, *cache.scales.values()):
            t = t.transpose(1, 2).contiguous()
            out.append(t.view(torch.uint8).reshape(t.shape[0] * t.shape[1], -1).clone())
    return out


@pytest.mark.parametrize("cache", ["bf16", "int8", "e4m3"])
def test_only_rows_out_of_place_move_and_as_they_are(serve, cache, monkeypatch):  # noqa: F811
    model = serve.Model(serve.Config(cache=cache), seed=4)
    prompts = prompts_of(model, (40, 3, 129, 20), 5)
    want = serve.generate(model, prompts, [6] * 4)
    server = serve.Server(model, 4)
    first = server.step(prompts).argmax(-1).tolist()
    wrong = lambda t: (t + 1) % model.cfg.vocab  # noqa: E731
    trees = []
    for r, (o, full) in enumerate(zip(first, want)):
        a, b = full[1], full[2]
        trees.append([[(-1, o), (0, wrong(a)), (0, a), (2, wrong(b)), (2, b)],   # the path's nodes are 0, 2, 4
                      [(-1, o), (0, a), (1, b)],                                  # in place
                      [(-1, o)], [(-1, o), (0, wrong(a)), (1, b)]][r])
    held, before = {}, []
    plan, move = server._plan, serve.Cache.move
    monkeypatch.setattr(server, "_plan", lambda new: held.setdefault("plan", plan(new)))

    def recorded(self, *slots):
        if not before:
            before.extend(state(model))
        move(self, *slots)

    monkeypatch.setattr(serve.Cache, "move", recorded)
    more = server.verify(trees)
    slots, at, source, target = held["plan"][3].tolist(), 0, [], []
    for nodes, m in zip(trees, more):
        path = [0]
        for t in m[:-1]:
            path.append(next(i for i, (p, token) in enumerate(nodes) if p == path[-1] and token == t))
        source += [slots[at + i] for i in path]
        target += slots[at:at + len(path)]
        at += len(nodes)
    assert source != target and before, "some path was out of place"
    for old, new in zip(before, state(model)):
        expect = old.clone()
        expect[target] = old[source]
        assert torch.equal(new, expect)
