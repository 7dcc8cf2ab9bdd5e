"""The serving example refuses a step that its block table has no room for, and goes on from where it was."""
import importlib.util
import sys
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_request_longer_than_the_table():
    path = Path(__file__).resolve().parent.parent / "examples" / "serve.py"
    spec = importlib.util.spec_from_file_location("serve_example_limits", path)
    serve = importlib.util.module_from_spec(spec)
    sys.modules["serve_example_limits"] = serve
    spec.loader.exec_module(serve)
    model = serve.Model(serve.Config(max_pages=3), seed=7)  # 48 positions a request
    g = torch.Generator().manual_seed(8)
    a = torch.randint(0, model.cfg.vocab, (48,), generator=g).tolist()
    server, alone = serve.Server(model, 2), serve.Server(model, 1)
    server.step([a[:40], a[:5]])
    free, past = list(server.free), list(server.past)
    with pytest.raises(RuntimeError):
        server.step([a[40:] + [1], [2]])
    assert server.free == free and server.past == past
    logits = server.step([a[40:], [2]])[0].float()
    want = alone.step([a])[0].float()
    assert (logits - want).abs().max() <= 16 * 2.0 ** -8 * want.abs().max()
