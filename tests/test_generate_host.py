"""The example of generation, on the CPU: the order of its streams' work."""
import contextlib
import importlib.util
import os

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_example_waits_for_its_weights(monkeypatch, capsys):
    """The model is made on the current stream and used on another, which
    waits for it first."""
    path = os.path.join(ROOT, "examples", "generate.py")
    spec = importlib.util.spec_from_file_location("generate_streams", path)
    gen = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(gen)
    done = []

    class Stream:
        def __init__(self, name="side"):
            self.name = name

        def wait_stream(self, other):
            done.append((self.name, "waits for", other.name))

        def synchronize(self):
            done.append((self.name, "synchronized"))

    now = [Stream("first")]

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    class Cache:
        seen = lens = torch.zeros(4)

    def decoder(**kw):
        done.append((now[-1].name, "makes the model"))

    def generate(*args, **kw):
        done.append((now[-1].name, "generates"))
        return torch.zeros(1, 4), torch.zeros(1, 4), Cache

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now[-1])
    monkeypatch.setattr(gen, "Decoder", decoder)
    monkeypatch.setattr(gen, "generate", generate)
    gen.main()
    assert done == [("first", "makes the model"),
                    ("side", "waits for", "first"), ("side", "generates"),
                    ("side", "synchronized")]
    assert "200 steps" in capsys.readouterr().out
