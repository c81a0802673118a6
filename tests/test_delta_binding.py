"""What the Python calls over include/hla_delta.h check and allocate, on tensors without memory (no GPU)."""
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import higher_order_linear_chunked_b200 as hla


def fake(*shape, dtype=torch.float32, device="cuda:0"):
    return torch.empty(*shape, dtype=dtype, device=device)


def delta_leaves():
    return [fake(1, 2, 8, 64, dtype=torch.bfloat16) for _ in range(3)] + [fake(1, 2, 8) for _ in range(2)]


def calls():
    x = delta_leaves()
    y, w = fake(4, 64), fake(64)
    return {"gated_delta": lambda ws: hla.gated_delta(*x, workspace=ws),
            "gated_delta_backward": lambda ws: hla.gated_delta_backward(*x, x[2], workspace=ws),
            "group_norm_backward": lambda ws: hla.group_norm_backward(y, y, 2, weight=w, workspace=ws)}


@pytest.mark.parametrize("name", ["gated_delta", "gated_delta_backward", "group_norm_backward"])
def test_workspace_of_another_kind(name):
    n = 1 << 24
    with FakeTensorMode():
        call = calls()[name]
        for ws, what in ((fake(n, dtype=torch.uint8, device="cpu"), "workspace must be a CUDA tensor"),
                         (fake(n, dtype=torch.uint8, device="cuda:1"), "workspace is on cuda:1"),
                         (fake(1, dtype=torch.uint8).expand(n), "workspace must be contiguous"),
                         (fake(2 * n, dtype=torch.uint8)[::2], "workspace must be contiguous")):
            with pytest.raises(ValueError, match=what):
                call(ws)


class Watch:
    """torch with its factories watched: what is allocated while which stream is current, and for which
    other stream it is kept."""

    def __init__(self, monkeypatch, module):
        self.current, self.side = SimpleNamespace(cuda_stream=0), SimpleNamespace(cuda_stream=1)
        self.stream, self.made, self.kept = self.current, [], []
        watch = self

        class Current:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, watch.stream = watch.stream, self.stream

            def __exit__(self, *_):
                watch.stream = self.before

        class Torch:
            def __getattr__(self, name):
                return getattr(torch, name)

            def empty(self, *a, **k):
                return watch.note(torch.empty(*a, **k))

            def empty_like(self, *a, **k):
                return watch.note(torch.empty_like(*a, **k))

        monkeypatch.setattr(torch.cuda, "stream", Current)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: watch.stream)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: watch.kept.append((id(t), s)))
        monkeypatch.setattr(hla, "_torch", Torch)
        if module is not hla:
            monkeypatch.setattr(module, "torch", Torch())
            monkeypatch.setattr(module, "_call", lambda *a: None)
            monkeypatch.setattr(module, "_stream_of", lambda *a: 0)
            monkeypatch.setattr(module, "_raw_stream", lambda device: 0)

    def note(self, t):
        self.made.append((t, self.stream))
        return t


def streamed(x, S, y, w):
    return {"gated_delta": lambda **k: hla.gated_delta(*x, return_state=True, **k),
            "gated_delta_step": lambda **k: (hla.gated_delta_step(S, *(t[:, :, 0].contiguous() for t in x), **k),),
            "gated_delta_backward": lambda **k: hla.gated_delta_backward(*x, x[2], initial_state=S, **k),
            "group_norm": lambda **k: (hla.group_norm(y, 2, **k),),
            "group_norm_backward": lambda **k: hla.group_norm_backward(y, y, 2, weight=w, bias=w, gate=y, **k)}


@pytest.mark.parametrize("name", ["gated_delta", "gated_delta_step", "gated_delta_backward", "group_norm", "group_norm_backward"])
def test_what_a_call_on_a_given_stream_allocates(name, monkeypatch):
    """From that stream's memory (a block of the current stream's may still be in use by work queued there),
    and kept for the current stream, on which the caller has the results."""
    from higher_order_linear_chunked_b200 import delta
    with FakeTensorMode():
        call = streamed(delta_leaves(), fake(1, 2, 64, 64), fake(4, 64), fake(64))[name]
        watch = Watch(monkeypatch, delta)
        out = call(stream=watch.side)
        assert watch.made and all(s is watch.side for _, s in watch.made)
        assert watch.stream is watch.current
        kept = {i for i, s in watch.kept if s is watch.current}
        assert all(id(t) in kept for t in out)
        watch.made.clear(), watch.kept.clear()
        call()
        assert watch.made and all(s is watch.current for _, s in watch.made) and not watch.kept


@pytest.mark.parametrize("name,results", [("hla2", 1), ("hla2_normalized", 1), ("ahla", 1), ("hla3", 1), ("hla2_unmasked", 1),
                                          ("hla2_backward", 3), ("ahla_backward", 3), ("state", 1), ("step", 1),
                                          ("forward_profiled", 1)])
def test_what_the_other_calls_allocate(name, results, monkeypatch):
    """The same of the HLA family's calls (which refuse these tensors, all at address 0, once they have allocated)."""
    with FakeTensorMode():
        x = [fake(1, 2, 8, 64) for _ in range(3)]
        args = {"hla2_backward": (*x, x[2]), "ahla_backward": (*x, x[2]), "state": ("hla2", *x), "forward_profiled": ("hla2", *x, ()),
                "step": ("hla2", fake(1, 2, 17000), *(t[:, :, 0].contiguous() for t in x))}.get(name, x)
        watch = Watch(monkeypatch, hla)
        for stream in (watch.side, None):
            watch.made.clear(), watch.kept.clear()
            with pytest.raises(hla.HLAError):
                getattr(hla, name)(*args, stream=stream)
            want = watch.side if stream else watch.current
            assert len(watch.made) >= results and all(s is want for _, s in watch.made)
            assert len(watch.kept) == (results if stream else 0) and all(s is watch.current for _, s in watch.kept)


def test_the_module_is_an_attribute_of_the_package():
    """Without an import of it, and before any of its calls was used."""
    code = "import higher_order_linear_chunked_b200 as hla; assert hla.delta.gated_delta is hla.gated_delta"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
