"""The captured step's hold on its weights, with a stand-in for the graph (no GPU)."""
import contextlib
import gc
import types
import weakref

import torch

from sync_protocols_amd import decode_layer as D
from sync_protocols_amd import ops


def test_captured_step_keeps_the_weights_it_was_captured_with(monkeypatch):
    none = contextlib.nullcontext
    stream = types.SimpleNamespace(wait_stream=lambda other: None)
    for name, value in (("Stream", lambda device: stream), ("current_stream", lambda device: stream), ("stream", lambda s: none()),
                        ("CUDAGraph", object), ("graph", lambda g: none())):
        monkeypatch.setattr(torch.cuda, name, value)
    monkeypatch.setattr(D.ExpertLayer, "workspace", lambda self, tokens: torch.empty(1))
    monkeypatch.setattr(D.ExpertLayer, "step", lambda self, *a: None)
    layer = D.random_layer(256, 64, 128, 4, 4, 2, group=32, device="cpu")
    tensors = [layer.gamma, layer.router] + [t for w in (layer.wo, layer.w1, layer.w2) for t in (w.q, w.scale)]
    refs = [weakref.ref(t) for t in tensors]
    del tensors
    captured = D.CapturedStep(layer, 3, 128)
    layer.w1 = layer.w2 = ops.W4Weight(torch.empty(0), torch.empty(0))      # replaced, then dropped
    del layer
    gc.collect()
    assert all(r() is not None for r in refs)
    del captured
    gc.collect()
    assert all(r() is None for r in refs)
