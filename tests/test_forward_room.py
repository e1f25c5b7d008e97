"""Forwards refuse tensors that hold less than they read or write (on the host: nothing is launched
here, and the refusals need no GPU)."""
import pytest
import torch

from weight_only_int4_moe_gb300 import layer, ops

E, H, I, K, M = 8, 384, 256, 2, 6
BF16, FP32, I32 = torch.bfloat16, torch.float32, torch.int32


class Launched(Exception):
    pass


@pytest.fixture
def no_library(monkeypatch):
    """The library's calls, left out: reaching one is an error of its own."""

    class Library:
        def __getattr__(self, name):
            raise Launched(name)

    monkeypatch.setattr(ops, "load_library", Library)


def tensors():
    return dict(x=torch.zeros(M, H, dtype=BF16), out=torch.zeros(M, H), topk_ids=torch.zeros(M, K, dtype=I32),
                topk_weights=torch.zeros(M, K))


SMALL = [dict(out=torch.zeros(M - 1, H)), dict(out=torch.zeros(M, H - 8)), dict(out=torch.zeros(0)),
         dict(x=torch.zeros(M, H - 8, dtype=BF16)), dict(topk_ids=torch.zeros(M, K - 1, dtype=I32)),
         dict(topk_weights=torch.zeros(M - 1, K))]


@pytest.mark.parametrize("small", SMALL)
def test_forward(no_library, small):
    t = {**tensors(), **small}
    w = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="expected 6 rows"):
        ops.moe_int4_forward(t["x"], w, w, w, w, t["topk_ids"], t["topk_weights"], ops.Shape.of(E, K, H, I),
                             out=t["out"], workspace=w)


@pytest.mark.parametrize("small", SMALL + [dict(logits=torch.zeros(M, E - 1))])
def test_forward_routed(no_library, small):
    t = {**tensors(), "logits": torch.zeros(M, E), **small}
    w = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="expected 6 rows"):
        ops.moe_int4_forward_routed(t["x"], w, w, w, w, t["logits"], ops.Shape.of(E, K, H, I), out=t["out"],
                                    topk_ids=t["topk_ids"], topk_weights=t["topk_weights"], workspace=w)


@pytest.mark.parametrize("out", [torch.zeros(M - 1, H), torch.zeros(M, H - 8)])
def test_forward_from_hidden_states(no_library, monkeypatch, out):
    """The call in front of it, with its product and routing left out."""

    class Experts:
        shape = ops.Shape.of(E, K, H, I)

        def forward(self, x, ids, weights, out=None, workspace=None, stream=None):
            w = torch.zeros(16, dtype=torch.uint8)
            return ops.moe_int4_forward(x, w, w, w, w, ids, weights, self.shape, out=out, workspace=workspace,
                                        stream=stream)

    class Router:
        N, K = E, H

    t = tensors()
    monkeypatch.setattr(layer, "moe_linear", lambda *a, **k: torch.zeros(M, E))
    monkeypatch.setattr(layer, "moe_route_experts", lambda *a, **k: (t["topk_ids"], t["topk_weights"]))
    with pytest.raises(ValueError, match="expected 6 rows"):
        layer.moe_int4_forward_hidden(t["x"], Experts(), Router(), out=out,
                                      workspace=torch.zeros(16, dtype=torch.uint8))
