"""Calls that are the first ones of their thread: nothing has made the device's context current
there (outputs are given, so that no allocation does it either)."""
import threading

import pytest
import torch

from weight_only_int4_moe_gb300 import inputs, ops

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


def in_a_new_thread(call):
    """What it raised, or None."""
    got = []

    def work():
        try:
            call()
            got.append(None)
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("m,n,k,out", [(1, 640, 512, BF16), (4000, 3008, 768, BF16), (1300, 3900, 1024, FP32)])
def test_product(layer, m, n, k, out, captured):
    x, w = (torch.randn(r, k, device="cuda").to(BF16) for r in (m, n))
    lin = layer.Linear(w)
    want = layer.moe_linear(x, lin, out_dtype=out)
    got, stream = torch.zeros_like(want), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def call():
        layer.moe_linear(x, lin, out=got, stream=stream)

    if captured:
        # the capture is another thread's; the call's thread has its part of it
        with torch.cuda.graph(graph, stream=stream, capture_error_mode="relaxed"):
            error = in_a_new_thread(call)
        assert error is None
        graph.replay()
    else:
        assert in_a_new_thread(call) is None
    torch.cuda.synchronize()
    assert torch.equal(got, want) and lin.errors() == 0


def test_norm_and_routing(layer):
    x = torch.randn(7, 384, device="cuda").to(BF16)
    want, ids = layer.moe_add_norm(x).out, layer.moe_route_experts(x, 4)
    got, got_ids, got_w, stream = torch.zeros_like(want), torch.zeros_like(ids[0]), torch.zeros_like(ids[1]), \
        torch.cuda.Stream()
    torch.cuda.synchronize()
    assert in_a_new_thread(lambda: layer.moe_add_norm(x, out=got, stream=stream)) is None
    assert in_a_new_thread(lambda: layer.moe_route_experts(x, 4, topk_ids=got_ids, topk_weights=got_w,
                                                           stream=stream)) is None
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_ids, ids[0]) and torch.equal(got_w, ids[1])


@pytest.mark.parametrize("m", [1, 40])
def test_experts_from_hidden_states(layer, m):
    e, h = 8, 384
    experts = ops.PackedWeights(inputs.make_weights(e, h, 256, 0), e, h, 256, 2)
    router = layer.Linear(torch.randn(e, h, device="cuda").to(BF16))
    x = torch.randn(m, h, device="cuda").to(BF16)
    ws, stream = ops.alloc_workspace(m, experts.shape), torch.cuda.Stream()
    want, ids, _ = layer.moe_int4_forward_hidden(x, experts, router, workspace=ws)
    got = torch.zeros_like(want)
    torch.cuda.synchronize()
    assert in_a_new_thread(lambda: layer.moe_int4_forward_hidden(x, experts, router, out=got, workspace=ws,
                                                                 stream=stream)) is None
    torch.cuda.synchronize()
    # (the experts add in an order of their own)
    assert (got.float() - want.float()).abs().max() <= 2e-2 * want.float().abs().max()
    assert router.errors() == 0 and ops.moe_int4_get_errors(ws)[0] == 0
