"""The operators between attention and experts used together and with the experts: a
block of a decoder layer against 64 bits, in graphs, on other streams, from several
threads."""
import threading

import numpy as np
import pytest
import torch

import layer_reference as ref
import oracle
from weight_only_int4_moe_gb300 import inputs, ops

pytestmark = pytest.mark.gpu
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E, K, H, I = 16, 4, 384, 256


@pytest.fixture(scope="module")
def layer():
    from weight_only_int4_moe_gb300 import layer as m
    m.load_library()
    return m


class Block:
    """Attention's output projection with the residual, norm, router, experts, and a shared
    expert (gate, up, down) on 8-bit codes."""

    def __init__(self, layer, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.layer = layer

        def weight(n, k):
            return (torch.randn(n, k, generator=g) / k ** 0.5).to(BF16)

        def codes(w):
            s = w.float().abs().amax(-1) / 448
            return (w.float() / s[:, None]).to(E4M3), s

        self.out, self.router = weight(H, 512), weight(E, H)
        self.gate, self.up, self.down = codes(weight(I, H)), codes(weight(I, H)), weight(H, I)
        self.norm = (1 + 0.1 * torch.randn(H, generator=g)).to(BF16)
        self.bias = 0.05 * torch.randn(E, generator=g)
        self.w = inputs.make_weights(E, H, I, seed)
        self.experts = ops.PackedWeights(self.w, E, H, I, K)
        L = layer.Linear
        self.l_out, self.l_router, self.l_down = (L(t.cuda()) for t in (self.out, self.router, self.down))
        self.l_gate, self.l_up = (L(c.cuda(), scale=s.cuda()) for c, s in (self.gate, self.up))
        self.norm_d, self.bias_d = self.norm.cuda(), self.bias.cuda()

    def run(self, a, x, ws=None, stream=None):
        """(new residual, y, ids, weights, experts' output, block output)."""
        m, s = self.layer, stream
        h = m.moe_linear(a, self.l_out, residual=x, stream=s)
        y = m.moe_add_norm(h, self.norm_d, codes=True, stream=s)
        out, ids, w = m.moe_int4_forward_hidden(
            y.out, self.experts, self.l_router, scoring="sigmoid", bias=self.bias_d, groups=4, top_groups=2,
            scale=1.5, workspace=ws, stream=s)
        up = m.moe_linear(y.codes, self.l_up, x_scale=y.scales, stream=s)
        act = m.moe_linear(y.codes, self.l_gate, "silu", gate=up, x_scale=y.scales, stream=s)
        shared = m.moe_linear(act, self.l_down, residual=out, out_dtype=FP32, stream=s)
        return h, y, ids, w, out, m.moe_add_norm(shared, residual=h, out_dtype=None, stream=s).residual


def tokens(m, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(m, n, generator=g).to(BF16).cuda() for n in (512, H)]


@pytest.fixture(scope="module")
def block(layer):
    return Block(layer)


@pytest.mark.parametrize("m", [1, 7, 130])
def test_block_against_64_bits(block, m):
    """Each step from what the step before it returned."""
    a, x = tokens(m, m)
    h, y, ids, w, out, last = block.run(a, x)
    torch.cuda.synchronize()
    want, bound = ref.linear(a.cpu(), block.out, residual=x.cpu())
    assert ((h.cpu().double() - want).abs() <= bound + ref.half_step(want.abs() + bound, BF16)).all()
    held, want = ref.add_norm(h.cpu(), block.norm, None, 1e-6)
    assert ((y.out.cpu().double() - want).abs() <= 6 * ref.U * want.abs() + ref.half_step(want, BF16) *
            (1 + 1e-6)).all()
    logits, bound = ref.linear(y.out.cpu(), block.router)
    got = block.layer.moe_linear(y.out, block.l_router, out_dtype=FP32)
    assert ((got.cpu().double() - logits).abs() <= bound + ref.U * logits.abs()).all()
    want_ids, want_w = ref.route_experts(got.cpu(), K, "sigmoid", block.bias, 4, 2, scale=1.5)
    assert torch.equal(ids.cpu(), want_ids)
    assert ((w.cpu().double() - want_w).abs() <= 100 * ref.U * want_w).all()
    bits = y.out.cpu().view(torch.int16).numpy().view(np.uint16)
    moe, _ = oracle.moe_forward(bits, block.w["q13"], block.w["s13"], block.w["q2"], block.w["s2"],
                                ids.cpu().numpy(), w.cpu().numpy())
    rms = np.sqrt((moe ** 2).mean())
    assert np.abs(out.cpu().numpy() - moe).max() <= 2e-2 * rms
    # the shared expert on the codes, then everything added up
    codes, s = y.codes.cpu().float(), y.scales.cpu()
    up, e_up = ref.linear(codes, block.up[0].float(), s, block.up[1])
    up_b = up.to(BF16)
    act, e_act = ref.linear(codes, block.gate[0].float(), s, block.gate[1], act="silu", gate=up_b)
    shared = act.to(BF16).double() @ block.down.double().T
    # (two intermediates rounded to bf16, each to the neighbour, a step of 2^-7, where the
    # kernel's sum fell to the other side of a border)
    room = ((act.abs() * 2.0 ** -6 + e_act + e_up * 4).abs() @ block.down.double().abs().T) * 1.1
    total = shared + out.cpu().double() + h.cpu().double()
    assert ((last.cpu().double() - total).abs() <= room + 2 * ref.half_step(total.abs() + room, BF16)).all()
    for lin in (block.l_out, block.l_router, block.l_gate, block.l_up, block.l_down):
        assert lin.errors() == 0


@pytest.mark.parametrize("m", [1, 90])
def test_block_in_a_graph(block, m):
    """Captured once, replayed on new tokens; two graphs over the same weights in turn."""
    ws = ops.alloc_workspace(m, block.experts.shape)
    graphs = []
    for seed in (1, 2):
        a, x = tokens(m, seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block.run(a, x, ws)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = block.run(a, x, ws)
        graphs.append((graph, a, x, got))
    for seed in (5, 6, 7):
        for graph, a, x, got in graphs:
            na, nx = tokens(m, seed)
            a.copy_(na)
            x.copy_(nx)
            graph.replay()
        for graph, a, x, got in graphs:
            want = block.run(a, x, ws)
            torch.cuda.synchronize()
            for i in (0, 2, 3):
                assert torch.equal(got[i], want[i])
            assert torch.equal(got[1].out, want[1].out)
            # (the experts add in an order of their own)
            assert (got[5].float() - want[5].float()).abs().max() <= 2e-2 * want[5].float().abs().max()
    assert ops.moe_int4_get_errors(ws)[0] == 0


def keep_busy():
    """Some 50 ms of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=BF16, device="cuda")
    for _ in range(80):
        a = torch.matmul(a, a).clamp_(-1, 1)
    return a


@pytest.mark.parametrize("m", [3, 600])
def test_block_on_another_stream(block, m):
    """What a call makes for itself belongs to the call's stream: the current one is busy and
    its freed memory full of ones."""
    a, x = tokens(m, 3)
    want = block.run(a, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block.run(a, x, stream=side)
    for _ in range(3):
        for n in (m * H * 2, m * H * 4, m * E * 4, m * K * 4, m * 4, m * I * 2):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        busy = keep_busy()
        got = block.run(a, x, stream=side)
        side.synchronize()
        for i in (0, 2, 3):
            assert torch.equal(got[i], want[i])
        assert torch.equal(got[1].codes.view(torch.uint8), want[1].codes.view(torch.uint8))
        del busy
        torch.cuda.synchronize()


def test_calls_from_several_threads(layer):
    """Eight threads, each on its own stream, with sizes that take every kernel."""
    sizes = [(1, 512, 2048), (90, 384, 4096), (300, 640, 512), (2600, 2048, 256), (1500, 3000, 768),
             (17, 77, 64), (5000, 256, 128), (64, 4096, 1024)]
    data, want = [], []
    for i, (m, n, k) in enumerate(sizes):
        g = torch.Generator().manual_seed(i)
        x = torch.randn(m, k, generator=g).to(BF16).cuda()
        lin = layer.Linear((torch.randn(n, k, generator=g) / k ** 0.5).to(BF16).cuda())
        data.append((x, lin))
        y = layer.moe_linear(x, lin, out_dtype=FP32)
        r = layer.moe_add_norm(y.to(BF16), residual=y, codes=n % 16 == 0)
        want.append((y, r.out, *layer.moe_route_experts(y[:, :min(n, 512)], 8, "sigmoid")))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            x, lin = data[i]
            stream = torch.cuda.Stream()
            for _ in range(20):
                y = layer.moe_linear(x, lin, out_dtype=FP32, stream=stream)
                with torch.cuda.stream(stream):
                    b = y.to(BF16)
                r = layer.moe_add_norm(b, residual=y, codes=lin.N % 16 == 0, stream=stream)
                ids, w = layer.moe_route_experts(y[:, :min(lin.N, 512)], 8, "sigmoid", stream=stream)
                stream.synchronize()
                if not all(torch.equal(p, q) for p, q in zip((y, r.out, ids, w), want[i])):
                    bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert all(lin.errors() == 0 for _, lin in data)


def test_forward_hidden_refuses(block):
    x = torch.zeros(2, H, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        block.layer.moe_int4_forward_hidden(x, block.experts, block.l_down)
    out, ids, w = block.layer.moe_int4_forward_hidden(x[:0], block.experts, block.l_router)
    assert out.shape == (0, H) and ids.shape == (0, K)
