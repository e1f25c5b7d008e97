"""A decoder layer served from this library: attention over the 4-bit paged cache,
then the INT4 expert MLP.

    python examples/decoder_layer.py

Prompts of different lengths are prefilled, streams are decoded one token at a time
from a captured CUDA graph, a stream is branched and verified against a tree of
drafts, and pages are freed and compacted.  Random weights.  The projection in front of
the attention takes 8-bit codes of the normed tokens; the experts are chosen by sigmoid
scores with a balance bias.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from weight_only_int4_moe_gb300 import inputs, kv4, layer, ops  # noqa: E402


class DecoderLayer:
    """x -> x + attention(x) -> y + experts(y), for the new tokens of a batch."""

    def __init__(self, hidden=256, q_heads=4, kv_heads=2, head_dim=64, experts=8, top_k=2,
                 inter=128, n_pages=64, page_size=16, max_pos=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") / cols ** 0.5
            return w.to(torch.bfloat16)

        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        # codes of the rows of one projection, with a scale each
        w = weight((q_heads + 2 * kv_heads) * head_dim, hidden).float()
        scale = w.abs().amax(-1) / 448
        self.w_qkv = layer.Linear((w / scale[:, None]).to(torch.float8_e4m3fn), scale=scale)
        self.w_out = layer.Linear(weight(hidden, q_heads * head_dim))
        self.w_router = layer.Linear(weight(experts, hidden))
        self.balance = 0.01 * torch.randn(experts, generator=g, device="cuda")
        self.norms = torch.ones(2, hidden, dtype=torch.bfloat16, device="cuda")
        self.q_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.k_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        angle = torch.arange(max_pos, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(head_dim // 2, device="cuda") * 2 / head_dim)
        self.cos, self.sin = angle.cos(), angle.sin()
        self.experts = ops.PackedWeights(inputs.make_weights(experts, hidden, inter, seed), experts,
                                         hidden, inter, top_k, out_dtype=ops.MOE_OUT_BF16)
        self.cache = kv4.Cache.empty(1, n_pages, kv_heads, head_dim, page_size)

    def workspaces(self, tokens):
        """What a caller keeps for steps of up to this many new tokens."""
        return (kv4.alloc_workspace(self.cache, None, self.q_heads),
                ops.alloc_workspace(tokens, self.experts.shape))

    def forward(self, x, batch, workspaces, tree=None, positions=None):
        """x bf16 [tokens, hidden], the batch's new tokens in order."""
        hq, hkv, d = self.q_heads, self.kv_heads, self.head_dim
        y = layer.moe_add_norm(x, self.norms[0], out_dtype=None, codes=True)
        qkv = layer.moe_linear(y.codes, self.w_qkv, x_scale=y.scales)
        q, k, v = qkv.unflatten(1, (hq + 2 * hkv, d)).split((hq, hkv, hkv), 1)
        q = kv4.moe_kv4_append(self.cache, batch, q, k, v, self.q_norm, self.k_norm, self.cos,
                               self.sin, positions)
        a = kv4.moe_kv4_attention(q, self.cache, batch, tree=tree, workspace=workspaces[0])
        x = layer.moe_linear(a.flatten(1), self.w_out, residual=x)
        y = layer.moe_add_norm(x, self.norms[1]).out
        out, _, _ = layer.moe_int4_forward_hidden(y, self.experts, self.w_router, scoring="sigmoid",
                                                  bias=self.balance, scale=2.0,
                                                  workspace=workspaces[1])
        # (a next layer would add and norm in one call)
        return layer.moe_add_norm(out, residual=x, out_dtype=None).residual


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def batch_of(seqs, ids, new):
    """The batch of sequences `ids` whose last new[i] tokens are to be computed."""
    ids = torch.as_tensor(ids, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    lens = seqs.lens[ids].contiguous()
    return kv4.Batch(cu, lens, seqs.tables[ids].contiguous(), int(sum(new)), max(new),
                     int(lens.max()))


def main():
    torch.cuda.set_device(0)
    block = DecoderLayer()
    seqs = kv4.Sequences.empty(8, 16, block.cache.shape.n_pages)
    g = torch.Generator(device="cuda").manual_seed(1)

    def tokens(n):
        return torch.randn(n, block.hidden, generator=g, device="cuda").to(torch.bfloat16)

    ws = block.workspaces(128)

    # three prompts at once
    prompts = [37, 5, 64]
    kv4.moe_kv4_reserve(block.cache, seqs, ints(0, 1, 2), ints(*prompts))
    out = block.forward(tokens(sum(prompts)), batch_of(seqs, [0, 1, 2], prompts), ws)
    print(f"prefill: {sum(prompts)} tokens of {len(prompts)} prompts, rms {out.float().std():.3f}")

    # decode: one token a stream, the layer captured once and replayed; the graph's
    # lengths and tables are the sequences' own tensors
    step = kv4.Batch(ints(0, 1, 2, 3), seqs.lens[:3], seqs.tables[:3], 3, 1,
                     seqs.tables.shape[1] * block.cache.shape.page_size)
    x, stream = torch.zeros(3, block.hidden, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()
    kv4.moe_kv4_reserve(block.cache, seqs, ints(0, 1, 2), seqs.lens[:3] + 1)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        x.copy_(tokens(3))
        eager = block.forward(x, step, ws)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = block.forward(x, step, ws)
    graph.replay()
    torch.cuda.synchronize()
    if not torch.equal(eager, replayed):
        raise RuntimeError("the replayed step differs from the eager one")
    for _ in range(20):
        kv4.moe_kv4_reserve(block.cache, seqs, ints(0, 1, 2), seqs.lens[:3] + 1)
        x.copy_(tokens(3))
        graph.replay()
    print(f"decode: lengths {seqs.lens.tolist()}")

    # branch stream 2, and let both go on with the same token: the same result
    kv4.moe_kv4_fork(block.cache, seqs, ints(2), ints(3))
    kv4.moe_kv4_reserve(block.cache, seqs, ints(2, 3), seqs.lens[2:4] + 1)
    pair = block.forward(tokens(1).repeat(2, 1), batch_of(seqs, [2, 3], [1, 1]), ws)
    if not torch.equal(pair[0], pair[1]):
        raise RuntimeError("a fork went on differently from its parent")

    # verify four drafts of stream 0 in one step, in a branch that is thrown away:
    # token 0, its children 1 and 2, and 3 below 2; each sees its ancestors and itself,
    # and has its depth's position
    base = int(seqs.lens[0])
    kv4.moe_kv4_fork(block.cache, seqs, ints(0), ints(4))
    kv4.moe_kv4_reserve(block.cache, seqs, ints(4), ints(base + 4))
    tree = torch.tensor([0b0001, 0b0011, 0b0101, 0b1101], device="cuda")
    drafts = tokens(4)
    positions = base + ints(0, 1, 1, 2)
    verified = block.forward(drafts, batch_of(seqs, [4], [4]), ws, tree=tree, positions=positions)
    kv4.moe_kv4_free(block.cache, seqs, ints(4))
    # the accepted path 0, 2, 3 as the stream's next tokens gives the same outputs
    path = torch.tensor([0, 2, 3], device="cuda")
    kv4.moe_kv4_reserve(block.cache, seqs, ints(0), ints(base + 3))
    accepted = block.forward(drafts[path], batch_of(seqs, [0], [3]), ws, positions=positions[path])
    worst = ((accepted - verified[path]).float().abs().max() / verified.float().std()).item()
    print(f"verify: path of {len(path)} drafts, tree against chain {worst:.1e} of the rms")
    if worst > 0.05:
        raise RuntimeError("the verified path differs from the chain")

    # stream 1 ends; the pool becomes dense again
    kv4.moe_kv4_free(block.cache, seqs, ints(1))
    before = block.forward(x[:1], batch_of(seqs, [2], [1]), ws)
    used = int(kv4.moe_kv4_compact(block.cache, seqs))
    after = block.forward(x[:1], batch_of(seqs, [2], [1]), ws)
    if not torch.equal(before, after):
        raise RuntimeError("compacting changed a result")
    print(f"pages: {used} in use, the highest {int(seqs.refs.nonzero().max())}")
    flags, _ = block.cache.errors()
    flags |= block.w_qkv.errors() | block.w_out.errors() | block.w_router.errors()
    if flags or ws[0][:8].any() or ops.moe_int4_get_errors(ws[1])[0]:
        raise RuntimeError("a device error was reported")
    print("ok")


if __name__ == "__main__":
    main()
