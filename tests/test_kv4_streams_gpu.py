"""Calls of the 4-bit cache on a stream other than the current one, which is busy
meanwhile: what a call makes for itself must belong to the call's stream."""
import numpy as np
import pytest
import torch

import kv4_gpu_reference as gref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from weight_only_int4_moe_gb300 import kv4 as m
    m.load_library()
    return m


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def keep_busy():
    """Some 50 ms of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(80):
        a = torch.matmul(a, a).clamp_(-1, 1)
    return a


def used_memory(*sizes):
    """Freed blocks of the current stream's memory that hold ones."""
    for n in sizes:
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def case(kv4):
    # decode, narrow and wide requests, items that several CTAs share
    kv, ql = [9000, 5000, 700, 300], [1, 40, 16, 100]
    hkv, group, d, ps = 2, 4, 128, 64
    pool, tables, cu, q = gref.make_case(3, kv, ql, hkv, group, d, ps)
    cache = kv4.Cache(pool[None], hkv, d, ps)
    batch = kv4.Batch(ints(cu), ints(kv), ints(tables), int(cu[-1]), max(ql), max(kv))
    return cache, batch, q


def test_attention_makes_its_workspace_on_the_given_stream(kv4):
    cache, batch, q = case(kv4)
    ws = kv4.alloc_workspace(cache, batch, q.shape[1])
    want, lse = kv4.moe_kv4_attention(q, cache, batch, return_lse=True, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kv4.moe_kv4_attention(q, cache, batch, return_lse=True, stream=side)  # its memory is there now
    shown = False
    for _ in range(3):
        used_memory(ws.numel(), q.numel() * 2, 4 * lse.numel())
        torch.cuda.synchronize()
        busy = keep_busy()
        done = torch.cuda.Event()
        done.record()
        out, out_lse = kv4.moe_kv4_attention(q, cache, batch, return_lse=True, stream=side)
        side.synchronize()
        shown |= not done.query()
        with torch.cuda.stream(side):
            same = torch.equal(out, want) and torch.equal(out_lse, lse)
        assert same
        torch.cuda.synchronize()
        del busy
    if not shown:
        pytest.skip("the current stream was never busy while the call ran: nothing is shown")


def test_workspace_of_a_stream(kv4):
    cache, batch, q = case(kv4)
    want = kv4.moe_kv4_attention(q, cache, batch)
    side = torch.cuda.Stream()
    n = kv4.alloc_workspace(cache, batch, q.shape[1]).numel()
    used_memory(n)
    torch.cuda.synchronize()
    busy = keep_busy()
    ws = kv4.alloc_workspace(cache, batch, q.shape[1], stream=side)
    out = kv4.moe_kv4_attention(q, cache, batch, workspace=ws, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        assert not ws[:kv4.MOE_KV4_WS_HEADER].any() and torch.equal(out, want)
    torch.cuda.synchronize()
    del busy


def test_outputs_on_the_given_stream(kv4):
    """append, read and the page calls write what they made, not memory that the
    current stream's pending work still uses."""
    cache, batch, _ = case(kv4)
    g = torch.Generator(device="cuda").manual_seed(1)
    t = batch.tokens
    q = torch.randn(t, 8, 128, device="cuda", generator=g).to(torch.bfloat16)
    k = torch.randn(t, 2, 128, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    want = kv4.moe_kv4_append(cache, batch, q, k, k, w, w)
    want_k, want_v = kv4.moe_kv4_read(cache, batch)
    seqs = kv4.Sequences.empty(4, 8, cache.shape.n_pages)
    one, length = ints([0]), ints([100])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = keep_busy()
    # memory that the current stream writes once its work is done: the calls' outputs
    # must not lie there
    late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
            (q.numel() * 2, k.numel() * 2, k.numel() * 2, 512, 1 << 20)]
    for x in late:
        x.fill_(255)
    del late, x
    got = kv4.moe_kv4_append(cache, batch, q, k, k, w, w, stream=side)
    got_k, got_v = kv4.moe_kv4_read(cache, batch, stream=side)
    kv4.moe_kv4_reserve(cache, seqs, one, length, stream=side)
    used = kv4.moe_kv4_compact(cache, seqs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_k, want_k) and torch.equal(got_v, want_v)
    assert int(used) == 2 and seqs.tables.tolist()[0][:3] == [0, 1, -1]
    del busy


def test_errors_wait_for_every_stream(kv4):
    cache, batch, q = case(kv4)
    side = torch.cuda.Stream()
    bad = torch.full((1, 2, 128), float("inf"), dtype=torch.bfloat16, device="cuda")
    one = kv4.Batch(ints([0, 1]), ints([5]), batch.tables[2:3].contiguous(), 1, 1, 5)
    assert cache.errors() == (0, 0)
    with torch.cuda.stream(side):
        busy = keep_busy()
    kv4.moe_kv4_append(cache, one, None, bad, bad, stream=side)
    assert cache.errors()[0] == kv4.MOE_KV4_DEVERR_RANGE
    del busy
