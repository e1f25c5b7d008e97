"""The attention kernels' bounded waits, on the GPU, through the debug-bounds build (run as
a child process by test_kv4_timeout_gpu.py; MOE_INT4_DEBUG_BOUNDS=1).

That build's host hook MOE_KV4_DEBUG_SKIP_TILE=i makes CTA 0 leave the copy of its first
warp's i-th tile out (decode kernel) or not say that V's i-th tile is there (prefill
kernel): the wait for it runs out (about 50 ms in this build), sets MOE_DEVERR_TIMEOUT
and the kernel winds down with its copies and products ended.  Nothing faults and nothing
traps.  The call must return, report the flag and leave the context usable: with the
workspace's header zeroed again, the next call gives what the first one gave."""
import os
import sys
import time

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import kv4_gpu_reference as gref  # noqa: E402
from weight_only_int4_moe_gb300 import build, kv4, ops  # noqa: E402


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def run(label, kv, ql, hkv, group, d, ps, skip):
    pool, tables, cu, q = gref.make_case(1, kv, ql, hkv, group, d, ps)
    cache = kv4.Cache(pool[None], hkv, d, ps)
    batch = kv4.Batch(ints(cu), ints(kv), ints(tables), int(cu[-1]), max(ql), max(kv))
    ws = kv4.alloc_workspace(cache, batch, hkv * group)
    want = kv4.moe_kv4_attention(q, cache, batch, workspace=ws)
    torch.cuda.synchronize()
    assert not ws[:kv4.MOE_KV4_WS_HEADER].any()
    os.environ["MOE_KV4_DEBUG_SKIP_TILE"] = str(skip)
    t0 = time.perf_counter()
    kv4.moe_kv4_attention(q, cache, batch, workspace=ws)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    del os.environ["MOE_KV4_DEBUG_SKIP_TILE"]
    flags = int(ws[:4].view(torch.int32)[0])
    assert flags == ops.MOE_DEVERR_TIMEOUT, hex(flags)
    assert dt < 20.0, dt
    ws[:kv4.MOE_KV4_WS_HEADER].zero_()
    again = kv4.moe_kv4_attention(q, cache, batch, workspace=ws)
    torch.cuda.synchronize()
    assert not ws[:kv4.MOE_KV4_WS_HEADER].any() and torch.equal(again, want)
    print(f"{label}: timeout reported after {dt * 1e3:.0f} ms, next call as before", flush=True)


def main():
    assert ops.debug_bounds(), "run with MOE_INT4_DEBUG_BOUNDS=1"
    ops.load_library()
    assert ops.library_path() == build.DEBUG_LIB
    run("decode, 8 rows", [150000], [1], 8, 4, 128, 64, 3)
    run("decode, 16 rows", [150000, 900], [1, 1], 8, 16, 64, 16, 5)
    run("prefill, items of 256 rows", [9000], [600], 4, 8, 128, 64, 4)
    run("prefill, items of up to 128 rows", [700] * 90, [14] * 90, 4, 8, 64, 32, 5)
    run("prefill, the first tile", [700] * 90, [14] * 90, 4, 8, 128, 64, 0)
    print("kv4 timeouts: all cases reported and recovered", flush=True)


if __name__ == "__main__":
    main()
