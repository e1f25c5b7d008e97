"""moe_linear's bounded waits, on the GPU, through the debug-bounds build (run as a child
process by test_linear_timeout_gpu.py; MOE_INT4_DEBUG_BOUNDS=1).

That build's host hook MOE_LINEAR_DEBUG_SKIP_LINE=i makes block 0 leave the copy of w for
its i-th line out: the wait for it runs out (about 50 ms in this build), sets
MOE_DEVERR_TIMEOUT and the kernel winds down with its copies and products ended.  Nothing
faults and nothing traps.  The call must return, report the flag and leave the context
usable: the next call gives what the first one gave."""
import os
import sys
import time

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

from weight_only_int4_moe_gb300 import build, layer, ops  # noqa: E402


def run(label, m, n, k, skip, dtype=torch.bfloat16, out=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = (torch.randn(r, k, generator=g, device="cuda").to(dtype) for r in (m, n))
    lin = layer.Linear(w)
    want = layer.moe_linear(x, lin, out_dtype=out)
    assert lin.errors() == 0
    os.environ["MOE_LINEAR_DEBUG_SKIP_LINE"] = str(skip)
    t0 = time.perf_counter()
    layer.moe_linear(x, lin, out_dtype=out)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    del os.environ["MOE_LINEAR_DEBUG_SKIP_LINE"]
    assert lin.errors() == ops.MOE_DEVERR_TIMEOUT, hex(lin.errors())
    assert dt < 20.0, dt
    lin.clear_errors()
    again = layer.moe_linear(x, lin, out_dtype=out)
    assert lin.errors() == 0 and torch.equal(again, want)
    print(f"{label}: timeout reported after {dt * 1e3:.0f} ms, next call as before", flush=True)


def main():
    assert ops.debug_bounds(), "run with MOE_INT4_DEBUG_BOUNDS=1"
    ops.load_library()
    assert ops.library_path() == build.DEBUG_LIB
    f32, e4m3 = torch.float32, torch.float8_e4m3fn
    run("one block a tile, the first line", 40, 512, 512, 0)
    run("a tile's k over several blocks", 5, 384, 7168, 9)
    run("more lines than stages", 100, 20000, 2048, 25)
    run("pairs", 2600, 2048, 1024, 7)
    run("pairs, in a later tile", 8192, 4096, 1024, 30)
    run("pairs, sums of fp32 results", 4096, 2048, 3000 // 8 * 8, 40, out=f32)
    run("pairs, codes", 4096, 4096, 2048, 11, e4m3)
    print("linear timeouts: all cases reported and recovered", flush=True)


if __name__ == "__main__":
    main()
