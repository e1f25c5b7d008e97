"""The decoder layer example: attention over the 4-bit cache and the expert MLP,
prefill, graph decode, fork, tree verification, free and compact together."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_decoder_layer_example():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py")],
                       capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.strip().endswith("ok")
