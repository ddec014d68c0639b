"""The package's host-side calls on a torch that lacks the functions by which a GPU build
is asked for its current stream (a CPU build, or another version)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import sparse_delta_codec_amd as pulse
ntiles, tile0, tile_seg = pulse.pulse_segment_tiles([5, 16385])
assert ntiles == 3
"""


def test_host_side_calls_need_no_stream():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
