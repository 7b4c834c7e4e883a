"""The MXFP4 binding on a torch without the internal calls that it prefers."""
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_block_scaled_linear_amd as nv
from gpu_helpers import device

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import nvfp4_block_scaled_linear_amd as nv
"""


def run_without(body):
    return subprocess.run([sys.executable, "-c", WITHOUT + body], cwd=ROOT, capture_output=True, text=True, timeout=100)


def test_imports_and_host_calls():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_linear_amd import build
        build.build()
    r = run_without("print(nv.status_string(0), nv.mxfp4_grouped_workspace_size(16, 8, 1536, 2048, 128, nv.OUT_COMBINE))")
    assert r.returncode == 0, r.stderr
    size = nv.mxfp4_grouped_workspace_size(16, 8, 1536, 2048, 128, nv.OUT_COMBINE)
    assert r.stdout.split()[-1] == str(size)


@pytest.mark.gpu
def test_public_forms_name_the_same_stream_and_device():
    device()
    from nvfp4_block_scaled_linear_amd import _mx
    assert _mx._public_device() == _mx._current_device() == 0
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert _mx._public_stream(0) == _mx._raw_stream(0) == stream.cuda_stream
