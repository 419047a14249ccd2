"""The binding's stream handle without torch's short way to it."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
from block_scaled_fp8_x1_gb300 import ops
class Stream:
    def __init__(self, device): self.cuda_stream = 0x1234 + (device.index or 0)
torch.cuda.current_stream = Stream
assert ops._stream(torch.device("cuda", 1)) == 0x1235
"""


def test_a_torch_without_the_raw_stream_call():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
