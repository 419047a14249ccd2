"""expert_rows at expert counts around the 48 KB of shared memory that a launch may have without asking."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

RUN = """
import sys
import numpy as np, torch
sys.path[:0] = [{root!r}, {tests!r}]
import expert_reference as ref
from block_scaled_fp8_x1_gb300 import ops
E = {E}
idx = np.random.default_rng(E).integers(0, E, ({T}, 3)).astype(np.int32)
for align in (1, 128):
    r = ops.expert_rows(torch.tensor(idx, device="cuda"), E, align)
    for got, want in zip(r[:4], ref.rows(idx, E, align)):
        assert np.array_equal(got.cpu().numpy(), want), align
"""


@pytest.mark.parametrize("E,T", [(680, 50), (681, 50), (682, 50), (682, 2000), (683, 50)])
def test_expert_rows_in_a_fresh_process(fp8lib, E, T):
    """A process of its own: a larger count before it would have raised the kernel's limit."""
    import os
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", RUN.format(root=os.path.dirname(tests), tests=tests, E=E, T=T)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
