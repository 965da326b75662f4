"""Host side of the operators between the GEMMs at their smallest sizes (CPU
only: no call here touches a device)."""
import subprocess
import sys

import pytest

from conftest import ROOT
from fp8_block_scaled_x128_amd import ops


def test_workspace_of_no_columns_in_a_process_of_its_own():
    """A fault in the library ends the process, so this one asks in a child."""
    code = ("from fp8_block_scaled_x128_amd import ops\n"
            "print(ops.fp8_block_norm_backward_ws_size(4, 0, 2, True, True, True))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "0", (r.returncode, r.stderr[-300:])


@pytest.mark.parametrize("rows", [0, 1, 5, 1 << 20])
@pytest.mark.parametrize("cols", [0, 8])
@pytest.mark.parametrize("gate_rows", [1, 3, 1 << 40])
def test_workspace_of_small_sizes(rows, cols, gate_rows):
    n = ops.fp8_block_norm_backward_ws_size(rows, cols, gate_rows, True, True, True)
    assert (n == 0) == (rows == 0 or cols == 0) and n % 16 == 0
    # never more than one partial row per row, each for the three sums, and
    # one per workgroup of at most four per compute unit
    assert n <= 3 * 4 * cols * max(1, min(rows, 4 * 256))
