"""The debug build (-DTXL_DEBUG) on the paged memory and the attention for drafted trees:
in a child process that loads it, their parity tests pass with every device-side index
check active (ring columns through which the nodes' depths shift the position products,
ancestors' distances, table slots, staged rows)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def test_paged_parity_tests_pass_with_index_checks():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_tree.py", "tests/test_gpu_paged.py"],
                       cwd=ROOT, env=dict(os.environ, TXL_DEBUG_LIB="1"), capture_output=True, text=True,
                       timeout=1800)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
